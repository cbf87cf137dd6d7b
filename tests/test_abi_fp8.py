"""Host validation of the FP8 block-128 and norm / residual entry points, and
the refusals of their Python helpers (no GPU needed, nothing launched)."""
import pytest
import torch

fp4 = pytest.importorskip("fp4_block_scaled_h16_b200.fp4", reason="libfp4.so not built")

A = 1 << 20      # a fake, 16-byte aligned address: validation fails before any use
INVALID, SHAPE, MISALIGNED, WORKSPACE, NO_DEVICE = 1, 2, 3, 4, 5
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="the fake addresses must never reach a GPU")


def test_scales_count():
    n = fp4.fp4_fp8_block_scales_count
    assert n(1, 1, 1) == 128 and n(129, 4096, 1) == 256 * 32 and n(129, 4097, 128) == 2 * 33
    assert n(0, 4096, 1) == 0 and n(5, 0, 128) == 0 and n(5, 5, 64) == 0


def q(**kw):
    a = dict(x=A, dt=fp4.FP4_IN_BF16, rows=100, cols=200, ld=200, lines=1, cr=A, lr=208, sr=A, cc=A, lc=112, sc=A)
    a.update(kw)
    return fp4._lib.fp4_fp8_block_quantize(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(dt=7), INVALID), (dict(lines=64), INVALID), (dict(rows=-1), INVALID), (dict(ld=100), INVALID),
    (dict(x=None), INVALID), (dict(cr=None, cc=None), INVALID), (dict(sr=None), INVALID), (dict(sc=None), INVALID),
    (dict(lr=192), INVALID), (dict(lc=96), INVALID), (dict(x=A + 8), MISALIGNED), (dict(ld=204), MISALIGNED),
    (dict(lr=200), MISALIGNED), (dict(lc=104), MISALIGNED), (dict(cr=A + 8), MISALIGNED), (dict(sc=A + 4), MISALIGNED),
    (dict(rows=1 << 33, lc=1 << 33), SHAPE),
    (dict(rows=0), 0), (dict(cols=0, ld=0), 0),
])
def test_quantize_validation(kw, status):
    assert q(**kw) == status


def g(**kw):
    a = dict(a=A, lda=208, sa=A, b=A, ldb=208, sb=A, lines=128, M=100, N=300, K=200, c=A, out=fp4.FP4_OUT_BF16, ldc=304)
    a.update(kw)
    return fp4._lib.fp4_fp8_block_gemm(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(out=2), INVALID), (dict(lines=16), INVALID), (dict(M=-1), INVALID), (dict(ldc=299), INVALID),
    (dict(lda=192), INVALID), (dict(ldb=64), INVALID), (dict(a=None), INVALID), (dict(sa=None), INVALID),
    (dict(sb=None), INVALID), (dict(c=None), INVALID), (dict(K=0), SHAPE), (dict(M=1 << 32), SHAPE),
    (dict(lda=200), MISALIGNED), (dict(a=A + 8), MISALIGNED), (dict(sb=A + 4), MISALIGNED), (dict(c=A + 2), MISALIGNED),
    (dict(ldc=301), MISALIGNED), (dict(M=0), 0), (dict(N=0, K=0), 0),
])
def test_gemm_validation(kw, status):
    assert g(**kw) == status


def n(**kw):
    a = dict(o=A, ldo=104, h=A, ldh=104, dt=fp4.FP4_IN_BF16, rows=10, cols=100, w_post=A, gate=A, ldg=104, per=4,
             alpha=1.0, w_pre=A, eps=1e-6, h_out=A, ldho=104, y=A, ldy=104, codes=None, ldc=0, scales=None, r1=A, r2=A)
    a.update(kw)
    return fp4._lib.fp4_norm_residual(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(dt=3), INVALID), (dict(rows=-1), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(alpha=float("inf")), INVALID), (dict(o=None), INVALID),
    (dict(o=None, gate=None), INVALID), (dict(y=None), INVALID), (dict(w_pre=None), INVALID), (dict(per=0), INVALID),
    (dict(h=None), INVALID), (dict(h_out=None), INVALID), (dict(r1=None), INVALID), (dict(r2=None), INVALID),
    (dict(codes=A, ldc=112), INVALID), (dict(ldo=96), INVALID), (dict(ldg=96), INVALID),
    (dict(o=None, w_post=None, gate=None, w_pre=None, y=None), INVALID),
    (dict(cols=16385, ldo=16392, ldh=16392, ldho=16392, ldg=16392, ldy=16392), SHAPE),
    (dict(ldo=102), MISALIGNED), (dict(h=A + 8), MISALIGNED), (dict(h_out=A + 4), MISALIGNED),
    (dict(gate=A + 2), MISALIGNED), (dict(w_post=A + 8), MISALIGNED), (dict(r2=A + 2), MISALIGNED),
    (dict(codes=A, ldc=104, scales=A), MISALIGNED), (dict(codes=A, ldc=112, scales=A + 4), MISALIGNED),
    (dict(rows=0), 0),
])
def test_norm_validation(kw, status):
    assert n(**kw) == status


def b(**kw):
    a = dict(dy=A, lddy=104, dhi=A, lddhi=104, h=A, ldh=104, o=A, ldo=104, dt=fp4.FP4_IN_BF16, rows=10, cols=100,
             w_post=A, gate=A, ldg=104, per=4, alpha=1.0, w_pre=A, r1=A, r2=A, dh=A, lddh=104, do=A, lddo=104, dwp=A,
             dwo=A, dg=A, ws=A, wsb=1 << 30)
    a.update(kw)
    return fp4._lib.fp4_norm_residual_backward(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(dt=3), INVALID), (dict(rows=-1), INVALID), (dict(alpha=float("nan")), INVALID), (dict(dwp=None), INVALID),
    (dict(dwo=None), INVALID), (dict(dg=None), INVALID), (dict(per=0), INVALID), (dict(dy=None), INVALID),
    (dict(h=None), INVALID), (dict(r2=None), INVALID), (dict(r1=None), INVALID), (dict(dh=None), INVALID),
    (dict(do=None), INVALID), (dict(o=None), INVALID), (dict(lddy=96), INVALID),
    (dict(dy=None, w_pre=None, dwp=None, dhi=None), INVALID),
    (dict(cols=16385), SHAPE), (dict(dwp=A + 4), MISALIGNED), (dict(dg=A + 8), MISALIGNED), (dict(ldo=102), MISALIGNED),
    (dict(dh=A + 2), MISALIGNED), (dict(ws=A + 4), MISALIGNED), (dict(ws=None), WORKSPACE), (dict(wsb=16), WORKSPACE),
])
def test_norm_backward_validation(kw, status):
    assert b(**kw) == status


@no_gpu
def test_valid_calls_without_a_gpu_report_no_device():
    assert q() == q(cr=None) == q(cc=None) == g() == n() == b() == NO_DEVICE


def test_backward_workspace():
    ws = fp4.fp4_norm_residual_backward_workspace_size
    assert ws(0, 100, 1, 1, 0, 0) == 0
    assert ws(1, 100, 1, 0, 0, 0) == 400 and ws(1, 101, 1, 1, 0, 0) == 2 * 416
    assert ws(5, 128, 0, 0, 1, 1) == 0                  # a gate per row: its gradient is written directly
    with pytest.raises(fp4.Fp4Error):
        ws(5, 100, 1, 1, 1, 0)
    with pytest.raises(fp4.Fp4Error):
        ws(5, 16385, 1, 1, 0, 0)


def cpu(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def test_python_refusals():
    with pytest.raises(ValueError):
        fp4.fp8_block_quantize(cpu(4, 128))              # a CPU tensor
    with pytest.raises(ValueError):
        fp4.fp8_block_quantize(cpu(4, 128), axis=2)
    with pytest.raises(ValueError):
        fp4.alloc_fp8_block(4, 128, 64, device="cpu")
    a = fp4.alloc_fp8_block(4, 128, device="cpu")
    with pytest.raises(ValueError):
        fp4.fp8_block_gemm(a, fp4.alloc_fp8_block(4, 256, device="cpu"))     # another K
    with pytest.raises(ValueError):
        fp4.fp8_block_gemm(fp4.alloc_fp8_block(4, 128, 128, device="cpu"), a)   # A in 128 x 128 blocks
    with pytest.raises(ValueError):
        fp4.fp8_block_gemm(a, a)                         # CPU tensors
    with pytest.raises(ValueError):
        fp4.norm_residual(cpu(4, 128), w_pre=cpu(128))
    with pytest.raises(ValueError):
        fp4.norm_residual_backward(None, None)


def test_helper_checks_refuse_wrong_buffers():
    bf16, f32, dev = torch.bfloat16, torch.float32, -1          # -1: CPU tensors, as the checks see them
    good = fp4.alloc_fp8_block(4, 100, device="cpu")
    assert fp4._fp8_tensor(good, "q", 4, 100, 1, dev)[1] == 112
    for bad in (dict(good, codes=good["codes"][:, :96]), dict(good, codes=good["codes"].t()),
                dict(good, codes=good["codes"].float()), dict(good, scales=good["scales"][:, ::2]),
                dict(good, scales=good["scales"][:, :64]), dict(good, lines=5), dict(good, K=99),
                dict(good, block_lines=128)):
        with pytest.raises((ValueError, TypeError)):
            fp4._fp8_tensor(bad, "q", 4, 100, 1, dev)
    with pytest.raises((ValueError, TypeError)):
        fp4._fp8_tensor(good, "q", 4, 100, 1, 0)                # another device
    with pytest.raises(TypeError):
        fp4._mat(cpu(4, 100), "o", (4, 100), f32, dev)
    with pytest.raises(ValueError):
        fp4._mat(cpu(4, 200)[:, ::2], "o", (4, 100), bf16, dev)
    assert fp4._mat(cpu(4, 112)[:, :100], "o", (4, 100), bf16, dev) == 112
    assert fp4._mat(cpu(1, 100), "o", (1, 100), bf16, dev) == 112    # any pitch does for one row
    with pytest.raises(ValueError):
        fp4._gate_of(cpu(2, 100), None, 4, 100, bf16, dev)
    with pytest.raises(ValueError):
        fp4._gate_of(cpu(3, 100), 2, 4, 100, bf16, dev)
    with pytest.raises(ValueError):
        fp4._flat(torch.zeros(5), "rstd", (4,), f32, dev)
    with pytest.raises(ValueError):
        fp4._flat(torch.zeros(8)[::2], "rstd", (4,), f32, dev)


@pytest.mark.parametrize("per", [10, 11, 2 ** 40, 2 ** 63 - 1])
def test_groups_longer_than_the_rows_are_one_group(per):
    """rows + rows_per_group may pass 63 bits."""
    want = fp4.fp4_norm_residual_backward_workspace_size(10, 8, True, True, True, 10)
    assert want > 0
    assert fp4.fp4_norm_residual_backward_workspace_size(10, 8, True, True, True, per) == want


@pytest.mark.parametrize("n", [2 ** 31 - 512, 2 ** 31, 2 ** 63 - 1])
def test_sizes_beyond_the_tile_coordinates_are_refused(n):
    assert fp4.fp4_fp8_block_scales_count(n, 128, 1) == 0
    assert fp4.fp4_fp8_block_scales_count(1, n, 128) == 0
    with pytest.raises(fp4.Fp4Error, match="UNSUPPORTED_SHAPE"):
        fp4.fp4_norm_residual_backward_workspace_size(n, 8, True, True, True, n)
    with pytest.raises(fp4.Fp4Error, match="UNSUPPORTED_SHAPE"):
        fp4.fp4_norm_residual(None, 0, A, 8, fp4.FP4_IN_F32, n, 8, None, None, 0, 1, 1.0, A, 1e-6, None, 0, A, 8, None,
                              0, None, None, A, stream=0)
    with pytest.raises(fp4.Fp4Error, match="UNSUPPORTED_SHAPE"):
        fp4.fp4_norm_residual_backward(A, 8, None, 0, A, 8, None, 0, fp4.FP4_IN_F32, n, 8, None, None, 0, 1, 1.0, A,
                                       None, A, A, 8, None, 0, A, None, None, A, 4096, stream=0)
    with pytest.raises(fp4.Fp4Error, match="UNSUPPORTED_SHAPE"):
        fp4.fp4_fp8_block_gemm(A, 128, A, A, 128, A, 1, n, 8, 128, A, fp4.FP4_OUT_F32, 8, stream=0)


@pytest.mark.parametrize("per", [5, 2 ** 63, 2 ** 64 + 1, 2 ** 70])
def test_groups_longer_than_the_rows_reach_the_library_as_one(per):
    """Python's integers are longer than the library's: 2^64 + 1 must not arrive as 1,
    which would read a gate row per row behind the only one there is."""
    address, pitch, got = fp4._gate_of(cpu(1, 104), per, 4, 104, torch.bfloat16, -1)
    assert got == 4 and pitch == 112
    assert fp4._gate_of(cpu(0, 104), per, 0, 104, torch.bfloat16, -1)[2] == 1


def test_outputs_of_a_norm_that_is_not_asked_for_are_refused():
    """Without w_pre there is no y: a buffer for it would come back unwritten."""
    h = cpu(4, 128)
    q = fp4.alloc_fp8_block(4, 128, device="cpu")
    for kw in (dict(quantize=True), dict(out=dict(y=h)), dict(out=dict(q=q)), dict(quantize=True, out=dict(h=h))):
        with pytest.raises(ValueError, match="w_pre"):
            fp4.norm_residual(h, o=h, **kw)


@no_gpu
def test_in_place_with_another_pitch_is_refused():
    """Rows would be written over rows that are still to be read."""
    assert n(ldho=112) == n(ldh=112) == INVALID
    assert n(ldho=112, rows=1) == n(ldho=112, h_out=2 * A) == NO_DEVICE
    assert b(lddh=112) == b(lddhi=112) == INVALID
    assert b(lddh=112, rows=1) == b(lddh=112, dh=2 * A) == NO_DEVICE
