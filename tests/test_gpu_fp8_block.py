"""FP8 with a scale per block of 128 on the GPU against the oracle: scales and
the codes of bf16 bit for bit, the codes of fp32 but for quotients within one
step of the middle of two codes, the GEMM within |C - C64| <= 1e-5 sum |a b| (+ half a bf16
step of the result for bf16 output), on both of its kernels.

The GEMM's bound: a chunk's tensor-core sum of 128 products takes part in at
most 5 binary32 roundings per K = 32 step and chunk, the scales in 2, and the
promotion in one per chunk; at K = 14336 (112 chunks) that is under 140
roundings of 2^-24, 8.4e-6 of sum |a b|.
"""
import numpy as np
import pytest
import torch

import oracle
from parity import assert_within_gemm_bound, oracle_input

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fp4(cuda_device):
    from fp4_block_scaled_h16_b200 import fp4 as m
    return m


def make(rows, cols, seed, dtype=torch.bfloat16, pad=0):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, (cols + 7) // 8 * 8 + pad)).astype(np.float32)
    x[:, rng.integers(0, cols, max(1, cols // 100))] *= 50.0
    x[rng.integers(0, rows)] = 0.0                       # a block of zeros
    x[rng.integers(0, rows)] *= np.float32(2.0 ** -130)  # subnormal quotients
    return torch.from_numpy(x).to(dtype)[:, :cols]


def assert_same(q, o, exact, what=""):
    codes, scales = q["codes"].cpu().numpy()[:, :q["K"]], q["scales"].cpu().numpy()
    n = o["scales"].shape[0]
    assert (scales[:, :n].T.view(np.uint32) == o["scales"].view(np.uint32)).all(), what + " scales"
    bad = codes != o["codes"]
    if exact:
        at = np.argwhere(bad)
        assert len(at) == 0, "%s: %d codes differ, first %s" % (what, len(at), at[:3].tolist())
    elif bad.any():
        # both quotients are roundings of nearly the same number: one step of
        # 2^-23 may lie between them, across the middle of two codes
        value = lambda c: oracle.fp8_dequantize(dict(codes=c.reshape(1, -1), scale=1.0))[0]  # noqa: E731
        got, want, quotient = codes[bad], o["codes"][bad], o["quotients"][bad].astype(np.float64)
        assert (np.abs(got.astype(int) - want.astype(int)) == 1).all(), what
        assert (np.abs(quotient - (value(got) + value(want)) / 2) <= 2.0 ** -23 * np.abs(quotient)).all(), what


SHAPES = [(1, 1), (1, 4096), (3, 130), (128, 128), (127, 129), (129, 127), (300, 513), (1000, 272), (257, 2000)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lines", [1, 128])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("pad", [0, 24])
def test_quantize_matches_oracle(fp4, dtype, lines, shape, pad):
    x = make(*shape, seed=shape[0] + shape[1], dtype=dtype, pad=pad)
    xd = torch.zeros((shape[0], x.stride(0) if shape[0] > 1 else shape[1] + (-shape[1]) % 8 + pad), dtype=dtype).cuda()
    xd[:, :shape[1]] = x.cuda()
    if xd.shape[1] > shape[1]:
        xd[:, shape[1]:] = 1e30                          # never read into a block
    xd = xd[:, :shape[1]]
    want = [oracle.fp8_block_quantize(oracle_input(x.contiguous()), lines, axis) for axis in (1, 0)]
    exact = dtype == torch.bfloat16
    assert_same(fp4.fp8_block_quantize(xd, 1, lines), want[0], exact, "rows")
    assert_same(fp4.fp8_block_quantize(xd, 0, lines), want[1], exact, "columns")
    qr, qc = fp4.fp8_block_quantize_both_axes(xd, lines)
    assert_same(qr, want[0], exact, "rows of both")
    assert_same(qc, want[1], exact, "columns of both")
    assert fp4.fp4_last_error() == fp4.FP4_OK


def test_quantize_writes_nothing_past_its_lines_and_columns(fp4):
    x = make(130, 200, 5).cuda()
    qr, qc = fp4.alloc_fp8_block(130, 200), fp4.alloc_fp8_block(200, 130)
    for q in (qr, qc):
        q["codes"].fill_(0xA5)
        q["scales"].fill_(-7.0)
    fp4.fp8_block_quantize_both_axes(x, out_rows=qr, out_cols=qc)
    torch.cuda.synchronize()
    for q in (qr, qc):
        assert (q["codes"][:, q["K"]:] == 0xA5).all()
        assert (q["scales"][:, q["lines"]:] == -7.0).all() and (q["scales"][:, :q["lines"]] > 0).all()


def test_empty_quantize_and_gemm(fp4):
    q = fp4.fp8_block_quantize(torch.zeros((0, 256), dtype=torch.bfloat16, device="cuda"))
    w = fp4.fp8_block_quantize(make(300, 256, 1).cuda(), 1, 128)
    assert fp4.fp8_block_gemm(q, w).shape == (0, 300)


def upload(fp4, o):
    q = fp4.alloc_fp8_block(o["codes"].shape[0], o["codes"].shape[1], o["block_lines"])
    q["codes"].fill_(0x7F)                               # NaN codes past K: never read into a sum
    q["codes"][:, :q["K"]] = torch.from_numpy(o["codes"]).cuda()
    q["scales"].fill_(float("nan"))                      # lines past the last: never in a stored element
    q["scales"][:, :o["scales"].shape[0]] = torch.from_numpy(np.ascontiguousarray(o["scales"].T)).cuda()
    return q


def check_gemm(fp4, M, N, K, b_lines, out_bf16, seed, pitch_extra=0):
    rng = np.random.default_rng(seed)
    a = rng.standard_normal((M, K)).astype(np.float32) * np.exp(rng.standard_normal((M, 1))).astype(np.float32)
    b = rng.standard_normal((N, K)).astype(np.float32) * 0.05
    oa, ob = oracle.fp8_block_quantize(a, 1), oracle.fp8_block_quantize(b, b_lines)
    ld = (N + 7) // 8 * 8 + pitch_extra
    buf = torch.full((M + 1, ld), -77.0, dtype=torch.bfloat16 if out_bf16 else torch.float32, device="cuda")
    fp4.fp8_block_gemm(upload(fp4, oa), upload(fp4, ob), fp4.FP4_OUT_BF16 if out_bf16 else fp4.FP4_OUT_F32,
                       out=buf[:M, :N])
    assert fp4.fp4_last_error() == fp4.FP4_OK
    C64, bound = oracle.fp8_block_gemm(oa, ob)
    assert_within_gemm_bound(buf[:M, :N].float().cpu().numpy(), C64, bound, out_bf16, "%s" % ((M, N, K, b_lines),))
    assert (buf[:M, N:] == -77.0).all() and (buf[M] == -77.0).all()


SMALL = [(1, 128, 128), (1, 1, 1), (1, 4096, 512), (2, 130, 257), (7, 300, 1000), (16, 256, 4096), (17, 129, 640),
         (33, 1000, 384), (64, 128, 2048), (65, 513, 130), (130, 100, 129), (200, 1000, 1536)]


@pytest.mark.parametrize("out_bf16", [False, True])
@pytest.mark.parametrize("b_lines", [1, 128])
@pytest.mark.parametrize("shape", SMALL)
def test_gemm_small(fp4, shape, b_lines, out_bf16):
    check_gemm(fp4, *shape, b_lines, out_bf16, seed=sum(shape))


# outputs that run on CTA pairs: whole and ragged tiles, one chunk and many,
# fewer tiles than pairs and several waves (1 x 128 blocks: the first and third on
# one round of 128 x 192 tiles)
LARGE = [(1280, 2048, 256), (2300, 1900, 130), (1111, 2999, 1025), (2560, 2560, 100), (4096, 2300, 640)]


@pytest.mark.parametrize("out_bf16", [False, True])
@pytest.mark.parametrize("b_lines", [1, 128])
@pytest.mark.parametrize("shape", LARGE)
def test_gemm_large(fp4, shape, b_lines, out_bf16):
    check_gemm(fp4, *shape, b_lines, out_bf16, seed=sum(shape), pitch_extra=16)


@pytest.mark.parametrize("b_lines", [1, 128])
def test_gemm_large_without_pairs(fp4, b_lines):
    fp4.fp4_set_gemm_cta_pairs(False)
    try:
        check_gemm(fp4, 1111, 2999, 1025, b_lines, True, seed=8)
    finally:
        fp4.fp4_set_gemm_cta_pairs(True)


@pytest.mark.parametrize("M,N,K", [(1, 512, 14336), (1300, 2100, 14336)])
def test_gemm_long_k(fp4, M, N, K):
    check_gemm(fp4, M, N, K, 128, False, seed=K)


@pytest.mark.parametrize("M,N,K", [(3, 640, 8192), (2048, 2304, 2048)])
def test_gemm_is_deterministic_and_row_independent(fp4, M, N, K):
    g = torch.Generator().manual_seed(2)
    x, w = torch.randn((M, K), generator=g).cuda(), torch.randn((N, K), generator=g).cuda()
    qa, qb = fp4.fp8_block_quantize(x), fp4.fp8_block_quantize(w, 1, 128)
    first = fp4.fp8_block_gemm(qa, qb)
    for _ in range(3):
        assert torch.equal(fp4.fp8_block_gemm(qa, qb), first)


@pytest.mark.parametrize("M,N,K,b_lines", [(4, 256, 8192, 128), (4, 256, 8192, 1), (2304, 2304, 8192, 128),
                                           (2304, 2304, 8192, 1)])
def test_gemm_wait_timeout_is_reported_and_recoverable(fp4, M, N, K, b_lines):
    g = torch.Generator().manual_seed(3)
    qa = fp4.fp8_block_quantize(torch.randn((M, K), generator=g).cuda())
    qb = fp4.fp8_block_quantize(torch.randn((N, K), generator=g).cuda(), 1, b_lines)
    before = fp4.fp8_block_gemm(qa, qb)
    assert fp4.fp4_last_error() == fp4.FP4_OK
    fp4.fp4_set_wait_limit(1)
    try:
        fp4.fp8_block_gemm(qa, qb)
        status = fp4.fp4_last_error()
    finally:
        fp4.fp4_set_wait_limit(0)
    assert status == fp4.FP4_ERR_TIMEOUT, fp4.fp4_status_string(status)
    after = fp4.fp8_block_gemm(qa, qb)
    assert fp4.fp4_last_error() == fp4.FP4_OK
    assert torch.equal(before, after)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantizer_over_the_range_of_magnitudes(fp4, dtype):
    """A block per power of two, the subnormal ones and the largest finite values among them."""
    e = np.repeat(np.arange(-140, 128), 2)
    rng = np.random.default_rng(11)
    x = rng.uniform(0.5, 1.0, (len(e), 256)) * rng.choice([-1.0, 1.0], (len(e), 256))
    x[:, 1::3] *= rng.uniform(0, 0.01, x[:, 1::3].shape)
    x = torch.from_numpy((x * np.exp2(e.astype(np.float64))[:, None]).astype(np.float32)).to(dtype)
    x[-1, :4] = torch.finfo(dtype).max
    assert torch.isfinite(x).all()
    o = oracle.fp8_block_quantize(oracle_input(x))
    assert_same(fp4.fp8_block_quantize(x.cuda()), o, dtype == torch.bfloat16)
    assert_same(fp4.fp8_block_quantize(x.t().contiguous().cuda(), 0), o, dtype == torch.bfloat16)


@pytest.mark.parametrize("b_lines", [1, 128])
def test_quantizer_recovers_from_a_wait_that_runs_out(fp4, b_lines):
    """One poll may or may not see the tile land; a call after it is right either way."""
    x = torch.randn((1500, 2100), generator=torch.Generator().manual_seed(6)).cuda()
    for t in (x, x.bfloat16()):
        t = torch.nn.functional.pad(t, (0, 12))[:, :2100]
        before = fp4.fp8_block_quantize_both_axes(t, b_lines)
        fp4.fp4_set_wait_limit(1)
        try:
            fp4.fp8_block_quantize_both_axes(t, b_lines)
            status = fp4.fp4_last_error()
        finally:
            fp4.fp4_set_wait_limit(0)
        assert status in (fp4.FP4_OK, fp4.FP4_ERR_TIMEOUT), fp4.fp4_status_string(status)
        after = fp4.fp8_block_quantize_both_axes(t, b_lines)
        assert fp4.fp4_last_error() == fp4.FP4_OK
        for a, b, n, k in zip(before, after, (1500, 2100), (2100, 1500)):
            assert torch.equal(a["codes"][:, :k], b["codes"][:, :k])
            m = n if b_lines == 1 else a["scales"].shape[1]
            assert torch.equal(a["scales"][:, :m], b["scales"][:, :m])


@pytest.mark.parametrize("out_bf16", [False, True])
@pytest.mark.parametrize("shape", [(1150, 4090, 256), (128, 14336, 512), (513, 6140, 300), (128, 4096, 2304)])
def test_gemm_tiles_of_192_and_256_lines(fp4, shape, out_bf16):
    """1 x 128 blocks on both widths, K whole and split: 256 for the first two."""
    check_gemm(fp4, *shape, 1, out_bf16, seed=sum(shape))


@pytest.mark.parametrize("M,N,out", [(3, 128 * 65536 + 40, "bf16"), (128 * 65536 + 40, 3, "f32")])
def test_gemm_with_more_tiles_than_a_grid_has_lines(fp4, M, N, out):
    """Beyond 65535 tiles along either side, on single CTAs."""
    K = 16
    g = torch.Generator(device="cuda").manual_seed(7)
    a = torch.randint(-3, 4, (M, K), generator=g, device="cuda").to(torch.bfloat16)
    b = torch.randint(-3, 4, (N, K), generator=g, device="cuda").to(torch.bfloat16)
    a[:, 0] = b[:, 0] = 7                                    # one scale, 7 / 448 = 2^-6, for every block
    qa, qb = fp4.fp8_block_quantize(a), fp4.fp8_block_quantize(b)
    fp4.fp4_set_gemm_cta_pairs(False)
    try:
        c = fp4.fp8_block_gemm(qa, qb, fp4.FP4_OUT_BF16 if out == "bf16" else fp4.FP4_OUT_F32)
    finally:
        fp4.fp4_set_gemm_cta_pairs(True)
    assert fp4.fp4_last_error() == fp4.FP4_OK
    want = a.float() @ b.float().T                           # integers below 2^8: exact
    assert torch.equal(c.float(), want)


def test_two_streams_at_once(fp4):
    g = torch.Generator().manual_seed(4)
    x, w = torch.randn((64, 4096), generator=g).cuda(), torch.randn((1024, 4096), generator=g).cuda()
    qb = fp4.fp8_block_quantize(w, 1, 128)
    want = fp4.fp8_block_gemm(fp4.fp8_block_quantize(x), qb)
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    for s in streams * 4:
        qa = fp4.fp8_block_quantize(x, stream=s)
        outs.append(fp4.fp8_block_gemm(qa, qb, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


# outputs of the pair kernel and of the split kernel's 16-, 64-, 192- and 256-line tiles
@pytest.mark.parametrize("M,N,K", [(4096, 2300, 200), (2300, 1900, 130), (1150, 4090, 256), (130, 300, 200), (40, 300, 260),
                                   (3, 200, 130)])
@pytest.mark.parametrize("b_lines", [1, 128])
@pytest.mark.parametrize("ea,eb", [(-110, 124), (118, -105)])
def test_gemm_with_scales_far_apart(fp4, M, N, K, b_lines, ea, eb):
    """The product of two scales lies near 1, but a partial product times one of them passes binary32."""
    rng = np.random.default_rng(M + N)
    a = (rng.standard_normal((M, K)) * 2.0 ** ea).astype(np.float32)
    b = (rng.standard_normal((N, K)) * 0.05 * 2.0 ** eb).astype(np.float32)
    oa, ob = oracle.fp8_block_quantize(a, 1), oracle.fp8_block_quantize(b, b_lines)
    assert np.isfinite(a).all() and np.isfinite(b).all()
    assert max(oa["scales"].max(), ob["scales"].max()) > 2.0 ** 108 and max(oa["scales"].min(), ob["scales"].min()) > 1
    C64, bound = oracle.fp8_block_gemm(oa, ob)
    for pairs in (True, False):
        fp4.fp4_set_gemm_cta_pairs(pairs)
        try:
            C = fp4.fp8_block_gemm(upload(fp4, oa), upload(fp4, ob))
        finally:
            fp4.fp4_set_gemm_cta_pairs(True)
        assert torch.isfinite(C).all()
        assert_within_gemm_bound(C.cpu().numpy(), C64, bound, False, "%s" % ((M, N, K, b_lines, ea, eb, pairs),))
    assert fp4.fp4_last_error() == fp4.FP4_OK


@pytest.mark.parametrize("M,N,K,b_lines", [(2300, 1900, 640, 1), (2300, 1900, 640, 128), (333, 1000, 1300, 128),
                                           (300, 1000, 1300, 1), (50, 700, 2050, 128), (9, 700, 2050, 1)])
def test_gemm_rows_and_columns_do_not_see_each_other(fp4, M, N, K, b_lines):
    """With other tokens around it a token keeps its row, bit for bit, and a line of the weight its column."""
    g = torch.Generator().manual_seed(M)
    x, w = torch.randn((M, K), generator=g), torch.randn((N, K), generator=g)
    C = fp4.fp8_block_gemm(fp4.fp8_block_quantize(padded(x)), fp4.fp8_block_quantize(padded(w), 1, b_lines))
    rows = [0, M // 2, M - 1]
    x2 = torch.randn((M, K), generator=g) * 100
    x2[rows] = x[rows]
    D = fp4.fp8_block_gemm(fp4.fp8_block_quantize(padded(x2)), fp4.fp8_block_quantize(padded(w), 1, b_lines))
    assert torch.equal(C[rows], D[rows]) and not torch.equal(C, D)
    block = slice(128, 256) if b_lines == 128 else slice(130, 131)       # lines that share a scale
    w2 = torch.randn((N, K), generator=g) * 100
    w2[block] = w[block]
    D = fp4.fp8_block_gemm(fp4.fp8_block_quantize(padded(x)), fp4.fp8_block_quantize(padded(w2), 1, b_lines))
    assert torch.equal(C[:, block], D[:, block]) and not torch.equal(C, D)


def padded(t):
    """On the GPU in fp32, with a row pitch of a multiple of 16 bytes."""
    room = torch.zeros((t.shape[0], (t.shape[1] + 3) // 4 * 4), device="cuda")
    room[:, :t.shape[1]] = t.cuda()
    return room[:, :t.shape[1]]
