"""The norms around a block with gate and residual update, and their gradients,
on the GPU against the float64 formulas of the oracle.

Tolerances count roundings of u = 2^-24 relative to the sum of the magnitudes
that enter.  A row sum adds at most 32 products in a thread, 5 steps of a warp
and 16 warps: 53 roundings, and the mean, eps, square root and reciprocal 4
more, halved by the square root in an inverse RMS: 31.  With the products after
it the forward results stay under 40 u.  Backward, a mean of products takes 56
and the values in it up to 6: 70 u for dh; do adds a second such mean of values
that are off by 70 u: 140 u.  A column sum adds, per CTA, the rows that 148
CTAs or more leave to it, 5 for up to 700 rows, and then every 32nd of at most
700 partial sums and 32 such, 54: 60 for the sizes here, 80 u for dw_pre, 220 u
for dw_post and dgate, whose terms hold dh.  A result in bf16 adds half a step,
2^-8 of it.
"""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def fp4(cuda_device):
    from fp4_block_scaled_h16_b200 import fp4 as m
    return m


def half_step(dtype):
    return 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24


def wide(t):
    return None if t is None else t.double().cpu().numpy()


def matrix(g, rows, cols, dtype, pad=0, scale=1.0):
    t = torch.full((rows, (cols + 7) // 8 * 8 + pad), 1e30, dtype=dtype, device="cuda")
    t[:, :cols] = (torch.randn((rows, cols), generator=g) * scale).to(dtype).cuda()
    return t[:, :cols]


def inputs(rows, cols, dtype, post, per, pad, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    vec = lambda: (1 + 0.2 * torch.randn(cols, generator=g)).to(dtype).cuda()  # noqa: E731
    return dict(h=matrix(g, rows, cols, dtype, pad, scale), o=matrix(g, rows, cols, dtype, pad, scale),
                w_post=vec() if post else None, w_pre=vec(),
                gate=matrix(g, (rows + per - 1) // per, cols, dtype, pad) if per else None)


def assert_close(got, want, tol, what):
    got = wide(got)
    assert got.shape == want.shape, what
    bad = np.argwhere(~(np.abs(got - want) <= tol))
    assert len(bad) == 0, "%s: %d of %d off, first %s got %r want %r tol %r" % (
        what, len(bad), got.size, bad[0].tolist(), got[tuple(bad[0])], want[tuple(bad[0])],
        np.broadcast_to(tol, want.shape)[tuple(bad[0])])


CASES = [(1, 1), (1, 8), (1, 4096), (5, 7), (3, 2048), (130, 1003), (300, 128), (17, 2056), (9, 5120), (6, 8200),
         (700, 264), (3, 16384), (2, 16377)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", CASES)
@pytest.mark.parametrize("post,per", [(True, 0), (True, 3), (False, 0), (False, 1), (True, 1000)])
def test_forward_and_backward(fp4, dtype, shape, post, per):
    rows, cols = shape
    alpha, eps = 0.75, 1e-5
    t = inputs(rows, cols, dtype, post, per, pad=16, seed=rows + cols)
    f = fp4.norm_residual(t["h"], w_pre=t["w_pre"], o=t["o"], w_post=t["w_post"], gate=t["gate"],
                          rows_per_group=per or None, alpha=alpha, eps=eps)
    w = {k: wide(v) for k, v in t.items()}
    ref = oracle.norm_residual(w["h"], w["o"], w["w_post"], w["gate"], per, alpha, None, eps)
    size = np.abs(w["h"]) + np.abs(ref["h"] - w["h"])
    half = half_step(dtype)
    assert_close(f["h"], ref["h"], 40 * U * size + half * np.abs(ref["h"]) * (1 + 40 * U), "h'")
    if post:
        assert_close(f["rstd_post"], ref["rstd_post"], 32 * U * ref["rstd_post"], "rstd_post")
    kept = wide(f["h"])                                  # the norm takes the stored stream
    ref2 = oracle.norm_residual(kept, w_pre=w["w_pre"], eps=eps)
    assert_close(f["rstd_pre"], ref2["rstd_pre"], 32 * U * ref2["rstd_pre"], "rstd_pre")
    assert_close(f["y"], ref2["y"], (40 * U + half) * np.abs(ref2["y"]), "y")

    g = torch.Generator().manual_seed(cols)
    dy, dh_in = (matrix(g, rows, cols, dtype, 16) for _ in range(2))
    b = fp4.norm_residual_backward(dy, f["h"], f["rstd_pre"], w_pre=t["w_pre"], dh_in=dh_in, o=t["o"],
                                   w_post=t["w_post"], rstd_post=f["rstd_post"], gate=t["gate"],
                                   rows_per_group=per or None, alpha=alpha)
    r = oracle.norm_residual_backward(wide(dy), kept, wide(f["rstd_pre"]), w["w_pre"], wide(dh_in), w["o"],
                                      w["w_post"], wide(f["rstd_post"]), w["gate"], per, alpha)
    for name, count in (("dh", 70), ("do", 140), ("dw_pre", 80), ("dw_post", 220), ("dgate", 220)):
        if r[name] is None:
            assert b[name] is None
            continue
        tol = count * U * r["size"][name] + (half * np.abs(r[name]) if name in ("dh", "do") else 0.0)
        assert_close(b[name], r[name], tol, name)
    assert fp4.fp4_last_error() == fp4.FP4_OK


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", [(4, 640), (2, 1000)])
def test_parts_of_the_operator(fp4, dtype, shape):
    """Each half alone: a norm without an update, an update without a norm, and their gradients."""
    rows, cols = shape
    t = inputs(rows, cols, dtype, True, 0, 0, 3)
    w = {k: wide(v) for k, v in t.items()}
    half = half_step(dtype)
    f = fp4.norm_residual(t["h"], w_pre=t["w_pre"])
    assert f["h"] is t["h"] and f["rstd_post"] is None
    ref = oracle.norm_residual(w["h"], w_pre=w["w_pre"])
    assert_close(f["y"], ref["y"], (40 * U + half) * np.abs(ref["y"]), "y")
    f2 = fp4.norm_residual(t["h"], o=t["o"], alpha=-2.0)
    ref2 = oracle.norm_residual(w["h"], w["o"], alpha=-2.0)
    assert "y" not in f2 and f2["rstd_pre"] is None
    assert_close(f2["h"], ref2["h"], 2 * U * (np.abs(w["h"]) + 2 * np.abs(w["o"])) + half * np.abs(ref2["h"]), "h'")
    b = fp4.norm_residual_backward(t["o"], t["h"], f["rstd_pre"], w_pre=t["w_pre"])
    r = oracle.norm_residual_backward(w["o"], w["h"], wide(f["rstd_pre"]), w["w_pre"], None, None, None, None, None, 0, 1)
    assert b["do"] is None and b["dgate"] is None
    assert_close(b["dh"], r["dh"], 70 * U * r["size"]["dh"] + half * np.abs(r["dh"]), "dh")
    assert_close(b["dw_pre"], r["dw_pre"], 80 * U * r["size"]["dw_pre"], "dw_pre")
    b = fp4.norm_residual_backward(None, None, dh_in=t["h"], o=t["o"], alpha=-2.0)
    assert torch.equal(b["dh"], t["h"]) and torch.equal(b["do"], (-2.0 * t["h"].float()).to(dtype))


def test_norm_into_the_fp8_operand(fp4):
    """Codes of the binary32 y: within one E4M3 step, and exact off the borders; y and codes may be asked for together."""
    rows, cols = 37, 1000
    t = inputs(rows, cols, torch.bfloat16, True, 5, 0, 9)
    out = dict(y=torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda"))
    f = fp4.norm_residual(t["h"], w_pre=t["w_pre"], o=t["o"], w_post=t["w_post"], gate=t["gate"], rows_per_group=5,
                          quantize=True, out=out)
    y = oracle.norm_residual(wide(f["h"]), w_pre=wide(t["w_pre"]))["y"]
    assert_close(f["y"], y, (40 * U + 2.0 ** -8) * np.abs(y), "y")
    o = oracle.fp8_block_quantize(y.astype(np.float32))
    s = f["q"]["scales"].cpu().numpy()[:, :rows].T
    assert (np.abs(s - o["scales"]) <= 42 * U * o["scales"]).all()
    codes = f["q"]["codes"].cpu().numpy()[:, :cols]
    # y is off by 40 u, its scale by 42 u, the reciprocal and the product by one
    # each, so a code may differ only by one step and only where the exact
    # quotient lies within 84 u of the middle between the two codes (ties are
    # common: rstd cancels in y / max y, and bf16 factors make short quotients)
    differ = codes != o["codes"]
    value = lambda c: oracle.fp8_dequantize(dict(codes=c.reshape(1, -1), scale=1.0))[0]  # noqa: E731
    got, want = codes[differ], o["codes"][differ]
    assert (np.abs(got.astype(int) - want.astype(int)) <= 1).all()
    top = np.stack([np.abs(y[:, k:k + 128]).max(axis=1) for k in range(0, cols, 128)], axis=1)
    quotient = (y / (np.repeat(top, 128, axis=1)[:, :cols] / 448))[differ]
    middle = (value(got) + value(want)) / 2
    assert (np.abs(quotient - middle) <= 84 * U * np.abs(quotient)).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tiny", [2.0 ** -98, 2.0 ** -120, 2.0 ** -124])
def test_blocks_of_tiny_values_in_the_fp8_operand(fp4, dtype, tiny):
    """A block far below its row's RMS: y is a normal number, 448 over the block's
    largest h' w is none.  A code is off by half a step, 2^-4 of it or 2^-10 of
    the scale below the smallest normal one, and by the roundings of y and s."""
    g = torch.Generator().manual_seed(9)
    h = torch.randn((40, 512), generator=g) * 2.0 ** -14
    h[:, 128:256] = torch.randn((40, 128), generator=g).clamp(0.25, 4) * tiny
    h = h.to(dtype).cuda()
    w = torch.ones(512, dtype=dtype, device="cuda")
    q = fp4.norm_residual(h, w_pre=w, eps=0.0, quantize=True)["q"]
    want = oracle.norm_residual(wide(h), w_pre=wide(w), eps=0.0)["y"]
    scales = np.repeat(wide(q["scales"][:, :40].t()), 128, 1)
    got = q["codes"].view(torch.float8_e4m3fn).double().cpu().numpy() * scales
    assert_close(torch.from_numpy(got), want, 2.0 ** -4 * np.abs(want) * (1 + 2.0 ** -18) + 2.0 ** -10 * scales, "y")


@pytest.mark.parametrize("rows,cols", [(3, 256), (1, 130)])
def test_zero_rows_and_eps_zero(fp4, rows, cols):
    h = torch.zeros((rows, (cols + 7) // 8 * 8), device="cuda")[:, :cols]
    w = torch.ones(cols, device="cuda")
    f = fp4.norm_residual(h, w_pre=w, eps=1e-6, quantize=True)
    assert (f["q"]["codes"][:, :cols] == 0).all() and (f["q"]["scales"][:, :rows] == 1).all()
    f = fp4.norm_residual(torch.ones_like(h), w_pre=w, eps=0.0)
    assert torch.equal(f["y"], torch.ones_like(h))


def test_in_place_stream_and_gradient(fp4):
    t = inputs(50, 520, torch.bfloat16, True, 0, 0, 12)
    kw = dict(w_pre=t["w_pre"], o=t["o"], w_post=t["w_post"])
    want = fp4.norm_residual(t["h"], **kw)
    h = t["h"].clone()
    got = fp4.norm_residual(h, out=dict(h=h), **kw)
    assert got["h"] is h and torch.equal(h, want["h"]) and torch.equal(got["y"], want["y"])
    dy, dh_in = torch.randn_like(t["h"]), torch.randn_like(t["h"])
    bw = dict(w_pre=t["w_pre"], o=t["o"], w_post=t["w_post"], rstd_post=want["rstd_post"])
    ref = fp4.norm_residual_backward(dy, want["h"], want["rstd_pre"], dh_in=dh_in, **bw)
    got = fp4.norm_residual_backward(dy, want["h"], want["rstd_pre"], dh_in=dh_in, out=dict(dh=dh_in), **bw)
    for k in ("dh", "do", "dw_pre", "dw_post"):
        assert torch.equal(got[k], ref[k]), k


def test_nothing_is_written_past_rows_and_columns(fp4):
    rows, cols = 11, 130
    t = inputs(rows, cols, torch.bfloat16, True, 4, 0, 13)
    room = lambda dt: torch.full((rows + 2, cols + 22), 5.0, dtype=dt, device="cuda")  # noqa: E731
    bufs = {k: room(torch.bfloat16) for k in ("h", "y", "dh", "do")}
    view = {k: b[1:rows + 1, :cols] for k, b in bufs.items()}
    # rows 1.. of a pitch of 152 elements start 304 bytes in: 16-byte aligned
    f = fp4.norm_residual(t["h"], w_pre=t["w_pre"], o=t["o"], w_post=t["w_post"], gate=t["gate"], rows_per_group=4,
                          out=dict(h=view["h"], y=view["y"]))
    flat = torch.full((3 * cols + 10,), 5.0, device="cuda")
    fp4.norm_residual_backward(t["h"], f["h"], f["rstd_pre"], w_pre=t["w_pre"], o=t["o"], w_post=t["w_post"],
                               rstd_post=f["rstd_post"], gate=t["gate"], rows_per_group=4,
                               out=dict(dh=view["dh"], do=view["do"], dgate=flat[:3 * cols].view(3, cols)))
    torch.cuda.synchronize()
    for k, b in bufs.items():
        assert (b[0] == 5).all() and (b[-1] == 5).all() and (b[:, cols:] == 5).all(), k
    assert (flat[3 * cols:] == 5).all()


def test_empty_batch(fp4):
    h = torch.zeros((0, 256), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    f = fp4.norm_residual(h, w_pre=w, o=h, w_post=w)
    assert f["y"].shape == (0, 256)
    dw = torch.full((256,), 3.0, device="cuda")
    b = fp4.norm_residual_backward(h, h, f["rstd_pre"], w_pre=w, o=h, w_post=w, rstd_post=f["rstd_post"],
                                   out=dict(dw_pre=dw))
    assert (dw == 0).all() and (b["dw_post"] == 0).all()


def test_gradients_do_not_depend_on_timing(fp4):
    t = inputs(4000, 1000, torch.bfloat16, True, 700, 0, 15)
    f = fp4.norm_residual(t["h"], w_pre=t["w_pre"], o=t["o"], w_post=t["w_post"], gate=t["gate"], rows_per_group=700)
    run = lambda: fp4.norm_residual_backward(t["o"], f["h"], f["rstd_pre"], w_pre=t["w_pre"], o=t["o"],  # noqa: E731
                                             w_post=t["w_post"], rstd_post=f["rstd_post"], gate=t["gate"],
                                             rows_per_group=700)
    first = run()
    for _ in range(3):
        again = run()
        assert all(torch.equal(first[k], again[k]) for k in first)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(5, 1), (40, 131), (33, 1003), (20, 2035), (9, 5501), (7, 8501)])
def test_what_lies_behind_a_row_is_not_seen(fp4, rows, cols, dtype):
    """NaN up to the row's pitch, and no bytes at all behind the last row."""
    def holed(t, fill):
        ld = (cols + 7) // 8 * 8 + 8
        flat = torch.full(((t.shape[0] - 1) * ld + cols,), fill, dtype=dtype, device="cuda")
        v = flat.as_strided(t.shape, (ld, 1))
        v.copy_(t)
        return v
    a = inputs(rows, cols, dtype, True, 4, 0, 31)
    g = torch.Generator().manual_seed(32)
    dy, dh_in = matrix(g, rows, cols, dtype), matrix(g, rows, cols, dtype)
    got = []
    for fill in (0.0, float("nan")):
        b = {k: holed(v, fill) if v.dim() == 2 else v for k, v in a.items()}
        f = fp4.norm_residual(alpha=0.5, rows_per_group=4, quantize=True, out=dict(y=holed(dy, fill)), **b)
        r = fp4.norm_residual_backward(holed(dy, fill), holed(f["h"], fill), f["rstd_pre"], w_pre=b["w_pre"],
                                       dh_in=holed(dh_in, fill), o=b["o"], w_post=b["w_post"],
                                       rstd_post=f["rstd_post"], gate=b["gate"], rows_per_group=4, alpha=0.5)
        got.append(dict(h=f["h"], y=f["y"], codes=f["q"]["codes"][:, :cols], scales=f["q"]["scales"][:, :rows], **r))
    for k, v in got[0].items():
        assert torch.isfinite(v.float()).all() and torch.equal(v, got[1][k]), k


def test_own_workspace_on_another_stream(fp4, monkeypatch):
    """The workspace that the helper allocates is not handed out again before the
    call has run on its stream."""
    a = inputs(600, 1024, torch.bfloat16, True, 200, 0, 77)
    f = fp4.norm_residual(alpha=0.5, rows_per_group=200, **a)
    dy = matrix(torch.Generator().manual_seed(78), 600, 1024, torch.bfloat16)
    kw = dict(rstd_pre=f["rstd_pre"], w_pre=a["w_pre"], o=a["o"], w_post=a["w_post"], rstd_post=f["rstd_post"],
              gate=a["gate"], rows_per_group=200, alpha=0.5)
    want = fp4.norm_residual_backward(dy, f["h"], **kw)
    size = fp4.fp4_norm_residual_backward_workspace_size(600, 1024, True, True, True, 200)
    used, call = [], fp4._lib.fp4_norm_residual_backward

    def spy(*args):
        used.append(args[-3])
        return call(*args)
    monkeypatch.setattr(fp4._lib, "fp4_norm_residual_backward", spy)
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        out = {k: torch.empty_like(v) for k, v in want.items()}
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(50_000_000)            # tens of milliseconds
        got = fp4.norm_residual_backward(dy, f["h"], out=out, stream=stream, **kw)
        others = [torch.full((size,), 0x7f, dtype=torch.uint8, device="cuda") for _ in range(8)]
        assert not side.query()                      # all of them were handed out before the call ran
        assert used[-1] not in [t.data_ptr() for t in others]
        torch.cuda.synchronize()
        for k in want:
            assert torch.equal(got[k], want[k]), k


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("eh,ew", [(50, 80), (-40, -90), (-70, -70)])
def test_stream_and_weight_far_from_one(fp4, dtype, eh, ew):
    """h' w passes binary32 at one end, while y does not."""
    rows, cols = 21, 1000
    g = torch.Generator().manual_seed(eh - ew)
    h = (torch.randn((rows, cols), generator=g) * 2.0 ** eh).to(dtype).cuda()
    w = ((1 + 0.2 * torch.randn(cols, generator=g)) * 2.0 ** ew).to(dtype).cuda()
    f = fp4.norm_residual(h, w_pre=w, eps=0.0, quantize=True, out=dict(y=torch.empty_like(h)))
    want = oracle.norm_residual(wide(h), w_pre=wide(w), eps=0.0)["y"]
    half = half_step(dtype)
    assert_close(f["y"], want, (40 * U + half) * np.abs(want), "y")
    scales = np.repeat(wide(f["q"]["scales"][:, :rows].t()), 128, 1)[:, :cols]
    got = f["q"]["codes"][:, :cols].view(torch.float8_e4m3fn).double().cpu().numpy() * scales
    assert_close(torch.from_numpy(got), want, 2.0 ** -4 * np.abs(want) * (1 + 2.0 ** -18) + 2.0 ** -10 * scales, "codes")


# Many rows per CTA, and more groups than CTAs.  A CTA sums at most 14 rows here, a
# column at most 2368 CTAs' partial sums, every 32nd of them (74) and then 32 such:
# with the product's 6 roundings 126, under 140 u for dw_pre and, with the 140 of
# the terms themselves, 280 u for dw_post and dgate.
LOOPS = [(3000, 2056, 0), (3000, 2056, 1), (3000, 2056, 7), (3000, 2056, 2000), (900, 4104, 1), (900, 4104, 3),
         (700, 8200, 1), (700, 8200, 3), (5000, 130, 0), (5000, 130, 1), (5000, 130, 7), (1500, 4096, 700)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols,per", LOOPS)
def test_many_rows_and_groups_per_cta(fp4, dtype, rows, cols, per):
    alpha, eps = 0.75, 1e-5
    t = inputs(rows, cols, dtype, True, per, pad=16, seed=rows + cols + per)
    f = fp4.norm_residual(t["h"], w_pre=t["w_pre"], o=t["o"], w_post=t["w_post"], gate=t["gate"],
                          rows_per_group=per or None, alpha=alpha, eps=eps)
    w = {k: wide(v) for k, v in t.items()}
    ref = oracle.norm_residual(w["h"], w["o"], w["w_post"], w["gate"], per, alpha, None, eps)
    size = np.abs(w["h"]) + np.abs(ref["h"] - w["h"])
    half = half_step(dtype)
    assert_close(f["h"], ref["h"], 40 * U * size + half * np.abs(ref["h"]) * (1 + 40 * U), "h'")
    kept = wide(f["h"])
    ref2 = oracle.norm_residual(kept, w_pre=w["w_pre"], eps=eps)
    assert_close(f["y"], ref2["y"], (40 * U + half) * np.abs(ref2["y"]), "y")
    g = torch.Generator().manual_seed(cols)
    dy, dh_in = (matrix(g, rows, cols, dtype, 16) for _ in range(2))
    want_in = wide(dh_in)
    # in place: dh takes dh_in's memory
    b = fp4.norm_residual_backward(dy, f["h"], f["rstd_pre"], w_pre=t["w_pre"], dh_in=dh_in, o=t["o"],
                                   w_post=t["w_post"], rstd_post=f["rstd_post"], gate=t["gate"],
                                   rows_per_group=per or None, alpha=alpha, out=dict(dh=dh_in))
    r = oracle.norm_residual_backward(wide(dy), kept, wide(f["rstd_pre"]), w["w_pre"], want_in, w["o"],
                                      w["w_post"], wide(f["rstd_post"]), w["gate"], per, alpha)
    for name, count in (("dh", 70), ("do", 140), ("dw_pre", 140), ("dw_post", 280), ("dgate", 280)):
        if r[name] is None:
            assert b[name] is None
            continue
        tol = count * U * r["size"][name] + (half * np.abs(r[name]) if name in ("dh", "do") else 0.0)
        assert_close(b[name], r[name], tol, name)
    assert fp4.fp4_last_error() == fp4.FP4_OK


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cols", [2056, 4096, 8192, 12288])
def test_parts_of_the_operator_at_model_widths(fp4, dtype, cols):
    """Each half alone, and the update with its norm but none after it; up to 5 rows per CTA."""
    rows, per = 700, 9
    t = inputs(rows, cols, dtype, True, per, 0, cols)
    w = {k: wide(v) for k, v in t.items()}
    half = half_step(dtype)
    g = torch.Generator().manual_seed(cols + 1)
    dy, dh_in = (matrix(g, rows, cols, dtype) for _ in range(2))

    def check(b, r):
        for name, count in (("dh", 70), ("do", 140), ("dw_pre", 140), ("dw_post", 280), ("dgate", 280)):
            assert (b[name] is None) == (r[name] is None), name
            if r[name] is not None:
                tol = count * U * r["size"][name] + (half * np.abs(r[name]) if name in ("dh", "do") else 0.0)
                assert_close(b[name], r[name], tol, name)

    # the norm alone, and its gradients with and without what reaches the stream besides
    f = fp4.norm_residual(t["h"], w_pre=t["w_pre"])
    ref = oracle.norm_residual(w["h"], w_pre=w["w_pre"])
    assert_close(f["y"], ref["y"], (40 * U + half) * np.abs(ref["y"]), "y")
    for extra in (None, dh_in):
        check(fp4.norm_residual_backward(dy, t["h"], f["rstd_pre"], w_pre=t["w_pre"], dh_in=extra),
              oracle.norm_residual_backward(wide(dy), w["h"], wide(f["rstd_pre"]), w["w_pre"], wide(extra), None, None,
                                            None, None, 0, 1))
    # the update alone: without its norm, with it, and with a gate
    for post, gated in ((False, False), (True, False), (False, True), (True, True)):
        kw = dict(w_post=t["w_post"] if post else None, gate=t["gate"] if gated else None,
                  rows_per_group=per if gated else None, alpha=-2.0)
        f = fp4.norm_residual(t["h"], o=t["o"], **kw)
        wp, wg = w["w_post"] if post else None, w["gate"] if gated else None
        ref = oracle.norm_residual(w["h"], w["o"], wp, wg, per, -2.0, None, 1e-6)
        size = np.abs(w["h"]) + np.abs(ref["h"] - w["h"])
        assert_close(f["h"], ref["h"], 40 * U * size + half * np.abs(ref["h"]) * (1 + 40 * U), "h'")
        check(fp4.norm_residual_backward(None, None, dh_in=dh_in, o=t["o"], rstd_post=f["rstd_post"], **kw),
              oracle.norm_residual_backward(None, None, None, None, wide(dh_in), w["o"], wp, wide(f["rstd_post"]), wg,
                                            per, -2.0))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cols", [130, 4096, 8200])
@pytest.mark.parametrize("eps", [0.0, 2.0 ** -140, 2.0 ** -100])
def test_rows_whose_squares_underflow(fp4, dtype, cols, eps):
    """Rows of normal numbers whose squares are subnormal or zero in binary32."""
    exps = np.array([-30, -45, -49, -50, -51, -60, -63, -68, -70, -75, -90, -110, -115])
    g = torch.Generator().manual_seed(cols)
    x = torch.randn((len(exps), cols), generator=g).double() * torch.from_numpy(2.0 ** exps)[:, None]
    x = torch.where(x.abs() < 2.0 ** -126, 2.0 ** -126, x).to(dtype)
    room = torch.zeros((2, len(exps), (cols + 7) // 8 * 8), dtype=dtype, device="cuda")
    h, o = room[0][:, :cols], room[1][:, :cols]
    o.copy_(x)
    w = (1 + 0.2 * torch.randn(cols, generator=g)).to(dtype).cuda()
    half = half_step(dtype)
    # before a block
    f = fp4.norm_residual(o, w_pre=w, eps=eps)
    ref = oracle.norm_residual(wide(o), w_pre=wide(w), eps=eps)
    assert_close(f["rstd_pre"], ref["rstd_pre"], 32 * U * ref["rstd_pre"], "rstd_pre")
    assert_close(f["y"], ref["y"], (40 * U + half) * np.abs(ref["y"]), "y")
    # after one, onto a stream of zeros, and before the next
    f = fp4.norm_residual(h, w_pre=w, o=o, w_post=w, eps=eps)
    ref = oracle.norm_residual(wide(h), wide(o), wide(w), eps=eps)
    assert_close(f["rstd_post"], ref["rstd_post"], 32 * U * ref["rstd_post"], "rstd_post")
    assert_close(f["h"], ref["h"], (40 * U + half * (1 + 40 * U)) * np.abs(ref["h"]), "h'")
    ref2 = oracle.norm_residual(wide(f["h"]), w_pre=wide(w), eps=eps)
    assert_close(f["rstd_pre"], ref2["rstd_pre"], 32 * U * ref2["rstd_pre"], "rstd_pre")
