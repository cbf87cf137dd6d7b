"""The FP8 operators together, as a linear between two blocks uses them:
norm -> FP8 operand -> Fprop -> norm, gate and residual, and back through the
gradients to Dgrad and Wgrad; eagerly, and captured into a CUDA graph."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fp4(cuda_device):
    from fp4_block_scaled_h16_b200 import fp4 as m
    return m


def dequantize(q):
    v = q["codes"][:, :q["K"]].view(torch.float8_e4m3fn).double()
    s = q["scales"].double().t().repeat_interleave(q["block_lines"], 0)[:q["lines"]]
    return v * s.repeat_interleave(128, 1)[:, :q["K"]]


def rel(a, b):
    return float((a.double() - b).norm() / b.norm())


def setup(rows, C, seed=0):
    g = torch.Generator().manual_seed(seed)
    draw = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    vec = lambda: (1 + 0.1 * torch.randn(C, generator=g)).to(torch.bfloat16).cuda()  # noqa: E731
    per = (rows + 1) // 2
    return dict(h=draw(rows, C), w1=vec(), w2=vec(), w3=vec(), gate=draw(2 if rows > 1 else 1, C), per=per,
                W=draw(C, C) * 0.03, dy=draw(rows, C) * 0.01, dh_in=draw(rows, C) * 0.01)


def step(fp4, t):
    """One linear between two norms, forward and backward; every tensor of the pass."""
    r = dict(fp4=None)
    f0 = fp4.norm_residual(t["h"], w_pre=t["w1"], quantize=True,
                           out=dict(y=torch.empty_like(t["h"])))         # the operand, and its input for Wgrad
    wr, wc = fp4.fp8_block_quantize_both_axes(t["W"], 128)
    o = fp4.fp8_block_gemm(f0["q"], wr, fp4.FP4_OUT_BF16)                 # Fprop
    f1 = fp4.norm_residual(t["h"], w_pre=t["w3"], o=o, w_post=t["w2"], gate=t["gate"], rows_per_group=t["per"], alpha=0.5)
    b1 = fp4.norm_residual_backward(t["dy"], f1["h"], f1["rstd_pre"], w_pre=t["w3"], dh_in=t["dh_in"], o=o,
                                    w_post=t["w2"], rstd_post=f1["rstd_post"], gate=t["gate"],
                                    rows_per_group=t["per"], alpha=0.5)
    gr, gc = fp4.fp8_block_quantize_both_axes(b1["do"])
    dx = fp4.fp8_block_gemm(gr, wc, fp4.FP4_OUT_BF16)                     # Dgrad
    dW = fp4.fp8_block_gemm(gc, fp4.fp8_block_quantize(f0["y"], 0), fp4.FP4_OUT_F32)   # Wgrad
    b0 = fp4.norm_residual_backward(dx, t["h"], f0["rstd_pre"], w_pre=t["w1"], dh_in=b1["dh"])
    r.update(q=f0["q"], y0=f0["y"], wr=wr, wc=wc, o=o, h1=f1["h"], y1=f1["y"], b1=b1, gr=gr, gc=gc, dx=dx, dW=dW, b0=b0)
    return r


@pytest.mark.parametrize("rows,C", [(1, 512), (130, 520), (700, 1024)])
def test_linear_between_norms(fp4, rows, C):
    t = setup(rows, C)
    r = step(fp4, t)
    assert fp4.fp4_last_error() == fp4.FP4_OK
    # each product against the float64 product of its own operands
    assert rel(r["o"], dequantize(r["q"]) @ dequantize(r["wr"]).t()) < 2.0 ** -8
    assert rel(r["dx"], dequantize(r["gr"]) @ dequantize(r["wc"]).t()) < 2.0 ** -8
    # the weight's two operands hold the same values
    assert torch.equal(dequantize(r["wr"]), dequantize(r["wc"]).t())
    # the whole pass against float64 autograd of the same formulas with the
    # quantized operands' values taken as given: E4M3 keeps 3 bits, so an
    # operand is within 2^-4 of its value, and the products of two within 2^-3
    h, w1, w2, w3, gate, W = (t[k].double().requires_grad_() for k in ("h", "w1", "w2", "w3", "gate", "W"))
    unit = lambda x: x / (x.pow(2).mean(1, keepdim=True) + 1e-6).sqrt()  # noqa: E731
    o = (unit(h) * w1) @ W.t()
    h1 = h + 0.5 * gate[torch.arange(rows, device="cuda") // t["per"]] * (unit(o) * w2)
    ((unit(h1) * w3 * t["dy"].double()).sum() + (h1 * t["dh_in"].double()).sum()).backward()
    bound = 2.0 ** -3
    assert rel(r["o"], o.detach()) < bound and rel(r["h1"], h1.detach()) < bound
    for got, leaf in ((r["b0"]["dh"], h), (r["b0"]["dw_pre"], w1), (r["b1"]["dw_post"], w2), (r["b1"]["dw_pre"], w3),
                      (r["b1"]["dgate"], gate), (r["dW"], W)):
        assert rel(got, leaf.grad) < bound


def flat(r):
    for k in sorted(r):
        v = r[k]
        if isinstance(v, dict):
            lines = v.get("lines")
            for kk in sorted(v):
                x = v[kk]
                if isinstance(x, torch.Tensor):
                    # padding of codes and scales is not written
                    if kk == "codes":
                        x = x[:, :v["K"]]
                    elif kk == "scales" and v["block_lines"] == 1:
                        x = x[:, :lines]
                    yield "%s.%s" % (k, kk), x
        elif isinstance(v, torch.Tensor):
            yield k, v


def test_captured_pass_replays_with_new_inputs(fp4):
    t = setup(300, 640, 1)
    step(fp4, t)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(s):
        step(fp4, t)
        torch.cuda.synchronize()
        for _ in range(2):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                held = step(fp4, t)
            graphs.append((graph, held))
    torch.cuda.current_stream().wait_stream(s)
    for scale in (1.0, -3.0):
        t["h"].mul_(scale)
        t["dy"].mul_(scale)
        want = {k: v.clone() for k, v in flat(step(fp4, t))}
        for graph, held in graphs:
            graph.replay()
            torch.cuda.synchronize()
            for k, v in flat(held):
                assert torch.equal(v.view(torch.uint8) if v.dtype == torch.uint8 else v, want[k]), k
    assert fp4.fp4_last_error() == fp4.FP4_OK


def test_serving_step_repeats_a_training_rows_result(fp4):
    """A token's result does not depend on the other tokens of its batch where the same kernel runs."""
    t = setup(16, 512, 2)
    wr = fp4.fp8_block_quantize(t["W"], 1, 128)
    whole = fp4.norm_residual(t["h"], w_pre=t["w1"], quantize=True)["q"]
    o = fp4.fp8_block_gemm(whole, wr, fp4.FP4_OUT_F32)
    for i in (0, 7, 15):
        one = fp4.norm_residual(t["h"][i:i + 1], w_pre=t["w1"], quantize=True)["q"]
        assert torch.equal(one["codes"], whole["codes"][i:i + 1])
        assert torch.equal(fp4.fp8_block_gemm(one, wr, fp4.FP4_OUT_F32), o[i:i + 1])


def tensors(r):
    """Every tensor of a helper's result."""
    if isinstance(r, torch.Tensor):
        return [r]
    return [t for v in (r.values() if isinstance(r, dict) else r) if isinstance(v, (torch.Tensor, dict)) for t in tensors(v)]


def calls(fp4):
    """Helpers that allocate, each as (name, call with a stream)."""
    g = torch.Generator().manual_seed(5)
    x = torch.randn((256, 512), generator=g).to(torch.bfloat16).cuda()
    w = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    qa, qb = fp4.fp8_block_quantize(x), fp4.fp8_block_quantize(x, 1, 128)
    n4, b4 = (fp4.quantize(x, fp4.FP4_NVFP4) for _ in range(2))
    f = fp4.norm_residual(x, w_pre=w, o=x, w_post=w)
    return [
        ("quantize", lambda s: fp4.fp8_block_quantize(x, stream=s)),
        ("quantize both", lambda s: fp4.fp8_block_quantize_both_axes(x, stream=s)),
        ("gemm", lambda s: fp4.fp8_block_gemm(qa, qb, stream=s)),
        ("norm", lambda s: fp4.norm_residual(x, w_pre=w, o=x, w_post=w, stream=s)),
        ("norm fp8", lambda s: fp4.norm_residual(x, w_pre=w, quantize=True, stream=s)),
        ("backward", lambda s: fp4.norm_residual_backward(x, f["h"], f["rstd_pre"], w_pre=w, o=x, w_post=w,
                                                          rstd_post=f["rstd_post"], stream=s)),
        ("fp4 quantize", lambda s: fp4.quantize(x, fp4.FP4_NVFP4, rotation=fp4.FP4_ROT_H16, stream=s)),
        ("fp4 gemm", lambda s: fp4.gemm(n4, b4, stream=s)),
        ("rotate", lambda s: fp4.rotate(x, fp4.FP4_ROT_H16, stream=s)),
    ]


def test_memory_of_another_stream_is_left_alone(fp4):
    """What a call on a side stream allocates is not memory that the current stream
    has freed but not finished with, and it is not handed out on the current stream
    while the side stream has yet to use it."""
    side = torch.cuda.Stream()
    for name, call in calls(fp4):
        want = [v.clone() for v in tensors(call(None))]
        for stream in (side, side.cuda_stream):
            torch.cuda.synchronize()
            sizes = [v.untyped_storage().nbytes() for v in want]
            old = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
            torch.cuda._sleep(50_000_000)                # tens of milliseconds
            for t in old:
                t.fill_(0x7f)                            # still to come when the memory goes back
            taken = [(t.untyped_storage().data_ptr(), t.numel()) for t in old]
            del old, t
            got = call(stream)
            assert not torch.cuda.current_stream().query()
            mine = [(v.untyped_storage().data_ptr(), v.untyped_storage().nbytes()) for v in tensors(got)]
            assert mine
            assert not [1 for a, n in mine for b, m in taken if a < b + m and b < a + n], name
            torch.cuda.synchronize()
            for v, w in zip(tensors(got), want):
                assert torch.equal(v, w), name


def test_stream_of_another_device_is_refused(fp4, monkeypatch):
    side = torch.cuda.Stream()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 7)
    with pytest.raises(ValueError, match="stream"):
        fp4.fp8_block_quantize(torch.zeros((1, 128)), stream=side)
