"""The 8-bit linear layer's operators, as cases to time and to compare.

Four operators are run here, each in its plain form (elementary torch
operations in 32 bits) or, with ``own`` set, through the library's calls:

  quantize   E4M3 codes with one FP32 scale per block of 128 along K, of one
             line or of 128 lines; along the rows, the columns, or both
  gemm       C = A B^T of two such tensors (Fprop / Dgrad: B in 128 x 128
             blocks; Wgrad: both operands in 1 x 128 blocks)
  norm       h' = h + alpha * gate * (o normalised), y = h' normalised, with y
             in the stream's type or as the FP8 operand of the product
  norm_bwd   the gradients of `norm`

Layouts (the library's): codes uint8 [lines, pitch >= K, a multiple of 16];
scales float [ceil(K / 128), lines rounded up to 128] for 1 x 128 blocks,
[ceil(K / 128), ceil(lines / 128)] for 128 x 128 blocks.
"""
import math

import torch

own = False

BLOCK = 128
EPS = 1e-6


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one decoded token's activation, the operand of a serving step's linear
        dict(name="quantize_token", op="quantize", rows=1, cols=4096, type="bf16", axes="rows", lines=1, pad=0),
        # activations of a training step: rows for Fprop, columns for Wgrad
        dict(name="quantize_x_both", op="quantize", rows=8192, cols=4096, type="bf16", axes="both", lines=1, pad=0),
        # a float32 master weight: rows for Fprop, columns for Dgrad
        dict(name="quantize_w_both", op="quantize", rows=4096, cols=14336, type="f32", axes="both", lines=128, pad=0),
        # the QKV projection of one token
        dict(name="gemm_decode", op="gemm", M=1, N=6144, K=4096, b_lines=128, out="bf16"),
        # the down projection of a short ragged batch
        dict(name="gemm_ragged", op="gemm", M=333, N=4096, K=14336, b_lines=128, out="bf16"),
        # the QKV projection of a training step
        dict(name="gemm_fprop", op="gemm", M=8192, N=6144, K=4096, b_lines=128, out="bf16"),
        # the weight gradient of the down projection, in float32
        dict(name="gemm_wgrad", op="gemm", M=4096, N=14336, K=8192, b_lines=1, out="f32"),
        # one decoded token between two blocks, straight into the FP8 operand
        dict(name="norm_token", op="norm", rows=1, cols=4096, type="bf16", post=True, gate_rows=0, pre=True, fp8=True, pad=0),
        # a training step's stream between two blocks, a gate per sequence
        dict(name="norm_block", op="norm", rows=8192, cols=4096, type="bf16", post=True, gate_rows=2048, pre=True, fp8=False, pad=0),
        # add and normalise into the FP8 operand
        dict(name="norm_fp8", op="norm", rows=8192, cols=4096, type="bf16", post=False, gate_rows=0, pre=True, fp8=True, pad=0),
        # the gradients of a training step's stream, a gate per sequence
        dict(name="norm_bwd", op="norm_bwd", rows=8192, cols=4096, type="bf16", post=True, gate_rows=2048, pre=True, pad=0),
        # odd sizes in float32, groups that end inside the batch
        dict(name="norm_bwd_odd", op="norm_bwd", rows=1031, cols=1003, type="f32", post=True, gate_rows=100, pre=True, pad=8),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "gemm", "norm", "norm_bwd"])
    if op == "gemm":
        wgrad = rng.random() < 0.35
        M = _log(rng, 16, 4096) if wgrad else _log(rng, 1, 8192)
        N, K = _log(rng, 64, 14336), _log(rng, 64, 8192)
        while M * N * K > 4096 * 14336 * 8192:
            M = (M + 1) // 2
        return dict(op=op, M=M, N=N, K=K, b_lines=1 if wgrad else BLOCK, out=rng.choice(["bf16", "f32"]))
    rows, cols = _log(rng, 1, 8192), _log(rng, 64, 14336)
    while rows * cols > 4096 * 14336:
        rows = (rows + 1) // 2
    kind = rng.choice(["bf16", "bf16", "f32"])
    pad = rng.choice([0, 0, 8, 64])
    if op == "quantize":
        return dict(op=op, rows=rows, cols=cols, type=kind, axes=rng.choice(["rows", "cols", "both"]),
                    lines=rng.choice([1, 1, BLOCK]), pad=pad)
    case = dict(op=op, rows=rows, cols=cols, type=kind, post=rng.random() < 0.6,
                gate_rows=rng.choice([0, 1, _log(rng, 2, 2048)]), pre=True, pad=pad)
    if op == "norm":
        case["fp8"] = rng.random() < 0.4
    return case


# ------------------------------------------------------------------ inputs

def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _up(n, m):
    return (n + m - 1) // m * m


def _matrix(g, rows, cols, kind, pad, scale=1.0):
    """[rows, cols] of N(0, scale) with a few large columns, row pitch a multiple of 16 bytes."""
    ld = _up(cols, 8) + pad
    x = torch.randn((rows, ld), generator=g, device="cuda") * scale
    loud = torch.randint(0, cols, (max(1, cols // 512),), generator=g, device="cuda")
    x[:, loud] *= 16.0
    return x.to(_dtype(kind))[:, :cols]


def _vector(g, cols, kind):
    return (1.0 + 0.1 * torch.randn(cols, generator=g, device="cuda")).to(_dtype(kind))


def _qbuffers(lines, K, block_lines):
    n = _up(lines, BLOCK) if block_lines == 1 else (lines + BLOCK - 1) // BLOCK
    return dict(codes=torch.zeros((lines, _up(K, 16)), dtype=torch.uint8, device="cuda"),
                scales=torch.zeros(((K + BLOCK - 1) // BLOCK, n), dtype=torch.float32, device="cuda"),
                lines=lines, K=K, block_lines=block_lines)


def _qtensor(x, block_lines):
    codes, scales = _plain_quantize(x.float(), block_lines)
    q = _qbuffers(x.shape[0], x.shape[1], block_lines)
    q["codes"][:, :x.shape[1]] = codes.view(torch.uint8)
    q["scales"][:, :scales.shape[1]] = scales
    return q


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case=case)
    if case["op"] == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        a = _matrix(g, M, K, "f32", 0)
        b = _matrix(g, N, K, "f32", 0, 0.02)
        s["a"], s["b"] = _qtensor(a, 1), _qtensor(b, case["b_lines"])
        s["out"] = torch.empty((M, _up(N, 8)), dtype=_dtype(case["out"]), device="cuda")[:, :N]
        return s
    rows, cols, kind, pad = case["rows"], case["cols"], case["type"], case["pad"]
    if case["op"] == "quantize":
        s["x"] = _matrix(g, rows, cols, kind, pad, 0.02 if case["lines"] > 1 else 1.0)
        s["rows"] = _qbuffers(rows, cols, case["lines"]) if case["axes"] != "cols" else None
        s["cols"] = _qbuffers(cols, rows, case["lines"]) if case["axes"] != "rows" else None
        return s
    s["h"] = _matrix(g, rows, cols, kind, pad)
    s["o"] = _matrix(g, rows, cols, kind, pad)
    s["alpha"] = 0.5
    s["w_post"] = _vector(g, cols, kind) if case["post"] else None
    s["w_pre"] = _vector(g, cols, kind) if case["pre"] else None
    per = case["gate_rows"]
    s["gate"] = _matrix(g, (rows + per - 1) // per, cols, kind, pad, 0.5) if per else None
    blank = lambda: torch.empty((rows, _up(cols, 8) + pad), dtype=_dtype(kind), device="cuda")[:, :cols]  # noqa: E731
    word = lambda *n: torch.empty(n, dtype=torch.float32, device="cuda")  # noqa: E731
    if case["op"] == "norm":
        s["into"] = dict(h=blank(), rstd_pre=word(rows), rstd_post=word(rows) if case["post"] else None)
        s["into"]["q" if case["fp8"] else "y"] = _qbuffers(rows, cols, 1) if case["fp8"] else blank()
        return s
    f = _plain_norm(s)
    s["h_out"] = _matrix(g, rows, cols, kind, pad)
    s["h_out"].copy_(f["h"])
    s["rstd_pre"], s["rstd_post"] = f["rstd_pre"], f["rstd_post"]
    s["dy"] = _matrix(g, rows, cols, kind, pad, 1e-3)
    s["dh_in"] = _matrix(g, rows, cols, kind, pad, 1e-3)
    s["into"] = dict(dh=blank(), do=blank(), dw_pre=word(cols),
                     dw_post=word(cols) if case["post"] else None,
                     dgate=word(*s["gate"].shape) if per else None)
    return s


# -------------------------------------------------------------- plain forms

def _plain_quantize(x, block_lines):
    """(codes float8 [L, K], scales [ceil(K / 128), L or ceil(L / 128)]) of a float32 [L, K]."""
    L, K = x.shape
    nk, nl = (K + BLOCK - 1) // BLOCK, (L + block_lines - 1) // block_lines
    p = x.new_zeros((nl * block_lines, nk * BLOCK))
    p[:L, :K] = x
    p = p.view(nl, block_lines, nk, BLOCK)
    s = p.abs().amax(dim=(1, 3)) / 448.0
    s = torch.where(s >= torch.finfo(torch.float32).tiny, s, torch.ones_like(s))
    v = (p * (1.0 / s)[:, None, :, None]).clamp(-448.0, 448.0)
    codes = v.to(torch.float8_e4m3fn).view(nl * block_lines, nk * BLOCK)[:L, :K]
    return codes, s.t().contiguous()


def _plain_dequantize(q):
    v = q["codes"][:, :q["K"]].view(torch.float8_e4m3fn).float()
    s = q["scales"].t().repeat_interleave(q["block_lines"], 0)[:q["lines"]]
    return v * s.repeat_interleave(BLOCK, 1)[:, :q["K"]]


def _spread(gate, per, rows):
    return gate.float().repeat_interleave(per, 0)[:rows]


def _plain_norm(s):
    """h, y, rstd_post and rstd_pre of one pass; y in float32, before any rounding."""
    case, h = s["case"], s["h"].float()
    r, rstd_post = s["o"].float(), None
    if s["w_post"] is not None:
        rstd_post = torch.rsqrt(r.square().mean(1) + EPS)
        r = r * rstd_post[:, None] * s["w_post"].float()
    if s["gate"] is not None:
        r = r * _spread(s["gate"], case["gate_rows"], h.shape[0])
    h = (h + s["alpha"] * r).to(s["h"].dtype)
    rstd_pre = torch.rsqrt(h.float().square().mean(1) + EPS)
    return dict(h=h, y=h.float() * rstd_pre[:, None] * s["w_pre"].float(), rstd_pre=rstd_pre, rstd_post=rstd_post)


def _plain_norm_bwd(s):
    case, kind = s["case"], s["dy"].dtype
    dy, h, o, alpha = s["dy"].float(), s["h_out"].float(), s["o"].float(), s["alpha"]
    n2 = h * s["rstd_pre"][:, None]
    dn = dy * s["w_pre"].float()
    dh = s["dh_in"].float() + s["rstd_pre"][:, None] * (dn - n2 * (dn * n2).mean(1, keepdim=True))
    out = dict(dh=dh.to(kind), dw_pre=(dy * n2).sum(0), dw_post=None, dgate=None)
    dr = alpha * dh
    n1, r = None, o
    if s["w_post"] is not None:
        n1 = o * s["rstd_post"][:, None]
        r = n1 * s["w_post"].float()
    if s["gate"] is not None:
        per, rows = case["gate_rows"], dh.shape[0]
        t = dr.new_zeros((_up(rows, per), dh.shape[1]))
        t[:rows] = dr * r
        out["dgate"] = t.view(-1, per, dh.shape[1]).sum(1)
        dr = dr * _spread(s["gate"], per, rows)
    if n1 is not None:
        out["dw_post"] = (dr * n1).sum(0)
        dn = dr * s["w_post"].float()
        dr = s["rstd_post"][:, None] * (dn - n1 * (dn * n1).mean(1, keepdim=True))
    out["do"] = dr.to(kind)
    return out


# --------------------------------------------------------------------- run

def _values(q):
    n = q["lines"] if q["block_lines"] == 1 else q["scales"].shape[1]
    return dict(codes=q["codes"][:, :q["K"]].view(torch.float8_e4m3fn), scales=q["scales"][:, :n])


def _run_own(s):
    from fp4_block_scaled_h16_b200 import fp4
    case = s["case"]
    if case["op"] == "quantize":
        if case["axes"] == "both":
            r, c = fp4.fp8_block_quantize_both_axes(s["x"], case["lines"], out_rows=s["rows"], out_cols=s["cols"])
            return dict(rows=_values(r), cols=_values(c))
        axis = 1 if case["axes"] == "rows" else 0
        return {case["axes"]: _values(fp4.fp8_block_quantize(s["x"], axis, case["lines"], out=s[case["axes"]]))}
    if case["op"] == "gemm":
        return fp4.fp8_block_gemm(s["a"], s["b"], fp4.FP4_OUT_BF16 if case["out"] == "bf16" else fp4.FP4_OUT_F32,
                                  out=s["out"])
    if case["op"] == "norm":
        f = fp4.norm_residual(s["h"], w_pre=s["w_pre"], o=s["o"], w_post=s["w_post"], gate=s["gate"],
                              rows_per_group=case["gate_rows"] or None, alpha=s["alpha"], eps=EPS,
                              quantize=case["fp8"], out=s["into"])
        got = dict(h=f["h"], rstd_pre=f["rstd_pre"], rstd_post=f["rstd_post"])
        got["y"] = _values(f["q"]) if case["fp8"] else f["y"]
        return got
    return fp4.norm_residual_backward(s["dy"], s["h_out"], s["rstd_pre"], w_pre=s["w_pre"], dh_in=s["dh_in"], o=s["o"],
                                      w_post=s["w_post"], rstd_post=s["rstd_post"], gate=s["gate"],
                                      rows_per_group=case["gate_rows"] or None, alpha=s["alpha"], out=s["into"])


def run(state):
    if own:
        return _run_own(state)
    s, case = state, state["case"]
    if case["op"] == "quantize":
        got = {}
        if case["axes"] != "cols":
            got["rows"] = dict(zip(("codes", "scales"), _plain_quantize(s["x"].float(), case["lines"])))
        if case["axes"] != "rows":
            got["cols"] = dict(zip(("codes", "scales"), _plain_quantize(s["x"].float().t(), case["lines"])))
        return got
    if case["op"] == "gemm":
        return (_plain_dequantize(s["a"]) @ _plain_dequantize(s["b"]).t()).to(_dtype(case["out"]))
    if case["op"] == "norm":
        f = _plain_norm(s)
        f["y"] = dict(zip(("codes", "scales"), _plain_quantize(f["y"], 1))) if case["fp8"] else f["y"].to(s["h"].dtype)
        return f
    return _plain_norm_bwd(s)


def work(case):
    if case["op"] == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        nk = (K + BLOCK - 1) // BLOCK
        scales = 4 * nk * (M + (N if case["b_lines"] == 1 else (N + BLOCK - 1) // BLOCK))
        return dict(bytes=(M + N) * K + scales + M * N * (2 if case["out"] == "bf16" else 4), flops=2 * M * N * K)
    rows, cols = case["rows"], case["cols"]
    n, size = rows * cols, 2 if case["type"] == "bf16" else 4
    if case["op"] == "quantize":
        axes = 2 if case["axes"] == "both" else 1
        return dict(bytes=n * size + axes * (n + 4 * n / (BLOCK * case["lines"])), flops=n * (1 + 2 * axes))
    groups = (rows + case["gate_rows"] - 1) // case["gate_rows"] if case["gate_rows"] else 0
    weights = cols * (1 + case["post"] + groups)
    if case["op"] == "norm":
        return dict(bytes=n * 3 * size + n * (1 + 4 / BLOCK if case["fp8"] else size) + weights * size + 8 * rows,
                    flops=n * (8 + 3 * case["post"]))
    return dict(bytes=n * 6 * size + weights * (size + 4) + 8 * rows, flops=n * (14 + 8 * case["post"]))


# ------------------------------------------------------------------- exact

def _fp8_from_64(x, lines):
    """The codes' values and the scales of a float64 [L, K], block by block along K."""
    L, K = x.shape
    codes, scales = torch.empty((L, K), dtype=torch.float8_e4m3fn, device=x.device), []
    for k in range(0, K, BLOCK):
        part = x[:, k:k + BLOCK]
        m = part.abs().max(dim=1).values
        if lines > 1:
            m = torch.stack([t.max() for t in m.split(lines)])
        s = m / 448.0
        s[s < 2.0 ** -126] = 1.0
        scales.append(s)
        wide = s if lines == 1 else s.repeat_interleave(lines)[:L]
        codes[:, k:k + BLOCK] = (part / wide[:, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return dict(codes=codes, scales=torch.stack(scales))


def _matrix_from_64(q):
    """The float64 matrix that codes and scales stand for, chunk by chunk."""
    m = torch.empty((q["lines"], q["K"]), dtype=torch.float64, device="cuda")
    for c, k in enumerate(range(0, q["K"], BLOCK)):
        e = min(q["K"], k + BLOCK)
        s = q["scales"][c].double()
        if q["block_lines"] > 1:
            s = s.repeat_interleave(q["block_lines"])
        m[:, k:e] = q["codes"][:, k:e].view(torch.float8_e4m3fn).double() * s[:q["lines"], None]
    return m


def _unit(x):
    return x / (x.pow(2).mean(dim=1, keepdim=True) + EPS).sqrt()


def _branch(o, w_post, gate, per, alpha):
    r = o if w_post is None else _unit(o) * w_post
    if gate is not None:
        r = r * gate[torch.arange(o.shape[0], device=o.device) // per]
    return alpha * r


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        got = {}
        if s["rows"] is not None:
            got["rows"] = _fp8_from_64(s["x"].double(), case["lines"])
        if s["cols"] is not None:
            got["cols"] = _fp8_from_64(s["x"].double().t(), case["lines"])
        return got
    if case["op"] == "gemm":
        return _matrix_from_64(s["a"]) @ _matrix_from_64(s["b"]).t()
    wide = lambda t: None if t is None else t.double()  # noqa: E731
    o, w_post, w_pre, gate = (wide(s[k]) for k in ("o", "w_post", "w_pre", "gate"))
    per = case["gate_rows"]
    if case["op"] == "norm":
        h = s["h"].double() + _branch(o, w_post, gate, per, s["alpha"])
        # the stored stream is what is normalised
        kept = h.to(_dtype(case["type"])).double()
        y = _unit(kept) * w_pre
        return dict(h=h, y=_fp8_from_64(y, 1) if case["fp8"] else y,
                    rstd_pre=(kept.pow(2).mean(dim=1) + EPS).pow(-0.5),
                    rstd_post=None if w_post is None else (o.pow(2).mean(dim=1) + EPS).pow(-0.5))
    # the gradients of <dy, y> and of <dh', h'>, by differentiation of the definition
    h, dy = s["h_out"].double().requires_grad_(), s["dy"].double()
    w_pre.requires_grad_()
    dh, dw_pre = torch.autograd.grad((_unit(h) * w_pre * dy).sum(), (h, w_pre))
    dh = dh + s["dh_in"].double()
    leaves = {k: t.requires_grad_() for k, t in (("do", o), ("dw_post", w_post), ("dgate", gate)) if t is not None}
    found = torch.autograd.grad((_branch(o, w_post, gate, per, s["alpha"]) * dh).sum(), list(leaves.values()))
    return dict(dict(dw_post=None, dgate=None), dh=dh, dw_pre=dw_pre, **dict(zip(leaves, found)))
