"""Pins of the oracle's FP8 block-128 quantizer, its GEMM and the norm /
residual gradients: torch's E4M3 cast, values that E4M3 holds exactly, exact
rationals on a tiny product, and central differences of the forward formula."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle


def e4m3_by_torch(x):
    return torch.from_numpy(x).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


@pytest.mark.parametrize("shape", [(1, 128), (3, 300), (130, 257), (200, 64)])
@pytest.mark.parametrize("lines", [1, 128])
@pytest.mark.parametrize("axis", [0, 1])
def test_codes_and_scales_against_torch(shape, lines, axis):
    rng = np.random.default_rng(shape[1] + lines)
    x = rng.standard_normal(shape).astype(np.float32)
    q = oracle.fp8_block_quantize(x, lines, axis)
    v = x if axis else np.ascontiguousarray(x.T)
    L, K = v.shape
    for b in range(-(-L // lines)):
        for k in range(-(-K // 128)):
            at = (slice(b * lines, min(L, (b + 1) * lines)), slice(128 * k, min(K, 128 * k + 128)))
            m = np.abs(v[at]).max()
            assert q["scales"][b, k] == np.float32(m) / np.float32(448)
            assert (q["codes"][at] == e4m3_by_torch((448.0 * v[at].astype(np.float64) / m).astype(np.float32))).all()


def test_block_maximum_takes_the_top_code_and_zeros_stay_zero():
    x = np.zeros((2, 256), np.float32)
    x[0, 5] = -3.5
    q = oracle.fp8_block_quantize(x)
    assert q["codes"][0, 5] == 0xFE and q["scales"][0, 0] == np.float32(3.5) / np.float32(448)
    assert (q["scales"][1] == 1).all() and q["scales"][0, 1] == 1
    assert (np.delete(q["codes"].ravel(), 5) == 0).all()


def test_a_quotient_below_the_smallest_normal_gives_scale_one():
    x = np.full((1, 128), np.float32(2.0 ** -120))
    q = oracle.fp8_block_quantize(x)
    assert q["scales"][0, 0] == 1 and (q["codes"] == 0).all()


def test_a_quotient_in_the_middle_of_two_codes_goes_to_the_even_one():
    # m = 7 / 4: 448 x / m = 256 x; 17/16 * 256 = 272 lies between 256 (0x78) and 288 (0x79)
    x = np.zeros((1, 128), np.float32)
    x[0, :3] = 1.75, 17 / 16, 19 / 16                     # 304: between 288 (0x79) and 320 (0x7A)
    assert oracle.fp8_block_quantize(x)["codes"][0, :3].tolist() == [0x7E, 0x78, 0x7A]


def test_values_that_e4m3_holds_come_back_exactly():
    x = np.array([[448, -448, 1, 0.5, -0.0625, 416, 240, 0] * 16], np.float32)
    assert (oracle.fp8_block_dequantize(oracle.fp8_block_quantize(x)) == x).all()


def test_gemm_is_the_exact_rational_product():
    rng = np.random.default_rng(3)
    a = oracle.fp8_block_quantize(rng.standard_normal((2, 130)).astype(np.float32))
    b = oracle.fp8_block_quantize(rng.standard_normal((3, 130)).astype(np.float32), 128)
    C, bound = oracle.fp8_block_gemm(a, b)
    value = lambda q, i, k: (Fraction(float(oracle.fp8_dequantize(dict(codes=q["codes"][i:i + 1, k:k + 1], scale=1.0))[0, 0]))  # noqa: E731
                             * Fraction(float(q["scales"][i // q["block_lines"], k // 128])))
    for i in range(2):
        for j in range(3):
            exact = sum(value(a, i, k) * value(b, j, k) for k in range(130))
            # 130 float64 products and sums, and each value's own product with its scale
            assert abs(Fraction(C[i, j]) - exact) <= Fraction(float(bound[i, j])) * 134 * Fraction(1, 2 ** 53)


def forward_scalar(p, dy, dh_in, per, alpha):
    f = oracle.norm_residual(p["h"], p["o"], p.get("w_post"), p.get("gate"), per, alpha, p.get("w_pre"))
    loss = (dh_in * f["h"]).sum()
    return loss + ((dy * f["y"]).sum() if f["y"] is not None else 0.0)


@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("pre", [True, False])
def test_gradients_against_central_differences(post, gate, pre):
    rng = np.random.default_rng(11)
    rows, cols, per, alpha = 5, 7, 2, 0.7
    p = dict(h=rng.standard_normal((rows, cols)), o=rng.standard_normal((rows, cols)))
    if post:
        p["w_post"] = rng.standard_normal(cols)
    if gate:
        p["gate"] = rng.standard_normal((3, cols))
    if pre:
        p["w_pre"] = rng.standard_normal(cols)
    dy, dh_in = (rng.standard_normal((rows, cols)) for _ in range(2))
    f = oracle.norm_residual(p["h"], p["o"], p.get("w_post"), p.get("gate"), per, alpha, p.get("w_pre"))
    g = oracle.norm_residual_backward(dy if pre else None, f["h"], f["rstd_pre"], p.get("w_pre"), dh_in, p["o"],
                                      p.get("w_post"), f["rstd_post"], p.get("gate"), per, alpha)
    for name, key in (("h", "dh"), ("o", "do"), ("w_post", "dw_post"), ("gate", "dgate"), ("w_pre", "dw_pre")):
        if name not in p:
            assert g[key] is None
            continue
        for _ in range(4):
            d = rng.standard_normal(p[name].shape)
            e = 1e-5
            diff = (forward_scalar({**p, name: p[name] + e * d}, dy, dh_in, per, alpha)
                    - forward_scalar({**p, name: p[name] - e * d}, dy, dh_in, per, alpha)) / (2 * e)
            # central differences at e = 1e-5: truncation about e^2, cancellation about 1e-16 / e, of sums of about 100
            assert abs(diff - (g[key] * d).sum()) <= 1e-8 * 100
