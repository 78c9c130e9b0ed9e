"""MXFP4 on the GPU at the edges of what its header allows: attention scales and scores near the ends
of f32, operands that are missing."""

from __future__ import annotations

import numpy as np
import pytest

import gpu_helpers as gh
from oracle import mxfp4
from test_gpu_mxfp4 import _case, _check, _dev, _qmm, _torch

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ attention
def _check_decided(c):
    """_check, and where a head's largest score is ahead by far more than f32 can be off (2 (d + 12) u
    of the largest sum of magnitudes, and 200 for the others to weigh nothing) its token's value: a
    weight and its sum are the same number there, so the output is off by the inverse, a product and
    the three parts, below 8 u of the value.  Returns how many heads were."""
    torch, qmm = _torch(), _qmm()
    _check(c)
    out = qmm.paged_attention(_dev(c["q"]), c["cache"], _dev(c["table"]),
                              torch.tensor(c["lens"], dtype=torch.int32, device="cuda"), scale=c["scale"]).cpu().numpy()
    b, n_q, d = c["q"].shape
    seen, u = 0, 2.0 ** -24
    for i in np.flatnonzero(c["lens"]):
        t = np.arange(c["lens"][i])
        at = (c["table"][i][t // c["page"]], slice(None), t % c["page"])
        k, v = (mxfp4.dequantize(c["host"][n][at], c["host"][n + "s"][at]) for n in ("k", "v"))
        for h in range(n_q):
            kh, q = k[:, h // (n_q // k.shape[1])], c["q"][i, h].astype(np.float64)
            s, reach = c["scale"] * (kh @ q), abs(c["scale"]) * (np.abs(kh) @ np.abs(q))
            order = np.argsort(s)
            if len(s) == 1 or s[order[-1]] - s[order[-2]] > 2 * (d + 12) * u * reach.max() + 200:
                want = v[order[-1], h // (n_q // k.shape[1])]
                assert np.all(np.abs(out[i, h] - want) <= 8 * u * np.abs(want)), (i, h)
                seen += 1
    return seen


@pytest.mark.parametrize("page", [16, 4])
@pytest.mark.parametrize("q_mul", [2.0 ** 24, 2.0 ** 29, 2.0 ** 30, 2.0 ** 31, 2.0 ** 33, 2.0 ** 60, 2.0 ** 110])
def test_attention_any_score(q_mul, page):
    """A score's own rounding, 64 and more from 2^30 on, does not enter the exponentials."""
    gh.note(f"attention mxfp4 q*{q_mul} page {page}")
    seen = 0
    for lens, tokens in (([70, 1, 0, 33], 0), ([700, 90], 1024), ([1] * 8, 0)):
        for sign in (1.0, -1.0):
            seen += _check_decided(_case(lens, 2, 4, 64, page, tokens=tokens, scale=0.125 * sign, q_mul=q_mul))
    assert seen > 50


@pytest.mark.parametrize("page", [16, 4])
@pytest.mark.parametrize("scale,q_mul,scales", [
    (2.0 ** -30, 2.0 ** 20, (238, 243)),      # sums of products beyond f32, scores of 2^110
    (-2.0 ** -100, 2.0 ** 60, (240, 245)),
    (2.0 ** 118, 1.0, (3, 9)),                # scale times 2^12 beyond f32, scores of some units
    (-3e38, 2.0 ** -3, (0, 3)),
    (3e38, 1e-37, (122, 129)),
    (2.0 ** 60, 2.0 ** 50, (10, 20)),
    (2.0 ** -126, 2.0 ** 100, (140, 150)),
    (2.0 ** -149, 2.0 ** 120, (145, 155)),
    (0.0, 2.0 ** 100, (120, 129)),
    (2.0 ** -126, 2.0 ** 120, (246, 252)),    # products of 2^244
    (3e38, 2.0 ** 60, (0, 3)),
])
def test_attention_any_scale(scale, q_mul, scales, page):
    """Finite elements and scores give finite outputs whatever the scale."""
    gh.note(f"attention mxfp4 scale {scale} q*{q_mul} key scales {scales} page {page}")
    for lens, tokens in (([70, 1, 0, 33], 0), ([700, 90], 1024)):
        c = _case(lens, 2, 4, 64, page, tokens=tokens, scales=scales, scale=scale, q_mul=q_mul)
        for name in ("v_scale",):             # values of ordinary size
            t = getattr(c["cache"], name)
            t.copy_(_torch().where(t == 255, t, 122 + t % 6))
            c["host"]["vs"] = t.cpu().numpy()
        _check_decided(c)


@pytest.mark.parametrize("scale,q_mul,k_mul", [
    (2.0 ** -30, 2.0 ** 20, 2.0 ** 115), (-2.0 ** -100, 2.0 ** 60, 2.0 ** 120), (2.0 ** 118, 1.0, 2.0 ** -118),
    (-3e38, 2.0 ** -3, 2.0 ** -120), (3e38, 1e-37, 0.1), (2.0 ** 60, 2.0 ** 50, 2.0 ** -110),
    (2.0 ** -149, 2.0 ** 120, 2.0 ** 26), (0.0, 2.0 ** 60, 1.0), (0.125, 2.0 ** 33, 1.0), (-0.125, 2.0 ** 100, 1.0)])
def test_attention_bf16_any_scale(scale, q_mul, k_mul):
    """The same of a bfloat16 cache."""
    import test_gpu_step as of_step
    gh.note(f"attention bf16 scale {scale} q*{q_mul} k*{k_mul}")
    for lens, tokens in (([70, 1, 0, 33], 0), ([700, 90], 1024)):
        c = of_step._case("bf16", lens, 2, 4, 64, 16, tokens=tokens, scale=scale, q_mul=q_mul)
        k = c["cache"].k
        k.copy_(_torch().where(_torch().isfinite(k), k.float() * k_mul, k.float()))
        of_step._check(c)


# ------------------------------------------------------------------ refusals
def test_missing_and_flat_operands_are_named():
    torch, qmm = _torch(), _qmm()
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")  # noqa: E731
    f32 = lambda *s: torch.zeros(s, device="cuda")  # noqa: E731
    q, e = u8(4, 32), u8(4, 2)
    for call, error, name in (
        (lambda: qmm.gemm_mxfp4(q, e, None, e), TypeError, "xq"), (lambda: qmm.gemm_mxfp4(q, e, q, None), TypeError, "xe"),
        (lambda: qmm.gemm_mxfp4(None, e, q, e), TypeError, "wq"), (lambda: qmm.gemm_mxfp4(q, None, q, e), TypeError, "we"),
        (lambda: qmm.gemm_mxfp4(q, e, u8(4)[0], e), ValueError, "xq"), (lambda: qmm.gemm_mxfp4(u8(4)[0], e, q, e), ValueError, "wq"),
        (lambda: qmm.gemm_mxfp4(q, e, u8(32), u8(2)), ValueError, "xq"), (lambda: qmm.gemm_mxfp4(q, e, q, e, x_scale=3.0), TypeError, "x_scale"),
        (lambda: qmm.quantize_mxfp4(None), TypeError, "x"), (lambda: qmm.quantize_mxfp4(f32(64)), ValueError, "x must"),
        (lambda: qmm.quantize_mxfp4(f32(4)[0]), ValueError, "x must"), (lambda: qmm.quantize_mxfp4(f32(2, 2, 32)), ValueError, "x must"),
        (lambda: qmm.dequantize_mxfp4(None, e), TypeError, "q"), (lambda: qmm.dequantize_mxfp4(q, None), TypeError, "e"),
        (lambda: qmm.dequantize_mxfp4(u8(4)[0], e), ValueError, "q must"),
        (lambda: qmm.add_rmsnorm_mxfp4(None, f32(64)), TypeError, "x"), (lambda: qmm.add_rmsnorm_mxfp4(f32(4, 64), None), TypeError, "weight"),
        (lambda: qmm.add_rmsnorm_mxfp4(f32(64), f32(64)), ValueError, "x must"),
        (lambda: qmm.add_rmsnorm_mxfp4(f32(4)[0], f32(64)), ValueError, "x must"),
        (lambda: qmm.add_rmsnorm_mxfp4(f32(1, 4, 64), f32(64)), ValueError, "x must"),
    ):
        with pytest.raises(error, match=name):
            call()
