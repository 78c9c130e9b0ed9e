"""The decode-step operators on the GPU at the edges of what their header allows: signed and far
apart scales, values near the type's range, NaN in appended rows, every norm kernel."""

from __future__ import annotations

import numpy as np
import pytest

import gpu_helpers as gh
from oracle import step
from test_gpu_step import _case, _check, _new_cache, _qmm, _torch

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ 8-bit scales
@pytest.mark.parametrize("q_mul", [0.0, 1.0])
@pytest.mark.parametrize("big", [-10.0, 10.0, -1e3])
def test_attention_signed_value_scales(big, q_mul):
    """One value scale that is the largest in magnitude, at every place of two tiles in turn (a
    sequence each), among scales of one and minus one; key scales of both signs.  A q of zeros
    gives every token the largest weight."""
    gh.note(f"attention value scale {big} q*{q_mul}")
    c = _case("q8", [70] * 64, 2, 3, 64, 16, q_mul=q_mul, stale=False)
    sign = 1.0 - 2.0 * (_torch().arange(16, device="cuda") % 3 == 1)
    c["cache"].k_scale.copy_(0.02 * sign.expand_as(c["cache"].k_scale))
    c["cache"].v_scale.copy_(sign.expand_as(c["cache"].v_scale))
    for i in range(64):
        c["cache"].v_scale[int(c["table"][i][i // 16]), :, i % 16] = big
    _check(c)


@pytest.mark.parametrize("tokens", [0, 9000])
@pytest.mark.parametrize("place", [0, 20, 64, 199])
def test_attention_far_value_scale_of_a_negligible_token(place, tokens):
    """A token of weight e^-60 whose value scale is 1e12 times the others': these decide the output
    and keep all their bits."""
    torch = _torch()
    gh.note(f"attention far scale at {place}, table for {tokens}")
    c = _case("q8", [200], 2, 1, 64, 16, stale=False, tokens=tokens)
    page, at = int(c["table"][0][place // 16]), place % 16
    for h in range(2):
        q = c["q"][0, h]
        c["cache"].k[page, h, at] = (-100 * torch.sign(q)).to(torch.int8)
        c["cache"].k_scale[page, h, at] = 60.0 / (c["scale"] * 100 * float(q.abs().sum()))
        c["cache"].v_scale[page, h, at] = 1e12 * float(c["cache"].v_scale[:, h].abs().max())
    _check(c)


@pytest.mark.parametrize("tokens", [0, 9000])
@pytest.mark.parametrize("q_mul,k_scale", [(0.0, 1.0), (1e34, 1e-36), (1e-34, 1e32), (1e-20, 1e18)])
@pytest.mark.parametrize("v_scale", [1e30, 1e35, 1e-30])
def test_attention_scales_near_the_f32_range(q_mul, k_scale, v_scale, tokens):
    """Elements far from one on either side: outputs stay finite where elements and scores are."""
    gh.note(f"attention q*{q_mul} key scales {k_scale} value scales {v_scale}, table for {tokens}")
    c = _case("q8", [9000, 40, 1] if tokens else [150, 40, 1], 1, 2, 64, 16, q_mul=q_mul, stale=False)
    c["cache"].k_scale.fill_(k_scale)
    c["cache"].v_scale.fill_(v_scale)
    c["cache"].v.abs_()
    _check(c)


# ------------------------------------------------------------------ 16-bit ranges
@pytest.mark.parametrize("tokens", [0, 9000])
@pytest.mark.parametrize("q_mul,kv_mul", [(0.0, 3e37), (1e-35, 1e35), (1e-37, 3e37), (1e30, 1e-30), (1e34, 1e-34)])
def test_attention_bf16_near_the_f32_range(q_mul, kv_mul, tokens):
    """Finite keys and values up to the type's largest, with ordinary scores; every weight the same
    (a q of zeros) makes the sum of weights times values the largest."""
    gh.note(f"attention bf16 q*{q_mul} kv*{kv_mul}, table for {tokens}")
    c = _case("bf16", [9000, 40, 1] if tokens else [150, 40, 1], 1, 2, 64, 16, q_mul=q_mul, kv_mul=kv_mul)
    c["cache"].v.abs_()
    _check(c)


@pytest.mark.parametrize("kind", ["f16", "bf16", "q8"])
def test_attention_largest_scale(kind):
    """A scale whose product with log2(e) passes the f32 range, on queries that bring the scores back."""
    gh.note(f"attention {kind} scale 3e38")
    _check(_case(kind, [70, 33, 1000], 2, 4, 64, 16, q_mul=1e-37, kv_mul=0.1, scale=3e38))


# ------------------------------------------------------------------ NaN and infinity
@pytest.mark.parametrize("d", [32, 96, 128, 256])
@pytest.mark.parametrize("bad", [np.nan, -np.nan, np.inf, -np.inf])
def test_append_8bit_keeps_a_row_that_is_not_finite_visible(bad, d):
    """One element of a key (then of a value) that is no number or infinite: its row's scale says
    so, the head's attention is not finite, and no other row or head changes."""
    torch, qmm = _torch(), _qmm()
    gh.note(f"append q8 {bad} d={d}")
    rng = np.random.default_rng(d)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    for which in range(2):
        rows = rng.normal(size=(2, 40, 3, d)).astype(np.float32)
        rows[which, 17, 1, d - 3] = bad
        cache, _ = _new_cache("q8", 3, 3, 16, d)
        qmm.kv_append(cache, gh.to_dev(rows[0]), gh.to_dev(rows[1]), torch.arange(40, dtype=torch.int32, device="cuda"))
        for i, (codes, scales) in enumerate(((cache.k, cache.k_scale), (cache.v, cache.v_scale))):
            got, sc = (t.transpose(1, 2).flatten(0, 1)[:40].cpu().numpy() for t in (codes, scales))
            want, ws = step.q8_rows(np.where(np.isfinite(rows[i]), rows[i], 0), d)
            ws = ws[..., 0]
            if i == which:
                assert not got[17, 1].any() and (np.isnan(sc[17, 1]) if np.isnan(bad) else sc[17, 1] == np.inf)
                got[17, 1], sc[17, 1] = want[17, 1], ws[17, 1]
            assert np.array_equal(got, want) and np.array_equal(sc, ws)
        q = gh.to_dev(rng.normal(size=(1, 6, d)).astype(np.float32))
        out = qmm.paged_attention(q, cache, i32(0, 1, 2)[None], i32(40))[0].cpu().numpy()
        assert not np.isfinite(out[2:4]).any() and np.isfinite(out[[0, 1, 4, 5]]).all()


@pytest.mark.parametrize("k", [32, 288, 1056, 4096, 20000])
def test_norm_q8_keeps_what_is_not_finite_visible(k):
    """A NaN or infinite weight shows in its block's scale alone; a NaN in x in all of its row's."""
    torch, qmm = _torch(), _qmm()
    gh.note(f"norm q8 not finite k={k}")
    x, w = torch.randn(3, k, device="cuda"), torch.rand(k, device="cuda") + 0.5
    good_q, good_d, _ = qmm.add_rmsnorm_q8(x, w)
    for bad in (np.nan, -np.nan, np.inf, -np.inf):
        for at in (0, k - 1):
            wb = w.clone()
            wb[at] = bad
            q, d, _ = qmm.add_rmsnorm_q8(x, wb)
            block = at // 32
            assert not torch.isfinite(d[:, block]).any() and not q[:, 32 * block:32 * block + 32].any()
            q[:, 32 * block:32 * block + 32], d[:, block] = good_q[:, 32 * block:32 * block + 32], good_d[:, block]
            assert torch.equal(q, good_q) and torch.equal(d, good_d)
    xb = x.clone()
    xb[1, k // 2] = np.nan
    q, d, _ = qmm.add_rmsnorm_q8(xb, w)
    assert torch.isnan(d[1]).all() and torch.equal(d[::2], good_d[::2]) and torch.equal(q[::2], good_q[::2])


# ------------------------------------------------------------------ streams
def test_a_stream_of_another_device_is_refused():
    """Every call with all outputs given; a stream that says it belongs to device 1."""
    torch, qmm = _torch(), _qmm()

    class Other:
        device_index, cuda_stream = 1, 0
        device = torch.device("cuda", 0)

    c = _case("f16", [20], 1, 1, 32, 16, stale=False)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    x, out, rows = torch.zeros(2, 32, device="cuda"), torch.full((2, 32), 5.0, device="cuda"), i32(7, 7)
    for call in (lambda: qmm.kv_append(c["cache"], x, x, rows, stream=Other()),
                 lambda: qmm.add_rmsnorm(x, x[0], y=out, stream=Other()),
                 lambda: qmm.paged_extend(rows[None], i32(0), i32(1), i32(0), 16, 1, rows[:1], rows[1:], i32(0), i32(0),
                                          stream=Other())):
        with pytest.raises(ValueError, match="device 1"):
            call()
    torch.cuda.synchronize()
    assert (out == 5).all() and (rows == 7).all()


def test_attention_of_no_sequences_is_the_same_refusal_on_any_stream():
    torch, qmm = _torch(), _qmm()
    c = _case("f16", [20], 1, 2, 32, 16, stale=False)
    table, lens = torch.zeros(0, 4, dtype=torch.int32, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda")
    for stream in (None, torch.cuda.Stream()):
        for q in (c["q"][:0], c["q"][:0].flatten(1)):
            with pytest.raises(qmm.QmmError) as e:
                qmm.paged_attention(q, c["cache"], table, lens, stream=stream)
            assert e.value.status == 1      # an empty tensor has no address, and that is checked first
        with pytest.raises(ValueError):
            qmm.paged_attention(c["q"].flatten(), c["cache"], table, lens, stream=stream)
    torch.cuda.synchronize()


def test_attention_with_own_outputs_takes_any_stream_handle():
    """Nothing is allocated for the call: a stream known by its handle alone will do."""
    import types
    torch, qmm = _torch(), _qmm()
    c = _case("f16", [300, 40], 2, 4, 64, 16, stale=False, tokens=4000)
    args = (c["q"], c["cache"], torch.from_numpy(c["table"]).cuda(),
            torch.tensor(c["lens"], dtype=torch.int32, device="cuda"))
    need = qmm.paged_attention_workspace_bytes(2, 8, c["cache"], args[2].shape[1])
    out, ws, side = torch.empty_like(c["q"]), torch.empty(need, dtype=torch.uint8, device="cuda"), torch.cuda.Stream()
    want = qmm.paged_attention(*args)
    torch.cuda.synchronize()
    qmm.paged_attention(*args, out=out, workspace=ws, stream=types.SimpleNamespace(cuda_stream=side.cuda_stream))
    side.synchronize()
    assert need > 0 and torch.equal(out, want)


# ------------------------------------------------------------------ norm
def _norm_inputs(n, k, residual, seed):
    rng = np.random.default_rng(seed)
    x, r, w = (rng.normal(size=s).astype(np.float32) for s in ((n, k), (n, k), (k,)))
    return x, r if residual else None, w


def _check_norm_rows(rows, x, r, w, y=None, q=None, d=None, h=None):
    """Rows of a norm's outputs against the oracle (x, r, w host arrays of all rows)."""
    hs = x[rows] if r is None else x[rows] + r[rows]
    want, inv = step.rmsnorm(hs, w, 1e-5)
    rel = step.rmsnorm_rel(hs.shape[1])
    if h is not None:
        assert np.array_equal(h[rows].cpu().numpy(), hs)
    if y is not None:
        assert (np.abs(y[rows].cpu().double().numpy() - want) <= rel * np.abs(want) + 1e-44).all()
    else:
        codes, d0 = step.q8_rows(hs * w, 32)
        assert np.array_equal(q[rows].cpu().numpy(), codes)
        assert (np.abs(d[rows].cpu().double().numpy() - d0 * inv) <= rel * d0 * inv).all()


# 257 rows are more than the device's CUs: 256 threads a row with 2 to 8 elements of four each, then 1024
NORM_WIDTHS = [1028, 1056, 2048, 2052, 2080, 3104, 4096, 4608, 5120, 5124, 6176, 7168, 7200, 8192, 8196, 8224, 16384, 16416]


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("k", NORM_WIDTHS)
def test_norm_of_more_rows_than_cus(k, residual):
    qmm = _qmm()
    gh.note(f"norm n=257 k={k} residual={residual}")
    x, r, w = _norm_inputs(257, k, residual, k)
    dev = [None if v is None else gh.to_dev(v) for v in (x, w, r)]
    rows = np.arange(257)
    y, h = qmm.add_rmsnorm(*dev)
    _check_norm_rows(rows, x, r, w, y=y, h=h)
    if k % 32 == 0:
        q, d, h = qmm.add_rmsnorm_q8(*dev)
        _check_norm_rows(rows, x, r, w, q=q, d=d, h=h)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("k", [1024, 2048, 2080, 4096, 4608, 6144, 7168, 8192, 12288])
def test_norm_of_large_inputs(k, residual):
    """More than 48 MB of input, read past the caches: rows against the oracle, and all of them equal
    to calls of 300 rows each, which are not (fewer rows than CUs would add in another order)."""
    torch, qmm = _torch(), _qmm()
    n = (50 << 20) // (k * (8 if residual else 4)) + 2
    gh.note(f"norm n={n} k={k} residual={residual}")
    x, r, w = _norm_inputs(n, k, residual, k)
    dx, dw, dr = (None if v is None else gh.to_dev(v) for v in (x, w, r))
    rows = np.unique(np.concatenate([[0, 1, n - 2, n - 1], np.random.default_rng(1).integers(0, n, 60)]))
    for f in (qmm.add_rmsnorm, qmm.add_rmsnorm_q8):
        got = f(dx, dw, dr)
        _check_norm_rows(rows, x, r, w, **dict(zip(("y", "h") if len(got) == 2 else ("q", "d", "h"), got)))
        for at in [*range(0, n - 300, 300), n - 300]:
            part = f(dx[at:at + 300], dw, None if dr is None else dr[at:at + 300])
            assert all(g is None or torch.equal(g[at:at + 300], p) for g, p in zip(got, part))


# ------------------------------------------------------------------ steps at the same time
def test_whole_steps_at_the_same_time_on_three_streams():
    """Page tables, append, attention and norm of three caches on three streams, without waiting between
    them: both equal their serial results."""
    torch, qmm = _torch(), _qmm()
    cases = [_case(k, [2500, 40, 0, 900], 4, 2, 64, 16, seed=s, tokens=4000, stale=False)
             for s, k in ((3, "f16"), (4, "q8"), (5, "bf16"))]
    w = torch.ones(512, device="cuda")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731

    def one(c, stream=None):
        lens, slots, pos, used = qmm.paged_extend(c["tab"], c["cached"], c["new"], c["free"], 16, 6, stream=stream)
        qmm.kv_append(c["cache"], c["rows"][0], c["rows"][1], slots, stream=stream)
        out = qmm.paged_attention(c["q"], c["cache"], c["tab"], lens, stream=stream)
        y, h = qmm.add_rmsnorm(out.flatten(1), w, out.flatten(1), stream=stream)
        return lens, slots, pos, used, out, y, h

    for c in cases:                     # the last token of each sequence is the step's new one
        c["tab"] = torch.from_numpy(c["table"]).cuda()
        c["cached"], c["new"] = i32([2499, 39, 0, 899]), i32([1, 1, 0, 1])
        c["free"] = i32([0, 1])         # never needed: those tokens' pages are there
        c["rows"] = torch.randn(2, 6, 4, 64, device="cuda")
        c["want"] = [t.clone() for t in one(c)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(20):
        got = [one(c, s) for c, s in zip(cases, streams)]
        for s in streams:
            s.synchronize()
        for c, g in zip(cases, got):
            assert c["want"][3].item() == 0 and all(torch.equal(x, y) for x, y in zip(g, c["want"]))
