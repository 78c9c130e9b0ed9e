"""MXFP4 on the GPU against the f64 oracle: quantization and back, the norm that writes it, the
product, the paged cache with its append and attention, and a run of them together."""

from __future__ import annotations

import math

import numpy as np
import pytest

import gpu_helpers as gh
from oracle import mxfp4, step

pytestmark = pytest.mark.gpu

MX_TILE_SHAPES = [  # (m, k, n): every kernel and its edges
    (1, 32, 1), (16, 32, 1), (17, 64, 3), (100, 96, 16), (64, 128, 17), (33, 160, 31), (257, 256, 5), (130, 512, 64),
    (48, 544, 33), (300, 1024, 129), (70, 1056, 200), (513, 640, 260), (1, 2048, 300), (260, 96, 1), (256, 1536, 256),
    (1000, 192, 500), (31, 1792, 40), (640, 288, 70),
]


def _torch():
    import torch
    return torch


def _qmm():
    import gemv_prefill_decode_amd as qmm
    return qmm


def _dev(a):
    return _torch().from_numpy(np.ascontiguousarray(a)).cuda()


# ------------------------------------------------------------------ quantization
def _hard_values(rng, rows, k):
    """Values on and beside the borders between codes, of every size."""
    mids = np.array([0.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.9])
    x = rng.choice(mids, size=(rows, k)) * rng.choice([-1.0, 1.0], size=(rows, k))
    x = x * np.repeat(2.0 ** rng.integers(-20, 20, size=(rows, k // 32)), 32, axis=1)
    x = x.astype(np.float32)
    side = rng.integers(-1, 2, size=x.shape)
    x = np.where(side == 0, x, np.nextafter(x, np.where(side > 0, np.float32(np.inf), np.float32(-np.inf)).astype(np.float32)))
    rand = rng.random((rows, k // 32)) < 0.5
    return np.where(np.repeat(rand, 32, axis=1), rng.normal(size=x.shape).astype(np.float32), x).astype(np.float32)


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("rows,k,pad", [(1, 32, 0), (3, 96, 0), (7, 1024, 16), (130, 160, 8), (1, 4096, 0), (65, 32, 32)])
def test_quantize_is_exact(dtype, rows, k, pad):
    torch, qmm = _torch(), _qmm()
    gh.note(f"quantize {dtype} {rows}x{k} pad {pad}")
    rng = np.random.default_rng(rows + k)
    x = torch.full((rows, k + pad), math.nan, dtype=getattr(torch, dtype), device="cuda")[:, :k]
    x.copy_(torch.from_numpy(_hard_values(rng, rows, k)))
    q, e = qmm.quantize_mxfp4(x)
    wq, we = mxfp4.quantize(x.cpu().double().numpy())
    assert np.array_equal(e.cpu().numpy(), we) and np.array_equal(q.cpu().numpy(), wq)
    # (some float16 rows overflow: NaN blocks)
    assert np.array_equal(qmm.dequantize_mxfp4(q, e).cpu().numpy(), mxfp4.dequantize(wq, we).astype(np.float32), equal_nan=True)


def test_quantize_ends_of_the_range():
    torch, qmm = _torch(), _qmm()
    big = 3.4028234663852886e38
    rows = [[0.0], [-0.0, 1.0], [2.0 ** -149, -2.0 ** -149], [2.0 ** -126, 2.0 ** -127, 2.0 ** -129], [2.0 ** -125, -2.0 ** -128],
            [big, -big, 1.0], [math.inf, 1.0], [1.0, -math.inf], [math.nan, 1.0], [math.inf, math.nan], [2.0 ** -124, 2.0 ** -127]]
    x = np.zeros((len(rows), 64), np.float32)
    for i, r in enumerate(rows):
        x[i, 5:5 + len(r)] = r
    x[:, 40] = 1.0          # the neighbour block is untouched
    q, e = qmm.quantize_mxfp4(_dev(x))
    wq, we = mxfp4.quantize(x)
    assert np.array_equal(e.cpu().numpy(), we) and np.array_equal(q.cpu().numpy(), wq)
    v = qmm.dequantize_mxfp4(q, e).cpu().numpy()
    assert np.array_equal(v, mxfp4.dequantize(wq, we).astype(np.float32), equal_nan=True)


def test_dequantize_every_scale_and_code():
    torch, qmm = _torch(), _qmm()
    codes = np.arange(256, dtype=np.uint8)
    q = np.tile(codes.reshape(16, 16), (16, 1)).reshape(256, 1, 16)         # 256 blocks of 16 bytes
    q = np.broadcast_to(q.reshape(1, 256 * 16), (256, 4096)).copy()
    e = np.broadcast_to(np.arange(256, dtype=np.uint8)[:, None], (256, 256)).copy()
    with np.errstate(over="ignore"):
        want = mxfp4.dequantize(q, e).astype(np.float32)
    assert np.array_equal(qmm.dequantize_mxfp4(_dev(q), _dev(e)).cpu().numpy(), want, equal_nan=True)
    # leading dimensions are the caller's
    got = qmm.dequantize_mxfp4(_dev(q.reshape(4, 8, 8, 4096)), _dev(e.reshape(4, 8, 8, 256)))
    assert got.shape == (4, 8, 8, 8192) and np.array_equal(got.cpu().numpy().reshape(256, 8192), want, equal_nan=True)


def test_quantize_more_items_than_one_grid_and_guards():
    """Rows behind the arrays stay as they were; a large array is whole."""
    torch, qmm = _torch(), _qmm()
    q, e = torch.full((6, 48), 7, dtype=torch.uint8, device="cuda"), torch.full((6, 3), 7, dtype=torch.uint8, device="cuda")
    x = torch.randn(5, 96, device="cuda")
    qmm.quantize_mxfp4(x, q=q[:5], e=e[:5])
    out = torch.full((6, 96), 7.0, device="cuda")
    qmm.dequantize_mxfp4(q[:5], e[:5], out=out[:5])
    assert (q[5] == 7).all() and (e[5] == 7).all() and (out[5] == 7).all()
    x = torch.randn(9000, 14336, device="cuda")
    v = qmm.dequantize_mxfp4(*qmm.quantize_mxfp4(x))
    # half a step of the grid: 1/8 of a value of at least the scale, 1/4 of the scale below, 2 above 6
    scale = torch.exp2(torch.floor(torch.log2(x.view(9000, -1, 32).abs().amax(-1))) - 2).repeat_interleave(32, 1)
    assert ((v - x).abs() <= 2 * scale).all() and ((v - x).abs().mean() < 0.2)


# ------------------------------------------------------------------ product
def _gemm_inputs(rng, m, k, n, spread):
    w, x = (rng.integers(0, 256, (r, k // 2), dtype=np.uint8) for r in (m, n))
    we, xe = (rng.integers(127 - spread, 128 + spread, (r, k // 32), dtype=np.uint8) for r in (m, n))
    return w, we, x, xe


@pytest.mark.parametrize("m,k,n", MX_TILE_SHAPES)
def test_gemm_is_exact_where_sums_are(m, k, n):
    """Products are multiples of 1/4 of the two scales, so with scales 2^0 and 2^1 any f32 sum of up
    to 2^24 / (144 * 4) of them is exact: no tolerance."""
    torch, qmm = _torch(), _qmm()
    gh.note(f"gemm_mxfp4 exact {m}x{k} n={n}")
    assert k * 144 * 4 < 2 ** 24
    rng = np.random.default_rng(m * 7 + k + n)
    w, x = (rng.integers(0, 256, (r, k // 2), dtype=np.uint8) for r in (m, n))
    we, xe = (rng.integers(127, 129, (r, k // 32), dtype=np.uint8) for r in (m, n))
    want = mxfp4.gemm(w, we, x, xe)[0]
    out = torch.full((n + 1, m + 3), 7.0, device="cuda")
    qmm.gemm_mxfp4(_dev(w), _dev(we), _dev(x), _dev(xe), out=out[:n, :m])
    got = out.cpu().numpy()
    assert np.array_equal(got[:n, :m], want) and (got[n] == 7).all() and (got[:, m:] == 7).all()
    s = (2.0 ** rng.integers(-3, 4, n)).astype(np.float32)
    got = qmm.gemm_mxfp4(_dev(w), _dev(we), _dev(x), _dev(xe), x_scale=_dev(s)).cpu().numpy()
    assert np.array_equal(got, want * s[:, None])


@pytest.mark.parametrize("kernel", range(11))
def test_gemm_every_kernel(kernel, monkeypatch):
    """Each kernel on the edges of every other's tiles: rows and tokens that end inside a tile, k that
    ends inside a stage, a group of 512 and a wave's share."""
    torch, qmm = _torch(), _qmm()
    monkeypatch.setenv("QMM_MX_KERNEL", str(kernel))
    for m, k, n in [(1, 32, 1), (17, 64, 3), (65, 480, 33), (130, 544, 257), (257, 1024, 129), (48, 1056, 64), (300, 2080, 20),
                    (256, 1536, 512), (33, 5120, 5), (520, 288, 300)]:
        gh.note(f"gemm_mxfp4 kernel {kernel} {m}x{k} n={n}")
        rng = np.random.default_rng(m + k + n)
        w, x = (rng.integers(0, 256, (r, k // 2), dtype=np.uint8) for r in (m, n))
        we, xe = (rng.integers(127, 129, (r, k // 32), dtype=np.uint8) for r in (m, n))
        out = torch.full((n + 1, m + 1), 7.0, device="cuda")
        qmm.gemm_mxfp4(_dev(w), _dev(we), _dev(x), _dev(xe), out=out[:n, :m])
        got = out.cpu().numpy()
        assert np.array_equal(got[:n, :m], mxfp4.gemm(w, we, x, xe)[0]), (m, k, n)
        assert (got[n] == 7).all() and (got[:, m] == 7).all()
        if k > 1000:        # a NaN scale at the row's end stays in its row
            we[m // 2, -1] = 255
            got = qmm.gemm_mxfp4(_dev(w), _dev(we), _dev(x), _dev(xe)).cpu().numpy()
            assert np.isnan(got[:, m // 2]).all() and np.isfinite(np.delete(got, m // 2, 1)).all()


@pytest.mark.parametrize("m,k,n", [(16, 64, 1 << 20), (7, 32, (1 << 20) - 3), ((1 << 22) + 5, 64, 1), ((1 << 20) + 16, 32, 17)])
def test_gemm_many_rows(m, k, n):
    """As many tokens as there may be, and as many rows as one kind of tile would need a grid too
    large for.  All products are multiples of 1/4 below 36, their sums exact."""
    torch, qmm = _torch(), _qmm()
    gh.note(f"gemm_mxfp4 {m}x{k} n={n}")
    torch.manual_seed(m % 97)
    (w, we), (x, xe) = (tuple((torch.randint(0, 256, (r, k // 2), dtype=torch.uint8, device="cuda"),
                               torch.full((r, k // 32), 127, dtype=torch.uint8, device="cuda"))) for r in (m, n))
    out = torch.full((n, m), math.nan, device="cuda")
    qmm.gemm_mxfp4(w, we, x, xe, out=out)
    for i in torch.randint(0, n, (8,)).tolist() + [0, n - 1]:
        assert torch.equal(out[i], (qmm.dequantize_mxfp4(w, we) * qmm.dequantize_mxfp4(x[i:i + 1], xe[i:i + 1])).sum(1))
    wf = qmm.dequantize_mxfp4(w, we)
    for i in torch.randint(0, m, (8,)).tolist() + [0, m - 1]:
        assert torch.equal(out[:, i], (qmm.dequantize_mxfp4(x, xe) * wf[i]).sum(1))


def test_gemm_malformed_kernel_choice(monkeypatch):
    qmm = _qmm()
    args = [_dev(np.zeros(s, np.uint8)) for s in ((2, 16), (2, 1), (3, 16), (3, 1))]
    for bad in ("11", "-1", "x", "1 2"):
        monkeypatch.setenv("QMM_MX_KERNEL", bad)
        with pytest.raises(qmm.QmmError, match="8"):
            qmm.gemm_mxfp4(*args)


@pytest.mark.parametrize("m,k,n", [(40, 4608, 20), (300, 4096, 70), (130, 14336, 3), (300, 2080, 300), (16, 64, 16)])
def test_gemm_is_within_its_bound(m, k, n):
    torch, qmm = _torch(), _qmm()
    gh.note(f"gemm_mxfp4 {m}x{k} n={n}")
    rng = np.random.default_rng(m + k + n)
    w, we, x, xe = _gemm_inputs(rng, m, k, n, 12)
    s = rng.uniform(0.1, 3.0, n).astype(np.float32)
    want, tol = mxfp4.gemm(w, we, x, xe, s)
    args = [_dev(a) for a in (w, we, x, xe, s)]
    got = qmm.gemm_mxfp4(*args)
    assert np.all(np.abs(got.cpu().numpy() - want) <= tol)
    assert torch.equal(got, qmm.gemm_mxfp4(*args))          # identical calls, identical bits


@pytest.mark.parametrize("n", [3, 40, 300])
def test_gemm_nan_and_extreme_scales(n):
    torch, qmm = _torch(), _qmm()
    rng = np.random.default_rng(n)
    m, k = 70, 1120
    w, we, x, xe = _gemm_inputs(rng, m, k, n, 2)
    we[5, 34] = xe[n - 1, 0] = 255
    want, tol = mxfp4.gemm(w, we, x, xe)
    got = qmm.gemm_mxfp4(*(_dev(a) for a in (w, we, x, xe))).cpu().numpy()
    nan = np.zeros((n, m), bool)
    nan[:, 5] = nan[n - 1] = True
    assert np.array_equal(np.isnan(got), nan)
    assert np.all(np.abs(got - want)[~nan] <= tol[~nan])
    # 2^-127 beside 2^125, and products below f32
    we[:], xe[:] = 252, 0
    want, tol = mxfp4.gemm(w, we, x, xe)
    got = qmm.gemm_mxfp4(*(_dev(a) for a in (w, we, x, xe))).cpu().numpy()
    assert np.all(np.abs(got - want) <= tol)
    we[:] = 0
    assert not qmm.gemm_mxfp4(*(_dev(a) for a in (w, we, x, xe))).cpu().numpy().any()


def test_gemm_follows_quantized_rows():
    """The layouts of quantize_mxfp4 and gemm_mxfp4 agree."""
    torch, qmm = _torch(), _qmm()
    rng = np.random.default_rng(8)
    w, x = rng.normal(size=(90, 224)).astype(np.float32), rng.normal(size=(37, 224)).astype(np.float32)
    got = qmm.gemm_mxfp4(*qmm.quantize_mxfp4(_dev(w).bfloat16()), *qmm.quantize_mxfp4(_dev(x))).cpu().numpy()
    wb = torch.from_numpy(w).bfloat16().double().numpy()
    want, tol = mxfp4.gemm(*mxfp4.quantize(wb), *mxfp4.quantize(x))
    assert np.all(np.abs(got - want) <= tol)


# ------------------------------------------------------------------ norm
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("n,k", [(1, 32), (3, 64), (5, 96), (9, 256), (4, 1024), (300, 1056), (2, 4096), (3, 8192),
                                 (290, 4608), (1, 16384), (2, 20000 // 32 * 32)])
def test_norm_matches_the_oracle(n, k, residual):
    torch, qmm = _torch(), _qmm()
    gh.note(f"add_rmsnorm_mxfp4 {n}x{k} residual={residual}")
    rng = np.random.default_rng(n + k)
    x, r = (rng.normal(size=(n, k + 8)).astype(np.float32) for _ in range(2))
    w = rng.normal(size=k).astype(np.float32)
    dx, dr = _dev(x)[:, :k], _dev(r)[:, :k] if residual else None
    q, e, s, h = qmm.add_rmsnorm_mxfp4(dx, _dev(w), dr, eps=1e-5)
    h32 = x[:, :k] + r[:, :k] if residual else x[:, :k]
    wq, we = mxfp4.quantize((h32 * w).astype(np.float32))
    assert np.array_equal(q.cpu().numpy(), wq) and np.array_equal(e.cpu().numpy(), we)
    inv = step.rmsnorm(h32, w, 1e-5)[1][:, 0]
    assert np.all(np.abs(s.cpu().numpy() - inv) <= step.rmsnorm_rel(k) * inv)
    assert h is None if not residual else np.array_equal(h.cpu().numpy(), h32)


def test_norm_keeps_a_nan_visible_and_its_neighbours_whole():
    torch, qmm = _torch(), _qmm()
    x = np.random.default_rng(1).normal(size=(3, 128)).astype(np.float32)
    x[1, 70] = np.nan
    q, e, s, _ = qmm.add_rmsnorm_mxfp4(_dev(x), torch.ones(128, device="cuda"))
    e, s = e.cpu().numpy(), s.cpu().numpy()
    assert e[1, 2] == 255 and (np.delete(e, 1, 0) < 255).all() and (e[1, [0, 1, 3]] < 255).all()
    assert np.isnan(s[1]) and np.isfinite(s[[0, 2]]).all()


# ------------------------------------------------------------------ cache
def _new_cache(rng, n_pages, n_kv, page, d, layout, fill=None):
    """(KVCache, tensors) with tensors k, v, ks, vs as [n_pages, n_kv, page, ..] views."""
    torch, qmm = _torch(), _qmm()
    views = {}
    widths = (("k", d // 2), ("v", d // 2), ("ks", d // 32), ("vs", d // 32))
    if layout == "block":       # a page's codes and scales side by side
        rows, gap = n_kv * page, -(n_kv * page * (d // 16)) % 16
        base = torch.zeros(n_pages, rows * (d + d // 16) + gap, dtype=torch.uint8, device="cuda")
        at = 0
        for name, w in widths:
            views[name] = base[:, at:at + rows * w].unflatten(1, (n_kv, page, w))
            at += rows * w
    else:
        for name, w in widths:
            shape = (n_pages, n_kv, page, w) if layout == "hnd" else (n_pages, page, n_kv, w)
            t = torch.zeros(shape, dtype=torch.uint8, device="cuda")
            views[name] = t if layout == "hnd" else t.transpose(1, 2)
    if fill is not None:
        for name, w in widths:
            t = views[name]
            lo, hi = (0, 256) if len(name) == 1 else fill
            t.copy_(torch.from_numpy(rng.integers(lo, hi, tuple(t.shape), dtype=np.uint8)))
    return qmm.KVCache(views["k"], views["v"], views["ks"], views["vs"]), views


@pytest.mark.parametrize("layout", ["hnd", "nhd", "block"])
@pytest.mark.parametrize("n,n_kv,d,page", [(1, 1, 32, 1), (5, 3, 96, 4), (33, 8, 64, 16), (300, 2, 160, 8), (64, 5, 256, 32),
                                           (17, 4, 128, 16), (9, 2, 192, 2), (40, 1, 224, 16)])
def test_append_is_exact(layout, n, n_kv, d, page):
    torch, qmm = _torch(), _qmm()
    gh.note(f"append mxfp4 {layout} n={n} n_kv={n_kv} d={d} page={page}")
    rng = np.random.default_rng(n * 7 + d)
    n_pages = -(-n // page) + 3
    cache, views = _new_cache(rng, n_pages, n_kv, page, d, layout, fill=(0, 256))
    slots = rng.permutation(n_pages * page)[:n].astype(np.int32)
    skip = rng.permutation(n)[: n // 4]
    slots[skip] = rng.choice([-1, -2 ** 31, n_pages * page, 2 ** 31 - 1], size=len(skip))
    fused = rng.normal(size=(n, (2 * n_kv + 1) * d)).astype(np.float32) * 3
    fused[0, :3] = [1e-9, -0.0, math.inf]
    dev = _dev(fused)
    k, v = (dev[:, i * n_kv * d:(i + 1) * n_kv * d] for i in range(2))
    want = {name: t.cpu().numpy().copy() for name, t in views.items()}
    for name, i in (("k", 0), ("v", 1)):
        q, e = mxfp4.quantize(fused[:, i * n_kv * d:(i + 1) * n_kv * d].reshape(n * n_kv, d))
        q, e = q.reshape(n, n_kv, -1), e.reshape(n, n_kv, -1)
        for j in np.nonzero((slots >= 0) & (slots < n_pages * page))[0]:
            p, a = divmod(int(slots[j]), page)
            want[name][p, :, a], want[name + "s"][p, :, a] = q[j], e[j]
    qmm.kv_append(cache, k.unflatten(1, (n_kv, d)) if n % 2 else k, v, _dev(slots))
    for name, t in views.items():
        assert np.array_equal(t.cpu().numpy(), want[name]), name


# ------------------------------------------------------------------ attention
def _case(lens, n_kv, group, d, page, layout="hnd", seed=0, tokens=0, scales=(122, 129), scale=None, q_mul=1.0):
    """Shuffled pages, room for `tokens` tokens per sequence; unused rows hold NaN scales, unused
    table entries pages outside the cache."""
    torch = _torch()
    rng = np.random.default_rng(seed + 17 * d + group)
    pages = [-(-n // page) for n in lens]
    n_pages = sum(pages) + 2
    cache, views = _new_cache(rng, n_pages, n_kv, page, d, layout, fill=scales)
    ids = rng.permutation(n_pages)
    table = rng.choice([-1, 2 ** 31 - 1, -2 ** 31, n_pages, 10 ** 6], size=(len(lens), max(max(pages) + 1, tokens // page)))
    at, used = 0, np.zeros((n_pages, page), bool)
    for i, (p, n) in enumerate(zip(pages, lens)):
        table[i, :p] = ids[at:at + p]
        for t in range(n):
            used[table[i, t // page], t % page] = True
        at += p
    for name in ("ks", "vs"):
        views[name].masked_fill_(_dev(~used)[:, None, :, None], 255)
    q = (rng.normal(size=(len(lens), n_kv * group, d)) * q_mul).astype(np.float32)
    host = {k: v.cpu().numpy() for k, v in views.items()}
    return dict(cache=cache, host=host, table=table.astype(np.int32), lens=list(lens), q=q, page=page,
                scale=d ** -0.5 if scale is None else scale)


def _want(c, i):
    t = np.arange(c["lens"][i])
    at = (c["table"][i][t // c["page"]], slice(None), t % c["page"])
    k, v = (mxfp4.dequantize(c["host"][n][at], c["host"][n + "s"][at]) for n in ("k", "v"))
    return step.attention(c["q"][i], k, v, c["scale"]) + (np.abs(k).max(initial=0), np.abs(v).max(initial=0))


def _flushed(n, vtop):
    """The oracle's bound is relative; a weight below f32's normal numbers may count as zero.  Weights
    are held as 2^-b of their size, 2^b < 2 n, so that is one below 2^(b - 126): n of them, times the
    largest value, over a sum of weights of at least 1."""
    return n * 2 * n * 2.0 ** -126 * vtop


def _check(c):
    torch, qmm = _torch(), _qmm()
    b, n_q, d = c["q"].shape
    lse = torch.empty(b, n_q, device="cuda")
    args = (_dev(c["q"]), c["cache"], _dev(c["table"]), torch.tensor(c["lens"], dtype=torch.int32, device="cuda"))
    out = qmm.paged_attention(*args, scale=c["scale"], lse=lse)
    assert torch.equal(out, qmm.paged_attention(*args, scale=c["scale"]))
    for i in range(b):
        want, wl, tol, top, vtop = _want(c, i)
        assert np.all(np.abs(out[i].cpu().numpy() - want) <= tol + _flushed(c["lens"][i], vtop)), i
        if c["lens"][i]:
            reach = abs(c["scale"]) * np.abs(c["q"][i]).sum(-1) * top
            assert np.all(np.abs(lse[i].cpu().numpy() - wl) <= step.lse_tol(wl, c["lens"][i], reach, d)), i
        else:
            assert np.isneginf(lse[i].cpu().numpy()).all()


@pytest.mark.parametrize("layout", ["hnd", "nhd", "block"])
@pytest.mark.parametrize("d", [32, 64, 96, 128, 160, 192, 224, 256])
def test_attention_every_head_dim(d, layout):
    gh.note(f"attention mxfp4 d={d} {layout}")
    _check(_case([1, 0, 33, 100, 31], 3, 2, d, 16, layout))
    _check(_case([700, 5, 0, 64], 2, 5, d, 8, layout, tokens=1024))


@pytest.mark.parametrize("group", [1, 3, 8, 16, 20])
@pytest.mark.parametrize("page", [1, 32, 128])
def test_attention_groups_and_pages(group, page):
    gh.note(f"attention mxfp4 group={group} page={page}")
    _check(_case([129, 1, 40], 2, group, 128, page))
    _check(_case([3000, 0, 77, 640], 1, group, 64, page, tokens=4096))


def test_attention_splits_and_many_units():
    _check(_case([20000], 2, 4, 128, 64))
    _check(_case([5 + 7 * (i % 40) for i in range(300)], 4, 2, 64, 16, tokens=2048))
    _check(_case([513] * 3, 8, 4, 128, 16, layout="nhd"))


def test_attention_scores_and_scales_far_apart():
    """Large scores, and blocks whose scales differ by many powers of two."""
    _check(_case([300, 90], 2, 4, 128, 16, scales=(100, 135), q_mul=0.05))
    _check(_case([300, 90], 2, 4, 64, 16, scales=(127, 131), q_mul=20.0))
    _check(_case([64], 1, 2, 96, 16, scales=(0, 40)))


@pytest.mark.parametrize("d", [64, 96, 128, 256])
@pytest.mark.parametrize("scale", [-0.25, 0.0, 2.0 ** -30])
def test_attention_query_blocks_far_apart(d, scale):
    """A query's block of 32 is kept to 2^-29 of its largest element, whatever the other blocks hold: a
    score is off by up to 2^-29 M sum|k| per block, M its largest |q|, which the oracle's (d + 12) 2^-24
    sum|q k| holds as long as M sum|k| is below 2^5 (d + 12) sum|q k|, here by far."""
    for page, tail in ((16, 37), (4, 6)):
        c = _case([tail, 0, 96 + tail], 2, 3, d, page, scales=(120, 127), scale=scale)
        c["q"] *= np.repeat(2.0 ** np.random.default_rng(d).integers(-25, 3, (3, 6, d // 32)), 32, axis=-1).astype(np.float32)
        _check(c)


def test_attention_query_that_is_not_finite():
    torch, qmm = _torch(), _qmm()
    for d in (32, 128, 160):
        c = _case([70, 40, 33], 2, 4, d, 16)
        args = lambda q: (_dev(q), c["cache"], _dev(c["table"]), torch.tensor(c["lens"], dtype=torch.int32, device="cuda"))  # noqa: E731
        good = qmm.paged_attention(*args(c["q"]))
        assert torch.isfinite(good).all()
        bad = c["q"].copy()
        bad[0, 1, 5], bad[1, 6, d - 1], bad[2, 0, 0] = np.inf, np.nan, -np.inf
        out = qmm.paged_attention(*args(bad))
        hit = torch.zeros(3, 8, dtype=torch.bool, device="cuda")
        hit[0, 1] = hit[1, 6] = hit[2, 0] = True
        assert not torch.isfinite(out[hit]).any() and torch.equal(out[~hit], good[~hit])


def test_attention_bad_data():
    torch, qmm = _torch(), _qmm()
    c = _case([70, 40, 30, 10], 2, 2, 64, 16)
    args = lambda table, lens: (_dev(c["q"]), c["cache"], _dev(np.asarray(table, np.int32)), torch.tensor(lens, dtype=torch.int32, device="cuda"))  # noqa: E731
    good = qmm.paged_attention(*args(c["table"], c["lens"]))
    bad = c["table"].copy()
    bad[1, 1] = 10 ** 8
    out = qmm.paged_attention(*args(bad, [70, 40, -3, 10 ** 6]))
    assert torch.equal(out[0], good[0]) and torch.isnan(out[1:]).all()
    # a NaN scale in a key row, in a value row: the heads that read it
    page, at = c["table"][0][1], 3
    c["cache"].k_scale[page, 0, at, 1] = 255
    out = qmm.paged_attention(*args(c["table"], c["lens"]))
    assert torch.isnan(out[0, :2]).all() and torch.equal(out[0, 2:], good[0, 2:]) and torch.equal(out[1:], good[1:])
    c["cache"].k_scale[page, 0, at, 1] = 120
    c["cache"].v_scale[page, 1, at, 0] = 255
    out = qmm.paged_attention(*args(c["table"], c["lens"]))
    assert torch.isnan(out[0, 2:, :32]).all() and torch.isfinite(out[0, 2:, 32:]).all()


# ------------------------------------------------------------------ together
def _layer(st, stream=None):
    """One attention block of a decode step in MXFP4, as a model runs it."""
    qmm = _qmm()
    kw = dict(stream=stream)
    q, e, s, h = qmm.add_rmsnorm_mxfp4(st["x"], st["norm"], st["r"], **kw)
    qkv = qmm.gemm_mxfp4(*st["w_qkv"], q, e, x_scale=s, **kw)
    n, d, nq, nkv = len(qkv), st["d"], st["n_q"], st["n_kv"]
    lens, slots, _, _ = qmm.paged_extend(st["table"], st["cached"], st["new"], st["free"], st["page"], n, **kw)
    k, v = (qkv[:, (nq + i * nkv) * d:(nq + (i + 1) * nkv) * d] for i in range(2))
    qmm.kv_append(st["cache"], k, v, slots, **kw)
    a = qmm.paged_attention(qkv[:, :nq * d], st["cache"], st["table"], lens, **kw)
    aq, ae = qmm.quantize_mxfp4(a, **kw)
    return qkv, a, qmm.gemm_mxfp4(*st["w_out"], aq, ae, **kw), h


def _layer_state(seed=0, batch=5, model=256, n_q=8, n_kv=2, d=64, page=16):
    torch, qmm = _torch(), _qmm()
    rng = np.random.default_rng(seed)
    cached = [0, 17, 40, 15, 31][:batch]
    have = [-(-c // page) for c in cached]
    cache, views = _new_cache(rng, 24, n_kv, page, d, "hnd", fill=(122, 127))
    ids = rng.permutation(24)
    table, at = np.full((batch, 5), -1), 0
    for i, p in enumerate(have):
        table[i, :p] = ids[at:at + p]
        at += p
    i32 = lambda v: torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")  # noqa: E731
    host = dict(x=rng.normal(size=(batch, model)).astype(np.float32), r=rng.normal(size=(batch, model)).astype(np.float32),
                norm=rng.normal(size=model).astype(np.float32), w_qkv=rng.normal(size=((n_q + 2 * n_kv) * d, model)),
                w_out=rng.normal(size=(model, n_q * d)), table=table, cached=cached,
                kv={k: v.cpu().numpy() for k, v in views.items()}, free=ids[at:])
    st = dict(x=_dev(host["x"]), r=_dev(host["r"]), norm=_dev(host["norm"]), table=i32(table), cached=i32(cached),
              new=i32([1] * batch), free=i32(ids[at:]), page=page, d=d, n_q=n_q, n_kv=n_kv, cache=cache)
    for name in ("w_qkv", "w_out"):
        host[name] = mxfp4.quantize(host[name].astype(np.float32))
        st[name] = tuple(_dev(a) for a in host[name])
    return st, host


def test_a_layer_matches_the_oracle_step_by_step():
    qmm, torch = _qmm(), _torch()
    st, host = _layer_state()
    qkv, a, y, h = (t.cpu().numpy() for t in _layer(st))
    h32 = host["x"] + host["r"]
    assert np.array_equal(h, h32)
    inv = step.rmsnorm(h32, host["norm"], 1e-5)[1][:, 0]
    want, tol = mxfp4.gemm(*host["w_qkv"], *mxfp4.quantize((h32 * host["norm"]).astype(np.float32)), inv)
    assert np.all(np.abs(qkv - want) <= tol + step.rmsnorm_rel(256) * np.abs(want))
    d, nq, nkv, page = st["d"], st["n_q"], st["n_kv"], st["page"]
    table, lens, slots, _, _ = step.extend(host["table"], host["cached"], [1] * 5, host["free"], page, 5)
    for i in range(5):
        for name, at in (("k", nq), ("v", nq + nkv)):
            cq, ce = mxfp4.quantize(qkv[i, at * d:(at + nkv) * d].reshape(nkv, d))
            host["kv"][name][slots[i] // page, :, slots[i] % page] = cq
            host["kv"][name + "s"][slots[i] // page, :, slots[i] % page] = ce
        t = np.arange(lens[i])
        k, v = (mxfp4.dequantize(host["kv"][n][table[i][t // page], :, t % page], host["kv"][n + "s"][table[i][t // page], :, t % page])
                for n in ("k", "v"))
        out, _, tol = step.attention(qkv[i, :nq * d].reshape(nq, d), k, v, d ** -0.5)
        assert np.all(np.abs(a[i].reshape(nq, d) - out) <= tol + _flushed(len(k), np.abs(v).max()))
    want, tol = mxfp4.gemm(*host["w_out"], *mxfp4.quantize(a))
    assert np.all(np.abs(y - want) <= tol)


def test_a_layer_on_another_stream_and_in_a_graph():
    torch = _torch()
    st, _ = _layer_state(seed=3)
    eager = [t.clone() for t in _layer(st)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = _layer(st, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, other))
    with torch.cuda.stream(side):
        _layer(st)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            held = _layer(st)
    for i in range(3):
        st["x"].mul_(-1.5 if i else 1.0)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        assert all(torch.equal(a, b) for a, b in zip(got, _layer(st)))
        torch.cuda.synchronize()


def test_python_refusals():
    torch, qmm = _torch(), _qmm()
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")  # noqa: E731
    f32 = lambda *s: torch.zeros(s, device="cuda")  # noqa: E731
    x = f32(4, 64)
    for call, error in (
        (lambda: qmm.quantize_mxfp4(x.double()), TypeError), (lambda: qmm.quantize_mxfp4(x[0]), (ValueError, IndexError)),
        (lambda: qmm.quantize_mxfp4(f32(4, 48)), qmm.QmmError), (lambda: qmm.quantize_mxfp4(x.t()), ValueError),
        (lambda: qmm.quantize_mxfp4(x, q=u8(4, 16)), ValueError), (lambda: qmm.quantize_mxfp4(x, e=u8(4, 3)), ValueError),
        (lambda: qmm.dequantize_mxfp4(u8(4, 32), u8(4, 1)), ValueError), (lambda: qmm.dequantize_mxfp4(u8(4, 32), u8(3, 2)), ValueError),
        (lambda: qmm.dequantize_mxfp4(x, u8(4, 2)), TypeError), (lambda: qmm.dequantize_mxfp4(u8(4, 32), u8(4, 2), out=f32(4, 32)), ValueError),
        (lambda: qmm.gemm_mxfp4(u8(8, 32), u8(8, 2), u8(4, 48), u8(4, 3)), ValueError),
        (lambda: qmm.gemm_mxfp4(u8(8, 32), u8(8, 2), u8(4, 32), u8(4, 2), x_scale=f32(5)), ValueError),
        (lambda: qmm.gemm_mxfp4(u8(8, 32), u8(8, 2), u8(4, 32), u8(4, 2), out=f32(4, 9)), ValueError),
        (lambda: qmm.gemm_mxfp4(u8(8, 32), u8(8, 2), u8(2, 2, 32), u8(2, 2, 2), out=f32(4, 8)), ValueError),
        (lambda: qmm.gemm_mxfp4(u8(64)[16:48].view(1, 32)[:, :32], u8(1, 2), u8(65)[1:33].view(1, 32), u8(1, 2)), qmm.QmmError),
        (lambda: qmm.add_rmsnorm_mxfp4(x, f32(32)), ValueError), (lambda: qmm.add_rmsnorm_mxfp4(x, f32(64), s=f32(3)), ValueError),
        (lambda: qmm.KVCache(u8(2, 1, 16, 16), u8(2, 1, 16, 16)), ValueError),
        (lambda: qmm.KVCache(u8(2, 1, 16, 16), u8(2, 1, 16, 16), u8(2, 1, 16, 2), u8(2, 1, 16, 2)), ValueError),
        (lambda: qmm.KVCache(u8(2, 1, 16, 16), u8(2, 1, 16, 16), f32(2, 1, 16, 1), f32(2, 1, 16, 1)), TypeError),
    ):
        with pytest.raises(error):
            call()
