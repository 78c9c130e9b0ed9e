"""MXFP4 on the GPU at the edges of what its header allows: attention scales, scores and queries,
products and arrays that pass a launch's limits, every kernel's tails, operands that are missing."""

from __future__ import annotations

import numpy as np
import pytest

import gpu_helpers as gh
from oracle import mxfp4, step
from test_gpu_mxfp4 import _case, _check, _dev, _flushed, _layer, _layer_state, _qmm, _torch, _want

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


def test_attention_heads_do_not_touch_each_other():
    """A head whose scores are far larger leaves the others' bits as they are."""
    torch, qmm = _torch(), _qmm()
    for page, tokens in ((16, 0), (4, 1024)):
        c = _case([700 if tokens else 70, 33], 2, 4, 64, page, tokens=tokens, scale=0.125)
        args = (c["cache"], _dev(c["table"]), torch.tensor(c["lens"], dtype=torch.int32, device="cuda"))
        alone = qmm.paged_attention(_dev(c["q"]), *args, scale=0.125)
        for head in (0, 3, 6):
            q = c["q"].copy()
            q[:, head] *= np.float32(2.0 ** 40)
            out = qmm.paged_attention(_dev(q), *args, scale=0.125)
            keep = [h for h in range(8) if h != head]
            assert torch.isfinite(out).all() and torch.equal(out[:, keep], alone[:, keep])


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
    (2.0 ** 126, 2.0 ** 118, (0, 1)),
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
    (2.0 ** -149, 2.0 ** 120, 2.0 ** 26), (2.0 ** 126, 2.0 ** 118, 2.0 ** -125),
    (0.0, 2.0 ** 60, 1.0), (0.125, 2.0 ** 33, 1.0), (-0.125, 2.0 ** 100, 1.0)])
def test_attention_bf16_any_scale(scale, q_mul, k_mul):
    """The same of a bfloat16 cache."""
    import test_gpu_step as of_step
    gh.note(f"attention bf16 scale {scale} q*{q_mul} k*{k_mul}")
    for lens, tokens in (([70, 1, 0, 33], 0), ([700, 90], 1024)):
        c = of_step._case("bf16", lens, 2, 4, 64, 16, tokens=tokens, scale=scale, q_mul=q_mul)
        k = c["cache"].k
        k.copy_(_torch().where(_torch().isfinite(k), k.float() * k_mul, k.float()))
        of_step._check(c)


@pytest.mark.parametrize("kind,scale,q_mul,kv_mul", [("f16", 2.0 ** 118, 2.0 ** 16, 2.0 ** -16), ("f16", -2.0 ** 30, 2.0 ** 100, 2.0 ** -14),
                                                     ("q8", 2.0 ** 118, 2.0 ** 16, 2.0 ** -16), ("q8", 2.0 ** 20, 2.0 ** 110, 2.0 ** -12)])
def test_attention_f16_and_8_bit_largest_products_of_scale_and_query(kind, scale, q_mul, kv_mul):
    import test_gpu_step as of_step
    gh.note(f"attention {kind} scale {scale} q*{q_mul}")
    for lens, tokens in (([70, 1, 0, 33], 0), ([700, 90], 1024)):
        of_step._check(of_step._case(kind, lens, 2, 4, 64, 16, tokens=tokens, scale=scale, q_mul=q_mul, kv_mul=kv_mul))


@pytest.mark.parametrize("far", [2.0 ** 6, 2.0 ** 10, 2.0 ** 14, 2.0 ** 20])
@pytest.mark.parametrize("d", [32, 96, 128, 256])
def test_attention_one_large_query_element(d, far):
    """One element of a block many times the others, where most keys hold a zero: an element is kept
    to 2^-29 of its block's largest, so a token's score is off by E = |scale| 2^-29 sum over blocks of
    max|q| sum|k| beside what the oracle allows, a weight by the factor exp(E), an output by
    (exp(2 E) - 1) max|v|, the log-sum-exp by E."""
    gh.note(f"attention mxfp4 d={d} an element *{far}")
    torch, qmm = _torch(), _qmm()
    for page in (16, 2):
        c = _case([70, 0, 33, 100], 2, 3, d, page, scales=(118, 123))
        at = (7 + 32 * np.arange(d // 32)) % d
        c["q"][:, :, at] *= np.float32(far)
        codes = c["host"]["k"]
        codes[..., at // 2] &= np.where(at % 2, 0x0f, 0xf0).astype(np.uint8)       # their keys' codes
        first = c["table"][0][0]
        codes[first, :, 1, at[0] // 2] |= np.uint8(2 << 4 * (at[0] % 2))           # but one
        c["cache"].k.copy_(_dev(codes))
        lse = torch.empty(4, 6, device="cuda")
        out = qmm.paged_attention(_dev(c["q"]), c["cache"], _dev(c["table"]),
                                  torch.tensor(c["lens"], dtype=torch.int32, device="cuda"), scale=c["scale"], lse=lse)
        for i, n in enumerate(c["lens"]):
            if n == 0:
                continue
            want, wl, tol, top, vtop = _want(c, i)
            t = np.arange(n)
            where = (c["table"][i][t // c["page"]], slice(None), t % c["page"])
            k = np.abs(mxfp4.dequantize(c["host"]["k"][where], c["host"]["ks"][where])).reshape(n, 2, d // 32, 32).sum(-1)
            m = np.abs(c["q"][i].astype(np.float64)).reshape(6, d // 32, 32).max(-1)
            e = 2.0 ** -29 * c["scale"] * (k[:, np.arange(6) // 3] * m).sum(-1).max(0)       # of each head
            assert np.all(np.abs(out[i].cpu().numpy() - want) <= tol + (np.expm1(2 * e) * vtop)[:, None]), i
            reach = c["scale"] * np.abs(c["q"][i]).sum(-1) * top
            assert np.all(np.abs(lse[i].cpu().numpy() - wl) <= step.lse_tol(wl, n, reach, d) + e), i


# ------------------------------------------------------------------ product
def _exact_check(m, k, n, seed=0, nan=True):
    """A product whose sums are exact (scales 1 and 2: multiples of 1/4, below 2^24 / 4)."""
    torch, qmm = _torch(), _qmm()
    rng = np.random.default_rng(seed + m * 7 + k + n)
    w, x = (rng.integers(0, 256, (r, k // 2), dtype=np.uint8) for r in (m, n))
    we, xe = (rng.integers(127, 129, (r, k // 32), dtype=np.uint8) for r in (m, n))
    out = torch.full((n + 1, m + 3), 7.0, device="cuda")
    qmm.gemm_mxfp4(_dev(w), _dev(we), _dev(x), _dev(xe), out=out[:n, :m])
    got = out.cpu().numpy()
    assert np.array_equal(got[:n, :m], mxfp4.gemm(w, we, x, xe)[0]), (m, k, n)
    assert (got[n] == 7).all() and (got[:, m:] == 7).all()
    if nan:         # a NaN scale at a row's and a token's end stays in them
        we[m // 2, -1] = xe[n // 2, -1] = 255
        got = qmm.gemm_mxfp4(*(_dev(a) for a in (w, we, x, xe))).cpu().numpy()
        bad = np.zeros((n, m), bool)
        bad[n // 2] = bad[:, m // 2] = True
        assert np.array_equal(np.isnan(got), bad), (m, k, n)


@pytest.mark.parametrize("kernel", range(11))
def test_gemm_every_kernel_where_each_can_run(kernel, monkeypatch):
    """k in whole 64s, which every kernel takes (8 and 9 take no other): whole passes and then part of
    one, in rows and tokens that end inside a tile."""
    monkeypatch.setenv("QMM_MX_KERNEL", str(kernel))
    for m, k, n in [(33, 320, 35), (1, 1088, 1), (47, 2112, 17), (130, 576, 70), (300, 1344, 257), (16, 4160, 33),
                    (31, 192, 64), (70, 3136, 290), (513, 640, 45)]:
        gh.note(f"gemm_mxfp4 kernel {kernel} {m}x{k} n={n}")
        _exact_check(m, k, n)


@pytest.mark.parametrize("kernel", [None, 5, 7, 8, 10])
def test_gemm_more_token_tiles_than_a_grid_axis(kernel, monkeypatch):
    """2^20 tokens are 65536 tiles of 16, one more than a grid's second axis takes: for one row and this
    k kernel 10 would be the fastest, and 8 and 10 may not be forced either."""
    if kernel is not None:
        monkeypatch.setenv("QMM_MX_KERNEL", str(kernel))
    torch, qmm = _torch(), _qmm()
    n, k = 1 << 20, 1024
    gh.note(f"gemm_mxfp4 kernel {kernel} 1x{k} n={n}")
    torch.manual_seed(5)
    w, x = (torch.randint(0, 256, (r, k // 2), dtype=torch.uint8, device="cuda") for r in (1, n))
    we, xe = (torch.randint(127, 129, (r, k // 32), dtype=torch.uint8, device="cuda") for r in (1, n))
    got = qmm.gemm_mxfp4(w, we, x, xe)
    want = torch.cat([(qmm.dequantize_mxfp4(x[i:i + 65536], xe[i:i + 65536]) * qmm.dequantize_mxfp4(w, we)).sum(1)
                      for i in range(0, n, 65536)])
    assert torch.equal(got[:, 0], want)


@pytest.mark.parametrize("kernel", [None, 5, 7, 8, 10])
def test_gemm_more_tiles_than_a_grid(kernel, monkeypatch):
    """66000 x 66000 outputs are 4125^2 tiles of 16 x 16 or half as many of 32 x 16, more than the 2^22
    work groups that a launch takes (2^32 threads and more of the smallest): those kernels leave it to
    others."""
    if kernel is not None:
        monkeypatch.setenv("QMM_MX_KERNEL", str(kernel))
    torch, qmm = _torch(), _qmm()
    m = n = 66000
    gh.note(f"gemm_mxfp4 kernel {kernel} {m}x64 n={n}")
    torch.manual_seed(6)
    w, x = (torch.randint(0, 256, (r, 32), dtype=torch.uint8, device="cuda") for r in (m, n))
    we, xe = (torch.randint(127, 129, (r, 2), dtype=torch.uint8, device="cuda") for r in (m, n))
    out = torch.full((n, m), float("nan"), device="cuda")
    qmm.gemm_mxfp4(w, we, x, xe, out=out)
    assert not torch.isnan(out).any()
    wf, xf = qmm.dequantize_mxfp4(w, we), qmm.dequantize_mxfp4(x, xe)
    at = torch.randint(0, n, (24,)).tolist() + [0, 15, 16, 32767, 32768, 65535, 65536, n - 1]
    for i in at:
        assert torch.equal(out[i], (wf * xf[i]).sum(1)), i
        assert torch.equal(out[:, i], (xf * wf[i]).sum(1)), i


@pytest.mark.parametrize("n", [3, 40, 300])
def test_gemm_codes_of_zero_under_far_scales(n):
    """0 times anything is 0, whatever the two scales' product: 2^254 where all codes of one side are
    zero, beside blocks of ordinary size."""
    torch, qmm = _torch(), _qmm()
    rng = np.random.default_rng(n)
    m, k = 70, 1152
    w, x = (rng.integers(0, 256, (r, k // 2), dtype=np.uint8) for r in (m, n))
    we, xe = (rng.integers(127, 129, (r, k // 32), dtype=np.uint8) for r in (m, n))
    for blk in range(0, k // 32, 3):
        we[:, blk] = xe[:, blk] = 254
        (w if blk % 2 else x)[:, 16 * blk:16 * blk + 16] &= 0x88        # zeros of either sign
    want = mxfp4.gemm(w, we, x, xe)[0]
    assert np.isfinite(want).all() and np.array_equal(qmm.gemm_mxfp4(*(_dev(a) for a in (w, we, x, xe))).cpu().numpy(), want)


# ------------------------------------------------------------------ cache
@pytest.mark.parametrize("page,n_pages,strides,scale_strides,at", [
    # pages a GiB apart, up to the 64 GiB that a cache may span: codes of both, then scales of both, in each
    (16, 63, (1 << 30, 1 << 12, 64), (1 << 30, 1 << 12, 16), (0, 1 << 28, 1 << 29, 3 << 28)),
    (4, 63, (1 << 30, 1 << 12, 64), (1 << 30, 1 << 12, 16), (0, 1 << 28, 1 << 29, 3 << 28)),
    # a page's tokens 128 MiB apart and a little less, beside and within what 32-bit offsets of 16 rows take
    (16, 4, (1 << 16, 1 << 12, 1 << 27), (1 << 16, 1 << 12, 1 << 27), (0, 1 << 20, 1 << 21, 3 << 20)),
    (16, 4, (1 << 16, 1 << 12, (1 << 27) - 64), (1 << 16, 1 << 12, (1 << 27) - 63), (0, 1 << 20, 1 << 21, 3 << 20)),
    (32, 4, (1 << 16, 1 << 12, (1 << 27) - 64), (1 << 16, 1 << 12, (1 << 27) - 63), (0, 1 << 20, 1 << 21, 3 << 20)),
])
def test_rows_far_apart(page, n_pages, strides, scale_strides, at):
    """Append and attention where rows and scales are as far apart as a cache may hold them."""
    torch, qmm = _torch(), _qmm()
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("less than 80 GiB of device memory free")
    gh.note(f"mxfp4 cache page {page} x {n_pages} strides {strides}")
    n_kv, group, d = 2, 3, 96
    sizes = (n_pages, n_kv, page)
    reach = max(sum((n - 1) * s for n, s in zip(sizes, st)) for st in (strides, scale_strides)) + max(at) + d
    base = torch.empty(reach, dtype=torch.uint8, device="cuda")
    k, v, ks, vs = (base.as_strided(sizes + (w,), st + (1,), o) for w, st, o in
                    zip((d // 2, d // 2, d // 32, d // 32), (strides, strides, scale_strides, scale_strides), at))
    cache = qmm.KVCache(k, v, ks, vs)
    rng = np.random.default_rng(page + n_pages)
    lens = [n_pages * page // 2 - 5, 7, n_pages * page // 4]
    pages = [-(-n // page) for n in lens]
    ids = rng.permutation(n_pages)
    ids = np.concatenate([[n_pages - 1, 0], ids[(ids != 0) & (ids != n_pages - 1)]])
    table, slots, used = np.full((3, max(pages)), -1, np.int32), [], 0
    for i, (n, p) in enumerate(zip(lens, pages)):
        table[i, :p] = ids[used:used + p]
        used += p
        t = np.arange(n)
        slots.append(table[i][t // page] * page + t % page)
    slots = np.concatenate(slots).astype(np.int32)
    kv = rng.normal(size=(2, len(slots), n_kv, d)).astype(np.float32)
    qmm.kv_append(cache, _dev(kv[0]), _dev(kv[1]), _dev(slots))
    p, s = _dev(slots // page).long(), _dev(slots % page).long()
    held = []
    for rows, codes, scales in ((kv[0], k, ks), (kv[1], v, vs)):
        wq, we = mxfp4.quantize(rows.reshape(-1, d))
        assert np.array_equal(codes[p, :, s].cpu().numpy().reshape(-1, d // 2), wq)
        assert np.array_equal(scales[p, :, s].cpu().numpy().reshape(-1, d // 32), we)
        held.append(mxfp4.dequantize(wq, we).reshape(rows.shape))
    q = rng.normal(size=(3, n_kv * group, d)).astype(np.float32)
    out = qmm.paged_attention(_dev(q), cache, _dev(table), torch.tensor(lens, dtype=torch.int32, device="cuda")).cpu().numpy()
    first = 0
    for i, n in enumerate(lens):
        want, _, tol = step.attention(q[i], held[0][first:first + n], held[1][first:first + n], d ** -0.5)
        assert np.all(np.abs(out[i] - want) <= tol + _flushed(n, np.abs(held[1]).max())), i
        first += n


# ------------------------------------------------------------------ quantization
def test_quantize_more_items_than_a_grid():
    """2^35 values and some are four times as many items of eight as a launch has threads, and more than
    32 bits count; 2^33 values back are twice as many items of four."""
    torch, qmm = _torch(), _qmm()
    k = 1 << 16
    rows = (1 << 19) + 3
    if torch.cuda.mem_get_info()[0] < 120 << 30:
        pytest.skip("less than 120 GiB of device memory free")
    gh.note(f"quantize bfloat16 {rows}x{k}")
    gen = torch.Generator(device="cuda").manual_seed(3)
    some = torch.randn(4099, k, device="cuda", generator=gen).bfloat16()       # rows that repeat at no power of two
    x = torch.empty(rows, k, dtype=torch.bfloat16, device="cuda")
    for i in range(0, rows, 4099):
        x[i:i + 4099] = some[:rows - i]
    q, e = qmm.quantize_mxfp4(x)
    del x
    sq, se = qmm.quantize_mxfp4(some)           # a launch of one step
    for i in range(0, rows, 4099):
        assert torch.equal(q[i:i + 4099], sq[:rows - i]) and torch.equal(e[i:i + 4099], se[:rows - i]), i
    wq, we = mxfp4.quantize(some[:2, :4096].float().cpu().numpy())
    assert np.array_equal(sq[:2, :2048].cpu().numpy(), wq) and np.array_equal(se[:2, :128].cpu().numpy(), we)
    rows = (1 << 17) + 3
    gh.note(f"dequantize {rows}x{k}")
    back, want = qmm.dequantize_mxfp4(q[:rows], e[:rows]), qmm.dequantize_mxfp4(sq, se)
    for i in range(0, rows, 4099):
        assert torch.equal(back[i:i + 4099], want[:rows - i]), i


# ------------------------------------------------------------------ together
def test_layers_at_the_same_time_and_in_two_graphs():
    """Three layers with inputs of their own on three streams at once, and two graphs replayed in turn:
    each as it is alone."""
    torch = _torch()
    states = [_layer_state(seed=s)[0] for s in (11, 12, 13)]
    alone = [[t.clone() for t in _layer(st)] for st in states]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in states]
    for _ in range(5):
        got = [_layer(st, stream=s) for st, s in zip(states, streams)]
        torch.cuda.synchronize()
        for mine, want in zip(got, alone):
            assert all(torch.equal(a, b) for a, b in zip(mine, want))
    graphs = []
    for st, s in zip(states[:2], streams):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            held = _layer(st)
        graphs.append((graph, held))
    for _ in range(3):
        for graph, _held in graphs:
            graph.replay()
        again = _layer(states[2])
        torch.cuda.synchronize()
        for mine, want in zip([held for _, held in graphs] + [again], alone):
            assert all(torch.equal(a, b) for a, b in zip(mine, want))


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
