"""The decode-step operators on the GPU against the f64 oracle: page tables, cache rows, paged
attention, RMS norm, alone and as one decode step."""

from __future__ import annotations

import math

import numpy as np
import pytest

import gpu_helpers as gh
from oracle import formats, ref, step
from synth import gen

pytestmark = pytest.mark.gpu

KINDS = ("f16", "bf16", "q8")


def _torch():
    import torch
    return torch


def _qmm():
    import gemv_prefill_decode_amd as qmm
    return qmm


# ------------------------------------------------------------------ page tables
def _check_extend(table, cached, new, free, page, n_rows):
    torch, qmm = _torch(), _qmm()
    gh.note(f"extend batch={len(cached)} page={page} rows={n_rows} free={len(free)}")
    want = step.extend(table, cached, new, free, page, n_rows)
    dev = [torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda") for v in (table, cached, new, free)]
    for _ in range(2):                  # the call may be repeated
        got = qmm.paged_extend(dev[0], dev[1], dev[2], dev[3], page, n_rows)
        for g, w in zip((dev[0],) + got, want[:4] + (np.array([want[4]]),)):
            assert np.array_equal(g.cpu().numpy(), w)


@pytest.mark.parametrize("batch,page,most,fresh,short", [
    (1, 1, 5, 1, 0), (1, 16, 0, 40, 0), (3, 4, 20, 9, 0), (64, 16, 500, 1, 0), (65, 32, 300, 33, 5), (1023, 8, 60, 3, 0),
    (1024, 16, 40, 2, 100), (1025, 64, 200, 1, 0), (2500, 2, 9, 7, 700), (7, 128, 5000, 3000, 0),
])
def test_extend_matches_the_oracle(batch, page, most, fresh, short):
    rng = np.random.default_rng(batch * 131 + page)
    cached, new = rng.integers(0, most + 1, batch), rng.integers(0, fresh + 1, batch)
    width = -(-(most + fresh) // page) + 1
    ids = rng.permutation(batch * width + 10)
    table = np.full((batch, width), -1)
    at = 0
    for i in range(batch):
        have = -(-int(cached[i]) // page)
        table[i, :have] = ids[at:at + have]
        at += have
    need = int((-(-(cached + new) // page) - -(-cached // page)).sum())
    _check_extend(table, cached, new, ids[at:at + max(0, need - short)], page, int(new.sum()) + 37)


def test_extend_refused_sequences_and_short_rows():
    # negative lengths, a row that is too short, a free list that runs dry in the middle, a negative page
    table = [[0, 1, -1], [2, -1, -1], [3, 4, 5], [-7, -1, -1], [6, -1, -1], [7, -1, -1]]
    cached, new = [17, -3, 40, 3, 4, 1000], [20, 5, 10, 2, 60, 2 ** 31 - 1]
    _check_extend(table, cached, new, [9, 8, 11], 16, 300)
    _check_extend(table, cached[:2] + [40, 3, 4, 5], [20, -5, 8, 2, 60, 30], [9], 16, 90)
    _check_extend(table, [0] * 6, [0] * 6, [], 16, 0)


def test_extend_writes_nothing_behind_its_outputs():
    torch, qmm = _torch(), _qmm()
    big = torch.full((4, 9), -5, dtype=torch.int32, device="cuda")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    rows = torch.full((64,), -5, dtype=torch.int32, device="cuda")
    _, slots, pos, _ = qmm.paged_extend(big[:3, :4], i32(0, 0, 0), i32(5, 6, 7), i32(1, 2, 3, 4, 5, 6), 4, 12,
                                        slots=rows[:12], positions=rows[32:44])
    assert (big[3] == -5).all() and (big[:3, 4:] == -5).all() and (rows[12:32] == -5).all() and (rows[44:] == -5).all()
    assert pos.tolist() == [0, 1, 2, 3, 4, 0, 1, 2, 3, 4, 5, 0]     # the rows past n_rows are dropped
    assert slots.tolist() == [4, 5, 6, 7, 8, 12, 13, 14, 15, 16, 17, 20]


# ------------------------------------------------------------------ caches
def _new_cache(kind, n_pages, n_kv, page, d, layout="hnd", fill=None, rng=None):
    """(KVCache, dense) with dense(name) the cache's values f64 [n_pages, n_kv, page, d]."""
    torch, qmm = _torch(), _qmm()
    dt = {"f16": torch.float16, "bf16": torch.bfloat16, "q8": torch.int8}[kind]
    if layout == "both":            # keys and values of a page side by side
        base = torch.zeros(n_pages, 2, n_kv, page, d, dtype=dt, device="cuda")
        views = [base[:, 0], base[:, 1]]
    elif layout == "nhd":
        views = [torch.zeros(n_pages, page, n_kv, d, dtype=dt, device="cuda").transpose(1, 2) for _ in range(2)]
    else:
        views = [torch.zeros(n_pages, n_kv, page, d, dtype=dt, device="cuda") for _ in range(2)]
    scales = []
    if kind == "q8":
        for _ in range(2):
            s = torch.zeros(n_pages, n_kv, page, device="cuda")
            scales.append(s if layout != "nhd" else torch.zeros(n_pages, page, n_kv, device="cuda").transpose(1, 2))
    if rng is not None:
        for i, t in enumerate(views):
            x = rng.normal(size=t.shape).astype(np.float32) * (fill or 1.0)
            if kind == "q8":
                codes, d0 = step.q8_rows(x, d)
                t.copy_(torch.from_numpy(codes))
                scales[i].copy_(torch.from_numpy(d0[..., 0]))
            else:
                t.copy_(torch.from_numpy(x))
    cache = qmm.KVCache(*views, *scales)

    def dense(which):
        t = views[which].cpu().double().numpy()
        return t if kind != "q8" else t * scales[which].cpu().double().numpy()[..., None]
    return cache, dense


@pytest.mark.parametrize("layout", ["hnd", "nhd", "both"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n,n_kv,d,page", [(1, 1, 32, 1), (5, 3, 96, 4), (33, 8, 64, 16), (300, 2, 160, 8), (64, 5, 256, 32),
                                           (17, 4, 128, 16), (9, 2, 192, 2), (40, 1, 224, 16)])
def test_append_is_exact(kind, layout, n, n_kv, d, page):
    torch, qmm = _torch(), _qmm()
    gh.note(f"append {kind} {layout} n={n} n_kv={n_kv} d={d} page={page}")
    rng = np.random.default_rng(n * 7 + d)
    n_pages = -(-n // page) + 3
    cache, _ = _new_cache(kind, n_pages, n_kv, page, d, layout, rng=rng)
    slots = rng.permutation(n_pages * page)[:n].astype(np.int32)
    skip = rng.permutation(n)[: n // 4]
    slots[skip] = rng.choice([-1, -2 ** 31, n_pages * page, 2 ** 31 - 1], size=len(skip))
    fused = torch.from_numpy(rng.normal(size=(n, (2 * n_kv + 1) * d)).astype(np.float32) * 3).cuda()
    fused[0, :3] = torch.tensor([1e-9, 0.0, -70000.0])      # f16: subnormal to zero, and out of range
    k, v = (fused[:, i * n_kv * d:(i + 1) * n_kv * d] for i in range(2))
    want = []
    live = (slots >= 0) & (slots < n_pages * page)
    for t, s, new in ((cache.k, cache.k_scale, k), (cache.v, cache.v_scale, v)):
        w, ws = t.clone().cpu(), None if s is None else s.clone().cpu()
        x = new.reshape(n, n_kv, d).cpu()
        for j in np.nonzero(live)[0]:
            p, a = divmod(int(slots[j]), page)
            if kind == "q8":
                codes, d0 = step.q8_rows(x[j].numpy(), d)
                w[p, :, a], ws[p, :, a] = torch.from_numpy(codes), torch.from_numpy(d0[:, 0])
            else:
                w[p, :, a] = x[j].to(w.dtype)
        want.append((w, ws))
    qmm.kv_append(cache, k.unflatten(1, (n_kv, d)) if n % 2 else k, v, torch.from_numpy(slots).cuda())
    for (w, ws), t, s in zip(want, (cache.k, cache.v), (cache.k_scale, cache.v_scale)):
        assert torch.equal(t.cpu(), w)
        if s is not None:
            assert torch.equal(s.cpu(), ws)


# ------------------------------------------------------------------ attention
def _case(kind, lens, n_kv, group, d, page, layout="hnd", seed=0, scale=None, q_mul=1.0, kv_mul=1.0, stale=True,
          tokens=0):
    """Inputs of a paged attention with shuffled pages and room for `tokens` tokens per sequence
    (a table for more than 512 makes the kernel split the tokens between work groups); stale table
    entries and unwritten rows are hostile: page ids far outside the cache, NaN and infinity."""
    torch = _torch()
    rng = np.random.default_rng(seed + 17 * d + group)
    pages = [-(-n // page) for n in lens]
    n_pages = sum(pages) + 2
    cache, dense = _new_cache(kind, n_pages, n_kv, page, d, layout, fill=kv_mul, rng=rng)
    ids = rng.permutation(n_pages)
    width = max(max(pages) + 1, tokens // page)
    table = rng.choice([-1, 2 ** 31 - 1, -2 ** 31, n_pages, 10 ** 6], size=(len(lens), width)).astype(np.int32)
    at, used = 0, np.zeros((n_pages, page), bool)
    for i, (p, n) in enumerate(zip(pages, lens)):
        table[i, :p] = ids[at:at + p]
        for t in range(n):
            used[table[i, t // page], t % page] = True
        at += p
    if stale:
        dead = torch.from_numpy(~used).cuda()
        for t, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
            if s is not None:
                s.masked_fill_(dead[:, None], math.nan)
            else:
                t.masked_fill_(dead[:, None, :, None], math.nan)
                t.masked_fill_(dead[:, None, :, None] & (torch.arange(d, device="cuda") % 3 == 1), math.inf)
    q = torch.from_numpy((rng.normal(size=(len(lens), n_kv * group, d)) * q_mul).astype(np.float32)).cuda()
    return dict(cache=cache, dense=dense, table=table, lens=list(lens), q=q, page=page, d=d, n_kv=n_kv,
                scale=d ** -0.5 if scale is None else scale)


def _rows(c, which, i, n):
    t = np.arange(n)
    return c["dense"](which)[c["table"][i][t // c["page"]], :, t % c["page"]]


def _want(c):
    k, v = c["dense"](0), c["dense"](1)
    out = []
    for i, n in enumerate(c["lens"]):
        t = np.arange(n)
        at = (c["table"][i][t // c["page"]], slice(None), t % c["page"])
        out.append(step.attention(c["q"][i].cpu().numpy(), k[at], v[at], c["scale"]))
    return out


def _run(c, **kw):
    torch, qmm = _torch(), _qmm()
    b, hq, _ = c["q"].shape
    lse = torch.full((b, hq), 7.0, device="cuda")
    out = qmm.paged_attention(c["q"], c["cache"], torch.from_numpy(c["table"]).cuda(),
                              torch.tensor(c["lens"], dtype=torch.int32, device="cuda"), scale=c["scale"], lse=lse, **kw)
    return out.cpu().double().numpy(), lse.cpu().double().numpy()


def _check(c, got=None):
    out, lse = _run(c) if got is None else got
    q = np.abs(c["q"].cpu().double().numpy())
    worst = 0.0
    for i, (w, wl, tol) in enumerate(_want(c)):
        n = c["lens"][i]
        if n == 0:
            assert not out[i].any() and (lse[i] == -np.inf).all()
            continue
        err = np.abs(out[i] - w)
        assert np.isfinite(out[i]).all(), f"sequence {i} ({n} tokens)"
        assert (err <= tol).all(), f"sequence {i} ({n} tokens): {np.max(err / np.maximum(tol, 1e-300)):.3g} of the bound"
        worst = max(worst, float(np.max(err / np.maximum(tol, 1e-300))))
        reach = abs(c["scale"]) * q[i].sum(axis=1) * np.abs(_rows(c, 0, i, n)).max()
        assert (np.abs(lse[i] - wl) <= step.lse_tol(wl, n, reach, c["d"])).all()
    return worst


LENS = [0, 1, 2, 31, 32, 33, 64, 65, 130, 0]


@pytest.mark.parametrize("tokens", [0, 9000])
@pytest.mark.parametrize("d", range(32, 257, 32))
@pytest.mark.parametrize("kind", KINDS)
def test_attention_every_head_dim(kind, d, tokens):
    gh.note(f"attention {kind} d={d} table for {tokens}")
    print("worst of the bound", _check(_case(kind, LENS, 2, 3, d, 16, tokens=tokens)))


@pytest.mark.parametrize("tokens", [0, 9000])
@pytest.mark.parametrize("group", [1, 2, 4, 8, 15, 16, 17, 20, 33])
@pytest.mark.parametrize("kind", KINDS)
def test_attention_every_group(kind, group, tokens):
    gh.note(f"attention {kind} group={group} table for {tokens}")
    _check(_case(kind, LENS, 2, group, 64, 8, "nhd", tokens=tokens))


@pytest.mark.parametrize("n_kv,batch,n", [(1, 1, 1), (1, 1, 40), (3, 1, 513), (8, 7, 129), (5, 3, 1000), (8, 64, 96), (2, 600, 33),
                                          (16, 40, 260)])
def test_attention_joins_of_every_kind(n_kv, batch, n):
    """From one unit over all work groups to many units per wave: a unit whole in a wave, joined in
    a work group, and over work groups by the wide and the narrow join, at the edges of chunks."""
    gh.note(f"attention n_kv={n_kv} batch={batch} n={n}")
    lens = [max(0, n - 13 * (i % 5)) for i in range(batch)]
    _check(_case("f16", lens, n_kv, 2, 32, 16, tokens=2000, seed=batch))


@pytest.mark.parametrize("page", [1, 2, 4, 8, 16, 32, 64, 128, 512])
@pytest.mark.parametrize("layout", ["hnd", "nhd", "both"])
def test_attention_pages_and_layouts(page, layout):
    gh.note(f"attention page={page} {layout}")
    for kind in KINDS:
        _check(_case(kind, LENS, 3, 2, 96, page, layout, seed=page))


@pytest.mark.parametrize("kind,lens,n_kv,group,d", [
    ("f16", [5000], 1, 4, 64),                                # one sequence over many work groups
    ("bf16", [12345, 3], 2, 8, 128),
    ("q8", [9001], 3, 5, 128),
    ("f16", [4096, 1, 4097, 0, 2000, 31], 4, 16, 256),
    ("bf16", [700] * 9, 2, 20, 224),
    ("q8", list(range(0, 300, 7)), 2, 3, 96),
])
def test_attention_split_over_work_groups(kind, lens, n_kv, group, d):
    gh.note(f"attention split {kind} {lens[:6]} n_kv={n_kv} group={group} d={d}")
    _check(_case(kind, lens, n_kv, group, d, 16, seed=len(lens)))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("seed", [1, 2, 3])
def test_attention_large_ragged_batches(kind, seed):
    """Enough tiles per wave for the split to count what a unit costs beside its tiles; empty, short
    and long sequences in any order."""
    rng = np.random.default_rng(seed)
    lens = np.concatenate([rng.integers(0, 70, 40 * seed), rng.integers(1000, 6000, 24), [0, 1, 32, 64]])
    rng.shuffle(lens)
    c = _case(kind, lens.tolist(), 8, 2, 32, 32, seed=seed)
    assert sum(max(1, -(-int(n) // 32)) for n in lens) * 8 > 512 * 4 * 6
    _check(c)


@pytest.mark.parametrize("kind", KINDS)
def test_attention_many_short_sequences(kind):
    """More units than waves: a wave crosses sequences and heads, parts lie in every place."""
    rng = np.random.default_rng(5)
    lens = rng.integers(0, 100, 1500).tolist()
    _check(_case(kind, lens, 2, 2, 32, 4))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("q_mul,kv_mul", [(1e-20, 1.0), (30.0, 1.0), (1.0, 1e-6), (1.0, 1e-4), (1e4, 1e-6), (1e-3, 1e3), (0.0, 1.0)])
def test_attention_magnitudes(kind, q_mul, kv_mul):
    """Tiny (f16 subnormal) and large queries and rows: operands in parts keep their bits at every magnitude, and a
    single dominating score is no overflow."""
    _check(_case(kind, [70, 33, 1000], 2, 4, 64, 16, q_mul=q_mul, kv_mul=kv_mul))


def test_attention_scale_and_zero_rows():
    torch = _torch()
    for kind in KINDS:
        _check(_case(kind, [40, 100], 1, 3, 64, 16, scale=-0.25))
        _check(_case(kind, [40, 100], 1, 3, 64, 16, scale=0.0))
        c = _case(kind, [64, 100], 1, 3, 64, 16)
        for t in (c["cache"].k, c["cache"].v):       # rows of zeros, an 8-bit row's scale zero with them
            t[:, :, ::2] = 0
        if kind == "q8":
            for s in (c["cache"].k_scale, c["cache"].v_scale):
                s[:, :, ::2] = 0
        _check(c)
    torch.cuda.synchronize()


def test_attention_value_scales_of_any_size():
    """8-bit value scales from 1e-30 to 1e30: the sums stay relative to the largest so far."""
    torch = _torch()
    for order in (1, -1):
        c = _case("q8", [200], 1, 2, 64, 16, stale=False)
        pos = torch.arange(200)
        sc = 10.0 ** (order * (pos.double() * 0.3 - 30))
        for t in range(200):
            c["cache"].v_scale[int(c["table"][0][t // 16]), 0, t % 16] = float(sc[t])
        _check(c)


@pytest.mark.parametrize("kind", KINDS)
def test_attention_bad_pages_and_lengths_poison_their_sequence_only(kind):
    torch = _torch()
    c = _case(kind, [100, 50, 3000, 20, 64, 10], 2, 3, 64, 16)
    good = _want(c)
    table = c["table"].copy()
    lens = list(c["lens"])
    table[0, 3] = -1                                  # a page in the middle
    table[2, 187] = c["cache"].n_pages                # the last page of a split sequence
    lens[3], lens[4] = -1, table.shape[1] * 16 + 1
    c2 = dict(c, table=table, lens=lens)
    out, lse = _run(c2)
    for i in range(6):
        if i in (0, 2, 3, 4):
            assert np.isnan(out[i]).all() and np.isnan(lse[i]).all(), i
        else:
            assert (np.abs(out[i] - good[i][0]) <= good[i][2]).all()
    torch.cuda.synchronize()


@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_attention_infinite_and_nan_rows_stay_in_their_heads(kind):
    c = _case(kind, [80], 2, 2, 64, 16, stale=False)
    page, at = int(c["table"][0, 1]), 5
    c["cache"].k[page, 0, at, 7] = math.nan
    c["cache"].v[page, 1, at, 9] = math.inf
    out, _ = _run(c)
    assert not np.isfinite(out[0, :2]).any()          # kv head 0: the score is NaN
    bad = np.zeros(64, bool)
    bad[9] = True
    assert not np.isfinite(out[0, 2:, bad]).any() and np.isfinite(out[0, 2:][:, ~bad]).all()


def test_attention_shared_pages_strided_rows_and_own_workspace():
    """Two sequences on one prefix; q, out and the table views of larger tensors."""
    torch, qmm = _torch(), _qmm()
    c = _case("f16", [96, 90, 40], 2, 4, 64, 16, stale=False)
    c["table"][1, :4] = c["table"][0, :4]
    c["table"][1, 4:6] = c["table"][0, 4:6]
    wide = torch.zeros(3, 8 * 64 + 100, device="cuda")
    wide[:, 4:4 + 512] = c["q"].flatten(1)
    out = torch.full((3, 8 * 64 + 60), 5.0, device="cuda")
    tab = torch.full((3, 600), -9, dtype=torch.int32, device="cuda")
    tab[:, 5:5 + c["table"].shape[1]] = torch.from_numpy(c["table"]).cuda()
    tab = tab[:, 5:505]                     # room for 8000 tokens: the split is made for those
    lens = torch.tensor(c["lens"], dtype=torch.int32, device="cuda")
    need = qmm.paged_attention_workspace_bytes(3, 8, c["cache"], tab.shape[1])
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")     # any contents
    qmm.paged_attention(wide[:, 4:516], c["cache"], tab, lens, out=out[:, 8:520], workspace=ws[:need])
    assert (out[:, :8] == 5).all() and (out[:, 520:] == 5).all() and (ws[need:] == 255).all()
    for i, (w, _, tol) in enumerate(_want(c)):
        assert (np.abs(out[i, 8:520].cpu().double().numpy().reshape(8, 64) - w) <= tol).all()
    with pytest.raises(qmm.QmmError) as e:
        qmm.paged_attention(wide[:, 4:516], c["cache"], tab, lens, workspace=ws[:need - 256])
    assert e.value.status == 9
    with pytest.raises(ValueError):
        qmm.paged_attention(c["q"][:, :, :32], c["cache"], tab, lens)
    with pytest.raises(TypeError):
        qmm.paged_attention(c["q"].half(), c["cache"], tab, lens)
    with pytest.raises(ValueError):                   # rows that overlap
        qmm.KVCache(c["cache"].k.expand(-1, -1, -1, -1).as_strided((4, 2, 16, 64), (64, 64, 64, 1)), c["cache"].v[:4])


def test_cache_offsets_past_32_bits():
    """Rows more than 2^32 bytes (and elements) from the first one."""
    torch, qmm = _torch(), _qmm()
    n_pages, page, d = 300000, 128, 128                # 9.8 GB in keys
    base = torch.empty(n_pages, 1, page, d, dtype=torch.float16, device="cuda")
    cache = qmm.KVCache(base, torch.empty_like(base))
    rng = np.random.default_rng(0)
    ids = [299999, 0, 270000, 131073]
    table = torch.tensor([ids], dtype=torch.int32, device="cuda")
    k, v = (rng.normal(size=(500, 1, d)).astype(np.float32) for _ in range(2))
    slots = torch.tensor([ids[t // page] * page + t % page for t in range(500)], dtype=torch.int32, device="cuda")
    qmm.kv_append(cache, gh.to_dev(k), gh.to_dev(v), slots)
    q = rng.normal(size=(1, 2, d)).astype(np.float32)
    out = qmm.paged_attention(gh.to_dev(q), cache, table, torch.tensor([500], dtype=torch.int32, device="cuda"))
    w, _, tol = step.attention(q[0], k.astype(np.float16), v.astype(np.float16), d ** -0.5)
    assert (np.abs(out[0].cpu().double().numpy() - w) <= tol).all()


def test_outputs_made_for_another_stream():
    """Outputs that a call allocates for a given stream belong to it: not memory whose last reader
    may still be under way on the current one."""
    torch, qmm = _torch(), _qmm()
    c = _case("f16", [300, 40], 2, 4, 64, 16, tokens=4000)
    table, lens = torch.from_numpy(c["table"]).cuda(), torch.tensor(c["lens"], dtype=torch.int32, device="cuda")
    w = torch.ones(512, device="cuda")
    want = qmm.paged_attention(c["q"], c["cache"], table, lens)
    wy, wh = qmm.add_rmsnorm(want.flatten(1), w, want.flatten(1))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    big = torch.randn(4096, 4096, device="cuda")
    for _ in range(5):
        old = torch.full_like(want, 2.0)
        slow = big @ big @ big                          # the current stream is busy
        total = old.sum()                               # ... and reads `old` after that
        del old
        got = qmm.paged_attention(c["q"], c["cache"], table, lens, stream=side)
        side.synchronize()
        y, h = qmm.add_rmsnorm(got.flatten(1), w, got.flatten(1), stream=side)
        side.synchronize()
        assert torch.equal(got, want) and torch.equal(y, wy) and torch.equal(h, wh)
        assert float(total) == 2.0 * want.numel() and bool(torch.isfinite(slow[0, 0]))


@pytest.mark.parametrize("kind,group,d", [("f16", 16, 256), ("q8", 3, 96), ("bf16", 20, 64)])
def test_attention_captured_with_every_launch(kind, group, d):
    """The largest LDS, two blocks of heads, both joins, and a short table, replayed."""
    torch, qmm = _torch(), _qmm()
    for lens, tokens in (([3000], 0), ([700] * 40, 0), ([60, 0, 33], 0)):
        c = _case(kind, lens, 2, group, d, 16, tokens=tokens)
        a = (c["q"], c["cache"], torch.from_numpy(c["table"]).cuda(), torch.tensor(c["lens"], dtype=torch.int32, device="cuda"))
        want = qmm.paged_attention(*a)
        out = torch.empty_like(want)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            qmm.paged_attention(*a, out=out)
        for _ in range(3):
            out.fill_(5)
            g.replay()
            qmm.paged_attention(*a)
            torch.cuda.synchronize()
            assert torch.equal(out, want)


def test_attention_is_deterministic_on_any_stream_and_under_capture():
    """Equal bits for equal calls: eager, on another stream, and replayed from two graphs that are
    interleaved with eager calls of other inputs."""
    torch, qmm = _torch(), _qmm()
    cases = [_case("bf16", [900, 0, 33, 2500], 2, 4, 128, 16, seed=s) for s in (1, 2)]
    dev = [(c["q"], c["cache"], torch.from_numpy(c["table"]).cuda(),
            torch.tensor(c["lens"], dtype=torch.int32, device="cuda")) for c in cases]
    eager = [qmm.paged_attention(*a).clone() for a in dev]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = [qmm.paged_attention(*a, stream=side) for a in dev]
    side.synchronize()
    for e, o in zip(eager, other):
        assert torch.equal(e, o)
    outs = [torch.empty_like(e) for e in eager]
    graphs = []
    for a, o in zip(dev, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            qmm.paged_attention(*a, out=o)
        graphs.append(g)
    for r in range(4):
        for o in outs:
            o.fill_(math.nan)
        for g in graphs if r % 2 else graphs[::-1]:
            g.replay()
        again = qmm.paged_attention(*dev[r % 2])
        torch.cuda.synchronize()
        assert torch.equal(again, eager[r % 2])
        for e, o in zip(eager, outs):
            assert torch.equal(e, o), f"replay {r}"
    # lengths and tables are read at replay
    lens = dev[0][3]
    lens.copy_(torch.tensor([10, 0, 5, 2400], dtype=torch.int32))
    want = qmm.paged_attention(*dev[0]).clone()
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(want, outs[0])


def test_calls_at_the_same_time_on_two_streams():
    """Steps of two caches on two streams, each with append, page tables, attention and norm: neither
    disturbs the other (own workspaces), and both equal their serial results."""
    torch, qmm = _torch(), _qmm()
    cases = [_case(k, [2500, 40, 0, 900], 4, 2, 64, 16, seed=s, tokens=4000) for s, k in ((3, "f16"), (4, "q8"))]
    w = torch.ones(512, device="cuda")

    def one(c, stream=None):
        table, lens = c["dev"]
        out = qmm.paged_attention(c["q"], c["cache"], table, lens, stream=stream)
        y, _ = qmm.add_rmsnorm(out.flatten(1), w, stream=stream)
        _, slots, pos, _ = qmm.paged_extend(c["tab2"], lens, c["new"], c["free"], 16, 8, stream=stream)
        return out, y, slots, pos

    for c in cases:
        c["dev"] = (torch.from_numpy(c["table"]).cuda(), torch.tensor(c["lens"], dtype=torch.int32, device="cuda"))
        c["tab2"], c["new"] = c["dev"][0].clone(), torch.tensor([1, 2, 3, 1], dtype=torch.int32, device="cuda")
        c["free"] = torch.arange(8, dtype=torch.int32, device="cuda")
        c["want"] = [t.clone() for t in one(c)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(20):
        got = [one(c, s) for c, s in zip(cases, streams)]
        for s in streams:
            s.synchronize()
        for c, g in zip(cases, got):
            for x, y in zip(g, c["want"]):
                assert torch.equal(x, y)


# ------------------------------------------------------------------ norm
NORM_SHAPES = [(1, 4), (1, 32), (3, 36), (7, 64), (5, 100), (9, 128), (4, 256), (33, 260), (2, 1024), (5, 1028), (3, 2048),
               (16, 4096), (2, 4608), (3, 8192), (2, 12000), (1, 16384), (2, 16388), (2, 40000), (1000, 32), (257, 512)]


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("n,k", NORM_SHAPES)
def test_norm_f32(n, k, residual):
    torch, qmm = _torch(), _qmm()
    gh.note(f"norm n={n} k={k} residual={residual}")
    rng = np.random.default_rng(k + n)
    x, r, w = (rng.normal(size=s).astype(np.float32) for s in ((n, k), (n, k), (k,)))
    x[0] *= 1e-12                                       # eps alone decides
    x[-1] *= 300
    wide = torch.full((n, 2 * k + 8), 3.0, device="cuda")
    wide[:, 4:4 + k] = gh.to_dev(x)
    out = torch.full((n, k + 8), 9.0, device="cuda")
    y, h = qmm.add_rmsnorm(wide[:, 4:4 + k], gh.to_dev(w), gh.to_dev(r) if residual else None, eps=1e-6, y=out[:, 4:4 + k])
    hs = x + r if residual else x
    if residual:
        assert np.array_equal(h.cpu().numpy(), hs)
    else:
        assert h is None
    want, _ = step.rmsnorm(hs, w, 1e-6)
    assert (np.abs(y.cpu().double().numpy() - want) <= step.rmsnorm_rel(k) * np.abs(want) + 1e-44).all()
    assert (out[:, :4] == 9).all() and (out[:, 4 + k:] == 9).all() and (wide[:, 4 + k:] == 3).all()


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("n,k", [(n, k) for n, k in NORM_SHAPES if k % 32 == 0])
def test_norm_q8(n, k, residual):
    torch, qmm = _torch(), _qmm()
    gh.note(f"norm q8 n={n} k={k} residual={residual}")
    rng = np.random.default_rng(k + n)
    x, r, w = (rng.normal(size=s).astype(np.float32) for s in ((n, k), (n, k), (k,)))
    w[:32] = 0                                          # a block of zeros
    q, d, h = qmm.add_rmsnorm_q8(gh.to_dev(x), gh.to_dev(w), gh.to_dev(r) if residual else None)
    hs = x + r if residual else x
    codes, d0 = step.q8_rows(hs * w, 32)
    _, inv = step.rmsnorm(hs, w, 1e-5)
    assert np.array_equal(q.cpu().numpy(), codes)
    want = d0 * inv
    assert (np.abs(d.cpu().double().numpy() - want) <= step.rmsnorm_rel(k) * want).all()
    if residual:
        assert np.array_equal(h.cpu().numpy(), hs)
    torch.cuda.synchronize()


@pytest.mark.parametrize("q8", [False, True])
def test_norm_of_more_rows_than_a_launch_holds(q8):
    """2^24 rows of a work group of 256 threads each pass a launch's 2^32 threads."""
    torch, qmm = _torch(), _qmm()
    n, k, step_rows = (1 << 24) + 3, 288, 1 << 22
    if torch.cuda.mem_get_info()[0] < 50 << 30:
        pytest.skip("needs 50 GB of free device memory")
    gh.note(f"norm n={n} k={k} q8={q8}")
    x, w = torch.randn(n, k, device="cuda"), torch.rand(k, device="cuda")
    f = qmm.add_rmsnorm_q8 if q8 else qmm.add_rmsnorm
    got = f(x, w)[:-1]
    for at in range(0, n, step_rows):
        for g, part in zip(got, f(x[at:at + step_rows], w)[:-1]):
            assert torch.equal(g[at:at + step_rows], part)
    del got, g, part, x
    torch.cuda.empty_cache()


def test_norm_refuses_what_it_cannot_take():
    torch, qmm = _torch(), _qmm()
    x, w = torch.zeros(2, 64, device="cuda"), torch.ones(64, device="cuda")
    for call, error in ((lambda: qmm.add_rmsnorm(x[:, :62], w[:62]), qmm.QmmError),
                        (lambda: qmm.add_rmsnorm_q8(x[:, :36], w[:36]), qmm.QmmError),
                        (lambda: qmm.add_rmsnorm(x, w, y=x), qmm.QmmError),
                        (lambda: qmm.add_rmsnorm(x, w[:32]), ValueError),
                        (lambda: qmm.add_rmsnorm(x.t(), w[:2]), ValueError),
                        (lambda: qmm.add_rmsnorm(x.half(), w), TypeError),
                        (lambda: qmm.add_rmsnorm(x, w, x[:1]), ValueError),
                        (lambda: qmm.add_rmsnorm(x, w, eps=-1.0), qmm.QmmError)):
        with pytest.raises(error):
            call()


# ------------------------------------------------------------------ a decode step
def test_decode_step_end_to_end():
    """Two steps of one layer on quantized weights: norm, QKV projection, page tables, append,
    attention, output projection, norm to Q8_1, MoE gate/up and down; eager against the f64 oracle
    stage by stage, then captured and replayed with equal bits."""
    torch, qmm = _torch(), _qmm()
    n_kv, group, d, page, hidden = 2, 2, 64, 16, 512
    n_q, batch, width = n_kv * group, 5, 8
    n_expert, n_used, n_ff = 8, 2, 128
    rows_qkv = (n_q + 2 * n_kv) * d
    rng = np.random.default_rng(11)
    wq = gh.weights("q4_0", rows_qkv, hidden, 1)
    wo = gh.weights("q8_0", hidden, n_q * d, 2)
    wg, wu = (np.concatenate([gen.nvfp4_rows(n_ff, hidden, 100 * p + e) for e in range(n_expert)]) for p in (1, 2))
    wd = np.concatenate([gen.nvfp4_rows(hidden, n_ff, 300 + e) for e in range(n_expert)])
    dw = {n: gh.to_dev(v) for n, v in dict(q=wq, o=wo, g=wg, u=wu, d=wd).items()}
    ids = gh.to_dev(gen.expert_ids(batch, n_used, n_expert))
    sc = gh.to_dev(gen.pair_scales(3 * batch * n_used))
    norm_w = [gh.to_dev((1 + 0.1 * rng.normal(size=hidden)).astype(np.float32)) for _ in range(2)]
    # the stand-in projections grow values: keep the step's activations near one
    keys = rng.normal(size=(batch, 40, n_kv, d)).astype(np.float32)
    values = rng.normal(size=(batch, 40, n_kv, d)).astype(np.float32)
    cached0 = np.array([15, 16, 0, 39, 31])
    pages = torch.zeros(batch * width, n_kv, page, d, dtype=torch.float16, device="cuda")
    cache = qmm.KVCache(pages, torch.zeros_like(pages))
    table = torch.full((batch, width), -1, dtype=torch.int32, device="cuda")
    free = torch.from_numpy(rng.permutation(batch * width).astype(np.int32)).cuda()
    i32 = lambda v: torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")  # noqa: E731
    # the prompt: appended through the same entry points
    _, slots, _, used = qmm.paged_extend(table, i32([0] * batch), i32(cached0), free, page, int(cached0.sum()))
    prompt = [np.concatenate([t[i, :n] for i, n in enumerate(cached0)]) for t in (keys, values)]
    qmm.kv_append(cache, gh.to_dev(prompt[0]), gh.to_dev(prompt[1]), slots)
    free = free[int(used):]
    hist = [[t[i, :n].astype(np.float16).astype(np.float64) for i, n in enumerate(cached0)] for t in (keys, values)]
    x = gh.to_dev(rng.normal(size=(batch, hidden)).astype(np.float32))
    res = gh.to_dev(rng.normal(size=(batch, hidden)).astype(np.float32))
    cached, new = i32(cached0), i32([1] * batch)

    def layer(cached, free):
        s = {}
        s["y"], s["h"] = qmm.add_rmsnorm(x, norm_w[0], res)
        s["qkv"] = qmm.gemm(dw["q"], s["y"], rows_qkv, "q4_0")
        # a real layer's projections are near one: so are these after the division
        s["qkv"] = s["qkv"] * 0.02
        q, k, v = (s["qkv"][:, a * d:b * d] for a, b in ((0, n_q), (n_q, n_q + n_kv), (n_q + n_kv, n_q + 2 * n_kv)))
        s["lens"], s["slots"], s["pos"], s["used"] = qmm.paged_extend(table, cached, new, free, page, batch)
        qmm.kv_append(cache, k, v, s["slots"])
        s["att"] = qmm.paged_attention(q, cache, table, s["lens"])
        s["o"] = qmm.gemm(dw["o"], s["att"], hidden, "q8_0")
        s["aq"], s["ad"], s["h2"] = qmm.add_rmsnorm_q8(s["o"], norm_w[1], s["h"])
        act = qmm.moe_gateup_act_q8(dw["g"], dw["u"], ids, sc[: 2 * batch * n_used], s["aq"], s["ad"], n_expert, n_ff)
        s["moe"], _ = qmm.moe_down(dw["d"], ids, sc[2 * batch * n_used:], act, n_expert, hidden)
        return s

    for turn in range(2):
        s = {n: t.clone() for n, t in layer(cached, free).items()}
        got = {n: t.cpu().numpy() for n, t in s.items()}
        assert np.array_equal(got["pos"], cached.cpu().numpy()) and np.array_equal(got["lens"], got["pos"] + 1)
        y, _ = step.rmsnorm(got["h"], norm_w[0].cpu().numpy(), 1e-5)
        assert (np.abs(got["y"] - y) <= step.rmsnorm_rel(hidden) * np.abs(y)).all()
        for i in range(batch):
            kv = got["qkv"][i, n_q * d:].reshape(2, n_kv, d).astype(np.float16).astype(np.float64)
            for j in range(2):
                hist[j][i] = np.concatenate([hist[j][i], kv[j][None]])
            w, _, tol = step.attention(got["qkv"][i, : n_q * d].reshape(n_q, d), hist[0][i], hist[1][i], d ** -0.5)
            assert (np.abs(got["att"][i].reshape(n_q, d) - w) <= tol).all(), (turn, i)
        r, S = ref.gemm_ref("q8_0", wo, got["att"], hidden, n_q * d, batch)
        assert ref.tolerance_check(got["o"], r, S, gh.TAU_F32)[0]
        codes, d0 = step.q8_rows(got["h2"] * norm_w[1].cpu().numpy(), 32)
        assert np.array_equal(got["h2"], got["o"] + got["h"]) and np.array_equal(got["aq"], codes)
        assert np.isfinite(got["moe"]).all()
        # the same step captured: equal bits on every replay (the step may be repeated)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            t = layer(cached, free)
        for _ in range(3):
            for v in t.values():
                v.fill_(3)
            g.replay()
            layer(cached, free)
            torch.cuda.synchronize()
            for n in s:
                assert torch.equal(s[n], t[n]), n
        free = free[int(s["used"]):]
        cached = s["lens"].clone()
    assert formats.block_elems("q4_0") == 32
