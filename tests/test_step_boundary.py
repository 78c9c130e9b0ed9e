"""The decode-step entry points' argument checks, on the CPU: every refusal returns its status
before anything is launched (fake pointers, no GPU)."""

import ctypes
import os

import pytest

NULL, SHAPE, K_ALIGN, QTYPE, ALIGN, RANGE, WORKSPACE, ALIAS = 1, 2, 3, 4, 5, 8, 9, 10
V = ctypes.c_void_p
P = [V((i + 1) << 36) for i in range(16)]        # far apart: no two ranges of the tests' sizes meet
Z = V(0)


def _lib():
    from gemv_prefill_decode_amd import load, lib_path
    if not os.path.exists(lib_path()):
        pytest.skip("libqmm.so not built")
    return load()


def _cache(kind=0, **over):
    from gemv_prefill_decode_amd import _KvCacheStruct
    c = dict(k=P[0].value, v=P[1].value, k_scale=P[2].value, v_scale=P[3].value, n_pages=10, n_kv=4, page_size=16,
             head_dim=64, page_stride=4 * 16 * 64, head_stride=16 * 64, slot_stride=64, scale_page_stride=64,
             scale_head_stride=16, scale_slot_stride=1, kind=kind)
    c.update(over)
    return _KvCacheStruct(**c)


BAD_CACHES = [
    (NULL, dict(k=None)), (NULL, dict(v=None)), (NULL, dict(kind=2, k_scale=None)), (NULL, dict(kind=2, v_scale=None)),
    (QTYPE, dict(kind=3)), (QTYPE, dict(kind=-1)),
    (SHAPE, dict(n_pages=0)), (SHAPE, dict(n_kv=0)), (SHAPE, dict(page_size=0)), (SHAPE, dict(page_size=24)),
    (SHAPE, dict(head_dim=0)), (K_ALIGN, dict(head_dim=48)), (RANGE, dict(head_dim=288)),
    (SHAPE, dict(slot_stride=32)), (SHAPE, dict(head_stride=0)), (SHAPE, dict(page_stride=-64)),
    (ALIGN, dict(slot_stride=68)), (ALIGN, dict(kind=2, slot_stride=72)), (ALIGN, dict(k=P[0].value + 8)),
    (ALIAS, dict(v=P[0].value)), (RANGE, dict(n_pages=1 << 27)), (RANGE, dict(n_kv=65536)),
    (RANGE, dict(n_pages=1 << 20, page_stride=1 << 20)),          # 2 TiB between the first and the last page
    (RANGE, dict(page_stride=1 << 60)), (SHAPE, dict(kind=2, scale_slot_stride=0)),
    (ALIGN, dict(kind=2, v_scale=P[3].value + 2)),
]


@pytest.mark.parametrize("status,over", BAD_CACHES)
def test_bad_caches_are_refused(status, over):
    lib = _lib()
    c = ctypes.byref(_cache(**over))
    assert lib.qmm_kv_append(c, P[4], 256, P[5], 256, P[6], 3, Z) == status
    assert lib.qmm_paged_attention(P[4], 512, Z, P[5], 512, c, P[6], 8, P[7], 2, 8, 8, 0.1, P[8], 1 << 30, Z) == status
    assert lib.qmm_kv_append(Z, P[4], 256, P[5], 256, P[6], 3, Z) == NULL


def test_append_refusals():
    lib = _lib()
    c = ctypes.byref(_cache())
    f = lib.qmm_kv_append
    assert f(c, Z, 256, P[5], 256, P[6], 3, Z) == NULL
    assert f(c, P[4], 256, Z, 256, P[6], 3, Z) == NULL
    assert f(c, P[4], 256, P[5], 256, Z, 3, Z) == NULL
    assert f(c, P[4], 256, P[5], 256, P[6], 0, Z) == SHAPE
    assert f(c, P[4], 252, P[5], 256, P[6], 3, Z) == SHAPE
    assert f(c, P[4], 256, P[5], 128, P[6], 3, Z) == SHAPE
    assert f(c, P[4], 258, P[5], 256, P[6], 3, Z) == ALIGN
    assert f(c, V(P[4].value + 4), 256, P[5], 256, P[6], 3, Z) == ALIGN
    assert f(c, P[4], 256, P[5], 256, V(P[6].value + 2), 3, Z) == ALIGN
    assert f(c, V(P[0].value + 256), 256, P[5], 256, P[6], 3, Z) == ALIAS
    assert f(c, P[4], 256, P[5], 256, V(P[1].value + 64), 3, Z) == ALIAS
    assert f(c, P[4], 1 << 62, P[5], 256, P[6], 3, Z) == SHAPE


def test_attention_refusals():
    lib = _lib()
    c = ctypes.byref(_cache())
    need = lib.qmm_paged_attention_workspace_bytes(64, 8, 4, 64, 128, 16)
    assert need > 0 and need % 256 == 0

    def f(out=P[4], ldo=512, lse=P[9], q=P[5], ldq=512, cache=c, table=P[6], ts=128, lens=P[7], batch=64, n_q=8,
          width=128, scale=0.1, ws=P[8], nbytes=1 << 30):
        return lib.qmm_paged_attention(out, ldo, lse, q, ldq, cache, table, ts, lens, batch, n_q, width, scale, ws,
                                       nbytes, Z)

    for name in ("out", "q", "table", "lens", "ws"):
        assert f(**{name: Z}) == NULL, name
    assert f(batch=0) == f(n_q=0) == f(width=0) == f(n_q=6) == SHAPE
    assert f(ldo=504) == f(ldq=504) == f(ts=127) == SHAPE
    assert f(ldo=514) == f(ldq=513) == f(out=V(P[4].value + 4)) == f(lse=V(P[9].value + 1)) == ALIGN
    assert f(ws=V(P[8].value + 16)) == ALIGN
    assert f(nbytes=need - 1) == WORKSPACE
    assert f(scale=float("nan")) == f(scale=float("inf")) == f(batch=1 << 21) == RANGE
    assert f(n_q=65536, ldo=1 << 23, ldq=1 << 23) == RANGE
    assert f(width=1 << 27, ts=1 << 27) == RANGE                    # more than 2^30 tokens per row
    assert f(batch=64, width=1 << 26, ts=1 << 26) == RANGE          # 64 * (2^25 + 2) tiles
    assert lib.qmm_paged_attention_workspace_bytes(63, 8, 4, 64, 1 << 26, 16) > 0
    for other in (P[5], P[0], P[1], P[6], P[7], P[8], P[9]):        # out over q, the cache, the table, ...
        assert f(out=other) == ALIAS
        if other is not P[9]:
            assert f(lse=other) == ALIAS
    assert f(ws=P[5]) == f(ws=P[1]) == ALIAS
    w = lib.qmm_paged_attention_workspace_bytes
    assert w(0, 8, 4, 64, 128, 16) == w(1, 7, 4, 64, 128, 16) == w(1, 8, 4, 64, 128, 12) == -SHAPE
    assert w(1, 8, 4, 60, 128, 16) == -K_ALIGN and w(1, 8, 4, 512, 128, 16) == -RANGE
    assert w(1, 8, 8, 64, 1, 1) >= 0


def test_extend_refusals():
    lib = _lib()

    def f(table=P[0], ts=8, lens=P[1], slots=P[2], pos=P[3], used=P[4], cached=P[5], new=P[6], free=P[7], batch=4,
          width=8, page=16, n_free=10, n_rows=12):
        return lib.qmm_paged_extend(table, ts, lens, slots, pos, used, cached, new, free, batch, width, page, n_free,
                                    n_rows, Z)

    for name in ("table", "lens", "slots", "pos", "used", "cached", "new", "free"):
        assert f(**{name: Z}) == NULL, name
    assert f(batch=0) == f(width=0) == f(n_free=-1) == f(n_rows=-1) == f(ts=7) == f(page=0) == f(page=12) == SHAPE
    assert f(slots=V(P[2].value + 2)) == ALIGN
    assert f(width=1 << 27, ts=1 << 27) == f(n_rows=(1 << 30) + 1) == f(n_free=(1 << 30) + 1) == RANGE
    assert f(batch=1 << 20, width=1 << 12, ts=1 << 12, page=1) == RANGE
    assert f(lens=P[5]) == ALIAS                                     # in place: the kernel still reads the old lengths
    assert f(table=P[7]) == f(slots=P[3]) == f(used=V(P[0].value + 16)) == ALIAS


@pytest.mark.parametrize("q8", [False, True])
def test_norm_refusals(q8):
    lib = _lib()
    unit = 32 if q8 else 4

    def f(y=P[0], d=P[1], h=P[2], ldh=96, x=P[3], ldx=96, r=P[4], ldr=96, w=P[5], n=3, k=96, eps=1e-5, ldy=96):
        if q8:
            return lib.qmm_add_rmsnorm_q8(y, d, h, ldh, x, ldx, r, ldr, w, n, k, eps, Z)
        return lib.qmm_add_rmsnorm(y, ldy, h, ldh, x, ldx, r, ldr, w, n, k, eps, Z)

    assert f(y=Z) == f(x=Z) == f(w=Z) == NULL
    assert f(n=0) == f(k=0) == f(ldx=92) == f(ldr=92) == f(ldh=92) == SHAPE
    assert f(k=96 - unit // 2) == K_ALIGN
    assert f(ldx=98) == f(ldr=98) == f(ldh=98) == f(x=V(P[3].value + 4)) == f(w=V(P[5].value + 8)) == ALIGN
    assert f(eps=-1.0) == f(eps=float("nan")) == f(eps=float("inf")) == RANGE
    big = (1 << 24) + 32
    assert f(k=big, ldx=big, ldr=big, ldh=big, ldy=big) == RANGE
    assert f(h=P[4]) == f(h=P[3]) == f(y=P[3]) == f(y=P[5]) == f(h=P[0]) == ALIAS
    if q8:
        assert f(d=Z) == NULL and f(d=V(P[1].value + 2)) == ALIGN and f(d=V(P[0].value + 16)) == ALIAS


def test_python_layer_refuses_host_tensors():
    import torch
    import gemv_prefill_decode_amd as qmm
    _lib()
    k = torch.zeros(2, 1, 16, 32, dtype=torch.float16)
    with pytest.raises(TypeError):
        qmm.KVCache(k, k.clone())
    x, i = torch.zeros(2, 32), torch.zeros(2, dtype=torch.int32)
    for call in (lambda: qmm.add_rmsnorm(x, x[0]), lambda: qmm.add_rmsnorm_q8(x, x[0]),
                 lambda: qmm.paged_extend(i[None].repeat(2, 1), i, i, i, 16, 2)):
        with pytest.raises(TypeError):
            call()


# ------------------------------------------------------------------ arrays of a cache that meet
def test_scales_and_codes_that_meet_are_refused():
    """k_scale and v_scale the same, a part apart, or either inside codes (codes inside scales):
    one call would write both."""
    lib = _lib()
    ks = P[2].value
    for over in (dict(v_scale=ks), dict(v_scale=ks + 4), dict(v_scale=ks + 64 * 4), dict(v_scale=ks - 4),
                 dict(v_scale=P[0].value), dict(k_scale=P[0].value + 1024), dict(k_scale=P[1].value - 4),
                 dict(k_scale=P[1].value + 10 * 4096 - 4), dict(v_scale=P[1].value - 10 * 64 * 4 + 4),
                 dict(v=P[0].value + 64), dict(v=P[0].value + 4096)):
        c = ctypes.byref(_cache(2, **over))
        assert lib.qmm_kv_append(c, P[4], 256, P[5], 256, P[6], 3, Z) == ALIAS, over
        assert lib.qmm_paged_attention(P[4], 512, Z, P[5], 512, c, P[6], 8, P[7], 2, 8, 8, 0.1, P[8], 1 << 30, Z) == ALIAS, over


def test_caches_whose_arrays_lie_between_each_other_are_taken():
    """Keys and values of a page, of a head or of a token side by side, with or without their scales
    behind them in one allocation (n = 0 is the refusal behind the cache's)."""
    lib = _lib()
    b, n_kv, page, d = P[0].value, 4, 16, 64

    def taken(c):
        return lib.qmm_kv_append(ctypes.byref(c), P[4], 256, P[5], 256, P[6], 0, Z) == SHAPE

    rows = n_kv * page
    assert taken(_cache(0, v=b + 2 * rows * d, page_stride=2 * rows * d))                                # per page
    assert taken(_cache(0, v=b + 2 * page * d, page_stride=2 * rows * d, head_stride=2 * page * d))       # per head
    assert taken(_cache(0, v=b + 2 * d, page_stride=2 * rows * d, head_stride=2 * page * d, slot_stride=2 * d))
    assert taken(_cache(0, v=b + 2 * d, page_stride=2 * rows * d, slot_stride=2 * n_kv * d, head_stride=2 * d))
    # 8 bits, one block a page: keys, values, key scales, value scales
    block = 2 * rows * (d + 4)
    for first in (0, 2 * rows * d):
        assert taken(_cache(2, k=b + (0 if first else 8 * rows), v=b + (0 if first else 8 * rows) + rows * d,
                            page_stride=block, k_scale=b + first, v_scale=b + first + 4 * rows,
                            scale_page_stride=block // 4))
    # one page: a stride that no second page has means nothing
    assert taken(_cache(0, n_pages=1, page_stride=1 << 62)) and taken(_cache(2, n_pages=1, scale_page_stride=1 << 62))


def test_keys_and_values_that_meet_are_found_exactly():
    """Random layouts and distances against the set of the rows' bytes."""
    import random
    lib, rng = _lib(), random.Random(5)
    seen = {True: 0, False: 0}
    for _ in range(3000):
        kind = rng.choice([0, 1, 2])
        es, d = (1 if kind == 2 else 2), 32 * rng.randint(1, 2)
        counts = dict(page=rng.randint(1, 4), head=rng.randint(1, 3), slot=rng.choice([1, 2, 4]))
        strides, reach = {}, d
        for axis in rng.sample(list(counts), 3):
            strides[axis] = reach + 16 * rng.choice([0, 0, 1, 2, d // 16, reach // 16])
            reach = strides[axis] * (counts[axis] - 1) + reach
        delta = 16 * rng.randint(-reach * es // 16 - 1, reach * es // 16 + 1)
        if rng.random() < 0.5:          # near a sum of strides
            delta = sum(s * es * rng.randint(-1, 1) for s in strides.values()) + 16 * rng.randint(-1, 1)
        offsets = [es * (p * strides["page"] + h * strides["head"] + s * strides["slot"])
                   for p in range(counts["page"]) for h in range(counts["head"]) for s in range(counts["slot"])]
        mine = {o // 16 + i for o in offsets for i in range(d * es // 16)}
        meet = any(o // 16 + i + delta // 16 in mine for o in offsets for i in range(d * es // 16))
        c = _cache(kind, v=P[0].value + delta, n_pages=counts["page"], n_kv=counts["head"], page_size=counts["slot"],
                   head_dim=d, page_stride=strides["page"], head_stride=strides["head"], slot_stride=strides["slot"],
                   scale_page_stride=100, scale_head_stride=10, scale_slot_stride=1)
        got = lib.qmm_kv_append(ctypes.byref(c), P[4], 256, P[5], 256, P[6], 0, Z)
        assert got == (ALIAS if meet else SHAPE), (kind, d, counts, strides, delta)
        seen[meet] += 1
    assert min(seen.values()) > 300


def test_python_layer_refuses_a_stream_of_another_device():
    import types
    import gemv_prefill_decode_amd as qmm
    called = []
    with pytest.raises(ValueError, match="device 1"):
        qmm._run(called.append, 0, types.SimpleNamespace(device_index=1, cuda_stream=0))
    assert not called
