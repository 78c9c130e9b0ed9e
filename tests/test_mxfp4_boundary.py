"""The MXFP4 entry points' argument checks, on the CPU: every refusal returns its status before
anything is launched (fake pointers, no GPU)."""

import ctypes
import os

import pytest

NULL, SHAPE, K_ALIGN, QTYPE, ALIGN, RANGE, WORKSPACE, ALIAS = 1, 2, 3, 4, 5, 8, 9, 10
V = ctypes.c_void_p
P = [V((i + 1) << 40) for i in range(16)]
Z = V(0)


def _lib():
    from gemv_prefill_decode_amd import load, lib_path
    if not os.path.exists(lib_path()):
        pytest.skip("libqmm.so not built")
    return load()


def _off(p, n):
    return V(p.value + n)


def test_quantize_refusals():
    lib = _lib()

    def f(q=P[0], e=P[1], x=P[2], type=0, ldx=96, rows=3, k=96):
        return lib.qmm_quantize_mxfp4(q, e, x, type, ldx, rows, k, Z)

    assert f(q=Z) == f(e=Z) == f(x=Z) == NULL
    assert f(type=3) == f(type=-1) == QTYPE
    assert f(rows=0) == f(k=0) == f(ldx=95) == f(rows=1 << 61) == SHAPE
    assert f(k=80) == K_ALIGN
    assert f(q=_off(P[0], 8)) == f(x=_off(P[2], 4)) == f(ldx=98) == f(type=1, ldx=100) == ALIGN
    assert f(k=1 << 31, ldx=1 << 31) == RANGE
    assert f(e=_off(P[0], 143)) == f(e=P[2]) == f(q=_off(P[2], 1136)) == f(x=_off(P[0], 128)) == ALIAS


def test_dequantize_refusals():
    lib = _lib()

    def f(x=P[0], q=P[1], e=P[2], rows=3, k=96):
        return lib.qmm_dequantize_mxfp4(x, q, e, rows, k, Z)

    assert f(x=Z) == f(q=Z) == f(e=Z) == NULL
    assert f(rows=0) == f(k=-32) == f(rows=1 << 60) == SHAPE
    assert f(k=16) == K_ALIGN
    assert f(x=_off(P[0], 8)) == f(q=_off(P[1], 4)) == ALIGN
    assert f(q=_off(P[0], 1136)) == f(e=_off(P[0], 1151)) == ALIAS


def test_gemm_refusals():
    lib = _lib()

    def f(dst=P[0], ldd=48, wq=P[1], we=P[2], xq=P[3], xe=P[4], s=P[5], m=48, k=96, n=5):
        return lib.qmm_gemm_mxfp4(dst, ldd, wq, we, xq, xe, s, m, k, n, Z)

    for name in ("dst", "wq", "we", "xq", "xe"):
        assert f(**{name: Z}) == NULL, name
    assert f(m=0) == f(n=0) == f(k=0) == f(ldd=47) == f(ldd=1 << 62) == SHAPE
    assert f(k=48) == K_ALIGN
    assert f(wq=_off(P[1], 8)) == f(xq=_off(P[3], 8)) == f(we=_off(P[2], 2)) == f(xe=_off(P[4], 1)) == ALIGN
    assert f(dst=_off(P[0], 2)) == f(s=_off(P[5], 2)) == ALIGN
    assert f(k=(1 << 23) + 32) == f(m=1 << 31, ldd=1 << 31) == f(n=(1 << 20) + 1) == RANGE
    assert f(m=(1 << 26) + 1, ldd=1 << 27) == f(m=1 << 26, ldd=1 << 26, n=(1 << 11) + 1) == RANGE
    for other in (P[1], P[2], P[3], P[4], P[5]):
        assert f(dst=other) == f(dst=_off(other, -4)) == ALIAS
    assert f(dst=_off(P[1], 48 * 48 - 4)) == f(dst=_off(P[4], 12)) == ALIAS


def test_norm_refusals():
    lib = _lib()

    def f(q=P[0], e=P[1], s=P[6], h=P[2], ldh=96, x=P[3], ldx=96, r=P[4], ldr=96, w=P[5], n=3, k=96, eps=1e-5):
        return lib.qmm_add_rmsnorm_mxfp4(q, e, s, h, ldh, x, ldx, r, ldr, w, n, k, eps, Z)

    for name in ("q", "e", "s", "x", "w"):
        assert f(**{name: Z}) == NULL, name
    assert f(n=0) == f(k=0) == f(ldx=92) == f(ldr=92) == f(ldh=92) == SHAPE
    assert f(k=80) == K_ALIGN
    assert f(q=_off(P[0], 8)) == f(s=_off(P[6], 2)) == f(ldx=98) == f(x=_off(P[3], 4)) == f(w=_off(P[5], 8)) == ALIGN
    assert f(eps=-1.0) == f(eps=float("nan")) == RANGE
    assert f(e=_off(P[0], 143)) == f(s=P[1]) == f(s=_off(P[2], 8)) == f(q=P[3]) == f(e=P[4]) == f(s=P[5]) == ALIAS
    assert f(h=P[4]) == f(h=P[0]) == ALIAS


# ------------------------------------------------------------------ the cache
def _cache(**over):
    from gemv_prefill_decode_amd import _KvCacheStruct
    c = dict(k=P[0].value, v=P[1].value, k_scale=P[2].value, v_scale=P[3].value, n_pages=10, n_kv=4, page_size=16,
             head_dim=64, page_stride=4 * 16 * 64, head_stride=16 * 64, slot_stride=64, scale_page_stride=128,
             scale_head_stride=32, scale_slot_stride=2, kind=4)
    c.update(over)
    return ctypes.byref(_KvCacheStruct(**c))


def _append(lib, c, n=3):
    return lib.qmm_kv_append(c, P[4], 256, P[5], 256, P[6], n, Z)


@pytest.mark.parametrize("status,over", [
    (NULL, dict(k_scale=None)), (NULL, dict(v_scale=None)), (QTYPE, dict(kind=5)), (K_ALIGN, dict(head_dim=48)),
    (RANGE, dict(head_dim=288)), (ALIGN, dict(slot_stride=80)), (ALIGN, dict(head_stride=16 * 64 + 16)),
    (ALIGN, dict(k=P[0].value + 8)), (SHAPE, dict(slot_stride=32)), (SHAPE, dict(scale_slot_stride=1)),
    (SHAPE, dict(scale_head_stride=0)), (RANGE, dict(scale_page_stride=1 << 41)), (RANGE, dict(page_stride=1 << 40)),
    (ALIAS, dict(v=P[0].value)), (ALIAS, dict(v=P[0].value + 32 * 16)), (ALIAS, dict(v_scale=P[2].value + 1)),
    (ALIAS, dict(v_scale=P[2].value + 10 * 128 - 1)), (ALIAS, dict(k_scale=P[0].value + 100)),
    (ALIAS, dict(v_scale=P[1].value + 10 * 2048 - 1)), (ALIAS, dict(v_scale=P[1].value - 10 * 128 + 1)),
])
def test_bad_caches_are_refused(status, over):
    lib = _lib()
    c = _cache(**over)
    assert _append(lib, c) == status
    assert lib.qmm_paged_attention(P[4], 512, Z, P[5], 512, c, P[6], 8, P[7], 2, 8, 8, 0.1, P[8], 1 << 30, Z) == status


def test_caches_whose_arrays_lie_between_each_other_are_taken():
    """n = 0 is the refusal behind the cache's."""
    lib = _lib()
    b, rows = P[0].value, 4 * 16
    assert _append(lib, _cache(), 0) == SHAPE
    assert _append(lib, _cache(v_scale=P[2].value + 10 * 128), 0) == SHAPE
    assert _append(lib, _cache(v=b + rows * 32, page_stride=2 * rows * 64), 0) == SHAPE        # side by side in a page
    # one block a page: keys, values, their scales
    block = 2 * rows * 34
    assert _append(lib, _cache(v=b + rows * 32, page_stride=2 * block, k_scale=b + 2 * rows * 32,
                               v_scale=b + 2 * rows * 33, scale_page_stride=block), 0) == SHAPE
    assert _append(lib, _cache(v=b + rows * 32, page_stride=2 * block, k_scale=b + 2 * rows * 32,
                               v_scale=b + 2 * rows * 33 - 1, scale_page_stride=block), 0) == ALIAS
    assert _append(lib, _cache(n_pages=1, page_stride=1 << 62, scale_page_stride=1 << 62), 0) == SHAPE


def test_python_layer_refuses_host_tensors():
    import torch
    import gemv_prefill_decode_amd as qmm
    _lib()
    x, q, e = torch.zeros(2, 32), torch.zeros(2, 16, dtype=torch.uint8), torch.zeros(2, 1, dtype=torch.uint8)
    for call in (lambda: qmm.quantize_mxfp4(x), lambda: qmm.dequantize_mxfp4(q, e), lambda: qmm.gemm_mxfp4(q, e, q, e),
                 lambda: qmm.add_rmsnorm_mxfp4(x, x[0])):
        with pytest.raises(TypeError):
            call()
    pages = torch.zeros(2, 1, 16, 16, dtype=torch.uint8)
    with pytest.raises(TypeError):
        qmm.KVCache(pages, pages.clone(), pages[..., :1], pages[..., :1])


def test_boundary_tests_pass_under_asan_and_ubsan():
    """This file again, against the library's host code built with the sanitizers."""
    import subprocess
    import sys
    if "QMM_LIBRARY" in os.environ:
        pytest.skip("this is that run")
    from gemv_prefill_decode_amd import build as b
    objects = [os.path.join(b.BUILD_DIR, s + ".o") for s in b.SOURCES]
    if not all(os.path.exists(o) for o in objects):
        pytest.skip("regular build objects missing (run __graft_entry__.build())")
    try:
        fresh = os.path.exists(b.SAN_OUT) and os.path.getmtime(b.SAN_OUT) > max(map(os.path.getmtime, objects))
        san = b.SAN_OUT if fresh else b.build_sanitized()
        rt = b.asan_runtime()
    except (RuntimeError, FileNotFoundError) as e:
        pytest.skip(f"no sanitizer toolchain: {e}")
    env = dict(os.environ, QMM_LIBRARY=san, LD_PRELOAD=rt,
               ASAN_OPTIONS="detect_leaks=0:halt_on_error=1:abort_on_error=0",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([sys.executable, "-m", "pytest", os.path.abspath(__file__), "-q", "-p", "no:cacheprovider"],
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))), env=env, capture_output=True,
                       text=True, timeout=600)
    out = r.stdout[-4000:] + r.stderr[-4000:]
    assert r.returncode == 0, out
    assert "ERROR: AddressSanitizer" not in r.stderr and "runtime error:" not in r.stderr, out
