"""gemv_prefill_decode_amd - dequant-fused projection matmul for MI355X (gfx950).

A thin binding over ``libqmm.so`` (the C-ABI declared in ``include/qmm.h``):
ctypes, and for a decode step's small calls the ``_step`` module.  Every step of the computation runs in the library's HIP
kernels; this module only checks tensor dtypes/devices and passes data
pointers and the current HIP stream.  PyTorch is used for device memory and
streams.

    out = gemm(w, x, m, "q4_k")            # dst[n, m] = x[n, k] @ deq(w)[m, k]^T
    g, u = moe_gateup(wg, wu, ids, scales, x, n_expert, n_ff, "nvfp4")

and, between a decode step's projections,

    y, h = add_rmsnorm(x, weight, residual)
    lens, slots, positions, used = paged_extend(block_table, cached, new, free, page_size, n_rows)
    cache = KVCache(k_pages, v_pages)      # kept; views of the caller's memory
    kv_append(cache, k, v, slots)
    out = paged_attention(q, cache, block_table, lens)

If the library has not been built, every call raises RuntimeError: there is
no fallback path.
"""

from __future__ import annotations

import ctypes
import os
import threading

__all__ = [
    "QTYPES", "PATHS", "QmmError", "lib_path", "load", "gemm", "workspace_bytes", "gemm_plan",
    "plan_kernel_name", "moe_gateup", "moe_down", "moe_gateup_act", "moe_gateup_act_q8", "moe_gateup_probe",
    "moe_down_q8",
    "stream_loadonly", "repack_nvfp4_v2", "quantize_q8_1", "moe_gateup_q8",
    "KV_KINDS", "KVCache", "paged_extend", "kv_append", "paged_attention", "paged_attention_workspace_bytes",
    "add_rmsnorm", "add_rmsnorm_q8",
    "row_bytes", "block_elems", "gemv_max_n", "status_str", "abi_version",
]

QTYPES = {"f32": 0, "q4_0": 1, "q8_0": 2, "q4_k": 3, "q6_k": 4, "nvfp4": 5, "nvfp4_v2": 6}
PATHS = {"auto": 0, "gemv": 1, "mfma": 2, "gemv_fma": 3, "gemv_matrix": 4}
KV_KINDS = {"f16": 0, "bf16": 1, "q8": 2}

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB = None
_LOCK = threading.Lock()


class QmmError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: qmm status {status} ({status_str(status)})")


def lib_path() -> str:
    """The in-tree libqmm.so, or the library QMM_LIBRARY names (the host-only
    sanitized build that the boundary tests also run against)."""
    return os.environ.get("QMM_LIBRARY") or os.path.join(_HERE, "libqmm.so")


def load() -> ctypes.CDLL:
    """Load libqmm.so (built in-tree by ``__graft_entry__.build()``)."""
    global _LIB
    with _LOCK:
        if _LIB is not None:
            return _LIB
        path = lib_path()
        if not os.path.exists(path):
            raise RuntimeError(
                f"{path} is not built: run `python -m gemv_prefill_decode_amd.build` "
                "(or __graft_entry__.build()); there is no non-HIP fallback")
        lib = ctypes.CDLL(path)
        i64, i32, vp = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p
        lib.qmm_gemm.argtypes = [vp, vp, vp, i64, i64, i64, i32, vp]
        lib.qmm_gemm.restype = i32
        lib.qmm_gemm_path.argtypes = [vp, vp, vp, i64, i64, i64, i32, i32, vp]
        lib.qmm_gemm_path.restype = i32
        lib.qmm_gemm_ws.argtypes = [vp, vp, vp, i64, i64, i64, i32, i32, vp, i64, vp]
        lib.qmm_gemm_ex.argtypes = [vp, i64, vp, vp, i64, i64, i64, i64, i32, i32, vp, i64, vp]
        lib.qmm_gemm_ex.restype = i32
        lib.qmm_gemm_ws.restype = i32
        lib.qmm_gemm_noalloc.argtypes = [vp, vp, vp, i64, i64, i64, i32, i32, vp]
        lib.qmm_gemm_noalloc.restype = i32
        lib.qmm_gemm_noalloc_max_bytes.argtypes = []
        lib.qmm_gemm_noalloc_max_bytes.restype = i64
        lib.qmm_gemm_workspace_bytes.argtypes = [i64, i64, i64, i32, i32]
        lib.qmm_gemm_workspace_bytes.restype = i64
        lib.qmm_gemm_plan.argtypes = [i64, i64, i64, i32, i32, i32, ctypes.POINTER(ctypes.c_int32)]
        lib.qmm_gemm_plan.restype = i32
        lib.qmm_moe_gateup.argtypes = [vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, i32, vp]
        lib.qmm_moe_gateup.restype = i32
        lib.qmm_moe_down.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, i32, vp]
        lib.qmm_moe_down.restype = i32
        f32 = ctypes.c_float
        lib.qmm_moe_gateup_act.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, i32, f32, vp]
        lib.qmm_moe_gateup_act.restype = i32
        lib.qmm_moe_gateup_act_q8.argtypes = [vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, i32, f32, vp]
        lib.qmm_moe_gateup_act_q8.restype = i32
        lib.qmm_moe_gateup_probe.argtypes = [i32, vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, i32, vp]
        lib.qmm_moe_gateup_probe.restype = i32
        lib.qmm_moe_down_q8.argtypes = [vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, i32, vp]
        lib.qmm_moe_down_q8.restype = i32
        lib.qmm_quantize_q8_1.argtypes = [vp, vp, vp, i64, i64, vp]
        lib.qmm_quantize_q8_1.restype = i32
        lib.qmm_moe_gateup_q8.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, i32, vp]
        lib.qmm_moe_gateup_q8.restype = i32
        lib.qmm_nvfp4_repack_v2.argtypes = [vp, vp, i64, i64, vp]
        lib.qmm_nvfp4_repack_v2.restype = i32
        lib.qmm_stream_loadonly.argtypes = [vp, vp, i64, i64, i32, vp]
        lib.qmm_stream_loadonly.restype = i32
        lib.qmm_paged_extend.argtypes = [vp, i64] + [vp] * 7 + [i64] * 5 + [vp]
        lib.qmm_paged_extend.restype = i32
        lib.qmm_kv_append.argtypes = [vp, vp, i64, vp, i64, vp, i64, vp]
        lib.qmm_kv_append.restype = i32
        lib.qmm_paged_attention.argtypes = [vp, i64, vp, vp, i64, vp, vp, i64, vp, i64, i64, i64, f32, vp, i64, vp]
        lib.qmm_paged_attention.restype = i32
        lib.qmm_paged_attention_workspace_bytes.argtypes = [i64] * 6
        lib.qmm_paged_attention_workspace_bytes.restype = i64
        lib.qmm_add_rmsnorm.argtypes = [vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, i64, f32, vp]
        lib.qmm_add_rmsnorm.restype = i32
        lib.qmm_add_rmsnorm_q8.argtypes = [vp, vp, vp, i64, vp, i64, vp, i64, vp, i64, i64, f32, vp]
        lib.qmm_add_rmsnorm_q8.restype = i32
        lib.qmm_row_bytes.argtypes = [i32, i64]
        lib.qmm_row_bytes.restype = i64
        lib.qmm_block_elems.argtypes = [i32]
        lib.qmm_block_elems.restype = i32
        lib.qmm_gemv_max_n.argtypes = []
        lib.qmm_gemv_max_n.restype = i32
        lib.qmm_status_str.argtypes = [i32]
        lib.qmm_status_str.restype = ctypes.c_char_p
        lib.qmm_abi_version.argtypes = []
        lib.qmm_abi_version.restype = i32
        _LIB = lib
        return lib


def _qt(qtype) -> int:
    if isinstance(qtype, str):
        if qtype not in QTYPES:
            raise ValueError(f"unknown qtype {qtype!r}")
        return QTYPES[qtype]
    return int(qtype)


def status_str(status: int) -> str:
    return load().qmm_status_str(int(status)).decode()


def abi_version() -> int:
    return load().qmm_abi_version()


def row_bytes(qtype, k: int) -> int:
    r = load().qmm_row_bytes(_qt(qtype), int(k))
    if r < 0:
        raise QmmError(-r, "qmm_row_bytes")
    return r


def block_elems(qtype) -> int:
    r = load().qmm_block_elems(_qt(qtype))
    if r < 0:
        raise QmmError(-r, "qmm_block_elems")
    return r


def gemv_max_n() -> int:
    return load().qmm_gemv_max_n()


def _stream(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dev(t, what, dtype=None):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{what} must be a device (cuda/hip) tensor")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    return ctypes.c_void_p(t.data_ptr())


def workspace_bytes(m: int, k: int, n: int, qtype, path: str = "auto") -> int:
    """Bytes of workspace qmm_gemm_ws uses for this product (0: none)."""
    v = load().qmm_gemm_workspace_bytes(m, k, n, _qt(qtype), PATHS[path])
    if v < 0:
        raise QmmError(-v, "qmm_gemm_workspace_bytes")
    return v


def gemm_plan(m: int, k: int, n: int, qtype, path: str = "auto", workspace: bool = True) -> dict:
    """The kernels qmm_gemm_ws (workspace=True) or qmm_gemm would run."""
    out = (ctypes.c_int32 * 6)()
    st = load().qmm_gemm_plan(m, k, n, _qt(qtype), PATHS[path], int(workspace), out)
    if st != 0:
        raise QmmError(st, "qmm_gemm_plan")
    if out[0] == PATHS["gemv"]:
        return {"path": "gemv", "stream": "matrix" if out[1] else "fma", "tokens_per_pass": out[2]}
    return {"path": "mfma", "x16": out[1], "tile_rows": out[2], "k_groups": out[3], "n_split": out[4],
            "steps_per_split": out[5]}


def plan_kernel_name(plan: dict, qtype) -> str:
    """Kernel symbol (as the profiler names it) of a gemm_plan() result."""
    qt = _qt(qtype)
    if plan["path"] == "gemv":
        return "gemv_mfma_kernel" if plan["stream"] == "matrix" else "gemv_kernel"
    if plan["x16"] == 7:
        return f"gemm_lds_tg_kernel<{qt}, 64, 256>"
    if plan["x16"] >= 2:
        cols = 256 if plan["x16"] == 3 else 64 if plan["x16"] in (5, 6) else 128
        return (f"gemm_lds_kernel<{qt}, {plan['tile_rows'] // 4}, {cols}, "
                f"{plan['k_groups']}, {'true' if plan['x16'] in (4, 6) else 'false'}>")
    return f"gemm_mfma_kernel<{qt}, {plan['k_groups']}>"


# Workspaces handed to qmm_gemm_ws by gemm(workspace="auto"): one buffer per
# (device, stream), grown when a product needs more.  Buffers are never
# freed, so a call captured in a graph keeps a valid workspace.
_WS = {}
_WS_ALL = []


def _auto_workspace(device, stream_handle: int, nbytes: int):
    import torch
    key = (device.index, stream_handle)
    buf = _WS.get(key)
    if buf is None or buf.numel() < nbytes:
        buf = torch.empty(max(nbytes, 1 << 20), dtype=torch.uint8, device=device)
        _WS[key] = buf
        _WS_ALL.append(buf)
    return buf


def gemm(w, x, m: int, qtype, out=None, path: str = "auto", stream=None, workspace="auto"):
    """dst[n, m] with dst[j, i] = sum_c deq(w)[i, c] * x[j, c].

    w: packed weights (uint8, m*row_bytes(qtype, k) bytes; float32 [m, k] for
    "f32"); x: float32 [n, k]; out: optional float32 [n, m].  x and out may
    be row-strided views (unit stride along a row, rows any stride apart:
    qmm_gemm_ex); otherwise they must be contiguous.
    workspace: "auto" (a buffer kept per device and stream), None (no k split
    on the matrix-core path), or a device tensor of at least
    workspace_bytes() bytes."""
    import torch
    lib = load()
    qt = _qt(qtype)
    if x.dim() != 2:
        raise ValueError("x must be [n, k]")
    n, k = x.shape
    if out is None:
        out = torch.empty((n, m), dtype=torch.float32, device=x.device)
    if tuple(out.shape) != (n, m):
        raise ValueError(f"out must be [{n}, {m}]")
    need = m * row_bytes(qt, k)
    if w.numel() * w.element_size() != need:
        raise ValueError(f"w holds {w.numel() * w.element_size()} bytes, expected {need}")
    sh = _stream(stream)
    ws_ptr, ws_len = None, 0
    if workspace is not None:
        nbytes = workspace_bytes(m, k, n, qt, path)
        if nbytes > 0:
            if isinstance(workspace, str):
                if workspace != "auto":
                    raise ValueError("workspace must be 'auto', None or a tensor")
                workspace = _auto_workspace(x.device, sh.value or 0, nbytes)
            ws_ptr = _dev(workspace, "workspace")
            ws_len = workspace.numel() * workspace.element_size()
    st = lib.qmm_gemm_ex(*_rows(out, "out"), _dev(w, "w"), *_rows(x, "x"), m, k, n, qt, PATHS[path],
                         ws_ptr, ws_len, sh)
    if st != 0:
        raise QmmError(st, "qmm_gemm_ex")
    return out


def _rows(t, what):
    """(pointer, row stride in elements) of a float32 [rows, cols] device
    tensor with unit stride along its rows."""
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{what} must be a device (cuda/hip) tensor")
    if t.dtype != torch.float32:
        raise TypeError(f"{what} must be torch.float32, got {t.dtype}")
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{what} must be 2-D with unit stride along its rows")
    ld = t.stride(0) if t.shape[0] > 1 else t.shape[1]
    if ld < t.shape[1]:
        raise ValueError(f"{what} rows overlap (row stride {ld} < {t.shape[1]})")
    return ctypes.c_void_p(t.data_ptr()), ld


def moe_gateup(w_gate, w_up, expert_ids, pair_scale, x, n_expert: int, n_ff: int,
               qtype="nvfp4", gate_out=None, up_out=None, stream=None):
    """Gate and up projections over routed experts; returns (gate, up), each
    float32 [t*n_used, n_ff].  expert_ids: int32 [t, n_used]; pair_scale:
    float32 [2*t*n_used] (gate plane then up plane); x: float32 [t, in_f]."""
    import torch
    lib = load()
    qt = _qt(qtype)
    t, n_used = expert_ids.shape
    t2, in_f = x.shape
    if t2 != t:
        raise ValueError("x and expert_ids disagree on t")
    n_pairs = t * n_used
    if pair_scale.numel() != 2 * n_pairs:
        raise ValueError("pair_scale must hold 2*t*n_used floats")
    if gate_out is None:
        gate_out = torch.empty((n_pairs, n_ff), dtype=torch.float32, device=x.device)
    if up_out is None:
        up_out = torch.empty((n_pairs, n_ff), dtype=torch.float32, device=x.device)
    st = lib.qmm_moe_gateup(_dev(gate_out, "gate_out", torch.float32),
                            _dev(up_out, "up_out", torch.float32), _dev(w_gate, "w_gate"),
                            _dev(w_up, "w_up"), _dev(expert_ids, "expert_ids", torch.int32),
                            _dev(pair_scale, "pair_scale", torch.float32),
                            _dev(x, "x", torch.float32), t, n_used, n_expert, in_f, n_ff, qt,
                            _stream(stream))
    if st != 0:
        raise QmmError(st, "qmm_moe_gateup")
    return gate_out, up_out


def moe_down(w_down, expert_ids, pair_scale, act, n_expert: int, d_model: int, qtype="nvfp4",
             y=None, pair_out=None, stream=None):
    """MoE down projection; returns (y, pair_out): y float32 [t, d_model] (the
    token's slots summed in order), pair_out float32 [t*n_used, d_model] (each
    pair's scaled projection).  expert_ids: int32 [t, n_used]; pair_scale:
    float32 [t*n_used] (the down plane's); act: float32 [t*n_used, n_ff]."""
    import torch
    lib = load()
    qt = _qt(qtype)
    t, n_used = expert_ids.shape
    n_pairs = t * n_used
    n_p2, n_ff = act.shape
    if n_p2 != n_pairs:
        raise ValueError("act must hold one row per pair (t*n_used rows)")
    if pair_scale.numel() != n_pairs:
        raise ValueError("pair_scale must hold t*n_used floats")
    if y is None:
        y = torch.empty((t, d_model), dtype=torch.float32, device=act.device)
    if pair_out is None:
        pair_out = torch.empty((n_pairs, d_model), dtype=torch.float32, device=act.device)
    st = lib.qmm_moe_down(_dev(y, "y", torch.float32), _dev(pair_out, "pair_out", torch.float32),
                          _dev(w_down, "w_down"), _dev(expert_ids, "expert_ids", torch.int32),
                          _dev(pair_scale, "pair_scale", torch.float32),
                          _dev(act, "act", torch.float32), t, n_used, n_expert, n_ff, d_model, qt,
                          _stream(stream))
    if st != 0:
        raise QmmError(st, "qmm_moe_down")
    return y, pair_out


def quantize_q8_1(x, q=None, d=None, stream=None):
    """Q8_1 activations of x (float32 [rows, k], k % 32 == 0): returns
    (q int8 [rows, k], d float32 [rows, k/32])."""
    import torch
    lib = load()
    rows, k = x.shape
    if q is None:
        q = torch.empty((rows, k), dtype=torch.int8, device=x.device)
    if d is None:
        d = torch.empty((rows, k // 32), dtype=torch.float32, device=x.device)
    st = lib.qmm_quantize_q8_1(_dev(q, "q", torch.int8), _dev(d, "d", torch.float32),
                               _dev(x, "x", torch.float32), rows, k, _stream(stream))
    if st != 0:
        raise QmmError(st, "qmm_quantize_q8_1")
    return q, d


def moe_gateup_q8(w_gate, w_up, expert_ids, pair_scale, xq, xd, n_expert: int, n_ff: int,
                  qtype="nvfp4", gate_out=None, up_out=None, stream=None):
    """moe_gateup on Q8_1 activations (xq int8 [t, in_f], xd float32
    [t, in_f/32] from quantize_q8_1); returns (gate, up)."""
    import torch
    lib = load()
    qt = _qt(qtype)
    t, n_used = expert_ids.shape
    t2, in_f = xq.shape
    if t2 != t or xd.numel() != t * (in_f // 32):
        raise ValueError("xq / xd do not match expert_ids")
    n_pairs = t * n_used
    if pair_scale.numel() != 2 * n_pairs:
        raise ValueError("pair_scale must hold 2*t*n_used floats")
    if gate_out is None:
        gate_out = torch.empty((n_pairs, n_ff), dtype=torch.float32, device=xq.device)
    if up_out is None:
        up_out = torch.empty((n_pairs, n_ff), dtype=torch.float32, device=xq.device)
    st = lib.qmm_moe_gateup_q8(_dev(gate_out, "gate_out", torch.float32),
                               _dev(up_out, "up_out", torch.float32), _dev(w_gate, "w_gate"),
                               _dev(w_up, "w_up"), _dev(expert_ids, "expert_ids", torch.int32),
                               _dev(pair_scale, "pair_scale", torch.float32),
                               _dev(xq, "xq", torch.int8), _dev(xd, "xd", torch.float32), t, n_used,
                               n_expert, in_f, n_ff, qt, _stream(stream))
    if st != 0:
        raise QmmError(st, "qmm_moe_gateup_q8")
    return gate_out, up_out


def moe_gateup_act(w_gate, w_up, expert_ids, pair_scale, x, n_expert: int, n_ff: int, qtype="nvfp4",
                   limit: float = 7.0, act=None, stream=None):
    """Gate and up projections fused with the SwiGLU/clamp activation:
    returns act float32 [t*n_used, n_ff] = silu(min(gate, limit)) *
    clamp(up, -limit, limit) (the down projection's input).  Arguments as
    moe_gateup; limit > 0 or inf."""
    import torch
    lib = load()
    qt = _qt(qtype)
    t, n_used = expert_ids.shape
    t2, in_f = x.shape
    if t2 != t:
        raise ValueError("x and expert_ids disagree on t")
    n_pairs = t * n_used
    if pair_scale.numel() != 2 * n_pairs:
        raise ValueError("pair_scale must hold 2*t*n_used floats")
    if act is None:
        act = torch.empty((n_pairs, n_ff), dtype=torch.float32, device=x.device)
    st = lib.qmm_moe_gateup_act(_dev(act, "act", torch.float32), _dev(w_gate, "w_gate"), _dev(w_up, "w_up"),
                                _dev(expert_ids, "expert_ids", torch.int32),
                                _dev(pair_scale, "pair_scale", torch.float32), _dev(x, "x", torch.float32),
                                t, n_used, n_expert, in_f, n_ff, qt, float(limit), _stream(stream))
    if st != 0:
        raise QmmError(st, "qmm_moe_gateup_act")
    return act


def moe_gateup_act_q8(w_gate, w_up, expert_ids, pair_scale, xq, xd, n_expert: int, n_ff: int,
                      qtype="nvfp4", limit: float = 7.0, act=None, stream=None):
    """moe_gateup_act on Q8_1 activations (xq, xd from quantize_q8_1)."""
    import torch
    lib = load()
    qt = _qt(qtype)
    t, n_used = expert_ids.shape
    t2, in_f = xq.shape
    if t2 != t or xd.numel() != t * (in_f // 32):
        raise ValueError("xq / xd do not match expert_ids")
    n_pairs = t * n_used
    if pair_scale.numel() != 2 * n_pairs:
        raise ValueError("pair_scale must hold 2*t*n_used floats")
    if act is None:
        act = torch.empty((n_pairs, n_ff), dtype=torch.float32, device=xq.device)
    st = lib.qmm_moe_gateup_act_q8(_dev(act, "act", torch.float32), _dev(w_gate, "w_gate"), _dev(w_up, "w_up"),
                                   _dev(expert_ids, "expert_ids", torch.int32),
                                   _dev(pair_scale, "pair_scale", torch.float32), _dev(xq, "xq", torch.int8),
                                   _dev(xd, "xd", torch.float32), t, n_used, n_expert, in_f, n_ff, qt,
                                   float(limit), _stream(stream))
    if st != 0:
        raise QmmError(st, "qmm_moe_gateup_act_q8")
    return act


def moe_gateup_probe(arm: str, w_gate, w_up, expert_ids, pair_scale, x, n_expert: int, n_ff: int,
                     qtype="nvfp4", gate_out=None, up_out=None, stream=None):
    """A measurement twin of moe_gateup: arm "loadonly" (the same loads, no
    arithmetic) or "mathonly" (the arithmetic on one cached unit per row
    group).  The outputs are not projections."""
    import torch
    lib = load()
    arms = {"loadonly": 1, "mathonly": 2}
    if arm not in arms:
        raise ValueError(f"unknown arm {arm!r}")
    qt = _qt(qtype)
    t, n_used = expert_ids.shape
    in_f = x.shape[1]
    n_pairs = t * n_used
    if gate_out is None:
        gate_out = torch.empty((n_pairs, n_ff), dtype=torch.float32, device=x.device)
    if up_out is None:
        up_out = torch.empty((n_pairs, n_ff), dtype=torch.float32, device=x.device)
    st = lib.qmm_moe_gateup_probe(arms[arm], _dev(gate_out, "gate_out", torch.float32),
                                  _dev(up_out, "up_out", torch.float32), _dev(w_gate, "w_gate"),
                                  _dev(w_up, "w_up"), _dev(expert_ids, "expert_ids", torch.int32),
                                  _dev(pair_scale, "pair_scale", torch.float32), _dev(x, "x", torch.float32),
                                  t, n_used, n_expert, in_f, n_ff, qt, _stream(stream))
    if st != 0:
        raise QmmError(st, "qmm_moe_gateup_probe")
    return gate_out, up_out


def moe_down_q8(w_down, expert_ids, pair_scale, aq, ad, n_expert: int, d_model: int, qtype="nvfp4",
                y=None, pair_out=None, stream=None):
    """moe_down on Q8_1 pair activations (aq int8 [t*n_used, n_ff], ad
    float32 [t*n_used, n_ff/32] from quantize_q8_1); returns (y, pair_out)."""
    import torch
    lib = load()
    qt = _qt(qtype)
    t, n_used = expert_ids.shape
    n_pairs = t * n_used
    n_p2, n_ff = aq.shape
    if n_p2 != n_pairs or ad.numel() != n_pairs * (n_ff // 32):
        raise ValueError("aq / ad must hold one row per pair (t*n_used rows)")
    if pair_scale.numel() != n_pairs:
        raise ValueError("pair_scale must hold t*n_used floats")
    if y is None:
        y = torch.empty((t, d_model), dtype=torch.float32, device=aq.device)
    if pair_out is None:
        pair_out = torch.empty((n_pairs, d_model), dtype=torch.float32, device=aq.device)
    st = lib.qmm_moe_down_q8(_dev(y, "y", torch.float32), _dev(pair_out, "pair_out", torch.float32),
                             _dev(w_down, "w_down"), _dev(expert_ids, "expert_ids", torch.int32),
                             _dev(pair_scale, "pair_scale", torch.float32), _dev(aq, "aq", torch.int8),
                             _dev(ad, "ad", torch.float32), t, n_used, n_expert, n_ff, d_model, qt,
                             _stream(stream))
    if st != 0:
        raise QmmError(st, "qmm_moe_down_q8")
    return y, pair_out


def repack_nvfp4_v2(w, rows: int, k: int, out=None, stream=None):
    """NVFP4 rows (uint8, rows*k/64*36 bytes) -> the same values in the
    NVFP4_V2 layout (a new uint8 tensor, or ``out``)."""
    import torch
    lib = load()
    nbytes = rows * (k // 64) * 36
    if w.numel() * w.element_size() < nbytes:
        raise ValueError("w holds fewer than rows*k/64*36 bytes")
    if out is None:
        out = torch.empty(nbytes, dtype=torch.uint8, device=w.device)
    st = lib.qmm_nvfp4_repack_v2(_dev(out, "out"), _dev(w, "w"), rows, k, _stream(stream))
    if st != 0:
        raise QmmError(st, "qmm_nvfp4_repack_v2")
    return out


def stream_loadonly(w, m: int, k: int, qtype, sink=None, stream=None):
    """Load-only twin of the GEMV: reads all of w, writes one checksum per row."""
    import torch
    lib = load()
    if sink is None:
        sink = torch.empty(m, dtype=torch.int32, device=w.device)
    st = lib.qmm_stream_loadonly(_dev(sink, "sink"), _dev(w, "w"), m, k, _qt(qtype), _stream(stream))
    if st != 0:
        raise QmmError(st, "qmm_stream_loadonly")
    return sink


# ------------------------------------------------------------------ decode step
class _KvCacheStruct(ctypes.Structure):
    """qmm_kv_cache."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("k", "v", "k_scale", "v_scale")] +
                [(n, ctypes.c_int64) for n in ("n_pages", "n_kv", "page_size", "head_dim", "page_stride", "head_stride",
                                               "slot_stride", "scale_page_stride", "scale_head_stride",
                                               "scale_slot_stride")] + [("kind", ctypes.c_int32)])


class KVCache:
    """A paged key-value cache: views k and v [n_pages, n_kv, page_size, head_dim] of the caller's
    device memory, which the object keeps alive, in any order of pages, heads and tokens with unit
    stride along head_dim (pages that hold tokens outermost: ``pages.transpose(1, 2)``).

    float16 or bfloat16, or int8 codes with k_scale and v_scale float32 [n_pages, n_kv, page_size].
    page_size: a power of two; head_dim: a multiple of 32 up to 256."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        import torch
        kinds = {torch.float16: "f16", torch.bfloat16: "bf16", torch.int8: "q8"}
        if not isinstance(k, torch.Tensor) or not isinstance(v, torch.Tensor) or not k.is_cuda or not v.is_cuda:
            raise TypeError("k and v must be device (cuda/hip) tensors")
        if k.dtype not in kinds or v.dtype != k.dtype:
            raise TypeError(f"k and v must both be float16, bfloat16 or int8, got {k.dtype} and {v.dtype}")
        if k.dim() != 4 or k.shape != v.shape:
            raise ValueError("k and v must both be [n_pages, n_kv, page_size, head_dim]")
        self.kind = kinds[k.dtype]
        strides = _view_strides(k, 3, "k")
        if strides != _view_strides(v, 3, "v"):
            raise ValueError("k and v must have the same strides")
        scale_strides = (1, 1, 1)
        if (k_scale is not None or v_scale is not None) != (self.kind == "q8"):
            raise ValueError("k_scale and v_scale belong to an int8 cache")
        if self.kind == "q8":
            for t, what in ((k_scale, "k_scale"), (v_scale, "v_scale")):
                if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != torch.float32:
                    raise TypeError(f"{what} must be a float32 device (cuda/hip) tensor")
                if t.shape != k.shape[:3]:
                    raise ValueError(f"{what} must be [n_pages, n_kv, page_size]")
            scale_strides = _view_strides(k_scale, 3, "k_scale", 1)
            if scale_strides != _view_strides(v_scale, 3, "v_scale", 1):
                raise ValueError("k_scale and v_scale must have the same strides")
        self.device = k.device
        for t in (v,) if k_scale is None else (v, k_scale, v_scale):
            if t.device != k.device:
                raise ValueError(f"tensors on {k.device} and {t.device}")
        self._index = k.get_device()
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.n_pages, self.n_kv, self.page_size, self.head_dim = k.shape
        self._struct = _KvCacheStruct(
            k.data_ptr(), v.data_ptr(), None if k_scale is None else k_scale.data_ptr(),
            None if v_scale is None else v_scale.data_ptr(), *k.shape, *strides, *scale_strides, KV_KINDS[self.kind])
        self._ptr = ctypes.addressof(self._struct)


def _view_strides(t, n: int, what: str, least=None):
    """Strides of t's first n axes, those of axes of one entry replaced by the smallest that is
    valid; unit stride along a last axis behind them."""
    least = t.shape[-1] if least is None else least
    if t.dim() > n and t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{what} must have unit stride along head_dim")
    strides = tuple(t.stride(i) if t.shape[i] > 1 else least for i in range(n))
    spans = sorted((s, t.shape[i]) for i, s in enumerate(strides) if t.shape[i] > 1)
    reach = least
    for stride, count in spans:
        if stride < reach:
            raise ValueError(f"{what}'s rows overlap (strides {strides})")
        reach = stride * (count - 1) + reach
    return strides


# The calls below are a decode step's small kernels, a few microseconds each: _step (csrc/step_bind.cpp,
# built beside the library) checks their tensors and calls the library.
_STEP = None


def _load_step():
    """The _step module, its calls bound to the loaded library."""
    global _STEP, _current_device, _current_stream
    import torch
    lib = load()
    path = os.path.join(_HERE, "_step.so")
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is not built: run `python -m gemv_prefill_decode_amd.build` "
                           "(or __graft_entry__.build())")
    from . import _step
    _step.bind(*(ctypes.cast(getattr(lib, "qmm_" + n), ctypes.c_void_p).value
                 for n in ("paged_extend", "kv_append", "paged_attention", "paged_attention_workspace_bytes",
                           "add_rmsnorm", "add_rmsnorm_q8")))
    _current_device = getattr(torch._C, "_cuda_getDevice", None)
    _current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    _STEP = _step
    return _step


def _run(f, dev, stream, *args):
    """f on device dev, on the given stream or the device's current one."""
    if stream is not None and getattr(stream, "device_index", dev) != dev:
        raise ValueError(f"the stream is on device {stream.device_index}, the tensors on device {dev}")
    if stream is None and _current_device() == dev:
        st = f(_current_stream(dev), dev, *args)
    else:
        import torch
        with torch.cuda.device(dev):
            st = f(_current_stream(dev) if stream is None else stream.cuda_stream, dev, *args)
    if st != 0:
        raise QmmError(st, "qmm_" + f.__name__)


def _new(shape, dtype, like, stream):
    """An output (or workspace) on like's device, allocated on the stream that writes it: memory of
    another stream may still be read there."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def paged_extend(block_table, cached_lens, new_lens, free_pages, page_size: int, n_rows: int, seq_lens=None,
                 slots=None, positions=None, pages_used=None, stream=None):
    """Page tables of a step: gives each sequence (cached_lens tokens in the cache, new_lens more)
    the pages it newly needs from free_pages, in order, written into block_table (int32
    [batch, max_pages], in place); returns (seq_lens [batch], slots [n_rows], positions [n_rows],
    pages_used [1]), all int32.  slots and positions are those of the new tokens' rows, sequence
    after sequence, -1 behind the last row and (slots) for a sequence that is refused because its
    table row or the free list is too short: its seq_lens entry stays cached_lens."""
    step = _STEP or _load_step()
    dev = step.device(block_table, "block_table")
    if seq_lens is None:
        seq_lens = _new(cached_lens.shape, cached_lens.dtype, block_table, stream)
    if slots is None:
        slots = _new(n_rows, cached_lens.dtype, block_table, stream)
    if positions is None:
        positions = _new(n_rows, cached_lens.dtype, block_table, stream)
    if pages_used is None:
        pages_used = _new(1, cached_lens.dtype, block_table, stream)
    _run(step.paged_extend, dev, stream, block_table, cached_lens, new_lens, free_pages, page_size, n_rows, seq_lens,
         slots, positions, pages_used)
    return seq_lens, slots, positions, pages_used


def kv_append(cache: KVCache, k, v, slots, stream=None):
    """Writes new keys and values (float32 [n, n_kv, head_dim], or [n, n_kv*head_dim]; rows any
    stride apart, as views of a fused projection's output) into their slots (int32 [n]; a slot
    outside the cache, such as -1, is skipped; the others must differ)."""
    step = _STEP or _load_step()
    _run(step.kv_append, cache._index, stream, cache._ptr, k, v, slots)


def paged_attention_workspace_bytes(batch: int, n_q: int, cache: KVCache, max_pages: int) -> int:
    """Bytes of workspace paged_attention uses for these sizes (0: none)."""
    import torch
    with torch.cuda.device(cache.device):
        r = load().qmm_paged_attention_workspace_bytes(batch, n_q, cache.n_kv, cache.head_dim, max_pages, cache.page_size)
    if r < 0:
        raise QmmError(-r, "qmm_paged_attention_workspace_bytes")
    return r


def paged_attention(q, cache: KVCache, block_table, seq_lens, scale=None, out=None, lse=None, workspace="auto",
                    stream=None):
    """Attention of one new token per sequence over its cached tokens; returns out (float32, q's
    shape).  q: float32 [batch, n_q, head_dim] or [batch, n_q*head_dim], rows any stride apart;
    block_table: int32 [batch, max_pages]; seq_lens: int32 [batch], the new token included, 0 for
    a padded row (its output is zero).  scale: 1/sqrt(head_dim) by default.  lse: a float32
    [batch, n_q] tensor that takes the log-sum-exp of the scores.  workspace: "auto" (allocated
    for the call, from the graph's own memory under capture) or a device tensor of at least
    paged_attention_workspace_bytes() bytes that no other call uses at the same time.  A caller
    that knows a bound on the lengths may pass fewer columns of a wider block_table: up to 384
    tokens per row mostly take one kernel and no workspace."""
    step = _STEP or _load_step()
    if out is None:
        out = _new(q.shape, q.dtype, q, stream)
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError("workspace must be 'auto', None or a tensor")
        workspace = True
    args = (cache._ptr, q, block_table, seq_lens, scale, out, lse, workspace)
    if stream is None or workspace is not True:
        _run(step.paged_attention, cache._index, stream, *args)
    else:
        import torch
        with torch.cuda.stream(stream):     # the workspace is allocated on it
            _run(step.paged_attention, cache._index, stream, *args)
    return out


def add_rmsnorm(x, weight, residual=None, eps: float = 1e-5, y=None, h=None, stream=None):
    """Residual addition and RMS norm; returns (y, h): h = x + residual (None without a residual,
    unless a tensor is given for it) and y = h * weight / sqrt(mean(h*h) + eps), float32 [n, k],
    k a multiple of 4.  Rows of any of them may be any multiple of 4 apart."""
    step = _STEP or _load_step()
    dev = step.device(x, "x")
    if y is None:
        y = _new(x.shape, x.dtype, x, stream)
    if h is None and residual is not None:
        h = _new(x.shape, x.dtype, x, stream)
    _run(step.add_rmsnorm, dev, stream, x, weight, residual, eps, y, h)
    return y, h


def add_rmsnorm_q8(x, weight, residual=None, eps: float = 1e-5, q=None, d=None, h=None, stream=None):
    """add_rmsnorm with y as Q8_1 activations; returns (q int8 [n, k], d float32 [n, k/32], h), q
    and d as moe_gateup_q8 takes them.  k a multiple of 32."""
    step = _STEP or _load_step()
    dev = step.device(x, "x")
    if q is None or d is None:
        import torch
        q = _new(x.shape, torch.int8, x, stream) if q is None else q
        d = _new((x.shape[0], x.shape[1] // 32), torch.float32, x, stream) if d is None else d
    if h is None and residual is not None:
        h = _new(x.shape, x.dtype, x, stream)
    _run(step.add_rmsnorm_q8, dev, stream, x, weight, residual, eps, q, d, h)
    return q, d, h
