"""Python binding of ``libmoe.so`` (include/moe.h, moe_dense.h, moe_mx.h, moe_grouped.h): argument marshalling only.

Every function with a ``moe_`` name calls the C entry point of the same name.
Tensors are passed as raw pointers (``torch.Tensor.data_ptr()`` for device
memory, numpy arrays for host memory); streams as ``torch.cuda.Stream`` handles.
The library does all the work; if it is missing this module raises on import.
"""
from __future__ import annotations

import ctypes
import os
import re
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe.so")
HEADERS = [os.path.join(os.path.dirname(_HERE), "include", h) for h in ("moe.h", "moe_dense.h", "moe_mx.h", "moe_grouped.h")]
HEADER = HEADERS[0]

MOE_OK, MOE_EINVAL, MOE_ENULL, MOE_EDTYPE, MOE_EWORKSPACE, MOE_ENOSLOT, MOE_ESTALE, MOE_EHIP, MOE_ELEASE = \
    0, -1, -2, -3, -4, -5, -6, -7, -8
MOE_F32, MOE_BF16 = 0, 1
MOE_WF_Q4_G32, MOE_WF_Q4_ROW, MOE_WF_Q8_ROW = 0, 1, 2
MOE_ROPE_HALF, MOE_ROPE_INTERLEAVED = 0, 1
MOE_MX_FLOOR, MOE_MX_UP = 0, 1
MOE_ROPE_PLAIN, MOE_ROPE_LINEAR, MOE_ROPE_NTK, MOE_ROPE_YARN = 0, 1, 2, 3


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = _lib.moe_status_string(status).decode()
        if status == MOE_EHIP:
            msg += ": " + _lib.moe_last_hip_error().decode()
        super().__init__(f"{where}: {msg} ({status})")


class moe_cfg(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("n_experts", ctypes.c_int32), ("n_group", ctypes.c_int32),
                ("topk_group", ctypes.c_int32), ("top_k", ctypes.c_int32), ("moe_inter", ctypes.c_int32),
                ("shared_inter", ctypes.c_int32), ("group_size", ctypes.c_int32),
                ("routed_scaling_factor", ctypes.c_float), ("norm_topk_prob", ctypes.c_int32),
                ("mfma_min_tokens", ctypes.c_int32), ("weight_format", ctypes.c_int32), ("act_int8", ctypes.c_int32)]


class moe_slot_view(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("slot_bytes", ctypes.c_int64), ("table", ctypes.c_void_p),
                ("n_slots", ctypes.c_int32), ("gen", ctypes.c_void_p), ("slot_gen", ctypes.c_void_p),
                ("lease", ctypes.c_uint64)]


class moe_layer_call(ctypes.Structure):
    _fields_ = [("cfg", ctypes.POINTER(moe_cfg)), ("x", ctypes.c_void_p), ("x_dtype", ctypes.c_int32),
                ("S", ctypes.c_int32), ("W_gate", ctypes.c_void_p), ("bias", ctypes.c_void_p),
                ("idx", ctypes.c_void_p), ("w", ctypes.c_void_p), ("experts", ctypes.POINTER(moe_slot_view)),
                ("shared", ctypes.c_void_p), ("y", ctypes.c_void_p), ("ws", ctypes.c_void_p),
                ("ws_bytes", ctypes.c_size_t)]


class moe_rope_tensor(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("out", ctypes.c_void_p), ("x_token", ctypes.c_int64),
                ("x_head", ctypes.c_int64), ("out_token", ctypes.c_int64), ("out_head", ctypes.c_int64),
                ("heads", ctypes.c_int32)]


class moe_mx_rows(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("e", ctypes.c_void_p), ("ldq", ctypes.c_int64), ("lde", ctypes.c_int64),
                ("expert_q", ctypes.c_int64), ("expert_e", ctypes.c_int64)]


class moe_groups(ctypes.Structure):
    _fields_ = [("first", ctypes.c_void_p), ("order", ctypes.c_void_p), ("n", ctypes.c_int32),
                ("top_k", ctypes.c_int32)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built: run __graft_entry__.build() (hipcc for gfx950)")
    # torch ships its own HIP runtime and loads it by path.  Loaded first, the
    # library would resolve libamdhip64.so.7 through its run path to a second
    # runtime in the same process, which sees no device and knows none of
    # torch's streams; with torch loaded first (above), the soname binds to torch's copy.
    L = ctypes.CDLL(LIB_PATH)
    p, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    f32, f64 = ctypes.c_float, ctypes.c_double
    cp = ctypes.POINTER(moe_cfg)
    sigs = {
        "moe_validate_cfg": (ctypes.c_int, [cp]),
        "moe_status_string": (ctypes.c_char_p, [ctypes.c_int]),
        "moe_last_hip_error": (ctypes.c_char_p, []),
        "moe_expert_bytes": (i64, [cp, i32]),
        "moe_workspace_bytes": (sz, [cp, i32]),
        "moe_workspace_init": (ctypes.c_int, [p, sz, p]),
        "moe_pack_expert": (ctypes.c_int, [cp, i32, p, p, p, p, p, p, p, i32, p]),
        "moe_unpack_expert": (ctypes.c_int, [cp, i32, p, p, p, p, p, p, p]),
        "moe_pack_expert_rows": (ctypes.c_int, [cp, i32, p, p, p, p, p, p, p, i32, p]),
        "moe_unpack_expert_rows": (ctypes.c_int, [cp, i32, p, p, p, p, p, p, p]),
        "moe_route": (ctypes.c_int, [cp, p, i32, i32, p, p, p, p, p, sz, p]),
        "moe_ffn": (ctypes.c_int, [cp, p, i32, i32, p, p, ctypes.POINTER(moe_slot_view), p, p, p, sz, p]),
        "moe_layer": (ctypes.c_int, [cp, p, i32, i32, p, p, p, p, ctypes.POINTER(moe_slot_view), p, p, p, sz, p]),
        "moe_layer_noalloc": (ctypes.c_int, [cp, p, i32, i32, p, p, p, p, ctypes.POINTER(moe_slot_view), p, p, p]),
        "moe_chain_create": (ctypes.c_int, [ctypes.POINTER(moe_layer_call), i32, ctypes.POINTER(p)]),
        "moe_chain_launch": (ctypes.c_int, [p, p]),
        "moe_chain_destroy": (None, [p]),
        "moe_pool_create": (ctypes.c_int, [cp, i32, i32, i32, ctypes.POINTER(p)]),
        "moe_pool_destroy": (None, [p]),
        "moe_pool_register_host": (ctypes.c_int, [p, i32, i32, p]),
        "moe_pool_acquire": (ctypes.c_int, [p, i32, p, i32, ctypes.POINTER(moe_slot_view), ctypes.POINTER(i32), p, p]),
        "moe_pool_release": (ctypes.c_int, [p, i32, p]),
        "moe_pool_prefetch": (ctypes.c_int, [p, i32, p, i32, ctypes.POINTER(i32), p]),
        "moe_pool_trace": (ctypes.c_int, [p, p, i32]),
        "moe_pool_stats": (ctypes.c_int, [p, ctypes.c_char_p, sz]),
        "moe_pool_check_view": (ctypes.c_int, [p, i32, ctypes.POINTER(moe_slot_view)]),
        "moe_norm_quant": (ctypes.c_int, [p, i32, i64, p, i64, p, i32, f32, i32, i32, p, i64, p, i32, i64, p, i64, p, p]),
        "moe_silu_quant": (ctypes.c_int, [p, p, i32, i64, i32, i32, p, i32, i64, p, i64, p, p]),
        "moe_qmatmul_workspace_bytes": (i64, [p, i64, p, i64, i32, i32, i32]),
        "moe_qmatmul": (ctypes.c_int, [p, i64, p, p, i64, p, i32, i32, i32, p, i32, i64, p, sz, p]),
        "moe_rope": (ctypes.c_int, [p, p, i32, i32, i32, i32, i32, i32, p, i32, p, f64, p]),
        "moe_rope_freqs": (ctypes.c_int, [i32, f64, i32, f64, i32, f64, f64, p, ctypes.POINTER(f64)]),
        "moe_mx_quant": (ctypes.c_int, [p, i32, i64, i32, i32, i32, p, i64, p, i64, p]),
        "moe_mx_silu_quant": (ctypes.c_int, [p, p, i32, i64, i32, i32, i32, p, i64, p, i64, p]),
        "moe_mx_values": (ctypes.c_int, [p, i64, p, i64, i32, i32, p, i32, i64, p]),
        "moe_mx_matmul_workspace_bytes": (i64, [p, p, i32, i32, i32]),
        "moe_mx_matmul": (ctypes.c_int, [p, p, i32, i32, i32, p, i32, i64, p, sz, p]),
        "moe_group_workspace_bytes": (i64, [i32, i32, i32]),
        "moe_group": (ctypes.c_int, [p, i32, i32, i32, p, p, p, p, sz, p]),
        "moe_grouped_matmul_workspace_bytes": (i64, [p, i64, i32, p, i64, i64, p, i32, i32, i32]),
        "moe_grouped_matmul": (ctypes.c_int, [p, i64, i32, p, i64, i64, p, i32, i32, i32, p, i32, i64, p, sz, p]),
        "moe_mx_grouped_matmul_workspace_bytes": (i64, [p, i32, p, p, i32, i32, i32]),
        "moe_mx_grouped_matmul": (ctypes.c_int, [p, i32, p, p, i32, i32, i32, p, i32, i64, p, sz, p]),
        "moe_combine": (ctypes.c_int, [p, i32, i64, i32, p, p, i32, i32, i32, p, i64, p, i32, i64, p]),
        "moe_profile_enable": (ctypes.c_int, [ctypes.c_int]),
        "moe_profile_report": (ctypes.c_int, [ctypes.c_char_p, sz]),
    }
    for name, (res, args) in sigs.items():
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args
    return L


_lib = _load()


def header_functions() -> list[str]:
    """Names of the functions that the library's headers declare."""
    text = "".join(open(h).read() for h in HEADERS)
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(moe_[a-z_]+)\s*\(", text)))


def lib() -> ctypes.CDLL:
    return _lib


MFMA_MIN_TOKENS = 3  # default threshold of the matrix-core path (tokens per expert)


def make_cfg(c, mfma_min_tokens: int = MFMA_MIN_TOKENS, act_int8: int = 0) -> moe_cfg:
    """moe_cfg from any object with the LayerConfig field names."""
    return moe_cfg(c.hidden, c.n_experts, c.n_group, c.topk_group, c.top_k, c.moe_inter, c.shared_inter,
                   c.group_size, c.routed_scaling_factor, c.norm_topk_prob, mfma_min_tokens,
                   getattr(c, "weight_format", MOE_WF_Q4_G32), act_int8)


def ptr(t) -> int | None:
    """Raw address of a torch tensor or numpy array, or an address given as an int (None passes NULL)."""
    if t is None or isinstance(t, int):
        return t
    if hasattr(t, "data_ptr"):
        return t.data_ptr()
    return t.ctypes.data


def stream_handle(stream=None) -> int | None:
    if stream is None:
        import torch
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def _check(rc: int, where: str) -> None:
    if rc != MOE_OK:
        raise MoeError(rc, where)


def moe_validate_cfg(cfg: moe_cfg) -> int:
    return _lib.moe_validate_cfg(ctypes.byref(cfg))


def moe_expert_bytes(cfg: moe_cfg, inter: int) -> int:
    return _lib.moe_expert_bytes(ctypes.byref(cfg), inter)


def moe_workspace_bytes(cfg: moe_cfg, max_S: int) -> int:
    return _lib.moe_workspace_bytes(ctypes.byref(cfg), max_S)


def moe_workspace_init(ws, ws_bytes: int | None = None, stream=None) -> None:
    """Write the workspace header (magic words, zeroed counters) on `stream`."""
    n = ws.numel() * ws.element_size() if ws_bytes is None else ws_bytes
    _check(_lib.moe_workspace_init(ptr(ws), n, stream_handle(stream)), "moe_workspace_init")


def workspace(cfg: moe_cfg, max_S: int, device="cuda", stream=None):
    """A device workspace for up to max_S tokens, initialised (torch uint8 tensor)."""
    import torch
    ws = torch.empty(moe_workspace_bytes(cfg, max_S), dtype=torch.uint8, device=device)
    moe_workspace_init(ws, stream=stream)
    return ws


def moe_pack_expert(cfg: moe_cfg, inter: int, qg, sg, qu, su, qd, sd, dst, where: int, stream=None) -> None:
    st = stream_handle(stream) if where == 1 else None
    _check(_lib.moe_pack_expert(ctypes.byref(cfg), inter, ptr(qg), ptr(sg), ptr(qu), ptr(su), ptr(qd), ptr(sd),
                                ptr(dst), where, st), "moe_pack_expert")


def moe_unpack_expert(cfg: moe_cfg, inter: int, src, qg, sg, qu, su, qd, sd) -> None:
    _check(_lib.moe_unpack_expert(ctypes.byref(cfg), inter, ptr(src), ptr(qg), ptr(sg), ptr(qu), ptr(su), ptr(qd),
                                  ptr(sd)), "moe_unpack_expert")


def moe_pack_expert_rows(cfg: moe_cfg, inter: int, qg, sg, qu, su, qd, sd, dst, where: int, stream=None) -> None:
    st = stream_handle(stream) if where == 1 else None
    _check(_lib.moe_pack_expert_rows(ctypes.byref(cfg), inter, ptr(qg), ptr(sg), ptr(qu), ptr(su), ptr(qd), ptr(sd),
                                     ptr(dst), where, st), "moe_pack_expert_rows")


def moe_unpack_expert_rows(cfg: moe_cfg, inter: int, src, qg, sg, qu, su, qd, sd) -> None:
    _check(_lib.moe_unpack_expert_rows(ctypes.byref(cfg), inter, ptr(src), ptr(qg), ptr(sg), ptr(qu), ptr(su),
                                       ptr(qd), ptr(sd)), "moe_unpack_expert_rows")


def pack_expert(cfg: moe_cfg, inter: int, qg, sg, qu, su, qd, sd, dst, where: int, stream=None) -> None:
    """moe_pack_expert or moe_pack_expert_rows, by cfg.weight_format."""
    f = moe_pack_expert if cfg.weight_format == MOE_WF_Q4_G32 else moe_pack_expert_rows
    f(cfg, inter, qg, sg, qu, su, qd, sd, dst, where, stream)


def moe_route(cfg: moe_cfg, x, x_dtype: int, S: int, W, bias, idx, w, ws, ws_bytes: int, stream=None) -> None:
    _check(_lib.moe_route(ctypes.byref(cfg), ptr(x), x_dtype, S, ptr(W), ptr(bias), ptr(idx), ptr(w), ptr(ws),
                          ws_bytes, stream_handle(stream)), "moe_route")


def moe_ffn(cfg: moe_cfg, x, x_dtype: int, S: int, idx, w, view: moe_slot_view, shared, y, ws, ws_bytes: int,
            stream=None) -> None:
    _check(_lib.moe_ffn(ctypes.byref(cfg), ptr(x), x_dtype, S, ptr(idx), ptr(w), ctypes.byref(view), ptr(shared),
                        ptr(y), ptr(ws), ws_bytes, stream_handle(stream)), "moe_ffn")


def moe_layer(cfg: moe_cfg, x, x_dtype: int, S: int, W, bias, idx, w, view: moe_slot_view, shared, y, ws,
              ws_bytes: int, stream=None) -> None:
    _check(_lib.moe_layer(ctypes.byref(cfg), ptr(x), x_dtype, S, ptr(W), ptr(bias), ptr(idx), ptr(w),
                          ctypes.byref(view), ptr(shared), ptr(y), ptr(ws), ws_bytes, stream_handle(stream)),
           "moe_layer")


def moe_layer_noalloc(cfg: moe_cfg, x, x_dtype: int, S: int, W, bias, idx, w, view: moe_slot_view, shared, y,
                      stream=None) -> None:
    _check(_lib.moe_layer_noalloc(ctypes.byref(cfg), ptr(x), x_dtype, S, ptr(W), ptr(bias), ptr(idx), ptr(w),
                                  ctypes.byref(view), ptr(shared), ptr(y), stream_handle(stream)), "moe_layer_noalloc")


MOE_SCRATCH_BYTES = 8 << 20  # the library's per-device workspace of moe_layer_noalloc


def _x_dtype(x, cfg: moe_cfg) -> int:
    """dtype code of the activations x, which must be a contiguous [S, hidden] fp32 or bf16 tensor."""
    import torch
    if x.dim() != 2 or x.shape[1] != cfg.hidden or not x.is_contiguous():
        raise ValueError(f"x must be a contiguous [S, {cfg.hidden}] tensor, not {tuple(x.shape)} "
                         f"with strides {tuple(x.stride())}")
    if x.dtype == torch.float32:
        return MOE_F32
    if x.dtype == torch.bfloat16:
        return MOE_BF16
    raise ValueError(f"x must be float32 or bfloat16, not {x.dtype}")


def _check_routing(idx, w, S: int, cfg: moe_cfg) -> None:
    import torch
    for name, t, dtype in (("idx", idx, torch.int32), ("w", w, torch.float32)):
        if tuple(t.shape) != (S, cfg.top_k) or t.dtype != dtype or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous [{S}, {cfg.top_k}] {dtype} tensor")


def route(x, W, bias, cfg: moe_cfg, ws=None, stream=None):
    """(idx [S, k] int32, w [S, k] fp32) for the tokens x ([S, H] fp32 or bf16 device tensor): moe_route with
    its outputs (and, when ws is None, an initialised workspace) allocated on x's device."""
    import torch
    dt = _x_dtype(x, cfg)
    S = x.shape[0]
    ws = workspace(cfg, S, device=x.device, stream=stream) if ws is None else ws
    idx = torch.empty((S, cfg.top_k), dtype=torch.int32, device=x.device)
    w = torch.empty((S, cfg.top_k), dtype=torch.float32, device=x.device)
    moe_route(cfg, x, dt, S, W, bias, idx, w, ws, ws.numel(), stream)
    return idx, w


def ffn(x, idx, w, view: moe_slot_view, shared, cfg: moe_cfg, ws=None, stream=None):
    """y [S, H] fp32: moe_ffn with its output (and, when ws is None, a workspace) allocated on x's device."""
    import torch
    dt = _x_dtype(x, cfg)
    S = x.shape[0]
    _check_routing(idx, w, S, cfg)
    ws = workspace(cfg, S, device=x.device, stream=stream) if ws is None else ws
    y = torch.empty((S, cfg.hidden), dtype=torch.float32, device=x.device)
    moe_ffn(cfg, x, dt, S, idx, w, view, shared, y, ws, ws.numel(), stream)
    return y


def layer(x, W, bias, view: moe_slot_view, shared, cfg: moe_cfg, ws=None, stream=None):
    """(idx, w, y): moe_layer with its outputs (and, when ws is None, a workspace) allocated on x's device."""
    import torch
    dt = _x_dtype(x, cfg)
    S = x.shape[0]
    ws = workspace(cfg, S, device=x.device, stream=stream) if ws is None else ws
    idx = torch.empty((S, cfg.top_k), dtype=torch.int32, device=x.device)
    w = torch.empty((S, cfg.top_k), dtype=torch.float32, device=x.device)
    y = torch.empty((S, cfg.hidden), dtype=torch.float32, device=x.device)
    moe_layer(cfg, x, dt, S, W, bias, idx, w, view, shared, y, ws, ws.numel(), stream)
    return idx, w, y


def layer_call(cfg: moe_cfg, x, x_dtype: int, S: int, W, bias, idx, w, view: moe_slot_view, shared, y, ws,
               ws_bytes: int) -> moe_layer_call:
    """The arguments of one moe_layer call, for moe_chain_create (raw addresses; the struct keeps
    references to the cfg and view it points to)."""
    return moe_layer_call(ctypes.pointer(cfg), ptr(x), x_dtype, S, ptr(W), ptr(bias), ptr(idx), ptr(w),
                          ctypes.pointer(view), ptr(shared), ptr(y), ptr(ws), ws_bytes)


def moe_chain_create(calls) -> int:
    """Records the moe_layer calls (a sequence of layer_call results) as one graph; returns the chain handle."""
    arr = (moe_layer_call * len(calls))(*calls) if len(calls) else None
    out = ctypes.c_void_p()
    _check(_lib.moe_chain_create(arr, len(calls), ctypes.byref(out)), "moe_chain_create")
    return out.value


def moe_chain_launch(chain: int, stream=None) -> None:
    _check(_lib.moe_chain_launch(chain, stream_handle(stream)), "moe_chain_launch")


def moe_chain_destroy(chain: int | None) -> None:
    _lib.moe_chain_destroy(chain)


_CODES = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16}
_ROWS = torch.contiguous_format
_empty_like = torch.empty_like


# ---- dense operators ---------------------------------------------------------------------------------------------------
# They serve: no call has a backward pass, and the allocating ones refuse inputs that ask for gradients while torch records
# them.  A tensor written over (norm_quant's h, rope's inplace) raises its version.
# The ABI's sizes are int32, and ctypes would pass on the low 32 bits of a larger one.

def _sizes(where: str, *sizes) -> None:
    for n in sizes:
        if not -0x80000000 <= n <= 0x7FFFFFFF:
            raise MoeError(MOE_EINVAL, where)


def moe_norm_quant(x, x_dtype: int, ldx: int, residual, ldr: int, gamma, g_dtype: int, eps: float, S: int, H: int, h,
                   ldh: int, y, y_dtype: int, ldy: int, q, ldq: int, d, stream=None) -> None:
    _sizes("moe_norm_quant", S, H)
    _check(_lib.moe_norm_quant(ptr(x), x_dtype, ldx, ptr(residual), ldr, ptr(gamma), g_dtype, eps, S, H, ptr(h), ldh,
                               ptr(y), y_dtype, ldy, ptr(q), ldq, ptr(d), stream_handle(stream)), "moe_norm_quant")


def moe_silu_quant(g, u, x_dtype: int, ldx: int, S: int, I: int, y, y_dtype: int, ldy: int, q, ldq: int, d,
                   stream=None) -> None:
    _sizes("moe_silu_quant", S, I)
    _check(_lib.moe_silu_quant(ptr(g), ptr(u), x_dtype, ldx, S, I, ptr(y), y_dtype, ldy, ptr(q), ldq, ptr(d),
                               stream_handle(stream)), "moe_silu_quant")


def moe_qmatmul_workspace_bytes(q, ldq: int, w, ldw: int, S: int, N: int, K: int) -> int:
    if max(S, N, K) > 0x7FFFFFFF or min(S, N, K) < 0:
        return MOE_EINVAL
    return _lib.moe_qmatmul_workspace_bytes(ptr(q), ldq, ptr(w), ldw, S, N, K)


def moe_qmatmul(q, ldq: int, d, w, ldw: int, dw, S: int, N: int, K: int, y, y_dtype: int, ldy: int, ws, ws_bytes: int,
                stream=None) -> None:
    _sizes("moe_qmatmul", S, N, K)
    _check(_lib.moe_qmatmul(ptr(q), ldq, ptr(d), ptr(w), ldw, ptr(dw), S, N, K, ptr(y), y_dtype, ldy, ptr(ws), ws_bytes,
                            stream_handle(stream)), "moe_qmatmul")


def moe_rope(q: moe_rope_tensor, k: moe_rope_tensor | None, x_dtype: int, S: int, D: int, rot: int, offset: int,
             layout: int, pos, pos_i64: int, freqs, factor: float, stream=None) -> None:
    _sizes("moe_rope", S, D, rot, offset)
    _check(_lib.moe_rope(ctypes.byref(q), None if k is None else ctypes.byref(k), x_dtype, S, D, rot, offset, layout,
                         ptr(pos), pos_i64, ptr(freqs), factor, stream_handle(stream)), "moe_rope")


def moe_rope_freqs(rot: int, theta: float, scaling: int, scale: float, trained_length: int, beta_fast: float,
                   beta_slow: float):
    """(float64 numpy array [rot / 2], factor)."""
    import numpy as np
    _sizes("moe_rope_freqs", rot, trained_length)
    out = np.empty(max(rot, 0) // 2, np.float64)
    factor = ctypes.c_double(0.0)
    _check(_lib.moe_rope_freqs(rot, theta, scaling, scale, trained_length, beta_fast, beta_slow, ptr(out),
                               ctypes.byref(factor)), "moe_rope_freqs")
    return out, factor.value


def _code(dtype, what: str) -> int:
    code = _CODES.get(dtype)
    if code is None:
        raise ValueError(f"{what} must be float32 or bfloat16, not {dtype}")
    return code


def _rows(t, shape, what: str) -> int:
    """Row stride of the matrix t, whose rows must be contiguous and whose shape must be `shape`."""
    if t.shape == shape and len(shape) == 2:
        if t.is_contiguous():
            return shape[1]
        row, col = t.stride()
        if col == 1 or shape[1] <= 1:
            return row if shape[0] > 1 else shape[1]
    raise ValueError(f"{what} must be a matrix with contiguous rows, of shape {tuple(shape)}, not {tuple(t.shape)} "
                     f"with strides {tuple(t.stride())}")


def _vector(t, n: int, dtype, what: str) -> None:
    if t.shape != (n,) or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} vector of {n}, not {tuple(t.shape)} {t.dtype}")


# The handle of a GPU's current stream.  Small calls are bound by this module's own time: the handle alone, where torch
# has it, comes twenty times as fast as a stream object.
_stream_of = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)
_current_gpu = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


_recording = torch.is_grad_enabled
_written = torch.autograd.graph.increment_version  # of a tensor that a call wrote over


def _gpu(*tensors) -> int:
    """The index of the GPU that every given tensor is on.  None may ask for gradients where torch records them: these
    calls have no backward pass, and their outputs would be cut off from the graph without a word."""
    i = tensors[0].get_device()
    recording = _recording()
    for t in tensors:
        if t is not None:
            if recording and t.requires_grad:
                raise ValueError("this call has no backward pass: make it under torch.no_grad(), or detach the tensors that "
                                 "require gradients")
            if t.get_device() != i:
                raise ValueError(f"the tensors must be on one GPU, not on {tensors[0].device} and {t.device}")
    if i < 0:
        raise ValueError(f"the tensors must be on a GPU, not on {tensors[0].device}")
    return i


def _elsewhere(gpu: int, stream, f, inputs, *args, **kw):
    """f(*args, **kw) with `gpu`, and `stream` where one is given, made current: the outputs that f allocates then belong
    to the stream that writes them, and the memory of its inputs is not given out again before that stream is done."""
    if getattr(stream, "device_index", gpu) != gpu:
        raise ValueError(f"the stream is one of GPU {stream.device_index}, the tensors are on GPU {gpu}")
    with torch.cuda.device(gpu):
        if stream is None:
            return f(*args, **kw)
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(stream)
        with torch.cuda.stream(stream):
            for t in inputs:
                if t is not None:
                    t.record_stream(stream)
            return f(*args, **kw)


def norm_quant(x, gamma, eps: float, residual=None, h=None, y_dtype=None, quant: bool = True, stream=None):
    """(h, y, q, d) of the rows x [S, H]: moe_norm_quant with its outputs allocated on x's GPU.  h is the residual
    sum (None without a residual; written over the tensor given as h, which may be residual or x), y the norm in
    y_dtype (None: not wanted), q int8 and d fp32 the norm's quantised rows (None with quant=False)."""
    dtype, shape = x.dtype, x.shape
    xd, gd = _code(dtype, "x"), _code(gamma.dtype, "gamma")
    ldx = _rows(x, shape, "x")
    S, H = shape
    _vector(gamma, H, gamma.dtype, "gamma")
    ldr = ldh = ldy = ldq = yd = 0
    if residual is not None:
        ldr = _rows(residual, shape, "residual")
        if residual.dtype != dtype:
            raise ValueError(f"residual must have x's type {dtype}, not {residual.dtype}")
    if h is not None:
        if residual is None:
            raise ValueError("h is the sum with a residual: none is given")
        ldh = _rows(h, shape, "h")
        if h.dtype != dtype:
            raise ValueError(f"h must have x's type {dtype}, not {h.dtype}")
    if y_dtype is not None:
        yd = _code(y_dtype, "y_dtype")
    elif residual is None and not quant:
        raise ValueError("no output is asked for")
    if (S | H) >> 31:
        _sizes("moe_norm_quant", S, H)
    gpu = _gpu(x, gamma, residual, h)
    if stream is not None or gpu != _current_gpu():
        return _elsewhere(gpu, stream, norm_quant, (x, gamma, residual, h), x, gamma, eps, residual, h, y_dtype, quant)
    y = q = d = None
    py = pq = pd = ph = pr = None
    over = h
    if residual is not None:
        pr = residual.data_ptr()
        if h is None:
            h = _empty_like(x, memory_format=_ROWS)
            ldh = H
        ph = h.data_ptr()
    if y_dtype is not None:
        y = _empty_like(x, dtype=y_dtype, memory_format=_ROWS)
        py = y.data_ptr()
    if quant:
        q, d = _empty_like(x, dtype=torch.int8, memory_format=_ROWS), x.new_empty(S, dtype=torch.float32)
        pq, pd = q.data_ptr(), d.data_ptr()
    rc = _lib.moe_norm_quant(x.data_ptr(), xd, ldx, pr, ldr, gamma.data_ptr(), gd, eps, S, H, ph, ldh, py, yd, H, pq, H, pd,
                             _stream_of(gpu))
    if rc:
        raise MoeError(rc, "moe_norm_quant")
    if over is not None:
        _written(over)
    return h, y, q, d


def silu_quant(g, u=None, y_dtype=None, quant: bool = True, stream=None):
    """(y, q, d) of silu(g) * u, both [S, I], or of the halves of g [S, 2 I] where u is None: moe_silu_quant with its
    outputs allocated on g's GPU.  y in y_dtype (None: not wanted), q int8 and d fp32 (None with quant=False)."""
    dtype, shape = g.dtype, g.shape
    xd, ldx = _code(dtype, "g"), _rows(g, shape, "g")
    S, I = shape
    up = g.data_ptr()
    if u is None:
        if I % 2:
            raise ValueError(f"g holds gate and up side by side: its width {I} must be even")
        I //= 2
        up += I * g.element_size()
    else:
        if u.dtype != dtype:
            raise ValueError(f"u must have g's type {dtype}, not {u.dtype}")
        if _rows(u, shape, "u") != ldx:
            raise ValueError(f"u must have g's row stride {ldx}, not {u.stride(0)}")
        up = u.data_ptr()
    yd = 0
    if y_dtype is not None:
        yd = _code(y_dtype, "y_dtype")
    elif not quant:
        raise ValueError("no output is asked for")
    if (S | I) >> 31:
        _sizes("moe_silu_quant", S, I)
    gpu = _gpu(g, u)
    if stream is not None or gpu != _current_gpu():
        return _elsewhere(gpu, stream, silu_quant, (g, u), g, u, y_dtype, quant)
    y = q = d = py = pq = pd = None
    if y_dtype is not None:
        y = g.new_empty((S, I), dtype=y_dtype)
        py = y.data_ptr()
    if quant:
        q, d = g.new_empty((S, I), dtype=torch.int8), g.new_empty(S, dtype=torch.float32)
        pq, pd = q.data_ptr(), d.data_ptr()
    rc = _lib.moe_silu_quant(g.data_ptr(), up, xd, ldx, S, I, py, yd, I, pq, I, pd, _stream_of(gpu))
    if rc:
        raise MoeError(rc, "moe_silu_quant")
    return y, q, d


def qmatmul(q, d, w, dw, out_dtype=None, ws=None, stream=None):
    """y [S, N] in out_dtype (bfloat16 unless given): moe_qmatmul of the int8 rows q [S, K] with scales d [S] and the
    int8 weights w [N, K] with scales dw [N], with its output (and, when ws is None, a workspace) allocated on q's
    GPU."""
    out_dtype = out_dtype or torch.bfloat16
    yd = _code(out_dtype, "out_dtype")
    shape = q.shape
    ldq = _rows(q, shape, "q")
    S, K = shape
    N = w.shape[0] if w.dim() else 0
    ldw = _rows(w, (N, K), "w")
    if q.dtype != torch.int8 or w.dtype != torch.int8:
        raise ValueError(f"q and w must be int8, not {q.dtype} and {w.dtype}")
    _vector(d, S, torch.float32, "d")
    _vector(dw, N, torch.float32, "dw")
    if ws is not None and not ws.is_contiguous():
        raise ValueError(f"ws must be contiguous, not of strides {tuple(ws.stride())}")
    if (S | N | K) >> 31:
        _sizes("moe_qmatmul", S, N, K)
    gpu = _gpu(q, d, w, dw, ws)
    if stream is not None or gpu != _current_gpu():
        return _elsewhere(gpu, stream, qmatmul, (q, d, w, dw, ws), q, d, w, dw, out_dtype, ws)
    pq, pw = q.data_ptr(), w.data_ptr()
    # operands on 16-byte boundaries take no workspace
    if ws is None and (pq | pw | ldq | ldw | K) & 15:
        need = _lib.moe_qmatmul_workspace_bytes(pq, ldq, pw, ldw, S, N, K)
        if need > 0:
            ws = q.new_empty(need)
    pws, nws = (None, 0) if ws is None else (ws.data_ptr(), ws.numel() * ws.element_size())
    y = d.new_empty((S, N), dtype=out_dtype)
    rc = _lib.moe_qmatmul(pq, ldq, d.data_ptr(), pw, ldw, dw.data_ptr(), S, N, K, y.data_ptr(), yd, N, pws, nws,
                          _stream_of(gpu))
    if rc:
        raise MoeError(rc, "moe_qmatmul")
    return y


_ROPE_TENSOR = struct.Struct("@PPqqqqi4x")  # moe_rope_tensor's bytes: packed, they cost a third of a ctypes structure
assert _ROPE_TENSOR.size == ctypes.sizeof(moe_rope_tensor)
_ROPE_SCALING = {"none": MOE_ROPE_PLAIN, "linear": MOE_ROPE_LINEAR, "ntk": MOE_ROPE_NTK, "yarn": MOE_ROPE_YARN}


def rope_freqs(rot: int, theta: float = 10000.0, scaling: str = "none", scale: float = 1.0, trained_length: int = 0,
               beta_fast: float = 32.0, beta_slow: float = 1.0, device="cuda"):
    """(freqs, factor) for rope: moe_rope_freqs with the frequencies as a float64 tensor on `device`."""
    if scaling not in _ROPE_SCALING:
        raise ValueError(f"scaling must be one of {sorted(_ROPE_SCALING)}, not {scaling!r}")
    f, factor = moe_rope_freqs(rot, theta, _ROPE_SCALING[scaling], scale, trained_length, beta_fast, beta_slow)
    return torch.from_numpy(f).to(device), factor


def _heads(t, S: int, D: int, what: str):
    if t.dim() == 3 and t.shape[0] == S and t.shape[2] == D and t.stride(2) == 1:
        return t.stride()
    raise ValueError(f"{what} must be [{S}, heads, {D}] with contiguous heads, not {tuple(t.shape)} "
                     f"with strides {tuple(t.stride())}")


def rope(q, k, pos, freqs, offset: int = 0, interleaved: bool = False, factor: float = 1.0, inplace: bool = False,
         stream=None):
    """(q, k) turned to their positions: moe_rope of q [S, heads, D] and k [S, kheads, D] (or None), with pos [S] int32
    or int64 and freqs [rot / 2] float64, into tensors allocated on q's GPU, or over q and k with inplace=True."""
    dtype = q.dtype
    xd = _code(dtype, "q")
    shape = q.shape
    S, D = shape[0], shape[-1]
    strides, counts = [_heads(q, S, D, "q"), None], [shape[1], 0]
    if k is not None:
        strides[1] = _heads(k, S, D, "k")
        counts[1] = k.shape[1]
        if k.dtype != dtype:
            raise ValueError(f"k must have q's type {dtype}, not {k.dtype}")
    wide = pos.dtype == torch.int64
    if not wide and pos.dtype != torch.int32:
        raise ValueError(f"pos must be int32 or int64, not {pos.dtype}")
    _vector(pos, S, pos.dtype, "pos")
    half = freqs.shape[0] if freqs.dim() == 1 else -1
    _vector(freqs, half, torch.float64, "freqs")
    if (S | D | 2 * half | offset | counts[0] | counts[1]) >> 31:
        _sizes("moe_rope", S, D, 2 * half, offset, *counts)
    gpu = _gpu(q, k, pos, freqs)
    if stream is not None or gpu != _current_gpu():
        return _elsewhere(gpu, stream, rope, (q, k, pos, freqs), q, k, pos, freqs, offset, interleaved, factor, inplace)
    outs, args = [q, k], [None, None]
    for i, t in enumerate((q, k)):
        if t is None:
            continue
        o = outs[i] = t if inplace else _empty_like(t, memory_format=_ROWS)
        s0, s1, _ = strides[i]
        heads = counts[i]
        o0, o1 = (s0, s1) if inplace else (heads * D, D)
        args[i] = _ROPE_TENSOR.pack(t.data_ptr(), o.data_ptr(), s0, s1, o0, o1, heads)
    rc = _lib.moe_rope(args[0], args[1], xd, S, D, 2 * half, offset,
                       MOE_ROPE_INTERLEAVED if interleaved else MOE_ROPE_HALF, pos.data_ptr(), wide, freqs.data_ptr(), factor,
                       _stream_of(gpu))
    if rc:
        raise MoeError(rc, "moe_rope")
    if inplace:
        _written(q)
        if k is not None:
            _written(k)
    return outs[0], outs[1]


# ---- microscaled rows, products grouped by expert -----------------------------------------------------------------------
# They serve too: no backward pass, inputs that require gradients are refused.

def _ref(s):
    return None if s is None else ctypes.byref(s)


def moe_mx_quant(x, x_dtype: int, ldx: int, S: int, H: int, rounding: int, q, ldq: int, e, lde: int, stream=None) -> None:
    _sizes("moe_mx_quant", S, H)
    _check(_lib.moe_mx_quant(ptr(x), x_dtype, ldx, S, H, rounding, ptr(q), ldq, ptr(e), lde, stream_handle(stream)),
           "moe_mx_quant")


def moe_mx_silu_quant(g, u, x_dtype: int, ldx: int, S: int, I: int, rounding: int, q, ldq: int, e, lde: int,
                      stream=None) -> None:
    _sizes("moe_mx_silu_quant", S, I)
    _check(_lib.moe_mx_silu_quant(ptr(g), ptr(u), x_dtype, ldx, S, I, rounding, ptr(q), ldq, ptr(e), lde,
                                  stream_handle(stream)), "moe_mx_silu_quant")


def moe_mx_values(q, ldq: int, e, lde: int, S: int, H: int, y, y_dtype: int, ldy: int, stream=None) -> None:
    _sizes("moe_mx_values", S, H)
    _check(_lib.moe_mx_values(ptr(q), ldq, ptr(e), lde, S, H, ptr(y), y_dtype, ldy, stream_handle(stream)), "moe_mx_values")


def moe_mx_matmul_workspace_bytes(x: moe_mx_rows, w: moe_mx_rows, S: int, N: int, B: int) -> int:
    _sizes("moe_mx_matmul_workspace_bytes", S, N, B)
    return _lib.moe_mx_matmul_workspace_bytes(_ref(x), _ref(w), S, N, B)


def moe_mx_matmul(x: moe_mx_rows, w: moe_mx_rows, S: int, N: int, B: int, y, y_dtype: int, ldy: int, ws, ws_bytes: int,
                  stream=None) -> None:
    _sizes("moe_mx_matmul", S, N, B)
    _check(_lib.moe_mx_matmul(_ref(x), _ref(w), S, N, B, ptr(y), y_dtype, ldy, ptr(ws), ws_bytes, stream_handle(stream)),
           "moe_mx_matmul")


def moe_group_workspace_bytes(S: int, k: int, E: int) -> int:
    _sizes("moe_group_workspace_bytes", S, k, E)
    return _lib.moe_group_workspace_bytes(S, k, E)


def moe_group(idx, S: int, k: int, E: int, first, order, place, ws, ws_bytes: int, stream=None) -> None:
    _sizes("moe_group", S, k, E)
    _check(_lib.moe_group(ptr(idx), S, k, E, ptr(first), ptr(order), ptr(place), ptr(ws), ws_bytes, stream_handle(stream)),
           "moe_group")


def moe_grouped_matmul_workspace_bytes(x, ldx: int, x_rows: int, w, ldw: int, expert: int, g: moe_groups, T: int, N: int,
                                       K: int) -> int:
    _sizes("moe_grouped_matmul_workspace_bytes", x_rows, T, N, K)
    return _lib.moe_grouped_matmul_workspace_bytes(ptr(x), ldx, x_rows, ptr(w), ldw, expert, _ref(g), T, N, K)


def moe_grouped_matmul(x, ldx: int, x_rows: int, w, ldw: int, expert: int, g: moe_groups, T: int, N: int, K: int, y,
                       y_dtype: int, ldy: int, ws, ws_bytes: int, stream=None) -> None:
    _sizes("moe_grouped_matmul", x_rows, T, N, K)
    _check(_lib.moe_grouped_matmul(ptr(x), ldx, x_rows, ptr(w), ldw, expert, _ref(g), T, N, K, ptr(y), y_dtype, ldy,
                                   ptr(ws), ws_bytes, stream_handle(stream)), "moe_grouped_matmul")


def moe_mx_grouped_matmul_workspace_bytes(x: moe_mx_rows, x_rows: int, w: moe_mx_rows, g: moe_groups, T: int, N: int,
                                          B: int) -> int:
    _sizes("moe_mx_grouped_matmul_workspace_bytes", x_rows, T, N, B)
    return _lib.moe_mx_grouped_matmul_workspace_bytes(_ref(x), x_rows, _ref(w), _ref(g), T, N, B)


def moe_mx_grouped_matmul(x: moe_mx_rows, x_rows: int, w: moe_mx_rows, g: moe_groups, T: int, N: int, B: int, y,
                          y_dtype: int, ldy: int, ws, ws_bytes: int, stream=None) -> None:
    _sizes("moe_mx_grouped_matmul", x_rows, T, N, B)
    _check(_lib.moe_mx_grouped_matmul(_ref(x), x_rows, _ref(w), _ref(g), T, N, B, ptr(y), y_dtype, ldy, ptr(ws), ws_bytes,
                                      stream_handle(stream)), "moe_mx_grouped_matmul")


def moe_combine(z, z_dtype: int, ldz: int, T: int, w, place, S: int, k: int, H: int, add, lda: int, y, y_dtype: int,
                ldy: int, stream=None) -> None:
    _sizes("moe_combine", T, S, k, H)
    _check(_lib.moe_combine(ptr(z), z_dtype, ldz, T, ptr(w), ptr(place), S, k, H, ptr(add), lda, ptr(y), y_dtype, ldy,
                            stream_handle(stream)), "moe_combine")


_MX_ROWS = struct.Struct("@PPqqqq")  # moe_mx_rows and moe_groups as bytes, as for rope
_GROUPS = struct.Struct("@PPii")
assert _MX_ROWS.size == ctypes.sizeof(moe_mx_rows) and _GROUPS.size == ctypes.sizeof(moe_groups)


def _codes(q, e, what: str):
    """(rows, blocks, row strides of q and e) of microscaled rows q [S, 16 B], e [S, B]."""
    if q.dtype != torch.uint8 or e.dtype != torch.uint8:
        raise ValueError(f"{what} and its scales must be uint8, not {q.dtype} and {e.dtype}")
    if e.dim() != 2:
        raise ValueError(f"{what}'s scales must be a matrix, not {tuple(e.shape)}")
    S, B = e.shape
    return S, B, _rows(q, (S, 16 * B), what), _rows(e, (S, B), f"{what}'s scales")


def _matrices(t, shape, what: str):
    """(row stride, matrix stride) of the matrices t [E, N, K], whose rows must be contiguous."""
    if t.shape == shape and len(shape) == 3:
        E, N, K = shape
        if t.is_contiguous():
            return K, N * K
        a, b, c = t.stride()
        if c == 1 or K <= 1:
            return b if N > 1 else K, a if E > 1 else 0
    raise ValueError(f"{what} must be [experts, rows, width] with contiguous rows, of shape {tuple(shape)}, not "
                     f"{tuple(t.shape)} with strides {tuple(t.stride())}")


def _workspace(ws):
    """(address, bytes) of the workspace given, if any."""
    if ws is None:
        return None, 0
    if not ws.is_contiguous():
        raise ValueError(f"ws must be contiguous, not of strides {tuple(ws.stride())}")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def _missing(rc: int, ws, need: int, like):
    """A new workspace, if that is what a call made without one was refused for (small calls need none, and are not asked)."""
    if rc == MOE_ENULL and ws is None and need > 0:
        return like.new_empty(need, dtype=torch.uint8)
    return None


def mx_quant(x, round_up: bool = False, stream=None):
    """(q [S, 16 B], e [S, B]) uint8 of the rows x [S, H], B = ceil(H / 32): moe_mx_quant with its outputs allocated on
    x's GPU.  round_up: MOE_MX_UP, scales under which no value is cut off."""
    xd, shape = _code(x.dtype, "x"), x.shape
    ldx = _rows(x, shape, "x")
    S, H = shape
    if (S | H) >> 31:
        _sizes("moe_mx_quant", S, H)
    gpu = _gpu(x)
    if stream is not None or gpu != _current_gpu():
        return _elsewhere(gpu, stream, mx_quant, (x,), x, round_up)
    B = (H + 31) // 32
    q, e = x.new_empty((S, 16 * B), dtype=torch.uint8), x.new_empty((S, B), dtype=torch.uint8)
    rc = _lib.moe_mx_quant(x.data_ptr(), xd, ldx, S, H, MOE_MX_UP if round_up else MOE_MX_FLOOR, q.data_ptr(), 16 * B,
                           e.data_ptr(), B, _stream_of(gpu))
    if rc:
        raise MoeError(rc, "moe_mx_quant")
    return q, e


def mx_silu_quant(g, u=None, round_up: bool = False, stream=None):
    """(q [S, 16 B], e [S, B]) of silu(g) * u, both [S, I], or of the halves of g [S, 2 I] where u is None:
    moe_mx_silu_quant with its outputs allocated on g's GPU."""
    xd, shape = _code(g.dtype, "g"), g.shape
    ldx = _rows(g, shape, "g")
    S, I = shape
    up = g.data_ptr()
    if u is None:
        if I % 2:
            raise ValueError(f"g holds gate and up side by side: its width {I} must be even")
        I //= 2
        up += I * g.element_size()
    else:
        if u.dtype != g.dtype:
            raise ValueError(f"u must have g's type {g.dtype}, not {u.dtype}")
        if _rows(u, shape, "u") != ldx:
            raise ValueError(f"u must have g's row stride {ldx}, not {u.stride(0)}")
        up = u.data_ptr()
    if (S | I) >> 31:
        _sizes("moe_mx_silu_quant", S, I)
    gpu = _gpu(g, u)
    if stream is not None or gpu != _current_gpu():
        return _elsewhere(gpu, stream, mx_silu_quant, (g, u), g, u, round_up)
    B = (I + 31) // 32
    q, e = g.new_empty((S, 16 * B), dtype=torch.uint8), g.new_empty((S, B), dtype=torch.uint8)
    rc = _lib.moe_mx_silu_quant(g.data_ptr(), up, xd, ldx, S, I, MOE_MX_UP if round_up else MOE_MX_FLOOR, q.data_ptr(),
                                16 * B, e.data_ptr(), B, _stream_of(gpu))
    if rc:
        raise MoeError(rc, "moe_mx_silu_quant")
    return q, e


def mx_values(q, e, width: int | None = None, dtype=None, stream=None):
    """The numbers [S, width] (32 B unless given) that the microscaled rows q, e stand for, in dtype (bfloat16 unless
    given): moe_mx_values with its output allocated on q's GPU."""
    S, B, ldq, lde = _codes(q, e, "q")
    dtype = dtype or torch.bfloat16
    yd = _code(dtype, "dtype")
    H = 32 * B if width is None else width
    if not 32 * (B - 1) < H <= 32 * B:
        raise ValueError(f"rows of {B} blocks hold {32 * (B - 1) + 1} to {32 * B} values, not {H}")
    if (S | H) >> 31:
        _sizes("moe_mx_values", S, H)
    gpu = _gpu(q, e)
    if stream is not None or gpu != _current_gpu():
        return _elsewhere(gpu, stream, mx_values, (q, e), q, e, width, dtype)
    y = q.new_empty((S, H), dtype=dtype)
    rc = _lib.moe_mx_values(q.data_ptr(), ldq, e.data_ptr(), lde, S, H, y.data_ptr(), yd, H, _stream_of(gpu))
    if rc:
        raise MoeError(rc, "moe_mx_values")
    return y


def mx_matmul(q, e, w, ew, out_dtype=None, ws=None, stream=None):
    """y [S, N] in out_dtype (bfloat16 unless given): moe_mx_matmul of the microscaled rows q [S, 16 B], e [S, B] with the
    microscaled weights w [N, 16 B], ew [N, B], with its output (and, when ws is None, a workspace) allocated on q's
    GPU."""
    out_dtype = out_dtype or torch.bfloat16
    yd = _code(out_dtype, "out_dtype")
    S, B, ldq, lde = _codes(q, e, "q")
    N, Bw, ldw, ldew = _codes(w, ew, "w")
    if Bw != B:
        raise ValueError(f"q has rows of {B} blocks, w of {Bw}")
    pws, nws = _workspace(ws)
    if (S | N | B) >> 31:
        _sizes("moe_mx_matmul", S, N, B)
    gpu = _gpu(q, e, w, ew, ws)
    if stream is not None or gpu != _current_gpu():
        return _elsewhere(gpu, stream, mx_matmul, (q, e, w, ew, ws), q, e, w, ew, out_dtype, ws)
    px = _MX_ROWS.pack(q.data_ptr(), e.data_ptr(), ldq, lde, 0, 0)
    pw = _MX_ROWS.pack(w.data_ptr(), ew.data_ptr(), ldw, ldew, 0, 0)
    y = q.new_empty((S, N), dtype=out_dtype)
    rc = _lib.moe_mx_matmul(px, pw, S, N, B, y.data_ptr(), yd, N, pws, nws, _stream_of(gpu))
    if rc == MOE_ENULL:
        ws = _missing(rc, ws, _lib.moe_mx_matmul_workspace_bytes(px, pw, S, N, B), q)
        if ws is not None:
            rc = _lib.moe_mx_matmul(px, pw, S, N, B, y.data_ptr(), yd, N, ws.data_ptr(), ws.numel(), _stream_of(gpu))
    if rc:
        raise MoeError(rc, "moe_mx_matmul")
    return y


def group(idx, n_experts: int, ws=None, stream=None):
    """(first [n_experts + 1], order [S k], place [S, k]) int32 of a routing idx [S, k] int32: moe_group with its outputs
    (and, when ws is None, a workspace) allocated on idx's GPU."""
    if idx.dim() != 2 or idx.dtype != torch.int32 or not idx.is_contiguous():
        raise ValueError(f"idx must be a contiguous int32 matrix, not {tuple(idx.shape)} {idx.dtype}")
    S, k = idx.shape
    pws, nws = _workspace(ws)
    if (S | k | n_experts) >> 31:
        _sizes("moe_group", S, k, n_experts)
    gpu = _gpu(idx, ws)
    if stream is not None or gpu != _current_gpu():
        return _elsewhere(gpu, stream, group, (idx, ws), idx, n_experts, ws)
    first, order, place = idx.new_empty(max(n_experts, 0) + 1), idx.new_empty(S * k), _empty_like(idx)
    args = idx.data_ptr(), S, k, n_experts, first.data_ptr(), order.data_ptr(), place.data_ptr()
    rc = _lib.moe_group(*args, pws, nws, _stream_of(gpu))
    if rc == MOE_ENULL:
        ws = _missing(rc, ws, _lib.moe_group_workspace_bytes(S, k, n_experts), idx)
        if ws is not None:
            rc = _lib.moe_group(*args, ws.data_ptr(), ws.numel(), _stream_of(gpu))
    if rc:
        raise MoeError(rc, "moe_group")
    return first, order, place


def _groups(first, order, top_k, E: int, x_rows: int):
    """(rows of the product, moe_groups as bytes)."""
    _vector(first, E + 1, torch.int32, "first")
    if order is None:
        if top_k is not None:
            raise ValueError("top_k goes with order: none is given")
        return x_rows, _GROUPS.pack(first.data_ptr(), 0, E, 0)
    if top_k is None or not 0 < top_k <= 0x7FFFFFFF:
        raise ValueError(f"order goes with top_k, the choices of a token, not {top_k}")
    T = order.shape[0] if order.dim() == 1 else -1
    _vector(order, T, torch.int32, "order")
    return T, _GROUPS.pack(first.data_ptr(), order.data_ptr(), E, top_k)


def _grouped_out(out, T: int, N: int, out_dtype, like):
    """(output, its row stride, its dtype code)."""
    if out is None:
        out = like.new_empty((T, N), dtype=out_dtype or torch.bfloat16)
        return out, N, _code(out.dtype, "out_dtype")
    if out_dtype is not None and out.dtype != out_dtype:
        raise ValueError(f"out must be of out_dtype {out_dtype}, not {out.dtype}")
    return out, _rows(out, (T, N), "out"), _code(out.dtype, "out")


def grouped_matmul(x, w, first, order=None, top_k: int | None = None, out_dtype=None, out=None, ws=None, stream=None):
    """y [T, N] in out_dtype (bfloat16 unless given): moe_grouped_matmul of bf16 rows with the bf16 weights w [E, N, K] of
    their experts, expert e's being rows first[e] .. first[e + 1] - 1 of y.  Row i's input is row i of x [T, K], or, where
    order [T] is given, row order[i] // top_k of x.  The output (unless `out` is given) and a workspace (when ws is None)
    are allocated on x's GPU; rows that no expert has are left as they were (of a new output: not initialised)."""
    if x.dtype != torch.bfloat16 or w.dtype != torch.bfloat16:
        raise ValueError(f"x and w must be bfloat16, not {x.dtype} and {w.dtype}")
    shape = x.shape
    ldx = _rows(x, shape, "x")
    rows, K = shape
    E, N = w.shape[:2] if w.dim() == 3 else (0, 0)
    ldw, expert = _matrices(w, (E, N, K), "w")
    T, plan = _groups(first, order, top_k, E, rows)
    pws, nws = _workspace(ws)
    if (rows | T | N | K) >> 31:
        _sizes("moe_grouped_matmul", rows, T, N, K)
    if out_dtype is not None:
        _code(out_dtype, "out_dtype")
    gpu = _gpu(x, w, first, order, out, ws)
    if stream is not None or gpu != _current_gpu():
        return _elsewhere(gpu, stream, grouped_matmul, (x, w, first, order, out, ws), x, w, first, order, top_k, out_dtype,
                          out, ws)
    over = out
    out, ldy, yd = _grouped_out(out, T, N, out_dtype, x)
    px, pw = x.data_ptr(), w.data_ptr()
    args = px, ldx, rows, pw, ldw, expert, plan, T, N, K
    rc = _lib.moe_grouped_matmul(*args, out.data_ptr(), yd, ldy, pws, nws, _stream_of(gpu))
    if rc == MOE_ENULL:
        ws = _missing(rc, ws, _lib.moe_grouped_matmul_workspace_bytes(*args), x)
        if ws is not None:
            rc = _lib.moe_grouped_matmul(*args, out.data_ptr(), yd, ldy, ws.data_ptr(), ws.numel(), _stream_of(gpu))
    if rc:
        raise MoeError(rc, "moe_grouped_matmul")
    if over is not None:
        _written(over)
    return out


def mx_grouped_matmul(q, e, w, ew, first, order=None, top_k: int | None = None, out_dtype=None, out=None, ws=None,
                      stream=None):
    """y [T, N]: grouped_matmul of microscaled rows q [T, 16 B], e [T, B] with microscaled weights w [E, N, 16 B],
    ew [E, N, B] (moe_mx_grouped_matmul)."""
    rows, B, ldq, lde = _codes(q, e, "q")
    if w.dtype != torch.uint8 or ew.dtype != torch.uint8:
        raise ValueError(f"w and its scales must be uint8, not {w.dtype} and {ew.dtype}")
    E, N = w.shape[:2] if w.dim() == 3 else (0, 0)
    ldw, expert = _matrices(w, (E, N, 16 * B), "w")
    ldew, expert_e = _matrices(ew, (E, N, B), "w's scales")
    T, plan = _groups(first, order, top_k, E, rows)
    pws, nws = _workspace(ws)
    if (rows | T | N | B) >> 31:
        _sizes("moe_mx_grouped_matmul", rows, T, N, B)
    if out_dtype is not None:
        _code(out_dtype, "out_dtype")
    gpu = _gpu(q, e, w, ew, first, order, out, ws)
    if stream is not None or gpu != _current_gpu():
        return _elsewhere(gpu, stream, mx_grouped_matmul, (q, e, w, ew, first, order, out, ws), q, e, w, ew, first, order,
                          top_k, out_dtype, out, ws)
    over = out
    out, ldy, yd = _grouped_out(out, T, N, out_dtype, q)
    px = _MX_ROWS.pack(q.data_ptr(), e.data_ptr(), ldq, lde, 0, 0)
    pw = _MX_ROWS.pack(w.data_ptr(), ew.data_ptr(), ldw, ldew, expert, expert_e)
    args = px, rows, pw, plan, T, N, B
    rc = _lib.moe_mx_grouped_matmul(*args, out.data_ptr(), yd, ldy, pws, nws, _stream_of(gpu))
    if rc == MOE_ENULL:
        ws = _missing(rc, ws, _lib.moe_mx_grouped_matmul_workspace_bytes(*args), q)
        if ws is not None:
            rc = _lib.moe_mx_grouped_matmul(*args, out.data_ptr(), yd, ldy, ws.data_ptr(), ws.numel(), _stream_of(gpu))
    if rc:
        raise MoeError(rc, "moe_mx_grouped_matmul")
    if over is not None:
        _written(over)
    return out


def combine(z, w, place, add=None, out_dtype=None, stream=None):
    """y [S, H] in out_dtype (z's type unless given), y[s] = sum_j w[s, j] z[place[s, j]] + add[s]: moe_combine of the
    experts' rows z [T, H] with the weights w [S, k] fp32 and the places of group, with its output allocated on z's
    GPU."""
    zd, shape = _code(z.dtype, "z"), z.shape
    ldz = _rows(z, shape, "z")
    T, H = shape
    if place.dim() != 2:
        raise ValueError(f"place must be a matrix, not {tuple(place.shape)}")
    pairs = place.shape
    for name, t, dtype in (("place", place, torch.int32), ("w", w, torch.float32)):
        if t.shape != pairs or t.dtype != dtype or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {tuple(pairs)} {dtype} tensor, not {tuple(t.shape)} {t.dtype}")
    S, k = pairs
    out_dtype = out_dtype or z.dtype
    yd = _code(out_dtype, "out_dtype")
    lda, pa = 0, None
    if add is not None:
        lda = _rows(add, (S, H), "add")
        if add.dtype != z.dtype:
            raise ValueError(f"add must have z's type {z.dtype}, not {add.dtype}")
        pa = add.data_ptr()
    if (T | S | k | H) >> 31:
        _sizes("moe_combine", T, S, k, H)
    gpu = _gpu(z, w, place, add)
    if stream is not None or gpu != _current_gpu():
        return _elsewhere(gpu, stream, combine, (z, w, place, add), z, w, place, add, out_dtype)
    y = z.new_empty((S, H), dtype=out_dtype)
    rc = _lib.moe_combine(z.data_ptr(), zd, ldz, T, w.data_ptr(), place.data_ptr(), S, k, H, pa, lda, y.data_ptr(), yd, H,
                          _stream_of(gpu))
    if rc:
        raise MoeError(rc, "moe_combine")
    return y


def moe_profile_enable(on: bool) -> None:
    _check(_lib.moe_profile_enable(int(on)), "moe_profile_enable")


def moe_profile_report() -> dict:
    """{kernel: (total_ms, launches)} since the last report."""
    import json
    buf = ctypes.create_string_buffer(1 << 16)
    _check(_lib.moe_profile_report(buf, len(buf)), "moe_profile_report")
    return {k: (v[0], v[1]) for k, v in json.loads(buf.value.decode()).items()}


MOE_POOL_NO_DEVICE, MOE_POOL_POISON = 1, 2


class Pool:
    """Owner of a moe_pool handle (the C calls, with errors raised as MoeError)."""

    def __init__(self, cfg: moe_cfg, n_layers: int, slots_per_layer: int, flags: int = 0):
        self.h = ctypes.c_void_p()
        self._src = {}  # (layer, expert) -> registered host buffer, kept alive while the pool may copy from it
        _check(_lib.moe_pool_create(ctypes.byref(cfg), n_layers, slots_per_layer, flags, ctypes.byref(self.h)),
               "moe_pool_create")

    def register_host(self, layer: int, expert: int, src) -> None:
        _check(_lib.moe_pool_register_host(self.h, layer, expert, ptr(src)), "moe_pool_register_host")
        self._src[(layer, expert)] = src

    def acquire(self, layer: int, idx_host, compute=None, side=None):
        """-> (moe_slot_view, n_miss); idx_host: int32 numpy array."""
        import numpy as np
        idx = np.ascontiguousarray(idx_host, np.int32).ravel()
        view = moe_slot_view()
        n_miss = ctypes.c_int32(0)
        c = stream_handle(compute) if compute is not None or side is not None else None
        s_ = stream_handle(side) if side is not None else c
        _check(_lib.moe_pool_acquire(self.h, layer, idx.ctypes.data, idx.size, ctypes.byref(view), ctypes.byref(n_miss),
                                     c, s_), "moe_pool_acquire")
        return view, n_miss.value

    def prefetch(self, layer: int, idx_host, side=None) -> int:
        """Predicted routing idx_host (int32 numpy array) of `layer`; -> copies enqueued."""
        import numpy as np
        idx = np.ascontiguousarray(idx_host, np.int32).ravel()
        n_fill = ctypes.c_int32(0)
        _check(_lib.moe_pool_prefetch(self.h, layer, idx.ctypes.data, idx.size, ctypes.byref(n_fill),
                                      stream_handle(side) if side is not None else None), "moe_pool_prefetch")
        return n_fill.value

    def release(self, layer: int, compute=None) -> None:
        c = stream_handle(compute) if compute is not None else None
        _check(_lib.moe_pool_release(self.h, layer, c), "moe_pool_release")

    def trace(self):
        import numpy as np
        out = np.zeros(3 * 4096, np.int32)
        n = _lib.moe_pool_trace(self.h, out.ctypes.data, out.size)
        if n < 0:
            raise MoeError(n, "moe_pool_trace")
        return [tuple(out[3 * i:3 * i + 3]) for i in range(n)]

    def stats(self) -> dict:
        import json
        buf = ctypes.create_string_buffer(1024)
        _check(_lib.moe_pool_stats(self.h, buf, len(buf)), "moe_pool_stats")
        return json.loads(buf.value.decode())

    def check_view(self, layer: int, view: moe_slot_view) -> int:
        """moe_pool_check_view: MOE_OK or MOE_ESTALE (other statuses raise)."""
        rc = _lib.moe_pool_check_view(self.h, layer, ctypes.byref(view))
        if rc not in (MOE_OK, MOE_ESTALE):
            raise MoeError(rc, "moe_pool_check_view")
        return rc

    def close(self) -> None:
        if self.h:
            _lib.moe_pool_destroy(self.h)
            self.h = ctypes.c_void_p()
        self._src = {}

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def slot_view(base, slot_bytes: int, table, n_slots: int, gen=None, slot_gen=None) -> moe_slot_view:
    """A view of caller-owned slots (generation tags optional: gen [E] and slot_gen [n_slots] uint32).
    The view stores raw addresses; it also holds references to the objects given, so that
    a table built inline is not freed (and its memory reused) while the view is alive."""
    v = moe_slot_view(ptr(base), slot_bytes, ptr(table), n_slots, ptr(gen), ptr(slot_gen), 0)
    v._refs = (base, table, gen, slot_gen)
    return v
