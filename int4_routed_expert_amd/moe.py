"""Python binding of ``libmoe.so`` (include/moe.h, include/moe_dense.h): argument marshalling only.

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
HEADERS = [os.path.join(os.path.dirname(_HERE), "include", h) for h in ("moe.h", "moe_dense.h")]
HEADER = HEADERS[0]

MOE_OK, MOE_EINVAL, MOE_ENULL, MOE_EDTYPE, MOE_EWORKSPACE, MOE_ENOSLOT, MOE_ESTALE, MOE_EHIP, MOE_ELEASE = \
    0, -1, -2, -3, -4, -5, -6, -7, -8
MOE_F32, MOE_BF16 = 0, 1
MOE_WF_Q4_G32, MOE_WF_Q4_ROW, MOE_WF_Q8_ROW = 0, 1, 2
MOE_ROPE_HALF, MOE_ROPE_INTERLEAVED = 0, 1
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
