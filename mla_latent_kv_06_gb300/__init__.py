"""Thin Python binding of libmla.so (the C ABI in include/mla.h).

Argument marshalling only: every step of the hot path runs in the library's
CUDA kernels.  PyTorch provides device memory and streams.  Functions take
CUDA tensors, check dtype/shape/contiguity, allocate outputs and workspace
with torch when the caller gives none, and enqueue on the current stream.
There is no CPU fallback: without the built library every call raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Tuple

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libmla.so")

MLA_F32, MLA_BF16 = 0, 1
MLA_OK, MLA_ERR_INVALID, MLA_ERR_UNSUPPORTED, MLA_ERR_CUDA, MLA_ERR_DEVICE = 0, -1, -2, -3, -4
MLA_DEV_BAD_LENGTH, MLA_DEV_BAD_INDEX, MLA_DEV_TIMEOUT, MLA_DEV_BAD_VALUE = 1, 2, 4, 8

# Every symbol declared in include/mla.h.
EXPORTS = (
    "mla_last_error", "mla_abi_version", "mla_device_status", "mla_set_wait_limit_ns",
    "mla_set_kernel_events", "mla_last_launch_names",
    "mla_decode_absorbed_workspace_size", "mla_decode_absorbed", "mla_decode_launch_count",
    "mla_sparse_decode_workspace_size", "mla_sparse_decode", "mla_sparse_decode_layers_workspace_size",
    "mla_sparse_decode_layers",
    "mla_prefill_naive_workspace_size", "mla_prefill_naive", "mla_prefill_naive_noalloc",
    "dsa_index_scores", "dsa_topk_select_workspace_size", "dsa_topk_select",
    "mla_cache_append", "dsa_index_key_append",
    "mla_decode_paged_workspace_size", "mla_decode_paged", "mla_sparse_decode_paged", "mla_cache_append_paged",
    "dsa_select_workspace_size", "dsa_select",
    "mla_o_proj_workspace_size", "mla_o_proj", "mla_decode_oproj_workspace_size", "mla_decode_oproj",
    "mla_decode_fp8_workspace_size", "mla_decode_fp8", "mla_decode_fp8_paged", "mla_cache_append_fp8",
    "mla_cache_append_fp8_paged",
    "mla_decode_tree_workspace_size", "mla_decode_tree", "mla_decode_tree_paged", "mla_cache_append_tree",
    "mla_cache_append_tree_paged", "mla_tree_verify", "mla_tree_commit", "mla_tree_commit_paged",
)


class MlaDims(ctypes.Structure):
    _fields_ = [("H", ctypes.c_int), ("qk_nope", ctypes.c_int), ("qk_rope", ctypes.c_int),
                ("kv_lora", ctypes.c_int), ("v_head", ctypes.c_int), ("scale", ctypes.c_float),
                ("rope_base", ctypes.c_float)]


class MlaError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"libmla status {code}: {msg}")
        self.code = code


_lib: Optional[ctypes.CDLL] = None

_P = ctypes.c_void_p
_I = ctypes.c_int
_SZ = ctypes.c_size_t
_DP = ctypes.POINTER(MlaDims)
_PP = ctypes.POINTER(ctypes.c_void_p)  # host array of device pointers
_LL = ctypes.c_longlong
_IP = ctypes.POINTER(ctypes.c_int)


def _declare(lib: ctypes.CDLL) -> None:
    sig = {
        "mla_last_error": (ctypes.c_char_p, []),
        "mla_abi_version": (_I, []),
        "mla_device_status": (_I, [_P, ctypes.POINTER(_I)]),
        "mla_set_wait_limit_ns": (None, [ctypes.c_longlong]),
        "mla_set_kernel_events": (_I, [ctypes.POINTER(ctypes.c_void_p), _I]),
        "mla_last_launch_names": (ctypes.c_char_p, []),
        "mla_decode_absorbed_workspace_size": (_SZ, [_DP, _I, _I, _I, _I]),
        "mla_decode_launch_count": (_I, [_DP, _I, _I, _I, _I]),
        "mla_decode_absorbed": (_I, [_DP, _I, _I, _I, _P, _P, _P, _I, _P, _P, _P, _P, _SZ, _P]),
        "mla_sparse_decode_workspace_size": (_SZ, [_DP, _I, _I, _I, _I]),
        "mla_sparse_decode": (_I, [_DP, _I, _I, _I, _P, _P, _P, _I, _P, _P, _P, _P, _I, _P, _P,
                                   _SZ, _P]),
        "mla_sparse_decode_layers_workspace_size": (_SZ, [_DP, _I, _I, _I, _I, _I]),
        "mla_sparse_decode_layers": (_I, [_DP, _I, _I, _I, _I, _PP, _PP, _PP, _I, _P, _PP, _P, _P, _I, _PP, _PP, _I,
                                          _PP, _P, _SZ, _P]),
        "mla_prefill_naive_workspace_size": (_SZ, [_DP, _I, _I, _I, _I]),
        "mla_prefill_naive": (_I, [_DP, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _SZ, _P]),
        "mla_prefill_naive_noalloc": (_I, [_DP, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P]),
        "dsa_index_scores": (_I, [_I, _I, _I, _I, _P, _P, _P, _I, _P, _P, _P]),
        "dsa_topk_select_workspace_size": (_SZ, [_I, _I, _I, _I]),
        "dsa_topk_select": (_I, [_I, _I, _P, _I, _P, _I, _P, _P, _P, _SZ, _P]),
        "mla_cache_append": (_I, [_DP, _I, _I, _I, _P, _P, ctypes.c_float, _I, _P, _P, _P, _P]),
        "dsa_index_key_append": (_I, [_I, _I, _I, _I, _P, _P, _P, ctypes.c_float, ctypes.c_float, _I, _P,
                                      _P, _P]),
        "mla_decode_paged_workspace_size": (_SZ, [_DP, _I, _I, _I, _I, _I]),
        "mla_decode_paged": (_I, [_DP, _I, _I, _I, _P, _P, _P, _I, _I, _P, _I, _P, _P, _P, _P, _SZ, _P]),
        "mla_sparse_decode_paged": (_I, [_DP, _I, _I, _I, _P, _P, _P, _I, _I, _P, _I, _P, _P, _P, _P, _I, _P,
                                         _P, _SZ, _P]),
        "mla_cache_append_paged": (_I, [_DP, _I, _I, _I, _P, _P, ctypes.c_float, _P, _P, _I, _I, _P, _I, _P, _P]),
        "dsa_select_workspace_size": (_SZ, [_I, _I, _I, _I, _I, _I]),
        "dsa_select": (_I, [_I, _I, _I, _I, _P, _P, _P, _I, _P, _I, _P, _P, _P, _P, _SZ, _P]),
        "mla_o_proj_workspace_size": (_SZ, [_I, _I, _I, _I]),
        "mla_o_proj": (_I, [_I, _I, _I, _I, _P, _P, _P, _P, _SZ, _P]),
        "mla_decode_oproj_workspace_size": (_SZ, [_DP, _I, _I, _I, _I, _I]),
        "mla_decode_oproj": (_I, [_DP, _I, _I, _I, _P, _P, _P, _I, _P, _P, _P, _I, _P, _P, _SZ, _P]),
        "mla_decode_fp8_workspace_size": (_SZ, [_DP, _I, _I, _I]),
        "mla_decode_fp8": (_I, [_DP, _I, _I, _P, _P, _P, ctypes.c_float, _I, _P, _P, _P, _P, _SZ, _P]),
        "mla_decode_fp8_paged": (_I, [_DP, _I, _I, _P, _P, _P, ctypes.c_float, _I, _I, _P, _I, _P, _P, _P, _P,
                                      _SZ, _P]),
        "mla_cache_append_fp8": (_I, [_DP, _I, _I, _P, _P, ctypes.c_float, ctypes.c_float, _I, _P, _P, _P, _P]),
        "mla_cache_append_fp8_paged": (_I, [_DP, _I, _I, _P, _P, ctypes.c_float, ctypes.c_float, _P, _P, _I, _I,
                                            _P, _I, _P, _P]),
        "mla_decode_tree_workspace_size": (_SZ, [_DP, _I, _I, _I, _I]),
        "mla_decode_tree": (_I, [_DP, _I, _I, _I, _P, _P, _P, _I, _P, _P, _P, _I, _P, _P, _SZ, _P]),
        "mla_decode_tree_paged": (_I, [_DP, _I, _I, _I, _P, _P, _P, _I, _I, _P, _I, _P, _P, _P, _I, _P, _P, _SZ, _P]),
        "mla_cache_append_tree": (_I, [_DP, _I, _I, _I, _P, _P, ctypes.c_float, _I, _P, _P, _P, _P, _P]),
        "mla_cache_append_tree_paged": (_I, [_DP, _I, _I, _I, _P, _P, ctypes.c_float, _P, _P, _I, _I, _P, _I, _P, _P,
                                             _P]),
        "mla_tree_verify": (_I, [_I, _I, _I, _P, _LL, _LL, _P, _LL, _LL, _P, _P, _P, _P, _P, _P, _P]),
        "mla_tree_commit": (_I, [_I, _PP, _IP, _I, _I, _I, _P, _P, _P, _P, _P]),
        "mla_tree_commit_paged": (_I, [_I, _PP, _IP, _I, _I, _I, _I, _P, _I, _P, _P, _P, _P, _P]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args


def load(path: Optional[str] = None) -> ctypes.CDLL:
    """Load libmla.so (built by __graft_entry__.build()); raises if it is missing."""
    global _lib
    if _lib is None:
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(f"{p} is missing: build it first (python -c 'import __graft_entry__ as g; g.build()')")
        lib = ctypes.CDLL(p)
        _declare(lib)
        _lib = lib
    return _lib


def lib() -> ctypes.CDLL:
    return load()


def _check(rc: int) -> None:
    if rc != MLA_OK:
        raise MlaError(rc, lib().mla_last_error().decode(errors="replace"))


def make_dims(dims) -> MlaDims:
    """Accepts workload.Dims or any object with the same fields."""
    scale = getattr(dims, "scale", None)
    return MlaDims(dims.H, dims.qk_nope, dims.qk_rope, dims.kv_lora, dims.v_head,
                   float(scale) if scale else 0.0, float(getattr(dims, "rope_base", 10000.0)))


# ------------------------------------------------------------------ helpers
def _torch():
    import torch
    return torch


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.float32:
        return MLA_F32
    if t.dtype == torch.bfloat16:
        return MLA_BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors must live on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _workspace(nbytes: int, device, ws):
    torch = _torch()
    if nbytes == 0:
        return ws, 0
    if ws is None or ws.numel() * ws.element_size() < nbytes:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return ws, ws.numel() * ws.element_size()


def device_status(stream=None) -> int:
    """Synchronises the stream and returns (and clears) the device flag word."""
    flags = _I(0)
    rc = lib().mla_device_status(_stream(stream), ctypes.byref(flags))
    if rc not in (MLA_OK, MLA_ERR_DEVICE):
        _check(rc)
    return flags.value


def set_wait_limit_ns(ns: int) -> None:
    lib().mla_set_wait_limit_ns(int(ns))


_event_array = None


def set_kernel_events(events) -> None:
    """Record these torch.cuda.Event objects around the kernels of every later
    call on this thread (see mla_set_kernel_events); None switches it off."""
    global _event_array
    if not events:
        _event_array = None
        lib().mla_set_kernel_events(None, 0)
        return
    for e in events:
        if not e.cuda_event:
            e.record()  # torch creates the CUDA event lazily
    _event_array = (ctypes.c_void_p * len(events))(*[e.cuda_event for e in events])
    lib().mla_set_kernel_events(_event_array, len(events))


def last_launch_names():
    """Kernels launched by the last call on this thread, in order."""
    return [n for n in lib().mla_last_launch_names().decode().split(",") if n]


# ------------------------------------------------------------------ ops
def kernels_per_call(kind: str, dims, B: int = 1, S: int = 1, dtype: int = MLA_BF16) -> int:
    """Kernels one decode ("decode") or sparse-decode ("sparse") call launches."""
    d = make_dims(dims)
    return lib().mla_decode_launch_count(ctypes.byref(d), dtype, B, S, 1 if kind == "sparse" else 0)


def decode_workspace_size(dims, dtype: int, B: int, S: int, T_cap: int) -> int:
    d = make_dims(dims)
    return lib().mla_decode_absorbed_workspace_size(ctypes.byref(d), dtype, B, S, T_cap)


def decode_absorbed(q, Lc, Rc, T, kv_b, dims, out=None, workspace=None, stream=None):
    """Weight-absorbed decode; q [B,S,H,qk], Lc [B,T_cap,kv_lora], Rc [B,T_cap,qk_rope]."""
    torch = _torch()
    B, S, H = q.shape[0], q.shape[1], q.shape[2]
    T_cap = Lc.shape[1]
    code = _dtype_code(q)
    if out is None:
        out = torch.empty(B, S, H, dims.v_head, dtype=torch.float32, device=q.device)
    d = make_dims(dims)
    need = lib().mla_decode_absorbed_workspace_size(ctypes.byref(d), code, B, S, T_cap)
    workspace, wsb = _workspace(need, q.device, workspace)
    _check(lib().mla_decode_absorbed(ctypes.byref(d), code, B, S, _ptr(q), _ptr(Lc), _ptr(Rc), T_cap,
                                     _ptr(T), _ptr(kv_b), _ptr(out), _ptr(workspace), wsb,
                                     _stream(stream)))
    return out


def sparse_decode(q, Lc, Rc, T, kv_b, sel, nsel, dims, out=None, workspace=None, stream=None):
    """Absorbed decode over the keys sel[b,s,:nsel[b,s]] (sel [B,S,topk] int32)."""
    torch = _torch()
    B, S, H = q.shape[0], q.shape[1], q.shape[2]
    T_cap = Lc.shape[1]
    topk = sel.shape[2]
    code = _dtype_code(q)
    if out is None:
        out = torch.empty(B, S, H, dims.v_head, dtype=torch.float32, device=q.device)
    d = make_dims(dims)
    need = lib().mla_sparse_decode_workspace_size(ctypes.byref(d), code, B, S, topk)
    workspace, wsb = _workspace(need, q.device, workspace)
    _check(lib().mla_sparse_decode(ctypes.byref(d), code, B, S, _ptr(q), _ptr(Lc), _ptr(Rc), T_cap,
                                   _ptr(T), _ptr(kv_b), _ptr(sel), _ptr(nsel), topk, _ptr(out),
                                   _ptr(workspace), wsb, _stream(stream)))
    return out


def sparse_decode_layers(layers, T, sel, nsel, dims, outs=None, w_o=None, ys=None, workspace=None, stream=None):
    """Sparse decode of L layers over one selection: layers is a list of
    (q, Lc, Rc, kv_b) per layer.  With w_o (a list of L [hidden, H*v_head]
    weights) each layer's output is also projected.  Returns the list of L
    outputs [B,S,H,v_head], and with w_o also the list of L projections
    [B*S, hidden]."""
    torch = _torch()
    L = len(layers)
    q0, Lc0 = layers[0][0], layers[0][1]
    B, S, H = q0.shape[0], q0.shape[1], q0.shape[2]
    T_cap = Lc0.shape[1]
    topk = sel.shape[2]
    code = _dtype_code(q0)
    for q, Lc, Rc, kv_b in layers:
        if q.shape != q0.shape or Lc.shape != Lc0.shape or q.dtype != q0.dtype:
            raise ValueError("every layer needs the shapes and dtype of layer 0")
    if outs is None:
        outs = [torch.empty(B, S, H, dims.v_head, dtype=torch.float32, device=q0.device) for _ in range(L)]
    hidden = 0
    if w_o is not None:
        if len(w_o) != L:
            raise ValueError("one projection weight per layer")
        hidden = w_o[0].shape[0]
        if ys is None:
            ys = [torch.empty(B * S, hidden, dtype=torch.float32, device=q0.device) for _ in range(L)]
    d = make_dims(dims)
    need = lib().mla_sparse_decode_layers_workspace_size(ctypes.byref(d), code, B, S, topk, hidden)
    workspace, wsb = _workspace(need, q0.device, workspace)

    def arr(ts):
        return (ctypes.c_void_p * L)(*[_ptr(t) for t in ts])

    _check(lib().mla_sparse_decode_layers(
        ctypes.byref(d), code, L, B, S, arr([x[0] for x in layers]), arr([x[1] for x in layers]),
        arr([x[2] for x in layers]), T_cap, _ptr(T), arr([x[3] for x in layers]), _ptr(sel), _ptr(nsel), topk,
        arr(outs), arr(w_o) if w_o is not None else None, hidden, arr(ys) if w_o is not None else None,
        _ptr(workspace), wsb, _stream(stream)))
    return (outs, ys) if w_o is not None else outs


def prefill_naive(q, Lc, Rc, kv_b, dims, pos_base: int, out=None, workspace=None, stream=None):
    """Non-absorbed prefill of S new tokens at pos_base; Lc/Rc hold Tk = pos_base + S rows."""
    torch = _torch()
    B, S, H = q.shape[0], q.shape[1], q.shape[2]
    code = _dtype_code(q)
    if out is None:
        out = torch.empty(B, S, H, dims.v_head, dtype=torch.float32, device=q.device)
    d = make_dims(dims)
    need = lib().mla_prefill_naive_workspace_size(ctypes.byref(d), code, B, S, pos_base)
    workspace, wsb = _workspace(need, q.device, workspace)
    _check(lib().mla_prefill_naive(ctypes.byref(d), code, B, S, pos_base, _ptr(q), _ptr(Lc), _ptr(Rc),
                                   _ptr(kv_b), _ptr(out), _ptr(workspace), wsb, _stream(stream)))
    return out


def index_scores(q_idx, w, Ic, T, out=None, stream=None):
    """DSA indexer scores [B,S,T_cap] (fp32; -inf past each query's position)."""
    torch = _torch()
    B, S, n_ih, hd = q_idx.shape
    T_cap = Ic.shape[1]
    if out is None:
        out = torch.empty(B, S, T_cap, dtype=torch.float32, device=q_idx.device)
    _check(lib().dsa_index_scores(B, S, n_ih, hd, _ptr(q_idx), _ptr(w), _ptr(Ic), T_cap, _ptr(T),
                                  _ptr(out), _stream(stream)))
    return out


def topk_select(scores, T, topk: int, S: Optional[int] = None, sel=None, nsel=None,
                workspace=None, stream=None) -> Tuple[object, object]:
    """Causal top-k selection: (sel [B,S,topk] ascending then -1, nsel [B,S])."""
    torch = _torch()
    B, S_, T_cap = scores.shape
    S = S_ if S is None else S
    if sel is None:
        sel = torch.empty(B, S, topk, dtype=torch.int32, device=scores.device)
    if nsel is None:
        nsel = torch.empty(B, S, dtype=torch.int32, device=scores.device)
    need = lib().dsa_topk_select_workspace_size(B, S, T_cap, topk)
    workspace, wsb = _workspace(need, scores.device, workspace)
    _check(lib().dsa_topk_select(B, S, _ptr(scores), T_cap, _ptr(T), topk, _ptr(sel), _ptr(nsel),
                                 _ptr(workspace), wsb, _stream(stream)))
    return sel, nsel


def cache_append(comp, kv_a_ln, T, Lc, Rc, dims, rms_eps: float, stream=None):
    """Writes the S new tokens of each sequence into Lc/Rc in place at rows
    T[b]-S+s: comp [B,S,kv_lora+qk_rope] (the kv_a output), kv_a_ln [kv_lora]."""
    B, S = comp.shape[0], comp.shape[1]
    T_cap = Lc.shape[1]
    code = _dtype_code(comp)
    for t in (kv_a_ln, Lc, Rc):
        if t.dtype != comp.dtype:
            raise TypeError("comp, kv_a_ln, Lc and Rc must share one dtype")
    d = make_dims(dims)
    _check(lib().mla_cache_append(ctypes.byref(d), code, B, S, _ptr(comp), _ptr(kv_a_ln), float(rms_eps),
                                  T_cap, _ptr(T), _ptr(Lc), _ptr(Rc), _stream(stream)))
    return Lc, Rc


def index_key_append(k_idx, ln_w, ln_b, T, Ic, rope_dim: int, ln_eps: float = 1e-6,
                     rope_base: float = 10000.0, stream=None):
    """Writes the indexer keys of the S new tokens (k_idx [B,S,index_hd] fp32)
    into Ic [B,T_cap,index_hd] in place: LayerNorm, then RoPE on the last rope_dim."""
    B, S, hd = k_idx.shape
    T_cap = Ic.shape[1]
    _check(lib().dsa_index_key_append(B, S, hd, int(rope_dim), _ptr(k_idx), _ptr(ln_w), _ptr(ln_b),
                                      float(ln_eps), float(rope_base), T_cap, _ptr(T), _ptr(Ic),
                                      _stream(stream)))
    return Ic


def o_proj(x, w_o, y=None, workspace=None, stream=None):
    """y [R, hidden] = x [R, in_dim] (fp32) times w_o [hidden, in_dim]^T."""
    torch = _torch()
    x2 = x.reshape(-1, x.shape[-1]) if x.dim() == 2 else x.reshape(x.shape[0] * x.shape[1], -1)
    R, in_dim = x2.shape
    hidden = w_o.shape[0]
    code = _dtype_code(w_o)
    if y is None:
        y = torch.empty(R, hidden, dtype=torch.float32, device=x.device)
    need = lib().mla_o_proj_workspace_size(R, in_dim, hidden, code)
    workspace, wsb = _workspace(need, x.device, workspace)
    _check(lib().mla_o_proj(R, in_dim, hidden, code, _ptr(w_o), _ptr(x2), _ptr(y), _ptr(workspace), wsb,
                            _stream(stream)))
    return y


def decode_oproj(q, Lc, Rc, T, kv_b, w_o, dims, y=None, workspace=None, stream=None):
    """mla_decode_absorbed then the output projection: y [B, S, hidden]."""
    torch = _torch()
    B, S = q.shape[0], q.shape[1]
    T_cap = Lc.shape[1]
    hidden = w_o.shape[0]
    code = _dtype_code(q)
    if y is None:
        y = torch.empty(B, S, hidden, dtype=torch.float32, device=q.device)
    d = make_dims(dims)
    need = lib().mla_decode_oproj_workspace_size(ctypes.byref(d), code, B, S, T_cap, hidden)
    workspace, wsb = _workspace(need, q.device, workspace)
    _check(lib().mla_decode_oproj(ctypes.byref(d), code, B, S, _ptr(q), _ptr(Lc), _ptr(Rc), T_cap, _ptr(T),
                                  _ptr(kv_b), _ptr(w_o), hidden, _ptr(y), _ptr(workspace), wsb, _stream(stream)))
    return y


def select(q_idx, w, Ic, T, topk: int, scores=None, sel=None, nsel=None, workspace=None, stream=None):
    """Fused DSA selection: index scores then causal top-k -> (scores, sel, nsel)."""
    torch = _torch()
    B, S, n_ih, hd = q_idx.shape
    T_cap = Ic.shape[1]
    dev = q_idx.device
    if scores is None:
        scores = torch.empty(B, S, T_cap, dtype=torch.float32, device=dev)
    if sel is None:
        sel = torch.empty(B, S, topk, dtype=torch.int32, device=dev)
    if nsel is None:
        nsel = torch.empty(B, S, dtype=torch.int32, device=dev)
    need = lib().dsa_select_workspace_size(B, S, n_ih, hd, T_cap, topk)
    workspace, wsb = _workspace(need, dev, workspace)
    _check(lib().dsa_select(B, S, n_ih, hd, _ptr(q_idx), _ptr(w), _ptr(Ic), T_cap, _ptr(T), topk, _ptr(scores),
                            _ptr(sel), _ptr(nsel), _ptr(workspace), wsb, _stream(stream)))
    return scores, sel, nsel


# ------------------------------------------------------------------ paged cache
def decode_paged(q, Lc_pages, Rc_pages, block_table, T, kv_b, dims, out=None, workspace=None, stream=None):
    """Absorbed decode over a page pool: Lc_pages [num_pages, page_size, kv_lora],
    Rc_pages [num_pages, page_size, qk_rope], block_table [B, max_pages] int32."""
    torch = _torch()
    B, S, H = q.shape[0], q.shape[1], q.shape[2]
    num_pages, page_size = Lc_pages.shape[0], Lc_pages.shape[1]
    max_pages = block_table.shape[1]
    code = _dtype_code(q)
    if out is None:
        out = torch.empty(B, S, H, dims.v_head, dtype=torch.float32, device=q.device)
    d = make_dims(dims)
    need = lib().mla_decode_paged_workspace_size(ctypes.byref(d), code, B, S, max_pages, page_size)
    workspace, wsb = _workspace(need, q.device, workspace)
    _check(lib().mla_decode_paged(ctypes.byref(d), code, B, S, _ptr(q), _ptr(Lc_pages), _ptr(Rc_pages), num_pages,
                                  page_size, _ptr(block_table), max_pages, _ptr(T), _ptr(kv_b), _ptr(out),
                                  _ptr(workspace), wsb, _stream(stream)))
    return out


def sparse_decode_paged(q, Lc_pages, Rc_pages, block_table, T, kv_b, sel, nsel, dims, out=None, workspace=None,
                        stream=None):
    """Absorbed decode over the selected keys of a paged cache (sel holds token indices)."""
    torch = _torch()
    B, S, H = q.shape[0], q.shape[1], q.shape[2]
    num_pages, page_size = Lc_pages.shape[0], Lc_pages.shape[1]
    max_pages = block_table.shape[1]
    topk = sel.shape[2]
    code = _dtype_code(q)
    if out is None:
        out = torch.empty(B, S, H, dims.v_head, dtype=torch.float32, device=q.device)
    d = make_dims(dims)
    need = lib().mla_sparse_decode_workspace_size(ctypes.byref(d), code, B, S, topk)
    workspace, wsb = _workspace(need, q.device, workspace)
    _check(lib().mla_sparse_decode_paged(ctypes.byref(d), code, B, S, _ptr(q), _ptr(Lc_pages), _ptr(Rc_pages),
                                         num_pages, page_size, _ptr(block_table), max_pages, _ptr(T), _ptr(kv_b),
                                         _ptr(sel), _ptr(nsel), topk, _ptr(out), _ptr(workspace), wsb,
                                         _stream(stream)))
    return out


def cache_append_paged(comp, kv_a_ln, block_table, T, Lc_pages, Rc_pages, dims, rms_eps: float, stream=None):
    """mla_cache_append into the page pools (in place)."""
    B, S = comp.shape[0], comp.shape[1]
    num_pages, page_size = Lc_pages.shape[0], Lc_pages.shape[1]
    code = _dtype_code(comp)
    for t in (kv_a_ln, Lc_pages, Rc_pages):
        if t.dtype != comp.dtype:
            raise TypeError("comp, kv_a_ln and the pools must share one dtype")
    d = make_dims(dims)
    _check(lib().mla_cache_append_paged(ctypes.byref(d), code, B, S, _ptr(comp), _ptr(kv_a_ln), float(rms_eps),
                                        _ptr(Lc_pages), _ptr(Rc_pages), num_pages, page_size, _ptr(block_table),
                                        block_table.shape[1], _ptr(T), _stream(stream)))
    return Lc_pages, Rc_pages


# ------------------------------------------------------------- FP8 latent cache
def _need_bf16(*ts):
    torch = _torch()
    for t in ts:
        if t.dtype != torch.bfloat16:
            raise TypeError("the FP8 cache entry points take bf16 q, Rc, kv_b and comp")


def _need_u8(t):
    torch = _torch()
    if t.dtype != torch.uint8:
        raise TypeError("the FP8 latent cache holds uint8 E4M3 codes")


def decode_fp8(q, Lc8, Rc, T, kv_b, dims, lat_scale: float, out=None, workspace=None, stream=None):
    """Absorbed decode over an FP8 latent cache: Lc8 [B, T_cap, kv_lora] uint8
    E4M3 codes (latent = lat_scale * code), Rc [B, T_cap, qk_rope] bf16."""
    torch = _torch()
    _need_bf16(q, Rc, kv_b)
    _need_u8(Lc8)
    B, S, H = q.shape[0], q.shape[1], q.shape[2]
    T_cap = Lc8.shape[1]
    if out is None:
        out = torch.empty(B, S, H, dims.v_head, dtype=torch.float32, device=q.device)
    d = make_dims(dims)
    need = lib().mla_decode_fp8_workspace_size(ctypes.byref(d), B, S, T_cap)
    workspace, wsb = _workspace(need, q.device, workspace)
    _check(lib().mla_decode_fp8(ctypes.byref(d), B, S, _ptr(q), _ptr(Lc8), _ptr(Rc), float(lat_scale), T_cap,
                                _ptr(T), _ptr(kv_b), _ptr(out), _ptr(workspace), wsb, _stream(stream)))
    return out


def decode_fp8_paged(q, Lc8_pages, Rc_pages, block_table, T, kv_b, dims, lat_scale: float, out=None,
                     workspace=None, stream=None):
    """decode_fp8 over page pools: Lc8_pages [num_pages, page_size, kv_lora] uint8,
    Rc_pages [num_pages, page_size, qk_rope] bf16, block_table [B, max_pages] int32."""
    torch = _torch()
    _need_bf16(q, Rc_pages, kv_b)
    _need_u8(Lc8_pages)
    B, S, H = q.shape[0], q.shape[1], q.shape[2]
    num_pages, page_size = Lc8_pages.shape[0], Lc8_pages.shape[1]
    max_pages = block_table.shape[1]
    if out is None:
        out = torch.empty(B, S, H, dims.v_head, dtype=torch.float32, device=q.device)
    d = make_dims(dims)
    need = lib().mla_decode_fp8_workspace_size(ctypes.byref(d), B, S, max_pages * page_size)
    workspace, wsb = _workspace(need, q.device, workspace)
    _check(lib().mla_decode_fp8_paged(ctypes.byref(d), B, S, _ptr(q), _ptr(Lc8_pages), _ptr(Rc_pages),
                                      float(lat_scale), num_pages, page_size, _ptr(block_table), max_pages, _ptr(T),
                                      _ptr(kv_b), _ptr(out), _ptr(workspace), wsb, _stream(stream)))
    return out


def cache_append_fp8(comp, kv_a_ln, T, Lc8, Rc, dims, rms_eps: float, lat_scale: float, stream=None):
    """mla_cache_append into the FP8 cache (in place): Lc8 uint8 codes, Rc bf16."""
    _need_bf16(comp, kv_a_ln, Rc)
    _need_u8(Lc8)
    B, S = comp.shape[0], comp.shape[1]
    d = make_dims(dims)
    _check(lib().mla_cache_append_fp8(ctypes.byref(d), B, S, _ptr(comp), _ptr(kv_a_ln), float(rms_eps),
                                      float(lat_scale), Lc8.shape[1], _ptr(T), _ptr(Lc8), _ptr(Rc), _stream(stream)))
    return Lc8, Rc


def cache_append_fp8_paged(comp, kv_a_ln, block_table, T, Lc8_pages, Rc_pages, dims, rms_eps: float,
                           lat_scale: float, stream=None):
    """cache_append_fp8 into the page pools (in place)."""
    _need_bf16(comp, kv_a_ln, Rc_pages)
    _need_u8(Lc8_pages)
    B, S = comp.shape[0], comp.shape[1]
    num_pages, page_size = Lc8_pages.shape[0], Lc8_pages.shape[1]
    d = make_dims(dims)
    _check(lib().mla_cache_append_fp8_paged(ctypes.byref(d), B, S, _ptr(comp), _ptr(kv_a_ln), float(rms_eps),
                                            float(lat_scale), _ptr(Lc8_pages), _ptr(Rc_pages), num_pages, page_size,
                                            _ptr(block_table), block_table.shape[1], _ptr(T), _stream(stream)))
    return Lc8_pages, Rc_pages


# ------------------------------------------------------------- drafted token trees
def _all_plain(index, dtype, *ts) -> bool:
    """Every tensor contiguous, of `dtype`, on GPU `index` (the calls below are short: the check
    that passes is one expression per tensor, _explain finds words for one that fails)."""
    for t in ts:
        if t.dtype is not dtype or t.get_device() != index or not t.is_contiguous():
            return False
    return True


def _explain(device, **named):
    for name, (t, dtype) in named.items():
        if t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if t.device != device:
            raise ValueError(f"{name} is on {t.device}, not on {device}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")


def _current_stream(torch, index):
    """Handle of the current stream for a call on GPU `index` (-1: the CPU), which has to be the
    current one.  A call with a stream= makes that stream current first, so that outputs and
    scratch it allocates belong to the stream that uses them."""
    if index < 0:
        raise ValueError("tensors must live on the GPU")
    if index != torch._C._cuda_getDevice():
        raise ValueError(f"tensors on GPU {index}: make it the current device")
    return torch._C._cuda_getCurrentRawStream(index)


def _want(name, t, *shape):
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")


def decode_tree_workspace_size(dims, dtype, B: int, S: int, T_cap: int) -> int:
    """Workspace bytes of decode_tree (dtype: torch.float32 or torch.bfloat16); the
    paged call takes T_cap = max_pages * page_size."""
    torch = _torch()
    code = MLA_BF16 if dtype in (torch.bfloat16, MLA_BF16) else MLA_F32
    d = make_dims(dims)
    return lib().mla_decode_tree_workspace_size(ctypes.byref(d), code, B, S, T_cap)


def _tree_args(torch, q, Lc, Rc, T, parent, kv_b, dims, out, out_dtype, workspace, T_cap):
    """Checks shared by the two tree attentions ->
    (dims struct, dtype code, out, its code, workspace, its bytes)."""
    B, S, H, qk = q.shape
    dtype, index = q.dtype, q.get_device()
    if H != dims.H or qk != dims.qk_nope + dims.qk_rope:
        raise ValueError(f"q has shape {tuple(q.shape)}, expected [B, S, {dims.H}, {dims.qk_nope + dims.qk_rope}]")
    code = _dtype_code(q)
    if out is None:
        out = torch.empty((B, S, H, dims.v_head), dtype=out_dtype or torch.float32, device=q.device)
    else:
        if out_dtype is not None and out.dtype != out_dtype:
            raise TypeError("out does not have out_dtype")
        _want("out", out, B, S, H, dims.v_head)
    out_code = _dtype_code(out)
    ls = Lc.shape
    if ls[2] != dims.kv_lora or Rc.shape != (ls[0], ls[1], dims.qk_rope):
        raise ValueError("cache shapes do not match dims")
    _want("T", T, B)
    _want("parent", parent, B, S)
    _want("kv_b", kv_b, H, dims.qk_nope + dims.v_head, dims.kv_lora)
    i32 = torch.int32
    if not (_all_plain(index, dtype, q, Lc, Rc, kv_b) and _all_plain(index, i32, T, parent)
            and _all_plain(index, out.dtype, out)):
        _explain(q.device, q=(q, dtype), Lc=(Lc, dtype), Rc=(Rc, dtype), kv_b=(kv_b, dtype), T=(T, i32), parent=(parent, i32),
                 out=(out, out.dtype))
    d = make_dims(dims)
    if workspace is None:  # the library checks the size of one that is given
        workspace, wsb = _workspace(lib().mla_decode_tree_workspace_size(ctypes.byref(d), code, B, S, T_cap), q.device, None)
    else:
        if workspace.get_device() != index or not workspace.is_contiguous():
            raise ValueError(f"workspace must be contiguous and on {q.device}")
        wsb = workspace.numel() * workspace.element_size()
    return d, code, out, out_code, None if workspace is None else workspace.data_ptr(), wsb


def decode_tree(q, Lc, Rc, T, parent, kv_b, dims, out=None, out_dtype=None, workspace=None, stream=None):
    """Absorbed decode of a drafted tree: q [B,S,H,qk] (node s at row T[b]-S+s), parent [B,S]
    int32 (-1 a child of the last committed token, -2 absent).  out [B,S,H,v_head] in
    out_dtype (float32 unless given; bfloat16 is rounded once).  A workspace that is given
    must have decode_tree_workspace_size() bytes."""
    torch = _torch()
    if stream is not None:
        with torch.cuda.stream(stream):
            return decode_tree(q, Lc, Rc, T, parent, kv_b, dims, out, out_dtype, workspace)
    B, S = q.shape[0], q.shape[1]
    T_cap = Lc.shape[1]
    if Lc.shape[0] != B:
        raise ValueError(f"cache of {Lc.shape[0]} sequences for {B} queries")
    d, code, out, out_code, ws, wsb = _tree_args(torch, q, Lc, Rc, T, parent, kv_b, dims, out, out_dtype, workspace, T_cap)
    st = _current_stream(torch, q.get_device())
    _check(lib().mla_decode_tree(ctypes.byref(d), code, B, S, q.data_ptr(), Lc.data_ptr(), Rc.data_ptr(), T_cap,
                                 T.data_ptr(), parent.data_ptr(), kv_b.data_ptr(), out_code, out.data_ptr(), ws, wsb, st))
    return out


def decode_tree_paged(q, Lc_pages, Rc_pages, block_table, T, parent, kv_b, dims, out=None, out_dtype=None,
                      workspace=None, stream=None):
    """decode_tree over page pools (layouts as for decode_paged)."""
    torch = _torch()
    if stream is not None:
        with torch.cuda.stream(stream):
            return decode_tree_paged(q, Lc_pages, Rc_pages, block_table, T, parent, kv_b, dims, out, out_dtype, workspace)
    B, S = q.shape[0], q.shape[1]
    num_pages, page_size = Lc_pages.shape[0], Lc_pages.shape[1]
    max_pages = block_table.shape[1]
    _want("block_table", block_table, B, max_pages)
    _explain(q.device, block_table=(block_table, torch.int32))
    d, code, out, out_code, ws, wsb = _tree_args(torch, q, Lc_pages, Rc_pages, T, parent, kv_b, dims, out, out_dtype, workspace,
                                       max_pages * page_size)
    st = _current_stream(torch, q.get_device())
    _check(lib().mla_decode_tree_paged(ctypes.byref(d), code, B, S, q.data_ptr(), Lc_pages.data_ptr(),
                                       Rc_pages.data_ptr(), num_pages, page_size, block_table.data_ptr(), max_pages,
                                       T.data_ptr(), parent.data_ptr(), kv_b.data_ptr(), out_code, out.data_ptr(), ws,
                                       wsb, st))
    return out


def _append_tree_args(torch, comp, kv_a_ln, T, parent, Lc, Rc, dims):
    B, S = comp.shape[0], comp.shape[1]
    dtype, index, i32 = comp.dtype, comp.get_device(), torch.int32
    _want("comp", comp, B, S, dims.kv_lora + dims.qk_rope)
    _want("kv_a_ln", kv_a_ln, dims.kv_lora)
    _want("T", T, B)
    _want("parent", parent, B, S)
    ls = Lc.shape
    if ls[2] != dims.kv_lora or Rc.shape != (ls[0], ls[1], dims.qk_rope):
        raise ValueError("cache shapes do not match dims")
    if not (_all_plain(index, dtype, comp, kv_a_ln, Lc, Rc) and _all_plain(index, i32, T, parent)):
        _explain(comp.device, comp=(comp, dtype), kv_a_ln=(kv_a_ln, dtype), Lc=(Lc, dtype), Rc=(Rc, dtype), T=(T, i32),
                 parent=(parent, i32))
    return B, S, make_dims(dims), _dtype_code(comp)


def cache_append_tree(comp, kv_a_ln, T, parent, Lc, Rc, dims, rms_eps: float, stream=None):
    """cache_append of a drafted tree: node s goes to row T[b]-S+s with the rotary
    position of its depth; rows of absent nodes (parent -2) are left as they were."""
    torch = _torch()
    if stream is not None:
        with torch.cuda.stream(stream):
            return cache_append_tree(comp, kv_a_ln, T, parent, Lc, Rc, dims, rms_eps)
    B, S, d, code = _append_tree_args(torch, comp, kv_a_ln, T, parent, Lc, Rc, dims)
    if Lc.shape[0] != B:
        raise ValueError(f"cache of {Lc.shape[0]} sequences for {B} rows")
    st = _current_stream(torch, comp.get_device())
    _check(lib().mla_cache_append_tree(ctypes.byref(d), code, B, S, comp.data_ptr(), kv_a_ln.data_ptr(), rms_eps,
                                       Lc.shape[1], T.data_ptr(), parent.data_ptr(), Lc.data_ptr(), Rc.data_ptr(), st))
    return Lc, Rc


def cache_append_tree_paged(comp, kv_a_ln, block_table, T, parent, Lc_pages, Rc_pages, dims, rms_eps: float,
                            stream=None):
    """cache_append_tree into the page pools (in place)."""
    torch = _torch()
    if stream is not None:
        with torch.cuda.stream(stream):
            return cache_append_tree_paged(comp, kv_a_ln, block_table, T, parent, Lc_pages, Rc_pages, dims, rms_eps)
    B, S, d, code = _append_tree_args(torch, comp, kv_a_ln, T, parent, Lc_pages, Rc_pages, dims)
    _want("block_table", block_table, B, block_table.shape[1])
    _explain(comp.device, block_table=(block_table, torch.int32))
    st = _current_stream(torch, comp.get_device())
    _check(lib().mla_cache_append_tree_paged(ctypes.byref(d), code, B, S, comp.data_ptr(), kv_a_ln.data_ptr(), rms_eps,
                                             Lc_pages.data_ptr(), Rc_pages.data_ptr(), Lc_pages.shape[0],
                                             Lc_pages.shape[1], block_table.data_ptr(), block_table.shape[1],
                                             T.data_ptr(), parent.data_ptr(), st))
    return Lc_pages, Rc_pages


def tree_verify(p, q, tokens, parent, u, path=None, n_acc=None, token=None, stream=None):
    """Accepts a path of each drafted tree and draws the token after it.

    p [B,S+1,V] float32: the target's probabilities after the last committed token (row 0)
    and after node s (row s+1); q likewise for the draft, or None for drafts without
    probabilities (rows may be strided, values within a row contiguous); tokens, parent
    [B,S] int32; u [B,S+1] float32 in [0,1).  Returns (path [B,S] accepted nodes then -1,
    n_acc [B], token [B]), all int32."""
    torch = _torch()
    if stream is not None:
        with torch.cuda.stream(stream):
            return tree_verify(p, q, tokens, parent, u, path, n_acc, token)
    B, S = shape = tokens.shape
    index, f32, i32 = p.get_device(), torch.float32, torch.int32
    want = (B, S + 1, p.shape[2])
    if p.shape != want or p.dtype is not f32 or (q is not None and (q.shape != want or q.dtype is not f32 or q.get_device() != index)):
        for name, x in (("p", p), ("q", p if q is None else q)):
            _want(name, x, *want)
            if x.dtype is not f32:
                raise TypeError(f"{name} must be torch.float32, got {x.dtype}")
        raise ValueError(f"q is on {q.device}, not on {p.device}")
    pb, pr, pv = p.stride()
    qp, qb, qr, qv = (None, 0, 0, 1) if q is None else (q.data_ptr(), *q.stride())
    if (pv != 1 or qv != 1) and want[2] > 1:
        raise ValueError("the values of a row of p and of q must be contiguous")
    if parent.shape != shape or u.shape != want[:2]:
        _want("parent", parent, B, S)
        _want("u", u, B, S + 1)
    if not (_all_plain(index, i32, tokens, parent) and _all_plain(index, f32, u)):
        _explain(p.device, tokens=(tokens, i32), parent=(parent, i32), u=(u, f32))
    st = _current_stream(torch, index)
    if path is None:
        path = torch.empty_like(tokens)
    else:
        _want("path", path, B, S)
        _explain(p.device, path=(path, i32))
    if n_acc is None:
        n_acc = tokens.new_empty(B)
    else:
        _want("n_acc", n_acc, B)
        _explain(p.device, n_acc=(n_acc, i32))
    if token is None:
        token = tokens.new_empty(B)
    else:
        _want("token", token, B)
        _explain(p.device, token=(token, i32))
    _check(lib().mla_tree_verify(B, S, want[2], p.data_ptr(), pr, pb, qp, qr, qb, tokens.data_ptr(), parent.data_ptr(),
                                u.data_ptr(), path.data_ptr(), n_acc.data_ptr(), token.data_ptr(), st))
    return path, n_acc, token


class CacheRows:
    """The caches that tree_commit moves rows in: every layer's tensors [B, T_cap, row]
    (any dtypes and row widths), or pools [num_pages, page_size, row] with their
    block_table [B, max_pages].  Holds the tensors, so it can be kept with them."""

    def __init__(self, caches, block_table=None):
        torch = _torch()
        self.caches = list(caches)
        if not self.caches:
            raise ValueError("no caches")
        first = self.caches[0]
        for c in self.caches:
            if c.dim() != 3 or c.shape[:2] != first.shape[:2] or c.shape[2] < 1:
                raise ValueError("caches need one shape [B, T_cap, row] up to the row width")
        for c in self.caches:
            if not c.is_cuda or c.device != first.device or not c.is_contiguous():
                raise ValueError("caches must be contiguous tensors on one GPU")
        self.device = first.device
        self.block_table = block_table
        if block_table is not None:
            if block_table.dtype != torch.int32 or block_table.device != self.device or not block_table.is_contiguous():
                raise ValueError("block_table must be a contiguous int32 tensor on the caches' GPU")
            if block_table.dim() != 2:
                raise ValueError("block_table must be [B, max_pages]")
        self.B = first.shape[0] if block_table is None else block_table.shape[0]
        self.rows, self.cap = first.shape[0], first.shape[1]
        self.index = first.get_device()
        n = len(self.caches)
        self.n = n
        self.pointers = (ctypes.c_void_p * n)(*[c.data_ptr() for c in self.caches])
        self.row_bytes = (ctypes.c_int * n)(*[c.shape[2] * c.element_size() for c in self.caches])


def tree_commit(rows: CacheRows, T, path, n_acc, T_out=None, stream=None):
    """Moves the rows of the accepted nodes (path, n_acc of tree_verify) to the front of the
    tree's rows in every cache of `rows`; returns T_out [B] int32 = T - S + n_acc."""
    torch = _torch()
    if stream is not None:
        with torch.cuda.stream(stream):
            return tree_commit(rows, T, path, n_acc, T_out)
    B, S = path.shape
    index, i32, shape = rows.index, torch.int32, (B,)
    if B != rows.B:
        raise ValueError(f"caches of {rows.B} sequences, path of {B}")
    if T.shape != shape or n_acc.shape != shape:
        _want("T", T, B)
        _want("n_acc", n_acc, B)
    if not _all_plain(index, i32, T, path, n_acc):
        _explain(rows.device, T=(T, i32), path=(path, i32), n_acc=(n_acc, i32))
    st = _current_stream(torch, index)
    if T_out is None:
        T_out = torch.empty_like(T)
    else:
        _want("T_out", T_out, B)
        _explain(rows.device, T_out=(T_out, i32))
    table = rows.block_table
    if table is None:
        rc = lib().mla_tree_commit(rows.n, rows.pointers, rows.row_bytes, B, S, rows.cap, T.data_ptr(), path.data_ptr(),
                                   n_acc.data_ptr(), T_out.data_ptr(), st)
    else:
        rc = lib().mla_tree_commit_paged(rows.n, rows.pointers, rows.row_bytes, B, S, rows.rows, rows.cap,
                                         table.data_ptr(), table.shape[1], T.data_ptr(), path.data_ptr(),
                                         n_acc.data_ptr(), T_out.data_ptr(), st)
    _check(rc)
    return T_out
