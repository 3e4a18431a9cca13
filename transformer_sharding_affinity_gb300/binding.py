"""ctypes binding of libaffinity (include/affinity.h).

Argument marshalling only: every function forwards to the C entry point of
the same name.  Device tensors are PyTorch CUDA tensors (PyTorch supplies
device memory and streams); nothing here computes any part of the scores.
Loading fails loudly if the compiled library is missing -- there is no
fallback implementation.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libaffinity.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "affinity.h")

AFF_OK = 0
AFF_ERR_INVALID_ARG = 1
AFF_ERR_UNSUPPORTED_SHAPE = 2
AFF_ERR_UNSUPPORTED_DTYPE = 3
AFF_ERR_ARCH = 4
AFF_ERR_WORKSPACE = 5
AFF_ERR_CUDA = 6
AFF_ERR_DEVICE_TIMEOUT = 7
AFF_ERR_RANGE = 8
AFF_ERR_ALIGNMENT = 9
AFF_ERR_NO_CONVERGENCE = 10

AFF_MODE_FO = 0
AFF_MODE_ADD = 1
AFF_MODE_LOO = 2
AFF_BF16 = 0
AFF_FP32 = 1
AFF_FLAG_ADD_DIRECT = 1
MODES = {"fo": AFF_MODE_FO, "add": AFF_MODE_ADD, "loo": AFF_MODE_LOO}


class aff_dims(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("D", ctypes.c_int64), ("H", ctypes.c_int64), ("G", ctypes.c_int64),
                ("d_head", ctypes.c_int64), ("I", ctypes.c_int64), ("eps", ctypes.c_float),
                ("dtype", ctypes.c_int32), ("flags", ctypes.c_uint32)]


class aff_assign_opts(ctypes.Structure):
    _fields_ = [("dual_iters", ctypes.c_int32), ("dual_decay", ctypes.c_double), ("max_cycles", ctypes.c_int64)]


class aff_layout_opts(ctypes.Structure):
    _fields_ = [("max_sweeps", ctypes.c_int32), ("freeze_heads", ctypes.c_int32),
                ("freeze_neurons", ctypes.c_int32), ("minimise", ctypes.c_int32),
                ("layer_mask", ctypes.c_void_p), ("assign", aff_assign_opts)]


class aff_kv_cache(ctypes.Structure):
    device = None   # of the tensors it was made from; not known of raw addresses
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("n_pages", ctypes.c_int64),
                ("page_stride", ctypes.c_int64), ("group_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("G", ctypes.c_int32), ("page_size", ctypes.c_int32), ("d_head", ctypes.c_int32),
                ("dtype", ctypes.c_int32)]


class aff_step(ctypes.Structure):
    device = None   # of the tensors it was made from; not known of raw addresses
    copied = None   # (a part of a wider page table, its dense copy)
    _fields_ = [("T", ctypes.c_int64), ("prefix_len", ctypes.c_int64), ("pages_stride", ctypes.c_int64),
                ("q_start", ctypes.c_void_p), ("kv_len", ctypes.c_void_p), ("pages", ctypes.c_void_p),
                ("prefix_pages", ctypes.c_void_p), ("B", ctypes.c_int32), ("H", ctypes.c_int32)]


class aff_rotary(ctypes.Structure):
    device = None   # of the tensors it was made from; not known of raw addresses
    _fields_ = [("cos", ctypes.c_void_p), ("sin", ctypes.c_void_p), ("q_gain", ctypes.c_void_p),
                ("k_gain", ctypes.c_void_p), ("n_pos", ctypes.c_int64), ("eps", ctypes.c_float),
                ("rot", ctypes.c_int32), ("interleaved", ctypes.c_int32)]


class aff_block_norm(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("f", ctypes.c_void_p), ("gate", ctypes.c_void_p),
                ("post_gain", ctypes.c_void_p), ("pre_gain", ctypes.c_void_p), ("y", ctypes.c_void_p),
                ("h", ctypes.c_void_p), ("T", ctypes.c_int64), ("D", ctypes.c_int64), ("x_stride", ctypes.c_int64),
                ("f_stride", ctypes.c_int64), ("gate_stride", ctypes.c_int64), ("y_stride", ctypes.c_int64),
                ("h_stride", ctypes.c_int64), ("rows_per_gate", ctypes.c_int64), ("scale", ctypes.c_float),
                ("eps", ctypes.c_float), ("dtype", ctypes.c_int32)]


class AffinityError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str = ""):
        self.status = status
        super().__init__(f"{where}: status {status}: {detail}")


_lib = None
_P = ctypes.c_void_p


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libaffinity.so (built by __graft_entry__.build()); raises if absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"libaffinity.so not found at {path}: run __graft_entry__.build() first")
    lib = ctypes.CDLL(path)
    st = ctypes.c_int32
    lib.affinity_workspace_size.argtypes = [ctypes.POINTER(aff_dims), ctypes.c_int32, ctypes.c_int32,
                                            ctypes.POINTER(ctypes.c_size_t)]
    lib.affinity_workspace_size.restype = st
    lib.affinity_up.argtypes = [_P] * 7 + [ctypes.POINTER(aff_dims), ctypes.c_int32, _P, _P, _P, ctypes.c_size_t, _P]
    lib.affinity_up.restype = st
    lib.affinity_up_static.argtypes = [_P] * 7 + [ctypes.POINTER(aff_dims), ctypes.c_int32, _P, _P, _P]
    lib.affinity_up_static.restype = st
    lib.affinity_down.argtypes = [_P] * 9 + [ctypes.POINTER(aff_dims), _P, _P, ctypes.c_size_t, _P]
    lib.affinity_down.restype = st
    lib.affinity_device_status.argtypes = [_P, _P]
    lib.affinity_device_status.restype = st
    lib.affinity_static_device_status.argtypes = [_P]
    lib.affinity_static_device_status.restype = st
    lib.affinity_score_partitions.argtypes = [_P, ctypes.c_int32, ctypes.c_int32, _P, ctypes.POINTER(ctypes.c_int64),
                                              ctypes.POINTER(ctypes.c_int64), _P]
    lib.affinity_score_partitions.restype = st
    lib.affinity_group_gain.argtypes = [_P, _P, _P, _P, ctypes.c_int32, ctypes.c_int64, ctypes.c_int32, _P]
    lib.affinity_group_gain.restype = st
    lib.affinity_objective.argtypes = [_P, _P, _P, _P, ctypes.c_int32, ctypes.c_int32, ctypes.c_int64, _P]
    lib.affinity_objective.restype = st
    lib.affinity_unit_mass.argtypes = [_P, ctypes.c_int64, _P]
    lib.affinity_unit_mass.restype = st
    lib.affinity_best_heads.argtypes = [_P, _P, _P, ctypes.c_int32, ctypes.c_int32, ctypes.c_int64, ctypes.c_int32,
                                        _P, _P]
    lib.affinity_best_heads.restype = st
    lib.affinity_combine_shards.argtypes = [_P, _P, ctypes.c_int32, ctypes.c_int64, _P]
    lib.affinity_combine_shards.restype = st
    lib.affinity_neuron_gain.argtypes = [_P, _P, _P, _P, ctypes.c_int32, ctypes.c_int64, ctypes.c_int32, _P, _P]
    lib.affinity_neuron_gain.restype = st
    lib.affinity_assign_neurons.argtypes = [_P, ctypes.c_int32, ctypes.c_int64, ctypes.c_int32,
                                            ctypes.POINTER(aff_assign_opts), _P, _P, _P, ctypes.c_size_t, _P]
    lib.affinity_assign_neurons.restype = st
    lib.affinity_layout_workspace_size.argtypes = [ctypes.c_int32, ctypes.c_int32, ctypes.c_int64, ctypes.c_int32,
                                                   ctypes.POINTER(ctypes.c_size_t)]
    lib.affinity_layout_workspace_size.restype = st
    lib.affinity_optimise_layout.argtypes = [_P, _P, ctypes.c_int32, ctypes.c_int32, ctypes.c_int64, ctypes.c_int32,
                                             ctypes.POINTER(aff_layout_opts), _P, _P, ctypes.POINTER(ctypes.c_double),
                                             ctypes.POINTER(ctypes.c_int32), _P, ctypes.c_size_t, _P]
    lib.affinity_optimise_layout.restype = st
    lib.affinity_selftest_timeout.argtypes = [_P, ctypes.c_size_t, ctypes.c_int64, _P]
    lib.affinity_selftest_timeout.restype = st
    lib.affinity_layout_orders.argtypes = [_P, _P, ctypes.c_int32, ctypes.c_int64, ctypes.c_int64, ctypes.c_int32,
                                           _P, _P, _P]
    lib.affinity_layout_orders.restype = st
    lib.affinity_gather_blocks.argtypes = [_P, _P, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, _P, _P,
                                           ctypes.c_size_t, _P]
    lib.affinity_gather_blocks.restype = st
    lib.affinity_step_plan_size.argtypes = [ctypes.POINTER(aff_step), ctypes.POINTER(aff_kv_cache),
                                            ctypes.POINTER(ctypes.c_size_t)]
    lib.affinity_step_plan_size.restype = st
    lib.affinity_step_plan.argtypes = [ctypes.POINTER(aff_step), ctypes.POINTER(aff_kv_cache), _P, ctypes.c_size_t, _P]
    lib.affinity_step_plan.restype = st
    lib.affinity_kv_append.argtypes = [_P, ctypes.c_int64, _P, ctypes.c_int64, _P, ctypes.c_int64,
                                       ctypes.POINTER(aff_kv_cache), ctypes.POINTER(aff_step),
                                       ctypes.POINTER(aff_rotary), _P, ctypes.c_int64, _P, ctypes.c_size_t, _P]
    lib.affinity_kv_append.restype = st
    lib.affinity_prefix_attention.argtypes = [_P, ctypes.c_int64, ctypes.POINTER(aff_kv_cache),
                                              ctypes.POINTER(aff_step), ctypes.c_float, _P, _P, _P, ctypes.c_size_t,
                                              _P]
    lib.affinity_prefix_attention.restype = st
    lib.affinity_block_norm.argtypes = [ctypes.POINTER(aff_block_norm), _P]
    lib.affinity_block_norm.restype = st
    lib.affinity_strerror.argtypes = [ctypes.c_int32]
    lib.affinity_strerror.restype = ctypes.c_char_p
    lib.affinity_last_cuda_error.argtypes = []
    lib.affinity_last_cuda_error.restype = ctypes.c_char_p
    lib.affinity_set_timing_events.argtypes = [_P, _P]
    lib.affinity_set_timing_events.restype = st
    lib.affinity_version.argtypes = []
    lib.affinity_version.restype = ctypes.c_int32
    _lib = lib
    return lib


def strerror(status: int) -> str:
    return load().affinity_strerror(status).decode()


def _check(status: int, where: str) -> None:
    if status != AFF_OK:
        lib = load()
        detail = strerror(status)
        if status == AFF_ERR_CUDA:
            detail += " -- " + lib.affinity_last_cuda_error().decode()
        raise AffinityError(status, where, detail)


def dims(T, D, H, G, d_head, I, eps=1e-6, dtype=AFF_BF16, flags=0) -> aff_dims:
    return aff_dims(int(T), int(D), int(H), int(G), int(d_head), int(I), float(eps), int(dtype), int(flags))


def workspace_size(d: aff_dims, mode: int = AFF_MODE_FO, down: bool = False) -> int:
    n = ctypes.c_size_t(0)
    _check(load().affinity_workspace_size(ctypes.byref(d), int(mode), int(bool(down)), ctypes.byref(n)),
           "affinity_workspace_size")
    return n.value


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        # the handle alone: building the Stream object of torch.cuda.current_stream() takes microseconds
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _ws_bytes(workspace, workspace_bytes):
    if workspace_bytes is not None:
        return int(workspace_bytes)
    if hasattr(workspace, "nbytes"):
        return workspace.nbytes
    raise ValueError("workspace_bytes is required when the workspace is a raw address")


def affinity_up(a, x, Wo, gamma, Wg, Wu, Wd, d: aff_dims, mode: int, S_out, S_head_out, workspace,
                stream=None, workspace_bytes=None) -> None:
    """Enqueue S_up (see include/affinity.h). Tensors are CUDA tensors (or raw device addresses)."""
    nbytes = _ws_bytes(workspace, workspace_bytes)
    _check(load().affinity_up(_ptr(a), _ptr(x), _ptr(Wo), _ptr(gamma), _ptr(Wg), _ptr(Wu), _ptr(Wd),
                              ctypes.byref(d), int(mode), _ptr(S_out), _ptr(S_head_out), _ptr(workspace), nbytes,
                              _stream(stream)), "affinity_up")


def affinity_up_static(a, x, Wo, gamma, Wg, Wu, Wd, d: aff_dims, mode: int, S_out, S_head_out,
                       stream=None) -> None:
    """Enqueue S_up using the library's built-in 64 MiB scratch instead of a workspace."""
    _check(load().affinity_up_static(_ptr(a), _ptr(x), _ptr(Wo), _ptr(gamma), _ptr(Wg), _ptr(Wu), _ptr(Wd),
                                     ctypes.byref(d), int(mode), _ptr(S_out), _ptr(S_head_out), _stream(stream)),
           "affinity_up_static")


def affinity_down(x, gamma, Wg, Wu, Wd, gamma_next, Wq_next, Wk_next, Wv_next, d: aff_dims, S_out, workspace,
                  stream=None, workspace_bytes=None) -> None:
    """Enqueue S_down (see include/affinity.h)."""
    nbytes = _ws_bytes(workspace, workspace_bytes)
    _check(load().affinity_down(_ptr(x), _ptr(gamma), _ptr(Wg), _ptr(Wu), _ptr(Wd), _ptr(gamma_next),
                                _ptr(Wq_next), _ptr(Wk_next), _ptr(Wv_next), ctypes.byref(d), _ptr(S_out),
                                _ptr(workspace), nbytes, _stream(stream)), "affinity_down")


def selftest_timeout(workspace, limit_ns: int = 5_000_000, stream=None, workspace_bytes=None) -> None:
    """Enqueue a kernel whose one bounded wait must time out (affinity_selftest_timeout)."""
    _check(load().affinity_selftest_timeout(_ptr(workspace), _ws_bytes(workspace, workspace_bytes), int(limit_ns),
                                            _stream(stream)), "affinity_selftest_timeout")


def device_status(workspace, stream=None) -> int:
    """Synchronise and return (then clear) the device-latched status of the last call."""
    return int(load().affinity_device_status(_ptr(workspace), _stream(stream)))


def static_device_status(stream=None) -> int:
    """As device_status, for the array affinity_up_static uses in place of a workspace."""
    return int(load().affinity_static_device_status(_stream(stream)))


def score_partitions(C: np.ndarray):
    """Score all balanced partitions: returns (scores, count, best_index, best_assign)."""
    lib = load()
    C = np.ascontiguousarray(C, dtype=np.float64)
    G, L = C.shape
    count, best = ctypes.c_int64(0), ctypes.c_int64(0)
    _check(lib.affinity_score_partitions(C.ctypes.data, G, L, None, ctypes.byref(count), ctypes.byref(best), None),
           "affinity_score_partitions")
    scores = np.empty(count.value, np.float64)
    assign = np.empty(G, np.int32)
    _check(lib.affinity_score_partitions(C.ctypes.data, G, L, scores.ctypes.data, ctypes.byref(count),
                                         ctypes.byref(best), assign.ctypes.data), "affinity_score_partitions")
    return scores, int(count.value), int(best.value), tuple(int(v) for v in assign)


def group_gain(Shat_up_i: np.ndarray, nu_i: Sequence[int], L: int, Shat_down_prev: Optional[np.ndarray] = None,
               nu_prev: Optional[Sequence[int]] = None) -> np.ndarray:
    S = np.ascontiguousarray(Shat_up_i, dtype=np.float64)
    G, I = S.shape
    nu = np.ascontiguousarray(nu_i, dtype=np.int32)
    C = np.zeros((G, L), np.float64)
    Sd = None if Shat_down_prev is None else np.ascontiguousarray(Shat_down_prev, dtype=np.float64)
    npv = None if nu_prev is None else np.ascontiguousarray(nu_prev, dtype=np.int32)
    _check(load().affinity_group_gain(S.ctypes.data, nu.ctypes.data, None if Sd is None else Sd.ctypes.data,
                                      None if npv is None else npv.ctypes.data, G, I, L, C.ctypes.data),
           "affinity_group_gain")
    return C


def objective(Shat_up: Sequence[np.ndarray], Shat_down: Sequence[np.ndarray], h: Sequence, nu: Sequence) -> float:
    N = len(Shat_up)
    G, I = np.asarray(Shat_up[0]).shape
    up = np.ascontiguousarray(np.stack([np.asarray(s, np.float64) for s in Shat_up]))
    dn = np.ascontiguousarray(np.stack([np.asarray(s, np.float64) for s in Shat_down])) if N > 1 else None
    hh = np.ascontiguousarray(np.stack([np.asarray(v, np.int32) for v in h]))
    nn = np.ascontiguousarray(np.stack([np.asarray(v, np.int32) for v in nu]))
    J = ctypes.c_double(0.0)
    _check(load().affinity_objective(up.ctypes.data, None if dn is None else dn.ctypes.data, hh.ctypes.data,
                                     nn.ctypes.data, N, G, I, ctypes.byref(J)), "affinity_objective")
    return J.value


def unit_mass(S: np.ndarray) -> np.ndarray:
    """S / sum(S) in fp64 (affinity_unit_mass); S is a host fp32 array of any shape."""
    S = np.ascontiguousarray(S, dtype=np.float32)
    out = np.empty(S.shape, np.float64)
    _check(load().affinity_unit_mass(S.ctypes.data, S.size, out.ctypes.data), "affinity_unit_mass")
    return out


def best_heads(Shat_up: Sequence[np.ndarray], Shat_down: Sequence[np.ndarray], nu: Sequence, L: int):
    """Best balanced KV-group map of every layer for fixed neuron maps (affinity_best_heads).

    Returns (h [N, G] int32, J of (h, nu))."""
    N = len(Shat_up)
    G, I = np.asarray(Shat_up[0]).shape
    up = np.ascontiguousarray(np.stack([np.asarray(s, np.float64) for s in Shat_up]))
    dn = np.ascontiguousarray(np.stack([np.asarray(s, np.float64) for s in Shat_down])) if N > 1 else None
    nn = np.ascontiguousarray(np.stack([np.asarray(v, np.int32) for v in nu]))
    h = np.empty((N, G), np.int32)
    J = ctypes.c_double(0.0)
    _check(load().affinity_best_heads(up.ctypes.data, None if dn is None else dn.ctypes.data, nn.ctypes.data, N, G,
                                      I, int(L), h.ctypes.data, ctypes.byref(J)), "affinity_best_heads")
    return h, J.value


def combine_shards(S_shards: Sequence[np.ndarray], T_shards: Sequence[int]) -> np.ndarray:
    """Token-weighted merge of S matrices from disjoint token shards (affinity_combine_shards)."""
    arrs = [np.ascontiguousarray(s, dtype=np.float32) for s in S_shards]
    shape = arrs[0].shape
    if any(a.shape != shape for a in arrs):
        raise ValueError("all shards must have the same shape")
    ptrs = (ctypes.c_void_p * len(arrs))(*[a.ctypes.data for a in arrs])
    T = np.ascontiguousarray(T_shards, dtype=np.int64)
    if T.shape != (len(arrs),):
        raise ValueError("one token count per shard")
    out = np.empty(shape, np.float32)
    _check(load().affinity_combine_shards(ctypes.cast(ptrs, ctypes.c_void_p), T.ctypes.data, len(arrs),
                                          arrs[0].size, out.ctypes.data), "affinity_combine_shards")
    return out


def neuron_gain(Shat_up_i, Shat_down_i, h_i, h_next, L: int, M_out, stream=None) -> None:
    """Enqueue M [I, L] (affinity_neuron_gain); Shat_* and M_out are CUDA fp64 tensors."""
    G, I = Shat_up_i.shape
    h = np.ascontiguousarray(h_i, dtype=np.int32)
    hn = None if h_next is None else np.ascontiguousarray(h_next, dtype=np.int32)
    _check(load().affinity_neuron_gain(_ptr(Shat_up_i), _ptr(Shat_down_i), h.ctypes.data,
                                       None if hn is None else hn.ctypes.data, G, I, int(L), _ptr(M_out),
                                       _stream(stream)), "affinity_neuron_gain")


def assign_opts(dual_iters: int = 0, dual_decay: float = 0.0, max_cycles: int = 0) -> aff_assign_opts:
    return aff_assign_opts(int(dual_iters), float(dual_decay), int(max_cycles))


def assign_neurons(M, L: int, nu_out, value_out, workspace, opts: Optional[aff_assign_opts] = None,
                   stream=None, workspace_bytes=None) -> None:
    """Enqueue the balanced neuron solver on M [n, I, L] (CUDA fp64) -> nu_out [n, I] int32, value_out [n] fp64."""
    n, I = (1, M.shape[0]) if M.dim() == 2 else (M.shape[0], M.shape[1])
    _check(load().affinity_assign_neurons(_ptr(M), n, I, int(L), None if opts is None else ctypes.byref(opts),
                                          _ptr(nu_out), _ptr(value_out), _ptr(workspace),
                                          _ws_bytes(workspace, workspace_bytes), _stream(stream)),
           "affinity_assign_neurons")


def layout_workspace_size(N: int, G: int, I: int, L: int) -> int:
    n = ctypes.c_size_t(0)
    _check(load().affinity_layout_workspace_size(int(N), int(G), int(I), int(L), ctypes.byref(n)),
           "affinity_layout_workspace_size")
    return n.value


def optimise_layout(Shat_up: Sequence[np.ndarray], Shat_down: Sequence[np.ndarray], L: int, h0, nu0, workspace,
                    max_sweeps: int = 0, freeze_heads: bool = False, freeze_neurons: bool = False,
                    minimise: bool = False, layer_mask=None, assign: Optional[aff_assign_opts] = None,
                    stream=None, workspace_bytes=None):
    """Alternating layout search (affinity_optimise_layout). Returns (h [N, G], nu [N, I], J, sweeps)."""
    N = len(Shat_up)
    G, I = np.asarray(Shat_up[0]).shape
    up = np.ascontiguousarray(np.stack([np.asarray(s, np.float64) for s in Shat_up]))
    dn = np.ascontiguousarray(np.stack([np.asarray(s, np.float64) for s in Shat_down])) if N > 1 else None
    h = np.ascontiguousarray(np.array(h0, dtype=np.int32).reshape(N, G))
    nu = np.ascontiguousarray(np.array(nu0, dtype=np.int32).reshape(N, I))
    mask = None if layer_mask is None else np.ascontiguousarray(layer_mask, dtype=np.uint8)
    opts = aff_layout_opts(int(max_sweeps), int(bool(freeze_heads)), int(bool(freeze_neurons)), int(bool(minimise)),
                           None if mask is None else mask.ctypes.data, assign or aff_assign_opts())
    J = ctypes.c_double(0.0)
    sweeps = ctypes.c_int32(0)
    _check(load().affinity_optimise_layout(up.ctypes.data, None if dn is None else dn.ctypes.data, N, G, I, int(L),
                                           ctypes.byref(opts), h.ctypes.data, nu.ctypes.data, ctypes.byref(J),
                                           ctypes.byref(sweeps), _ptr(workspace),
                                           _ws_bytes(workspace, workspace_bytes), _stream(stream)),
           "affinity_optimise_layout")
    return h, nu, J.value, sweeps.value


def layout_orders(h, nu, H: int, L: int):
    """(group_order [G], head_order [H], neuron_order [I]) realising a balanced layout (affinity_layout_orders)."""
    hh = np.ascontiguousarray(h, dtype=np.int32)
    nn = np.ascontiguousarray(nu, dtype=np.int32)
    go = np.empty(hh.size, np.int32)
    ho = np.empty(int(H), np.int32)
    no = np.empty(nn.size, np.int32)
    _check(load().affinity_layout_orders(hh.ctypes.data, nn.ctypes.data, hh.size, int(H), nn.size, int(L),
                                         go.ctypes.data, ho.ctypes.data, no.ctypes.data), "affinity_layout_orders")
    return go, ho, no


def gather_blocks(src, dst, rows: int, n_blocks: int, block_bytes: int, order, workspace, stream=None,
                  workspace_bytes=None) -> None:
    """Enqueue dst[r][j] = src[r][order[j]] over byte blocks (affinity_gather_blocks); order is a host array."""
    o = np.ascontiguousarray(order, dtype=np.int32)
    _check(load().affinity_gather_blocks(_ptr(src), _ptr(dst), int(rows), int(n_blocks), int(block_bytes),
                                         o.ctypes.data, _ptr(workspace), _ws_bytes(workspace, workspace_bytes),
                                         _stream(stream)), "affinity_gather_blocks")


_types = {}     # torch dtype -> aff_dtype, filled at first use (importing this module does not import torch)


def _dtype(t) -> int:
    code = _types.get(t.dtype)
    if code is None:
        import torch
        _types.update({torch.bfloat16: AFF_BF16, torch.float32: AFF_FP32})
        if t.dtype not in _types:
            raise TypeError("tensors must be bfloat16 or float32")
        code = _types[t.dtype]
    return code


def _row_stride(t, width: int, name: str) -> int:
    """Elements between the rows of a [T, ...] tensor whose rows are dense and `width` elements wide."""
    shape, stride = t.shape, t.stride()
    n = len(shape)
    if n == 3:
        ok = shape[1] * shape[2] == width and (stride[2] == 1 or shape[2] == 1) and \
            (stride[1] == shape[2] or shape[1] == 1)
    else:
        ok = n == 2 and shape[1] == width and (stride[1] == 1 or width == 1)
    if not ok:
        raise ValueError(f"{name}: dense rows of {width} elements expected, got shape {tuple(shape)} with strides "
                         f"{tuple(stride)}")
    return stride[0] if shape[0] > 1 else width


def _same_type(like, **tensors) -> None:
    for name, t in tensors.items():
        if t is not None and (t.dtype != like.dtype or t.device != like.device):
            raise TypeError(f"{name} must be {like.dtype} on {like.device}")


def _one_gpu(structs, *tensors) -> None:
    """All of a call's tensors on one GPU: the kernels would follow a host address too.  Raw addresses are not looked
    at.  `structs` carry the device index of the tensors that they were made from, -1 for the host."""
    dev = None
    for s in structs:
        if dev is None:
            dev = s.device
        elif s.device is not None and s.device != dev:
            raise TypeError("all tensors of a call must be on one GPU")
    for t in tensors:
        if t is None or t.__class__ is int:
            continue
        at = t.get_device()
        if at != dev:
            if dev is not None:
                raise TypeError("all tensors of a call must be on one GPU")
            dev = at
    if dev is not None and dev < 0:
        raise TypeError("tensors must be on a GPU")


def _device_of(*tensors) -> int:
    where = {t.get_device() for t in tensors if t is not None}
    if len(where) != 1:
        raise TypeError("all tensors must be on one device")
    return where.pop()


def kv_cache(k, v) -> aff_kv_cache:
    """A layer's paged cache from its pools, [n_pages, G, page_size, d_head] in any order of the first three."""
    if k.shape != v.shape or k.dim() != 4:
        raise ValueError("k and v must be [n_pages, G, page_size, d_head]")
    if k.stride() != v.stride() or k.stride(3) != 1:
        raise ValueError("k and v must have the same strides and dense rows")
    _same_type(k, v=v)
    c = aff_kv_cache(k.data_ptr(), v.data_ptr(), k.shape[0], k.stride(0), k.stride(1), k.stride(2), k.shape[1],
                     k.shape[2], k.shape[3], _dtype(k))
    c.keep, c.device = (k, v), k.get_device()
    return c


def step(T: int, H: int, q_start, kv_len, pages, prefix_pages=None, prefix_len: int = 0) -> aff_step:
    """A step of T query tokens with H heads: q_start [B+1], kv_len [B], pages [B, n], prefix_pages (CUDA int32).
    Their contents are taken by step_plan: changed in place, they count from the next step_plan on.  The rows of pages
    may be a part of a wider table's."""
    import torch
    for name, t in (("q_start", q_start), ("kv_len", kv_len), ("pages", pages), ("prefix_pages", prefix_pages)):
        if t is not None and (t.dtype != torch.int32 or (t.dim() and t.stride(-1) != 1 and t.shape[-1] > 1)):
            raise ValueError(f"{name} must be dense int32")
    if kv_len.dim() != 1 or (prefix_pages is not None and prefix_pages.dim() != 1):
        raise ValueError("kv_len and prefix_pages must be vectors")
    B = kv_len.shape[0]
    if q_start.shape != (B + 1,) or pages.dim() != 2 or pages.shape[0] != B:
        raise ValueError("q_start must be [B+1], kv_len [B] and pages [B, n]")
    if B > 1 and pages.stride(0) < pages.shape[1]:
        raise ValueError("the rows of pages must not overlap")
    table = pages
    if B > 1 and pages.stride(0) != pages.shape[1]:
        pages = pages.contiguous()
    s = aff_step(int(T), int(prefix_len), pages.shape[1], q_start.data_ptr(), kv_len.data_ptr(), pages.data_ptr(),
                 _ptr(prefix_pages), B, int(H))
    s.keep = (q_start, kv_len, pages, prefix_pages)
    s.copied = None if pages is table else (table, pages)
    s.n_prefix_pages = 0 if prefix_pages is None else prefix_pages.shape[0]
    s.device = _device_of(q_start, kv_len, pages, prefix_pages)
    return s


def _prefix_covered(s: aff_step, c: aff_kv_cache) -> None:
    n = getattr(s, "n_prefix_pages", None)
    if n is not None and n * c.page_size < s.prefix_len:
        raise ValueError("prefix_pages does not cover prefix_len")


def step_plan_size(s: aff_step, c: aff_kv_cache) -> int:
    n = ctypes.c_size_t(0)
    _check(load().affinity_step_plan_size(ctypes.byref(s), ctypes.byref(c), ctypes.byref(n)),
           "affinity_step_plan_size")
    return n.value


def _copy_pages(table, pages, stream) -> None:
    """A step's dense copy of a part of a wider page table, as that is now."""
    if stream is None:
        pages.copy_(table)
        return
    import torch
    with torch.cuda.stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream):
        pages.copy_(table)


def step_plan(s: aff_step, c: aff_kv_cache, plan, stream=None, plan_bytes=None) -> None:
    """Enqueue the plan of a step (affinity_step_plan) into `plan`, a CUDA uint8 tensor of step_plan_size bytes."""
    _prefix_covered(s, c)
    _one_gpu((s, c), plan)
    if s.copied is not None:
        _copy_pages(*s.copied, stream)
    _check(load().affinity_step_plan(ctypes.byref(s), ctypes.byref(c), _ptr(plan), _ws_bytes(plan, plan_bytes),
                                     _stream(stream)), "affinity_step_plan")


def rotary(cos, sin, interleaved: bool = False, q_gain=None, k_gain=None, eps: float = 1e-6) -> aff_rotary:
    """Rotation tables [n_pos, rot / 2] (CUDA fp32) and the optional per-head norm gains of kv_append."""
    import torch
    if cos.shape != sin.shape or cos.dim() != 2 or cos.dtype != torch.float32 or sin.dtype != torch.float32:
        raise ValueError("cos and sin must be fp32 [n_pos, rot / 2]")
    if not (cos.is_contiguous() and sin.is_contiguous()):
        raise ValueError("cos and sin must be dense")
    for t in (q_gain, k_gain):
        if t is not None and (t.dim() != 1 or not t.is_contiguous()):
            raise ValueError("q_gain and k_gain must be dense [d_head]")
    r = aff_rotary(cos.data_ptr(), sin.data_ptr(), _ptr(q_gain), _ptr(k_gain), cos.shape[0], float(eps),
                   2 * cos.shape[1], int(bool(interleaved)))
    r.keep, r.gains, r.device = (cos, sin), (q_gain, k_gain), _device_of(cos, sin, q_gain, k_gain)
    return r


def kv_append(q, k, v, c: aff_kv_cache, s: aff_step, r: aff_rotary, q_out, plan, stream=None,
              plan_bytes=None) -> None:
    """Enqueue affinity_kv_append: q [T, H, d_head], k and v [T, G, d_head] (rows may be strided), q_out like q."""
    T, d, code = s.T, c.d_head, c.dtype
    hd, gd = s.H * d, c.G * d
    if not (q.shape[0] == k.shape[0] == v.shape[0] == q_out.shape[0] == T):
        raise ValueError(f"q, k, v and q_out must have {T} rows")
    if not (_dtype(q) == _dtype(k) == _dtype(v) == _dtype(q_out) == code):
        raise TypeError("q, k, v and q_out must be of the cache's type")
    for t in r.gains:
        if t is not None and (t.shape != (d,) or _dtype(t) != code):
            raise ValueError("q_gain and k_gain must be [d_head] of the cache's type")
    strides = _row_stride(q, hd, "q"), _row_stride(k, gd, "k"), _row_stride(v, gd, "v"), _row_stride(q_out, hd, "q_out")
    _one_gpu((c, s, r), q, k, v, q_out, plan)
    _check(load().affinity_kv_append(q.data_ptr(), strides[0], k.data_ptr(), strides[1], v.data_ptr(), strides[2], c, s, r,
                                     q_out.data_ptr(), strides[3], _ptr(plan), _ws_bytes(plan, plan_bytes),
                                     _stream(stream)), "affinity_kv_append")


def prefix_attention(q, c: aff_kv_cache, s: aff_step, scale: float, out, lse, plan, stream=None,
                     plan_bytes=None) -> None:
    """Enqueue affinity_prefix_attention: q and out [T, H, d_head], lse fp32 [T, H] or None."""
    T, H, code = s.T, s.H, c.dtype
    hd = H * c.d_head
    if not (q.shape[0] == out.shape[0] == T):
        raise ValueError(f"q and out must have {T} rows")
    if not (_dtype(q) == _dtype(out) == code):
        raise TypeError("q and out must be of the cache's type")
    if _row_stride(out, hd, "out") != hd:
        raise ValueError("out must be dense")
    if lse is not None and (_dtype(lse) != AFF_FP32 or lse.shape != (T, H) or not lse.is_contiguous()):
        raise ValueError("lse must be dense fp32 [T, H]")
    q_stride = _row_stride(q, hd, "q")
    _one_gpu((c, s), q, out, lse, plan)
    _check(load().affinity_prefix_attention(q.data_ptr(), q_stride, c, s, scale, out.data_ptr(),
                                            _ptr(lse), _ptr(plan), _ws_bytes(plan, plan_bytes), _stream(stream)),
           "affinity_prefix_attention")


def block_norm(x, f, y, h=None, post_gain=None, pre_gain=None, gate=None, rows_per_gate: int = 1, scale: float = 1.0,
               eps: float = 1e-6, stream=None) -> None:
    """Enqueue affinity_block_norm: x, f, y, h [T, D] (rows may be strided), gains [D], gate [n, D]."""
    shape, dtype = x.shape, x.dtype
    T, D = shape
    if f.shape != shape or y.shape != shape or (h is not None and h.shape != shape):
        raise ValueError(f"x, f, y and h must all be [{T}, {D}]")
    if gate is not None and (gate.dim() != 2 or rows_per_gate < 1 or gate.shape[1] != D or
                             gate.shape[0] * rows_per_gate < T):
        raise ValueError("gate must be [n, D] with n * rows_per_gate >= T")
    ptrs = []
    for t in (x, f, gate, post_gain, pre_gain, y, h):
        if t is None:
            ptrs.append(None)
            continue
        if t.dtype != dtype:
            raise TypeError(f"all tensors must be {dtype}")
        ptrs.append(t.data_ptr())
    for t in (post_gain, pre_gain):
        if t is not None and (t.shape != (D,) or not t.is_contiguous()):
            raise ValueError(f"gains must be dense [{D}]")
    a = aff_block_norm(*ptrs, T, D, _row_stride(x, D, "x"), _row_stride(f, D, "f"),
                       0 if gate is None else _row_stride(gate, D, "gate"), _row_stride(y, D, "y"),
                       0 if h is None else _row_stride(h, D, "h"), rows_per_gate, scale, eps, _dtype(x))
    _one_gpu((), x, f, gate, post_gain, pre_gain, y, h)
    _check(load().affinity_block_norm(a, _stream(stream)), "affinity_block_norm")


def set_timing_events(start_event, stop_event) -> None:
    """Record torch.cuda.Event pairs around the dominant kernel of later calls (None, None stops)."""
    h0 = None if start_event is None else start_event.cuda_event
    h1 = None if stop_event is None else stop_event.cuda_event
    _check(load().affinity_set_timing_events(h0, h1), "affinity_set_timing_events")


def version() -> int:
    return int(load().affinity_version())
