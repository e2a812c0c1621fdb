"""ctypes binding of libikbo.so (include/ikbo.h), same names as the C ABI.

Argument marshalling only: torch tensors are checked for device, dtype and
contiguity, their shapes become the C size arguments and their data
pointers the C pointers.  Every step of the hot path runs in the library's
CUDA kernels.  If the library is missing this module raises; there is no
fallback.
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libikbo.so")

STATUS_NAMES = {0: "IKBO_OK", 1: "IKBO_ERR_INVALID_ARG", 2: "IKBO_ERR_UNSUPPORTED", 3: "IKBO_ERR_CUDA",
                4: "IKBO_ERR_MAP_OUT_OF_RANGE", 5: "IKBO_ERR_TIMEOUT", 6: "IKBO_ERR_NOT_PLANNED",
                7: "IKBO_ERR_INTERNAL", 8: "IKBO_ERR_OUT_OF_PAGES", 9: "IKBO_ERR_CACHE"}
IKBO_OK = 0
IKBO_ERR_INVALID_ARG = 1
IKBO_ERR_UNSUPPORTED = 2
IKBO_ERR_CUDA = 3
IKBO_ERR_MAP_OUT_OF_RANGE = 4
IKBO_ERR_TIMEOUT = 5
IKBO_ERR_NOT_PLANNED = 6
IKBO_ERR_INTERNAL = 7
IKBO_ERR_OUT_OF_PAGES = 8
IKBO_ERR_CACHE = 9
DEBUG_WITHHOLD_USER_PARTIAL = 1
DEBUG_NO_COOPERATIVE = 2
DEBUG_WITHHOLD_KEYS = 4

# every function the header declares: name -> (restype, argtypes)
_vp, _i, _u64, _f64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_uint64, ctypes.c_double
SIGNATURES = {
    "ikbo_plan_create": (_i, [ctypes.POINTER(_vp), _i, _i, _i]),
    "ikbo_plan": (_i, [_vp, _vp, _i, _i, _i, _i, _vp]),
    "ikbo_plan_segments": (_i, [_vp, ctypes.POINTER(_vp), ctypes.POINTER(_vp), ctypes.POINTER(_vp)]),
    "ikbo_plan_worklist": (_i, [_vp, ctypes.POINTER(_vp), ctypes.POINTER(_vp), ctypes.POINTER(_i),
                                ctypes.POINTER(_i)]),
    "ikbo_lce_forward": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _vp]),
    "ikbo_lce_forward_staged": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp]),
    "ikbo_lce_forward_noalloc": (_i, [_vp, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _vp]),
    "ikbo_lce_backward": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _vp]),
    "ikbo_attn_forward": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, ctypes.c_float, _vp]),
    "ikbo_attn_forward_lse": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, ctypes.c_float, _vp]),
    "ikbo_attn_backward": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, ctypes.c_float,
                                _vp]),
    "ikbo_attn_self_target_forward": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, ctypes.c_float, _vp]),
    "ikbo_rope_frequencies": (_i, [_vp, _i, _f64, _i, _f64, _f64, _f64, _f64]),
    "ikbo_rope_create": (_i, [ctypes.POINTER(_vp), _i, _vp, _i, ctypes.c_float]),
    "ikbo_rope_destroy": (None, [_vp]),
    "ikbo_rope_forward": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp]),
    "ikbo_rope_backward": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp]),
    "ikbo_qcache_bytes": (_u64, [_i, _i, _i]),
    "ikbo_qcache_resize": (_i, [_vp, _vp, _vp, _i, _vp, _i, _i, _vp, _vp, _i, _vp, _vp, _vp, _i, _vp]),
    "ikbo_qcache_append": (_i, [_vp, _vp, _vp, ctypes.c_int64, _vp, _i, _i, _i, _vp, _i, _i, _vp]),
    "ikbo_qcache_load": (_i, [_vp, _vp, _i, _i, _i, _i, _vp, _i, _vp, _i, _vp, _vp, _vp, _i, _vp]),
    "ikbo_attn_qcache_forward": (_i, [_vp, _vp, _vp, _i, _i, _i, _vp, _i, _vp, _vp, _vp, _i, _i, ctypes.c_float,
                                      _vp]),
    "ikbo_plan_get_status": (_i, [_vp, _vp]),
    "ikbo_plan_set_debug": (_i, [_vp, ctypes.c_uint]),
    "ikbo_plan_set_timeout_ns": (_i, [_vp, _u64]),
    "ikbo_plan_set_lce_schedule": (_i, [_vp, _i]),
    "ikbo_plan_launch_count": (_u64, [_vp]),
    "ikbo_status_string": (ctypes.c_char_p, [_i]),
    "ikbo_plan_destroy": (None, [_vp]),
    "ikbo_version": (_i, []),
}

_lib = None


class IkboError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {STATUS_NAMES.get(code, code)}")


def load(path: str = LIB_PATH):
    """Load libikbo.so (raises OSError / RuntimeError if it is absent)."""
    global _lib
    if _lib is None:
        if not os.path.exists(path):
            raise RuntimeError(f"libikbo.so not built ({path}); run "
                               "`python -m broadcast_gemm_attention_gb300.build`")
        lib = ctypes.CDLL(path)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(lib, name)
            f.restype = res
            f.argtypes = args
        _lib = lib
    return _lib


def _check(rc: int, what: str):
    if rc != IKBO_OK:
        raise IkboError(rc, what)


def _stream(stream) -> Optional[int]:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _dev(t: torch.Tensor, dtype, name: str) -> int:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


# ---------------------------------------------------------------- the ABI
def ikbo_version() -> int:
    return int(load().ikbo_version())


def ikbo_status_string(code: int) -> str:
    return load().ikbo_status_string(code).decode()


def ikbo_plan_create(max_cand: int, max_users: int, max_heads: int = 1) -> int:
    h = ctypes.c_void_p()
    _check(load().ikbo_plan_create(ctypes.byref(h), max_cand, max_users, max_heads), "ikbo_plan_create")
    return h.value


def ikbo_plan_destroy(plan: int) -> None:
    load().ikbo_plan_destroy(plan)


def ikbo_plan(plan: int, map_: torch.Tensor, n_users: int, H: int = 1, Lq: int = 8, stream=None) -> None:
    ptr = _dev(map_, torch.int32, "map")
    _check(load().ikbo_plan(plan, ptr, map_.numel(), n_users, H, Lq, _stream(stream)), "ikbo_plan")


def ikbo_plan_segments(plan: int):
    """(counts_ptr, offsets_ptr, perm_ptr) device addresses (borrowed)."""
    c, o, p = ctypes.c_void_p(), ctypes.c_void_p(), ctypes.c_void_p()
    _check(load().ikbo_plan_segments(plan, ctypes.byref(c), ctypes.byref(o), ctypes.byref(p)), "ikbo_plan_segments")
    return c.value, o.value, p.value


def ikbo_plan_worklist(plan: int):
    """(work_ptr, n_units_ptr, cands_per_unit, max_units)."""
    w, n = ctypes.c_void_p(), ctypes.c_void_p()
    cpu, mu = ctypes.c_int(), ctypes.c_int()
    _check(load().ikbo_plan_worklist(plan, ctypes.byref(w), ctypes.byref(n), ctypes.byref(cpu), ctypes.byref(mu)),
           "ikbo_plan_worklist")
    return w.value, n.value, cpu.value, mu.value


def ikbo_lce_forward(plan: int, U: torch.Tensor, C: torch.Tensor, Wu: torch.Tensor, Wc: torch.Tensor,
                     b: Optional[torch.Tensor], Y: torch.Tensor, stream=None) -> None:
    """Y[i] = Wu^T U[map[i]] + Wc^T C[i] + b for the planned request."""
    bf = torch.bfloat16
    n_users, K_u, D = U.shape
    n_cand, K_c, D2 = C.shape
    N = Wu.shape[1]
    if D2 != D or tuple(Wu.shape) != (K_u, N) or tuple(Wc.shape) != (K_c, N) or tuple(Y.shape) != (n_cand, N, D):
        raise ValueError("inconsistent LCE shapes")
    bptr = None
    if b is not None:
        if tuple(b.shape) != (N,):
            raise ValueError("b must be [N]")
        bptr = _dev(b, bf, "b")
    _check(load().ikbo_lce_forward(plan, _dev(U, bf, "U"), _dev(C, bf, "C"), _dev(Wu, bf, "Wu"), _dev(Wc, bf, "Wc"),
                                   bptr, _dev(Y, bf, "Y"), K_u, K_c, D, N, _stream(stream)), "ikbo_lce_forward")


def ikbo_lce_backward(plan: int, U: torch.Tensor, C: torch.Tensor, Wu: torch.Tensor, Wc: torch.Tensor,
                      dY: torch.Tensor, dU: Optional[torch.Tensor], dC: Optional[torch.Tensor],
                      dWu: Optional[torch.Tensor], dWc: Optional[torch.Tensor], db: Optional[torch.Tensor],
                      stream=None) -> None:
    """Gradients of the LCE for upstream dY (any output may be None to skip it):
    dU/dC bf16, dWu/dWc/db fp32, all overwritten."""
    bf, f32 = torch.bfloat16, torch.float32
    n_users, K_u, D = U.shape
    n_cand, K_c, D2 = C.shape
    N = Wu.shape[1]
    if D2 != D or tuple(Wu.shape) != (K_u, N) or tuple(Wc.shape) != (K_c, N) or tuple(dY.shape) != (n_cand, N, D):
        raise ValueError("inconsistent LCE shapes")
    want = {"dU": (dU, (n_users, K_u, D), bf), "dC": (dC, (n_cand, K_c, D), bf), "dWu": (dWu, (K_u, N), f32),
            "dWc": (dWc, (K_c, N), f32), "db": (db, (N,), f32)}
    ptrs = {}
    for name, (t, shape, dt) in want.items():
        if t is None:
            ptrs[name] = None
            continue
        if tuple(t.shape) != shape:
            raise ValueError(f"{name} must be {list(shape)}")
        ptrs[name] = _dev(t, dt, name)
    _check(load().ikbo_lce_backward(plan, _dev(U, bf, "U"), _dev(C, bf, "C"), _dev(Wu, bf, "Wu"), _dev(Wc, bf, "Wc"),
                                    _dev(dY, bf, "dY"), ptrs["dU"], ptrs["dC"], ptrs["dWu"], ptrs["dWc"], ptrs["db"],
                                    K_u, K_c, D, N, _stream(stream)), "ikbo_lce_backward")


def ikbo_lce_forward_staged(plan: int, U: torch.Tensor, C: torch.Tensor, Wu: torch.Tensor, Wc: torch.Tensor,
                            b: Optional[torch.Tensor], Y: torch.Tensor, stage: int, stream=None) -> None:
    """The LCE as stage 1 (decomposed, unfused), 3 (fused epilogue, one
    accumulator) or 4 (the full kernel) of the pages' stage ladder."""
    bf = torch.bfloat16
    n_users, K_u, D = U.shape
    n_cand, K_c, D2 = C.shape
    N = Wu.shape[1]
    if D2 != D or tuple(Wu.shape) != (K_u, N) or tuple(Wc.shape) != (K_c, N) or tuple(Y.shape) != (n_cand, N, D):
        raise ValueError("inconsistent LCE shapes")
    bptr = None if b is None else _dev(b, bf, "b")
    _check(load().ikbo_lce_forward_staged(plan, _dev(U, bf, "U"), _dev(C, bf, "C"), _dev(Wu, bf, "Wu"),
                                          _dev(Wc, bf, "Wc"), bptr, _dev(Y, bf, "Y"), K_u, K_c, D, N, int(stage),
                                          _stream(stream)), "ikbo_lce_forward_staged")


def ikbo_lce_forward_noalloc(map_: torch.Tensor, n_users: int, U: torch.Tensor, C: torch.Tensor,
                             Wu: torch.Tensor, Wc: torch.Tensor, b: Optional[torch.Tensor], Y: torch.Tensor,
                             stream=None) -> None:
    """The fused LCE without a plan: its scratch lives in the library's own
    fixed device array, so the call allocates nothing (for callers whose
    device memory belongs to another allocator).  Calls share that scratch:
    do not overlap them on the GPU."""
    bf = torch.bfloat16
    n_u, K_u, D = U.shape
    n_cand, K_c, D2 = C.shape
    N = Wu.shape[1]
    if n_u != n_users or D2 != D or tuple(Wu.shape) != (K_u, N) or tuple(Wc.shape) != (K_c, N) or \
            tuple(Y.shape) != (n_cand, N, D) or map_.numel() != n_cand:
        raise ValueError("inconsistent LCE shapes")
    bptr = None
    if b is not None:
        if tuple(b.shape) != (N,):
            raise ValueError("b must be [N]")
        bptr = _dev(b, bf, "b")
    _check(load().ikbo_lce_forward_noalloc(_dev(map_, torch.int32, "map"), n_cand, n_users, _dev(U, bf, "U"),
                                           _dev(C, bf, "C"), _dev(Wu, bf, "Wu"), _dev(Wc, bf, "Wc"), bptr,
                                           _dev(Y, bf, "Y"), K_u, K_c, D, N, _stream(stream)),
           "ikbo_lce_forward_noalloc")


def ikbo_attn_forward(plan: int, Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor,
                      kv_offsets: Optional[torch.Tensor], O: torch.Tensor, scale: Optional[float] = None,
                      stream=None) -> None:
    """O[i,h] = softmax(Q[i,h] K[map[i],h]^T scale) V[map[i],h] for the planned request."""
    bf = torch.bfloat16
    d = Q.shape[-1]
    if kv_offsets is None:
        Lkv = K.shape[2]
        optr = None
    else:
        Lkv = K.shape[0]
        optr = _dev(kv_offsets, torch.int32, "kv_offsets")
    if K.shape != V.shape or O.shape != Q.shape:
        raise ValueError("inconsistent attention shapes")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    _check(load().ikbo_attn_forward(plan, _dev(Q, bf, "Q"), _dev(K, bf, "K"), _dev(V, bf, "V"), optr,
                                    _dev(O, bf, "O"), Lkv, d, float(scale), _stream(stream)), "ikbo_attn_forward")


def ikbo_attn_forward_lse(plan: int, Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor,
                          kv_offsets: Optional[torch.Tensor], O: torch.Tensor, lse: torch.Tensor,
                          scale: Optional[float] = None, stream=None) -> None:
    """ikbo_attn_forward that also writes each query row's natural-log
    log-sum-exp into lse (fp32 [n_cand, H, Lq])."""
    bf = torch.bfloat16
    d = Q.shape[-1]
    if kv_offsets is None:
        Lkv = K.shape[2]
        optr = None
    else:
        Lkv = K.shape[0]
        optr = _dev(kv_offsets, torch.int32, "kv_offsets")
    if K.shape != V.shape or O.shape != Q.shape or tuple(lse.shape) != tuple(Q.shape[:3]):
        raise ValueError("inconsistent attention shapes")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    _check(load().ikbo_attn_forward_lse(plan, _dev(Q, bf, "Q"), _dev(K, bf, "K"), _dev(V, bf, "V"), optr,
                                        _dev(O, bf, "O"), _dev(lse, torch.float32, "lse"), Lkv, d, float(scale),
                                        _stream(stream)), "ikbo_attn_forward_lse")


def ikbo_attn_backward(plan: int, Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, O: torch.Tensor,
                       dO: torch.Tensor, kv_offsets: Optional[torch.Tensor], dQ: torch.Tensor, dK: torch.Tensor,
                       dV: torch.Tensor, scale: Optional[float] = None, stream=None,
                       lse: Optional[torch.Tensor] = None) -> None:
    """Gradients of broadcast attention for upstream dO: dQ (Q's layout), and dK,
    dV (K's layout) summed over each user's candidates; all bf16, overwritten.
    lse: the forward's log-sum-exp (ikbo_attn_forward_lse), or None."""
    bf = torch.bfloat16
    d = Q.shape[-1]
    if kv_offsets is None:
        Lkv = K.shape[2]
        optr = None
    else:
        Lkv = K.shape[0]
        optr = _dev(kv_offsets, torch.int32, "kv_offsets")
    if K.shape != V.shape or O.shape != Q.shape or dO.shape != Q.shape or dQ.shape != Q.shape or \
            dK.shape != K.shape or dV.shape != V.shape:
        raise ValueError("inconsistent attention shapes")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    lptr = None
    if lse is not None:
        if tuple(lse.shape) != tuple(Q.shape[:3]):
            raise ValueError("inconsistent lse shape")
        lptr = _dev(lse, torch.float32, "lse")
    _check(load().ikbo_attn_backward(plan, _dev(Q, bf, "Q"), _dev(K, bf, "K"), _dev(V, bf, "V"), _dev(O, bf, "O"),
                                     _dev(dO, bf, "dO"), lptr, optr, _dev(dQ, bf, "dQ"), _dev(dK, bf, "dK"),
                                     _dev(dV, bf, "dV"), Lkv, d, float(scale), _stream(stream)),
           "ikbo_attn_backward")


def ikbo_attn_self_target_forward(plan: int, Q: torch.Tensor, Q_user: torch.Tensor, K: torch.Tensor,
                                  V: torch.Tensor, kv_offsets: Optional[torch.Tensor], O: torch.Tensor,
                                  O_user: torch.Tensor, scale: Optional[float] = None, stream=None) -> None:
    """Target attention (as ikbo_attn_forward) and the users' own queries
    O_user[u,h] = softmax(Q_user[u,h] K[u,h]^T scale) V[u,h], in one launch.
    Q and O both None: the self part alone."""
    bf = torch.bfloat16
    d = Q_user.shape[-1]
    if kv_offsets is None:
        Lkv = K.shape[2]
        optr = None
    else:
        Lkv = K.shape[0]
        optr = _dev(kv_offsets, torch.int32, "kv_offsets")
    if (Q is None) != (O is None):
        raise ValueError("Q and O are given together or not at all")
    if K.shape != V.shape or (Q is not None and O.shape != Q.shape) or O_user.shape != Q_user.shape \
            or Q_user.dim() != 4:
        raise ValueError("shape mismatch among Q/O, Q_user/O_user, K/V")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    qp = None if Q is None else _dev(Q, bf, "Q")
    op = None if O is None else _dev(O, bf, "O")
    _check(load().ikbo_attn_self_target_forward(plan, qp, _dev(Q_user, bf, "Q_user"), _dev(K, bf, "K"),
                                                _dev(V, bf, "V"), optr, op, _dev(O_user, bf, "O_user"),
                                                Q_user.shape[2], Lkv, d, float(scale), _stream(stream)),
           "ikbo_attn_self_target_forward")


# ------------------------------------------------- rotary positions, 4-bit cache
ROPE_SCALINGS = {"none": 0, "linear": 1, "base": 2, "turns": 3}
ROPE_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
QCACHE_BLOCK_BYTES = 2560  # 16 tokens of one head
QCACHE_MAX_USERS = 8192


def _current_device(t: torch.Tensor, name: str) -> int:
    """The current device, for a call whose argument t is on a CUDA device at all."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return torch._C._cuda_getDevice()


def _raw_stream(stream, dev: int) -> int:
    """_stream for the calls that take single tokens: the current stream without a Python object for it."""
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)


def _here(t: torch.Tensor, dtype, name: str, dev: int) -> int:
    """_dev, and the tensor lies on device dev (the current one, where the call launches)."""
    if t.get_device() != dev or t.dtype is not dtype or not t.is_contiguous():
        _dev(t, dtype, name)
        raise ValueError(f"{name} is on {t.device}, not on the current device")
    return t.data_ptr()


def ikbo_rope_frequencies(rot_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                          original_len: float = 1.0, low_turns: float = 0.0, high_turns: float = 1.0):
    """The rot_dim / 2 frequencies (radians per position, floats) of a rotation:
    scaling "none", "linear", "base" or "turns"."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(ROPE_SCALINGS)}")
    out = (ctypes.c_double * max(1, rot_dim // 2))()
    _check(load().ikbo_rope_frequencies(ctypes.addressof(out), rot_dim, base, ROPE_SCALINGS[scaling], factor,
                                        original_len, low_turns, high_turns), "ikbo_rope_frequencies")
    return list(out)


def ikbo_rope_create(rot_dim: int, freqs, interleaved: bool = False, magnitude: float = 1.0) -> int:
    if len(freqs) != rot_dim // 2:
        raise ValueError(f"freqs must hold rot_dim / 2 = {rot_dim // 2} values")
    table = (ctypes.c_double * max(1, len(freqs)))(*freqs)
    h = ctypes.c_void_p()
    _check(load().ikbo_rope_create(ctypes.byref(h), rot_dim, ctypes.addressof(table), int(interleaved), magnitude),
           "ikbo_rope_create")
    return h.value


def ikbo_rope_destroy(rope: int) -> None:
    load().ikbo_rope_destroy(rope)


_I64X3 = ctypes.c_int64 * 3


def _rope(fn, name: str, plan: int, rope: int, X: torch.Tensor, Y: torch.Tensor, start, broadcast: bool, stream) -> None:
    dev = _current_device(X, "input")
    if X.get_device() != dev or Y.get_device() != dev:
        raise ValueError(f"input and output are on {X.device} and {Y.device}, not on the current device")
    shape = X.shape
    dtype = ROPE_DTYPES.get(X.dtype)
    if dtype is None or Y.dtype is not X.dtype:
        raise ValueError("input and output must share a dtype: bfloat16, float16 or float32")
    if shape != Y.shape or len(shape) not in (3, 4):
        raise ValueError("input and output must share a shape [n, H, L, d] or [rows, H, d]")
    if len(shape) == 4:
        n, H, L, d = shape
    else:
        n, H, d = shape
        L = 1
    cx = cy = None  # NULL: contiguous
    if not (X.is_contiguous() and Y.is_contiguous()):
        if d > 1 and (X.stride(-1) != 1 or Y.stride(-1) != 1):
            raise ValueError("the last dimension must be contiguous")
        cx, cy = (_I64X3(*(t.stride()[:3] if len(shape) == 4 else t.stride()[:2] + (0,))) for t in (X, Y))
    sptr = None
    if start is not None:
        sptr = _here(start, torch.int32, "start", dev)
        if start.dim() != 1 or (not broadcast and start.numel() != n):
            raise ValueError("start must be [n], or [n_users] with broadcast")
    rc = fn(plan, rope, X.data_ptr(), cx, Y.data_ptr(), cy, sptr, broadcast, dtype, n, H, L, d, _raw_stream(stream, dev))
    if rc != IKBO_OK:
        raise IkboError(rc, name)


def ikbo_rope_forward(plan: int, rope: int, X: torch.Tensor, Y: torch.Tensor, start: Optional[torch.Tensor] = None,
                      broadcast: bool = False, stream=None) -> None:
    """Y = X [n, H, L, d] (or [rows, H, d]: one token each) with its pairs rotated by the
    angles of positions start[i] + l; with broadcast start[map[i]] + l of the planned
    request (start then holds one position per user).  Y may be X."""
    _rope(load().ikbo_rope_forward, "ikbo_rope_forward", plan, rope, X, Y, start, broadcast, stream)


def ikbo_rope_backward(plan: int, rope: int, dY: torch.Tensor, dX: torch.Tensor, start: Optional[torch.Tensor] = None,
                       broadcast: bool = False, stream=None) -> None:
    """Gradient of ikbo_rope_forward: dX from dY."""
    _rope(load().ikbo_rope_backward, "ikbo_rope_backward", plan, rope, dY, dX, start, broadcast, stream)


def ikbo_qcache_bytes(n_pages: int, page: int, H: int) -> int:
    """Bytes of a cache's data (0 for sizes outside the limits)."""
    return int(load().ikbo_qcache_bytes(n_pages, page, H))


def _qcache(data: torch.Tensor, page: int, dev: int):
    ptr = _here(data, torch.uint8, "data", dev)
    shape = data.shape
    if len(shape) != 4 or page < 16 or shape[2] * 16 != page or shape[3] != QCACHE_BLOCK_BYTES:
        raise ValueError(f"data must be [n_pages, H, page // 16, {QCACHE_BLOCK_BYTES}]")
    return ptr, shape[0], shape[1]


def _qtable(table: torch.Tensor, lens: torch.Tensor, dev: int):
    tptr, lptr = _here(table, torch.int32, "table", dev), _here(lens, torch.int32, "lens", dev)
    shape = table.shape
    if len(shape) != 2 or lens.dim() != 1 or lens.numel() != shape[0]:
        raise ValueError("table must be [n_users, max_blocks] and lens [n_users]")
    return tptr, lptr, shape[0], shape[1]


def ikbo_qcache_resize(plan: int, lens: torch.Tensor, new_lens: torch.Tensor, table: torch.Tensor, page: int,
                       free: torch.Tensor, n_free: torch.Tensor, slots: torch.Tensor, slot_offsets: torch.Tensor,
                       positions: Optional[torch.Tensor] = None, stream=None) -> None:
    """Set every user's length: pages are taken from and given back to the free list,
    and each added token gets its slot (and position).  lens, table, free and n_free
    change in place; all or nothing."""
    dev, i32 = _current_device(lens, "lens"), torch.int32
    tptr, lptr, n_users, max_blocks = _qtable(table, lens, dev)
    if new_lens.shape != lens.shape or slot_offsets.dim() != 1 or slot_offsets.numel() != n_users + 1 or \
            n_free.numel() != 1 or free.dim() != 1 or slots.dim() != 1 or \
            (positions is not None and positions.shape != slots.shape):
        raise ValueError("inconsistent cache shapes")
    _check(load().ikbo_qcache_resize(plan, lptr, _here(new_lens, i32, "new_lens", dev), n_users, tptr, max_blocks, page,
                                     _here(free, i32, "free", dev), _here(n_free, i32, "n_free", dev), free.numel(),
                                     _here(slots, i32, "slots", dev), _here(slot_offsets, i32, "slot_offsets", dev),
                                     None if positions is None else _here(positions, i32, "positions", dev),
                                     slots.numel(), _raw_stream(stream, dev)), "ikbo_qcache_resize")


def ikbo_qcache_append(plan: int, K: torch.Tensor, V: torch.Tensor, slots: torch.Tensor, data: torch.Tensor,
                       page: int, stream=None) -> None:
    """Quantise row r of K and V ([n_rows, H, 128] bf16; rows may be strided, both
    alike) into slot slots[r] of the cache (-1: skipped)."""
    dev, bf = _current_device(data, "data"), torch.bfloat16
    dptr, n_pages, H = _qcache(data, page, dev)
    shape = K.shape
    if len(shape) != 3 or shape != V.shape or shape[1] != H or slots.dim() != 1 or slots.numel() != shape[0]:
        raise ValueError("K and V must be [n_rows, H, d] and slots [n_rows]")
    n, _, d = shape
    for t, name in ((K, "K"), (V, "V")):
        if t.get_device() != dev or t.dtype is not bf:
            raise ValueError(f"{name} must be a tensor of bfloat16 on the current CUDA device")
    stride = (H * d + 7) // 8 * 8
    if not (K.is_contiguous() and V.is_contiguous()):
        for t in (K, V):
            if n and (t.stride(2) != 1 or (H > 1 and t.stride(1) != d)):
                raise ValueError("the heads of a row must be contiguous")
        if n > 1:
            stride = K.stride(0)
            if V.stride(0) != stride:
                raise ValueError("K and V must have the same row stride")
    _check(load().ikbo_qcache_append(plan, K.data_ptr(), V.data_ptr(), stride, _here(slots, torch.int32, "slots", dev), n,
                                     H, d, dptr, n_pages, page, _raw_stream(stream, dev)), "ikbo_qcache_append")


def ikbo_qcache_load(plan: int, data: torch.Tensor, page: int, table: torch.Tensor, lens: torch.Tensor,
                     kv_offsets: torch.Tensor, K: Optional[torch.Tensor], V: Optional[torch.Tensor],
                     stream=None) -> None:
    """Read histories back as jagged bf16 rows: token t of user u to row
    kv_offsets[u] + t of K and V [rows, H, 128] (either may be None)."""
    dev, bf = _current_device(data, "data"), torch.bfloat16
    dptr, n_pages, H = _qcache(data, page, dev)
    tptr, lptr, n_users, max_blocks = _qtable(table, lens, dev)
    if kv_offsets.dim() != 1 or kv_offsets.numel() != n_users + 1:
        raise ValueError("kv_offsets must be [n_users + 1]")
    some = K if K is not None else V
    if some is None:
        raise ValueError("K, V or both must be given")
    for t in (K, V):
        if t is not None and (t.dim() != 3 or t.shape != some.shape or t.shape[1] != H):
            raise ValueError("K and V must be [rows, H, d]")
    kptr = None if K is None else _here(K, bf, "K", dev)
    vptr = None if V is None else _here(V, bf, "V", dev)
    _check(load().ikbo_qcache_load(plan, dptr, n_pages, page, H, some.shape[2], tptr, max_blocks, lptr, n_users,
                                   _here(kv_offsets, torch.int32, "kv_offsets", dev), kptr, vptr, some.shape[0],
                                   _raw_stream(stream, dev)), "ikbo_qcache_load")


def ikbo_attn_qcache_forward(plan: int, Q: torch.Tensor, data: torch.Tensor, page: int, table: torch.Tensor,
                             lens: torch.Tensor, O: torch.Tensor, lse: Optional[torch.Tensor] = None,
                             Lkv: Optional[int] = None, scale: Optional[float] = None, stream=None) -> None:
    """ikbo_attn_forward's definition over the cache: user u's keys are the lens[u]
    tokens of its pages.  Lkv: a bound on the sum of the lengths (default: what the
    table can hold); the call's workspace and variant go by it."""
    dev, bf = _current_device(data, "data"), torch.bfloat16
    dptr, n_pages, H_kv = _qcache(data, page, dev)
    tptr, lptr, n_users, max_blocks = _qtable(table, lens, dev)
    shape = Q.shape
    if len(shape) != 4 or O.shape != shape or shape[1] % H_kv != 0 or (lse is not None and lse.shape != shape[:3]):
        raise ValueError("inconsistent attention shapes")
    d = shape[3]
    if Lkv is None:
        Lkv = n_users * max_blocks * page
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    _check(load().ikbo_attn_qcache_forward(plan, _here(Q, bf, "Q", dev), dptr, n_pages, page, H_kv, tptr, max_blocks,
                                           lptr, _here(O, bf, "O", dev),
                                           None if lse is None else _here(lse, torch.float32, "lse", dev),
                                           min(max(1, int(Lkv)), 2**31 - 1), d, scale, _raw_stream(stream, dev)),
           "ikbo_attn_qcache_forward")


def ikbo_plan_get_status(plan: int, stream=None) -> int:
    """Synchronises the stream; returns the device-detected status code (and clears it)."""
    return int(load().ikbo_plan_get_status(plan, _stream(stream)))


def ikbo_plan_set_debug(plan: int, flags: int) -> None:
    _check(load().ikbo_plan_set_debug(plan, flags), "ikbo_plan_set_debug")


def ikbo_plan_set_lce_schedule(plan: int, schedule: int) -> None:
    """0 = chosen from the shape, 1 = two launches, 2 = one launch."""
    _check(load().ikbo_plan_set_lce_schedule(plan, int(schedule)), "ikbo_plan_set_lce_schedule")


def ikbo_plan_set_timeout_ns(plan: int, ns: int) -> None:
    _check(load().ikbo_plan_set_timeout_ns(plan, ns), "ikbo_plan_set_timeout_ns")


def ikbo_plan_launch_count(plan: int) -> int:
    return int(load().ikbo_plan_launch_count(plan))


# ------------------------------------------------------------ convenience
class Plan:
    """Owns one ikbo_plan_t; `with Plan(...) as p:` destroys it on exit."""

    def __init__(self, max_cand: int, max_users: int, max_heads: int = 1):
        self._map = None
        self._request = None  # (n_cand, H, Lq) and n_users of the last plan()
        self.handle = ikbo_plan_create(max_cand, max_users, max_heads)

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def close(self):
        if self.handle:
            ikbo_plan_destroy(self.handle)
            self.handle = None
        self._map = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def plan(self, map_, n_users, H=1, Lq=8, stream=None):
        ikbo_plan(self.handle, map_, n_users, H, Lq, stream)
        # the plan borrows the map for every later call of this request: hold
        # the tensor so that a temporary passed here stays allocated
        self._map = map_
        self._request = ((map_.numel(), H, Lq), n_users)

    def lce_forward(self, U, C, Wu, Wc, b, Y, stream=None):
        ikbo_lce_forward(self.handle, U, C, Wu, Wc, b, Y, stream)

    def lce_backward(self, U, C, Wu, Wc, dY, dU=None, dC=None, dWu=None, dWc=None, db=None, stream=None):
        ikbo_lce_backward(self.handle, U, C, Wu, Wc, dY, dU, dC, dWu, dWc, db, stream)

    def lce_forward_staged(self, U, C, Wu, Wc, b, Y, stage, stream=None):
        ikbo_lce_forward_staged(self.handle, U, C, Wu, Wc, b, Y, stage, stream)

    def attn_forward(self, Q, K, V, kv_offsets, O, scale=None, stream=None):
        ikbo_attn_forward(self.handle, Q, K, V, kv_offsets, O, scale, stream)

    def attn_forward_lse(self, Q, K, V, kv_offsets, O, lse, scale=None, stream=None):
        ikbo_attn_forward_lse(self.handle, Q, K, V, kv_offsets, O, lse, scale, stream)

    def attn_backward(self, Q, K, V, O, dO, kv_offsets, dQ, dK, dV, scale=None, stream=None, lse=None):
        ikbo_attn_backward(self.handle, Q, K, V, O, dO, kv_offsets, dQ, dK, dV, scale, stream, lse)

    def attn_self_target_forward(self, Q, Q_user, K, V, kv_offsets, O, O_user, scale=None, stream=None):
        ikbo_attn_self_target_forward(self.handle, Q, Q_user, K, V, kv_offsets, O, O_user, scale, stream)

    def _check_start(self, start, broadcast):
        if broadcast and start is not None and self._request is not None and start.numel() != self._request[1]:
            raise ValueError(f"with broadcast, start must hold a position for each of the plan's {self._request[1]} users")

    def rope_forward(self, rope, X, Y, start=None, broadcast=False, stream=None):
        self._check_start(start, broadcast)
        ikbo_rope_forward(self.handle, rope.handle, X, Y, start, broadcast, stream)

    def rope_backward(self, rope, dY, dX, start=None, broadcast=False, stream=None):
        self._check_start(start, broadcast)
        ikbo_rope_backward(self.handle, rope.handle, dY, dX, start, broadcast, stream)

    def qcache_resize(self, lens, new_lens, table, page, free, n_free, slots, slot_offsets, positions=None, stream=None):
        ikbo_qcache_resize(self.handle, lens, new_lens, table, page, free, n_free, slots, slot_offsets, positions, stream)

    def qcache_append(self, K, V, slots, data, page, stream=None):
        ikbo_qcache_append(self.handle, K, V, slots, data, page, stream)

    def qcache_load(self, data, page, table, lens, kv_offsets, K, V, stream=None):
        ikbo_qcache_load(self.handle, data, page, table, lens, kv_offsets, K, V, stream)

    def attn_qcache_forward(self, Q, data, page, table, lens, O, lse=None, Lkv=None, scale=None, stream=None):
        if self._request is not None and (Q.shape[:3] != self._request[0] or lens.numel() != self._request[1]):
            raise ValueError("Q and lens must have the sizes of the planned request")
        ikbo_attn_qcache_forward(self.handle, Q, data, page, table, lens, O, lse, Lkv, scale, stream)

    def status(self, stream=None) -> int:
        return ikbo_plan_get_status(self.handle, stream)

    def set_lce_schedule(self, schedule: int) -> None:
        ikbo_plan_set_lce_schedule(self.handle, schedule)

    def launches(self) -> int:
        return ikbo_plan_launch_count(self.handle)

    def segments(self, n_cand: int, n_users: int):
        """Copies of (counts, offsets, perm) as CPU int32 tensors (synchronises)."""
        c, o, p = ikbo_plan_segments(self.handle)
        return (_copy_i32(c, n_users), _copy_i32(o, n_users + 1), _copy_i32(p, n_cand))

    def worklist(self):
        """Copy of the work list as a CPU int32 tensor [n_units, 4] (synchronises)."""
        w, n, cpu, mu = ikbo_plan_worklist(self.handle)
        n_units = int(_copy_i32(n, 1)[0])
        return _copy_i32(w, 4 * n_units).view(n_units, 4), cpu


class Rope:
    """Owns one ikbo_rope_t: the first rot_dim elements of a head, rotated by freqs
    (radians per position; ikbo_rope_frequencies makes the usual ones)."""

    def __init__(self, rot_dim: int, freqs=None, interleaved: bool = False, magnitude: float = 1.0):
        self.handle = None
        self.handle = ikbo_rope_create(rot_dim, ikbo_rope_frequencies(rot_dim) if freqs is None else freqs, interleaved,
                                       magnitude)

    def __del__(self):
        try:
            if self.handle:
                ikbo_rope_destroy(self.handle)
                self.handle = None
        except Exception:
            pass


class _DeviceArray:
    """Exposes a borrowed device int32 array through __cuda_array_interface__."""

    def __init__(self, ptr: int, count: int):
        self.__cuda_array_interface__ = {"shape": (count,), "typestr": "<i4", "data": (ptr, False),
                                         "version": 3, "strides": None}


def _copy_i32(dev_ptr: int, count: int) -> torch.Tensor:
    """Device int32 array at a borrowed address -> CPU tensor (synchronises)."""
    if count == 0:
        return torch.empty(0, dtype=torch.int32)
    torch.cuda.synchronize()
    return torch.as_tensor(_DeviceArray(dev_ptr, count), device="cuda").cpu().clone()
