"""Python binding of libpopffn.so: partition-guided online structured pruning (POP) of a gated-MLP FFN.

This module only marshals arguments: every step of prefill, partition and decode
runs in the library's sm_103a kernels. PyTorch supplies device memory
(``tensor.data_ptr()``) and streams (``torch.cuda.current_stream().cuda_stream``).
There is no CPU fallback: importing fails loudly when the library is missing.

The names mirror the C ABI in ``include/pop_ffn.h`` (``pop_ffn_create``,
``pop_prefill_partition``, ``pop_decode_step``, ``pop_ffn_dense_ref``, ...);
``PopFFN`` wraps a handle for convenience. Routing (``PopRouter``, ``include/pop_route.h``) and the
8-bit operators (``quantize_rows``, ``PopQLinear``, ``PopQMoE``, ``include/pop_quant.h``) follow below.
"""
from __future__ import annotations

import ctypes
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libpopffn.so")

POP_OK, POP_ERR_INVALID_ARG, POP_ERR_STATE, POP_ERR_CUDA, POP_ERR_OOM, POP_ERR_TIMEOUT, POP_ERR_UNSUPPORTED, \
    POP_ERR_DEVICE = range(8)
POP_MAX_D, POP_MAX_D_FF, POP_MAX_BATCH, POP_STATIC_MAX_D_FF = 16384, 49152, 64, 49152
POP_ROUTE_SOFTMAX, POP_ROUTE_SIGMOID = 0, 1
POP_ROUTE_MAX_EXPERTS, POP_ROUTE_MAX_TOP_K = 256, 16
POP_QUANT_BLOCK, POP_QUANT_MAX_DIM, POP_QMOE_MAX_EXPERTS, POP_QMOE_MAX_TOP_K = 128, 65536, 256, 16


class pop_config(ctypes.Structure):
    _fields_ = [("D", ctypes.c_int), ("D_FF", ctypes.c_int), ("r", ctypes.c_double), ("gamma", ctypes.c_double),
                ("period", ctypes.c_int), ("max_batch", ctypes.c_int), ("max_prefill_tokens", ctypes.c_int),
                ("out_f32", ctypes.c_int), ("skip", ctypes.c_int)]


class pop_counts(ctypes.Structure):
    _fields_ = [("n_P", ctypes.c_int), ("n_R", ctypes.c_int), ("n_C", ctypes.c_int), ("keep", ctypes.c_int),
                ("k", ctypes.c_int)]

    def as_dict(self):
        return {f: getattr(self, f) for f, _ in self._fields_}


class pop_route_config(ctypes.Structure):
    _fields_ = [("n_experts", ctypes.c_int), ("top_k", ctypes.c_int), ("score", ctypes.c_int),
                ("n_groups", ctypes.c_int), ("top_groups", ctypes.c_int), ("group_sum", ctypes.c_int),
                ("renorm", ctypes.c_int), ("scale", ctypes.c_float)]


class pop_qlinear_config(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int), ("K", ctypes.c_int), ("max_tokens", ctypes.c_int), ("out_f32", ctypes.c_int)]


class pop_qmoe_config(ctypes.Structure):
    _fields_ = [("n_experts", ctypes.c_int), ("top_k", ctypes.c_int), ("D", ctypes.c_int), ("D_FF", ctypes.c_int),
                ("max_tokens", ctypes.c_int), ("out_f32", ctypes.c_int)]


class PopError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{status_name(status)}: {message}")
        self.status = status


_vp, _i32, _f64, _u64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_double, ctypes.c_uint64
_i64 = ctypes.c_longlong
_ip, _fp = ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_float)
SIGNATURES = {
    "pop_region_counts": (_i32, [_i32, _f64, _f64, ctypes.POINTER(pop_counts)]),
    "pop_ffn_create": (_i32, [ctypes.POINTER(pop_config), _vp, _vp, _vp, _vp, ctypes.POINTER(_vp)]),
    "pop_ffn_destroy": (None, [_vp]),
    "pop_ffn_counts": (_i32, [_vp, ctypes.POINTER(pop_counts)]),
    "pop_prefill_partition": (_i32, [_vp, _vp, _i32, _vp, _vp]),
    "pop_partition_from_importance": (_i32, [_vp, _vp, _vp]),
    "pop_set_partition": (_i32, [_vp, _ip, _ip, _ip, _vp]),
    "pop_decode_step": (_i32, [_vp, _vp, _i32, _vp, _vp]),
    "pop_ffn_dense_ref": (_i32, [_vp, _vp, _i32, _vp, _vp]),
    "pop_get_partition": (_i32, [_vp, _ip, _ip, _ip]),
    "pop_get_importance": (_i32, [_vp, _fp, _fp]),
    "pop_get_selected": (_i32, [_vp, _ip, _ip]),
    "pop_get_scores": (_i32, [_vp, _fp, _fp]),
    "pop_get_step": (_i32, [_vp, _ip]),
    "pop_set_wait_limit": (_i32, [_vp, _u64]),
    "pop_profile_enable": (_i32, [_vp, _i32]),
    "pop_profile_read": (_i32, [_vp, ctypes.POINTER(ctypes.c_double), _ip]),
    "pop_ffn_dense_token_noalloc": (_i32, [_vp, _vp, _vp, _i32, _i32, _vp, _vp, _i32, _vp]),
    "pop_check": (_i32, [_vp]),
    "pop_last_error": (ctypes.c_char_p, [_vp]),
    "pop_status_string": (ctypes.c_char_p, [_i32]),
    # MoE layer (include/pop_moe.h)
    "pop_moe_create": (_i32, [ctypes.POINTER(pop_config), _i32, ctypes.POINTER(_vp), ctypes.POINTER(_vp),
                              ctypes.POINTER(_vp), _vp, ctypes.POINTER(_vp)]),
    "pop_moe_destroy": (None, [_vp]),
    "pop_moe_prefill_partition": (_i32, [_vp, _vp, _vp, _i32, _vp, _vp]),
    "pop_moe_decode_step": (_i32, [_vp, _vp, _vp, _i32, _vp, _vp]),
    "pop_moe_get_routing": (_i32, [_vp, _ip, _ip, _fp]),
    "pop_moe_get_counts": (_i32, [_vp, _ip]),
    "pop_moe_expert": (_vp, [_vp, _i32]),
    "pop_moe_num_experts": (_i32, [_vp]),
    "pop_moe_check": (_i32, [_vp]),
    "pop_moe_set_concurrent": (_i32, [_vp, _i32]),
    "pop_moe_last_error": (ctypes.c_char_p, [_vp]),
    # routing (include/pop_route.h)
    "pop_route": (_i32, [ctypes.POINTER(pop_route_config), _vp, _i32, _i64, _vp, _i32, _vp, _vp, _vp, _vp]),
    "pop_route_last_error": (ctypes.c_char_p, []),
    # 8-bit operators (include/pop_quant.h)
    "pop_quantize_rows": (_i32, [_vp, _i32, _i64, _i32, _i32, _vp, _i64, _vp, _vp]),
    "pop_qlinear_create": (_i32, [ctypes.POINTER(pop_qlinear_config), _vp, _vp, _vp, ctypes.POINTER(_vp)]),
    "pop_qlinear_destroy": (None, [_vp]),
    "pop_qlinear_forward": (_i32, [_vp, _vp, _i64, _i32, _vp, _i64, _vp]),
    "pop_qlinear_forward_quantized": (_i32, [_vp, _vp, _i64, _vp, _i64, _i32, _vp, _i64, _vp]),
    "pop_qlinear_set_wait_limit": (_i32, [_vp, _u64]),
    "pop_qlinear_check": (_i32, [_vp]),
    "pop_qmoe_create": (_i32, [ctypes.POINTER(pop_qmoe_config)] + [ctypes.POINTER(_vp)] * 6 + [_vp, ctypes.POINTER(_vp)]),
    "pop_qmoe_destroy": (None, [_vp]),
    "pop_qmoe_forward": (_i32, [_vp, _vp, _i64, _vp, _vp, _i32, _vp, _i64, _vp]),
    "pop_qmoe_set_wait_limit": (_i32, [_vp, _u64]),
    "pop_qmoe_check": (_i32, [_vp]),
    "pop_quant_last_error": (ctypes.c_char_p, []),
}

_lib = None


def load_library(path: str = LIB_PATH):
    """Loads libpopffn.so and declares its signatures. Raises ImportError when it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'`")
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    _lib = lib
    return lib


def status_name(s: int) -> str:
    names = ["POP_OK", "POP_ERR_INVALID_ARG", "POP_ERR_STATE", "POP_ERR_CUDA", "POP_ERR_OOM", "POP_ERR_TIMEOUT",
             "POP_ERR_UNSUPPORTED", "POP_ERR_DEVICE"]
    return names[s] if 0 <= s < len(names) else f"status {s}"


def _check(status: int, handle=None):
    if status != POP_OK:
        msg = load_library().pop_last_error(handle)
        raise PopError(status, msg.decode() if msg else "")


def _check_moe(status: int, handle=None):
    if status != POP_OK:
        msg = load_library().pop_moe_last_error(handle)
        raise PopError(status, msg.decode() if msg else "")


def _ptr(t):
    """Device address of a tensor (or an int already holding one, or None)."""
    if t is None or isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _expect(t, name, dtype, shape, min_rows=0):
    """Checks a tensor argument before its address goes to the C ABI: dtype, contiguity and shape
    (None in `shape` accepts any extent; an output may have more rows than it receives, at least
    `min_rows`). Raises PopError(POP_ERR_INVALID_ARG)."""
    if t is None:
        return
    ok = (t.dtype == dtype and t.is_contiguous() and t.dim() == len(shape)
          and all(want is None or got == want for got, want in zip(t.shape, shape))
          and (t.dim() == 0 or t.shape[0] >= min_rows))
    if not ok:
        raise PopError(POP_ERR_INVALID_ARG, f"{name}: expected a contiguous {dtype} tensor of shape "
                                            f"{tuple('*' if w is None else w for w in shape)}, got "
                                            f"{t.dtype} {tuple(t.shape)}{'' if t.is_contiguous() else ' (strided)'}")


def _int_array(a):
    import numpy as np
    arr = np.ascontiguousarray(a, dtype=np.int32)
    if arr.size == 0:
        arr = np.zeros(1, dtype=np.int32)
    return arr, arr.ctypes.data_as(_ip)


# ------------------------------------------------------------------ C-ABI mirrors

def pop_region_counts(N: int, r: float, gamma: float) -> pop_counts:
    out = pop_counts()
    _check(load_library().pop_region_counts(N, r, gamma, ctypes.byref(out)))
    return out


def pop_ffn_create(cfg: pop_config, Wg, W1, W2, stream=None) -> int:
    h = ctypes.c_void_p()
    _check(load_library().pop_ffn_create(ctypes.byref(cfg), _ptr(Wg), _ptr(W1), _ptr(W2), _stream(stream),
                                         ctypes.byref(h)))
    return h.value


def pop_ffn_destroy(h) -> None:
    load_library().pop_ffn_destroy(h)


def pop_ffn_counts(h) -> pop_counts:
    out = pop_counts()
    _check(load_library().pop_ffn_counts(h, ctypes.byref(out)), h)
    return out


def pop_prefill_partition(h, X, M: int, Y=None, stream=None) -> None:
    _check(load_library().pop_prefill_partition(h, _ptr(X), M, _ptr(Y), _stream(stream)), h)


def pop_partition_from_importance(h, importance, stream=None) -> None:
    _check(load_library().pop_partition_from_importance(h, _ptr(importance), _stream(stream)), h)


def pop_set_partition(h, R, C, P, stream=None) -> None:
    (_r, rp), (_c, cp), (_p, pp) = _int_array(R), _int_array(C), _int_array(P)
    _check(load_library().pop_set_partition(h, rp, cp, pp, _stream(stream)), h)


def pop_decode_step(h, x, B: int, y, stream=None) -> None:
    _check(load_library().pop_decode_step(h, _ptr(x), B, _ptr(y), _stream(stream)), h)


def pop_ffn_dense_ref(h, X, M: int, Y, stream=None) -> None:
    _check(load_library().pop_ffn_dense_ref(h, _ptr(X), M, _ptr(Y), _stream(stream)), h)


def pop_get_partition(h):
    import numpy as np
    c = pop_ffn_counts(h)
    R, C, P = (np.zeros(max(n, 1), dtype=np.int32) for n in (c.n_R, c.n_C, c.n_P))
    _check(load_library().pop_get_partition(h, R.ctypes.data_as(_ip), C.ctypes.data_as(_ip), P.ctypes.data_as(_ip)),
           h)
    return R[:c.n_R], C[:c.n_C], P[:c.n_P]


def pop_get_importance(h):
    import numpy as np
    c = pop_ffn_counts(h)
    N = c.n_P + c.n_R + c.n_C
    I, ss = np.zeros(N, dtype=np.float32), np.zeros(N, dtype=np.float32)
    _check(load_library().pop_get_importance(h, I.ctypes.data_as(_fp), ss.ctypes.data_as(_fp)), h)
    return I, ss


def pop_get_selected(h):
    import numpy as np
    c = pop_ffn_counts(h)
    S = np.zeros(max(c.k, 1), dtype=np.int32)
    k = ctypes.c_int()
    _check(load_library().pop_get_selected(h, ctypes.byref(k), S.ctypes.data_as(_ip)), h)
    return S[:k.value]


def pop_get_scores(h):
    import numpy as np
    c = pop_ffn_counts(h)
    a, m = np.zeros(max(c.n_C, 1), dtype=np.float32), np.zeros(max(c.n_C, 1), dtype=np.float32)
    _check(load_library().pop_get_scores(h, a.ctypes.data_as(_fp), m.ctypes.data_as(_fp)), h)
    return a[:c.n_C], m[:c.n_C]


def pop_get_step(h) -> int:
    s = ctypes.c_int()
    _check(load_library().pop_get_step(h, ctypes.byref(s)), h)
    return s.value


def pop_set_wait_limit(h, ns: int) -> None:
    _check(load_library().pop_set_wait_limit(h, ns), h)


def pop_profile_enable(h, enable: bool = True) -> None:
    _check(load_library().pop_profile_enable(h, 1 if enable else 0), h)


def pop_profile_read(h):
    """(ms per kernel [gate/up, select, down, reduce] summed since the last read, decode steps)."""
    ms = (ctypes.c_double * 4)()
    steps = ctypes.c_int()
    _check(load_library().pop_profile_read(h, ms, ctypes.byref(steps)), h)
    return list(ms), steps.value


def pop_check(h) -> None:
    _check(load_library().pop_check(h), h)


# ------------------------------------------------------------------ convenience wrapper

class PopFFN:
    """One gated-MLP layer with POP pruning, backed by a pop_ffn handle.

    Wg, W1: torch bf16 [D_FF, D] on the current CUDA device; W2: bf16 [D, D_FF].
    """

    def __init__(self, Wg, W1, W2, r: float, gamma: float = 0.1, period: int = 1, max_batch: int = 1,
                 max_prefill_tokens: int = 2048, out_f32: bool = True, skip: bool = False, stream=None):
        N, D = Wg.shape
        self.handle = None
        self.cfg = pop_config(D=D, D_FF=N, r=r, gamma=gamma, period=period, max_batch=max_batch,
                              max_prefill_tokens=max_prefill_tokens, out_f32=1 if out_f32 else 0,
                              skip=1 if skip else 0)
        self.D, self.N = D, N
        self.handle = pop_ffn_create(self.cfg, Wg, W1, W2, stream)
        self.counts = pop_ffn_counts(self.handle)

    def close(self):
        if getattr(self, "handle", None):
            if not getattr(self, "_borrowed", False):
                pop_ffn_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def out_dtype(self):
        import torch
        return torch.float32 if self.cfg.out_f32 else torch.bfloat16

    def prefill_partition(self, X, Y=None, stream=None):
        import torch
        _expect(X, "X", torch.bfloat16, (None, self.D))
        _expect(Y, "Y", self.out_dtype(), (None, self.D), X.shape[0])
        pop_prefill_partition(self.handle, X, X.shape[0], Y, stream)

    def partition_from_importance(self, importance, stream=None):
        import torch
        _expect(importance, "importance", torch.float32, (self.N,))
        pop_partition_from_importance(self.handle, importance, stream)

    def set_partition(self, R, C, P, stream=None):
        pop_set_partition(self.handle, R, C, P, stream)

    def decode_step(self, x, y=None, stream=None):
        import torch
        _expect(x, "x", torch.bfloat16, (None, self.D))
        if y is None:
            y = torch.empty((x.shape[0], self.D), dtype=self.out_dtype(), device=x.device)
        _expect(y, "y", self.out_dtype(), (None, self.D), x.shape[0])
        pop_decode_step(self.handle, x, x.shape[0], y, stream)
        return y

    def dense_ref(self, X, Y=None, stream=None):
        import torch
        _expect(X, "X", torch.bfloat16, (None, self.D))
        if Y is None:
            Y = torch.empty((X.shape[0], self.D), dtype=self.out_dtype(), device=X.device)
        _expect(Y, "Y", self.out_dtype(), (None, self.D), X.shape[0])
        pop_ffn_dense_ref(self.handle, X, X.shape[0], Y, stream)
        return Y

    def partition(self):
        return pop_get_partition(self.handle)

    def importance(self):
        return pop_get_importance(self.handle)

    def selected(self):
        return pop_get_selected(self.handle)

    def scores(self):
        return pop_get_scores(self.handle)

    def step_count(self):
        return pop_get_step(self.handle)

    def set_wait_limit(self, ns: int):
        pop_set_wait_limit(self.handle, ns)

    def profile(self, enable: bool = True):
        pop_profile_enable(self.handle, enable)

    def profile_read(self):
        return pop_profile_read(self.handle)

    def check(self):
        pop_check(self.handle)

    @classmethod
    def _borrow(cls, handle, cfg):
        """A view of a layer handle owned elsewhere (an MoE expert): close() leaves it alone."""
        v = cls.__new__(cls)
        v.cfg, v.D, v.N, v.handle, v._borrowed = cfg, cfg.D, cfg.D_FF, handle, True
        v.counts = pop_ffn_counts(handle)
        return v


# ------------------------------------------------------------------ MoE layer

def pop_moe_create(cfg: pop_config, Wg, W1, W2, stream=None) -> int:
    E = len(Wg)
    arr = [(_vp * E)(*[_ptr(w) for w in ws]) for ws in (Wg, W1, W2)]
    out = _vp()
    _check_moe(load_library().pop_moe_create(ctypes.byref(cfg), E, arr[0], arr[1], arr[2], _stream(stream),
                                             ctypes.byref(out)))
    return out.value


class PopMoE:
    """An MoE layer of POP-pruned gated-MLP experts (top-2 routing), backed by a pop_moe handle.

    Wg, W1: lists of torch bf16 [D_FF, D] (one per expert); W2: list of bf16 [D, D_FF].
    """

    def __init__(self, Wg, W1, W2, r: float, gamma: float = 0.1, period: int = 1, max_batch: int = 1,
                 max_prefill_tokens: int = 2048, out_f32: bool = True, stream=None):
        N, D = Wg[0].shape
        self.handle = None
        self.cfg = pop_config(D=D, D_FF=N, r=r, gamma=gamma, period=period, max_batch=max_batch,
                              max_prefill_tokens=max_prefill_tokens, out_f32=1 if out_f32 else 0)
        self.D, self.N, self.E = D, N, len(Wg)
        self.handle = pop_moe_create(self.cfg, Wg, W1, W2, stream)
        self.experts = [PopFFN._borrow(load_library().pop_moe_expert(self.handle, e), self.cfg)
                        for e in range(self.E)]
        self.counts = self.experts[0].counts

    def close(self):
        if getattr(self, "handle", None):
            self.experts = []
            load_library().pop_moe_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def out_dtype(self):
        import torch
        return torch.float32 if self.cfg.out_f32 else torch.bfloat16

    def prefill_partition(self, X, logits, Y=None, stream=None):
        """X: bf16 [M, D]; logits: float32 [M, E]; Y (optional): [M, D] of out_dtype()."""
        import torch
        _expect(X, "X", torch.bfloat16, (None, self.D))
        _expect(logits, "logits", torch.float32, (None, self.E), X.shape[0])
        _expect(Y, "Y", self.out_dtype(), (None, self.D), X.shape[0])
        _check_moe(load_library().pop_moe_prefill_partition(self.handle, _ptr(X), _ptr(logits), X.shape[0], _ptr(Y),
                                                            _stream(stream)), self.handle)

    def decode_step(self, x, logits, y=None, stream=None):
        import torch
        _expect(x, "x", torch.bfloat16, (None, self.D))
        _expect(logits, "logits", torch.float32, (None, self.E), x.shape[0])
        if y is None:
            y = torch.empty((x.shape[0], self.D), dtype=self.out_dtype(), device=x.device)
        _expect(y, "y", self.out_dtype(), (None, self.D), x.shape[0])
        _check_moe(load_library().pop_moe_decode_step(self.handle, _ptr(x), _ptr(logits), x.shape[0], _ptr(y),
                                                      _stream(stream)), self.handle)
        return y

    def routing(self):
        """(experts [T, 2] int32, weights [T, 2] float32) of the last call. Syncs."""
        import numpy as np
        lib = load_library()
        T = ctypes.c_int(0)
        _check_moe(lib.pop_moe_get_routing(self.handle, ctypes.byref(T), None, None), self.handle)
        ex = np.zeros((max(T.value, 1), 2), dtype=np.int32)
        w = np.zeros((max(T.value, 1), 2), dtype=np.float32)
        _check_moe(lib.pop_moe_get_routing(self.handle, ctypes.byref(T), ex.ctypes.data_as(_ip),
                                           w.ctypes.data_as(_fp)), self.handle)
        return ex[:T.value], w[:T.value]

    def token_counts(self):
        import numpy as np
        c = np.zeros(self.E, dtype=np.int32)
        _check_moe(load_library().pop_moe_get_counts(self.handle, c.ctypes.data_as(_ip)), self.handle)
        return c

    def check(self):
        _check_moe(load_library().pop_moe_check(self.handle), self.handle)

    def set_concurrent(self, on: bool):
        """Experts' decode kernels on streams of their own (True, the default) or one after another
        on the caller's stream (False: for per-kernel timing)."""
        _check_moe(load_library().pop_moe_set_concurrent(self.handle, 1 if on else 0), self.handle)


# ------------------------------------------------------------------ routing

def _check_with(last_error: str, status: int):
    if status != POP_OK:
        msg = getattr(load_library(), last_error)()
        raise PopError(status, msg.decode() if msg else "")


def _bad(what: str):
    raise PopError(POP_ERR_INVALID_ARG, what)


def _rows_arg(t, name, dtypes, cols, align):
    """Checks a [rows, cols] CUDA tensor whose elements of a row are contiguous (the rows may lie
    farther apart). Returns (rows, row stride in elements)."""
    shape = t.shape
    if len(shape) != 2 or shape[1] != cols or t.dtype not in dtypes or not t.is_cuda:
        _bad(f"{name}: expected a CUDA tensor of shape (*, {cols}) and type {' or '.join(map(str, dtypes))}, got "
             f"{t.dtype} {tuple(shape)} on {t.device}")
    rows = shape[0]
    ld, step = t.stride()
    if (cols > 1 and step != 1) or (rows > 1 and ld < cols):
        _bad(f"{name}: the elements of a row must be contiguous, its rows apart; strides are {tuple(t.stride())}")
    if rows <= 1:
        ld = -(-cols // 8) * 8
    if align > 1 and rows > 0 and (t.data_ptr() % align or (ld * t.element_size()) % align):
        _bad(f"{name}: rows must start on {align}-byte boundaries")
    return rows, ld


def _whole_arg(t, name, dtype, shape):
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous() or not t.is_cuda:
        _bad(f"{name}: expected a contiguous CUDA {dtype} tensor of shape {tuple(shape)}, got {t.dtype} "
             f"{tuple(t.shape)} on {t.device}")


_gpus = None  # that this process sees, once it has been asked


def _one_device(t, *others):
    """Checks that all of a call's tensors are on the current device: the library launches there."""
    global _gpus
    import torch
    if _gpus is None:
        _gpus = torch.cuda.device_count()
    dev = t.get_device()
    for x in others:
        if x is not None and x.get_device() != dev:
            _bad(f"tensors of one call on {t.device} and {x.device}")
    if dev != torch._C._cuda_getDevice():
        _bad(f"tensors on {t.device}, which is not the current device")


def _on(stream, t, *others):
    """The stream of a call, whose tensors are all on the current device: (raw handle, what new outputs are to be
    made under, or None for the current stream). New outputs belong to the call's stream, and inputs that another
    stream allocated are not given to others before it is done with them."""
    import torch
    dev = t.get_device()
    if _gpus != 1:  # (with one there is no other, and the check takes a fraction of a microsecond)
        _one_device(t, *others)
    raw = torch._C._cuda_getCurrentRawStream(dev)
    if stream is None:
        return raw, None
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
    if getattr(stream, "device_index", dev) != dev:
        _bad(f"a stream of cuda:{stream.device_index} for tensors on cuda:{dev}")
    if stream.cuda_stream == raw:
        return raw, None
    for x in (t, *others):
        if x is not None:
            x.record_stream(stream)
    return stream.cuda_stream, stream


def _empty(under, shape, dtype, device):
    import torch
    if under is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(under):
        return torch.empty(shape, dtype=dtype, device=device)


class PopRouter:
    """Routes tokens to experts (``pop_route``): softmax or sigmoid scores, an optional bias for
    balance, groups of experts, the ``top_k`` best, their weights. ``include/pop_route.h`` has the
    formulas and what masked experts, ties and rows without an expert give."""

    def __init__(self, n_experts: int, top_k: int, score: str = "softmax", n_groups: int = 1, top_groups: int = 1,
                 group_sum: int = 1, renorm: bool = True, scale: float = 1.0):
        kinds = {"softmax": POP_ROUTE_SOFTMAX, "sigmoid": POP_ROUTE_SIGMOID}
        if score not in kinds:
            _bad(f"score must be 'softmax' or 'sigmoid', got {score!r}")
        self.cfg = pop_route_config(n_experts=n_experts, top_k=top_k, score=kinds[score], n_groups=n_groups,
                                    top_groups=top_groups, group_sum=group_sum, renorm=1 if renorm else 0, scale=scale)
        self._cfg_ref = ctypes.byref(self.cfg)

    def route(self, logits, bias=None, counts=None, stream=None):
        """logits: [T, n_experts] float32 or bf16 (rows may be strided); bias: float32 [n_experts];
        counts: int32 [n_experts] that receives the slots given to each expert.
        Returns (experts int32 [T, top_k], weights float32 [T, top_k])."""
        import torch
        E, k = self.cfg.n_experts, self.cfg.top_k
        T, ld = _rows_arg(logits, "logits", (torch.float32, torch.bfloat16), E, 1)
        if bias is not None:
            _whole_arg(bias, "bias", torch.float32, (E,))
        if counts is not None:
            _whole_arg(counts, "counts", torch.int32, (E,))
        raw, under = _on(stream, logits, bias, counts)
        device = logits.device
        experts = _empty(under, (T, k), torch.int32, device)
        weights = _empty(under, (T, k), torch.float32, device)
        st = _lib.pop_route(self._cfg_ref, logits.data_ptr(), 1 if logits.dtype == torch.bfloat16 else 0, ld, _ptr(bias),
                            T, experts.data_ptr(), weights.data_ptr(), _ptr(counts), raw)
        if st != POP_OK:
            _check_with("pop_route_last_error", st)
        return experts, weights


# ------------------------------------------------------------------ 8-bit operators

def _check_quant(status: int):
    _check_with("pop_quant_last_error", status)


def _blocks(n: int) -> int:
    return -(-n // POP_QUANT_BLOCK)


def quantize_rows(x, stream=None):
    """x: [M, K] bf16 or float32, K a multiple of 8 (rows may be strided). Returns (q float8_e4m3fn
    [M, K], scales float32 [M, ceil(K/128)]): element (m, k) stands for scales[m, k // 128] * q[m, k]."""
    import torch
    if x.dim() != 2:
        _bad(f"x: expected two dimensions, got {tuple(x.shape)}")
    K = x.shape[1]
    M, ld = _rows_arg(x, "x", (torch.bfloat16, torch.float32), K, 16)
    raw, under = _on(stream, x)
    device = x.device
    q = _empty(under, (M, K), torch.float8_e4m3fn, device)
    s = _empty(under, (M, _blocks(K)), torch.float32, device)
    st = _lib.pop_quantize_rows(x.data_ptr(), 1 if x.dtype == torch.float32 else 0, ld, M, K, q.data_ptr(), K,
                                s.data_ptr(), raw)
    if st != POP_OK:
        _check_quant(st)
    return q, s


class _QHandle:
    """Owns a handle of include/pop_quant.h."""
    _destroy = _checker = _limiter = ""
    handle = None

    def close(self):
        if self.handle:
            getattr(load_library(), self._destroy)(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def out_dtype(self):
        import torch
        return torch.float32 if self.cfg.out_f32 else torch.bfloat16

    def set_wait_limit(self, ns: int):
        """Limit of every device-side wait of the handle's products, in nanoseconds (2 s unless set)."""
        _check_quant(getattr(load_library(), self._limiter)(self.handle, ns))

    def check(self):
        """Syncs and raises the first device-side failure since the last check."""
        _check_quant(getattr(load_library(), self._checker)(self.handle))

    def _output(self, y, rows, cols, device, under, align):
        """(y, its row stride): a new [rows, cols] tensor, or the caller's, checked."""
        if y is None:
            return _empty(under, (rows, cols), self.out_dtype(), device), cols
        got, ld = _rows_arg(y, "y", (self.out_dtype(),), cols, align)
        if got != rows:
            _bad(f"y: expected {rows} rows, got {tuple(y.shape)}")
        return y, ld


def _matrix_arg(W, S, name):
    """Checks one matrix: bf16 [N, K] (S None), or e4m3 [N, K] with float32 scales S."""
    import torch
    if W.dim() != 2:
        _bad(f"{name}: expected a matrix, got {tuple(W.shape)}")
    _whole_arg(W, name, torch.bfloat16 if S is None else torch.float8_e4m3fn, W.shape)
    if S is not None:
        _whole_arg(S, name + " scales", torch.float32, (_blocks(W.shape[0]), _blocks(W.shape[1])))


class PopQLinear(_QHandle):
    """y = x W^T with W kept in e4m3 and a scale per 128 x 128 block (``pop_qlinear``).

    W: torch bf16 [N, K], quantised here, or float8_e4m3fn [N, K] with float32 scales S
    [ceil(N/128), ceil(K/128)]. The handle keeps its own copy. max_tokens: rows that the workspace is
    made for; longer calls run in chunks."""
    _destroy, _checker, _limiter = "pop_qlinear_destroy", "pop_qlinear_check", "pop_qlinear_set_wait_limit"

    def __init__(self, W, S=None, max_tokens: int = 2048, out_f32: bool = False, stream=None):
        _matrix_arg(W, S, "W")
        _one_device(W, S)
        self.N, self.K = W.shape
        self.cfg = pop_qlinear_config(N=self.N, K=self.K, max_tokens=max_tokens, out_f32=1 if out_f32 else 0)
        h = _vp()
        _check_quant(load_library().pop_qlinear_create(ctypes.byref(self.cfg), _ptr(W), _ptr(S), _stream(stream),
                                                       ctypes.byref(h)))
        self.handle = h.value

    def forward(self, x, y=None, stream=None):
        """x: bf16 [M, K], quantised on the way. Returns y [M, N] of out_dtype()."""
        import torch
        M, ld = _rows_arg(x, "x", (torch.bfloat16,), self.K, 16)
        raw, under = _on(stream, x, y)
        y, ldy = self._output(y, M, self.N, x.device, under, 1)
        st = _lib.pop_qlinear_forward(self.handle, x.data_ptr(), ld, M, y.data_ptr(), ldy, raw)
        if st != POP_OK:
            _check_quant(st)
        return y

    def forward_q(self, xq, xs, y=None, stream=None):
        """The same for rows that quantize_rows gave: xq float8_e4m3fn [M, K], xs float32."""
        import torch
        M, ldq = _rows_arg(xq, "xq", (torch.float8_e4m3fn,), self.K, 8)
        rows, lds = _rows_arg(xs, "xs", (torch.float32,), _blocks(self.K), 1)
        if rows != M:
            _bad(f"xs: expected {M} rows, got {rows}")
        raw, under = _on(stream, xq, xs, y)
        y, ldy = self._output(y, M, self.N, xq.device, under, 1)
        st = _lib.pop_qlinear_forward_quantized(self.handle, xq.data_ptr(), ldq, xs.data_ptr(), lds, M, y.data_ptr(), ldy,
                                                raw)
        if st != POP_OK:
            _check_quant(st)
        return y


class PopQMoE(_QHandle):
    """Gated-MLP experts in e4m3 with a scale per block (``pop_qmoe``), for tokens that a router has
    given experts and weights.

    Wg, W1: [D_FF, D] per expert, W2: [D, D_FF] per expert. Each is a sequence (or a stacked tensor) of
    bf16 matrices, quantised here, or a pair of such sequences: float8_e4m3fn matrices and their scales."""
    _destroy, _checker, _limiter = "pop_qmoe_destroy", "pop_qmoe_check", "pop_qmoe_set_wait_limit"

    def __init__(self, Wg, W1, W2, top_k: int, max_tokens: int = 2048, out_f32: bool = False, stream=None):
        scaled = [isinstance(w, tuple) and len(w) == 2 and w[0][0].dim() == 2 for w in (Wg, W1, W2)]
        if any(scaled) and not all(scaled):
            _bad("Wg, W1 and W2 must all be bf16 or all be (e4m3, scales) pairs")
        mats = [list(w[0]) if all(scaled) else list(w) for w in (Wg, W1, W2)]
        scales = [list(w[1]) for w in (Wg, W1, W2)] if all(scaled) else [[None] * len(m) for m in mats]
        self.E = len(mats[0])
        if self.E < 1 or any(len(m) != self.E for m in mats + scales):
            _bad("Wg, W1, W2 and their scales must have one entry per expert")
        self.N, self.D = mats[0][0].shape
        for name, ms, ss, shape in zip(("Wg", "W1", "W2"), mats, scales,
                                       ((self.N, self.D), (self.N, self.D), (self.D, self.N))):
            for m, s in zip(ms, ss):
                _matrix_arg(m, s, name)
                if tuple(m.shape) != shape:
                    _bad(f"{name}: expected matrices of shape {shape}, got {tuple(m.shape)}")
        _one_device(*(t for ts in mats + scales for t in ts))
        self.cfg = pop_qmoe_config(n_experts=self.E, top_k=top_k, D=self.D, D_FF=self.N, max_tokens=max_tokens,
                                   out_f32=1 if out_f32 else 0)
        arrays = [(_vp * self.E)(*[_ptr(m) for m in ms]) for ms in mats]
        arrays += [(_vp * self.E)(*[_ptr(s) for s in ss]) if all(scaled) else None for ss in scales]
        h = _vp()
        _check_quant(load_library().pop_qmoe_create(ctypes.byref(self.cfg), *arrays, _stream(stream), ctypes.byref(h)))
        self.handle = h.value

    def forward(self, x, experts, weights, y=None, stream=None):
        """x: bf16 [T, D]; experts int32 and weights float32 [T, top_k], as PopRouter.route gives them.
        Returns y [T, D] of out_dtype()."""
        import torch
        T, ld = _rows_arg(x, "x", (torch.bfloat16,), self.D, 16)
        _whole_arg(experts, "experts", torch.int32, (T, self.cfg.top_k))
        _whole_arg(weights, "weights", torch.float32, (T, self.cfg.top_k))
        raw, under = _on(stream, x, experts, weights, y)
        y, ldy = self._output(y, T, self.D, x.device, under, 16)
        st = _lib.pop_qmoe_forward(self.handle, x.data_ptr(), ld, experts.data_ptr(), weights.data_ptr(), T, y.data_ptr(),
                                   ldy, raw)
        if st != POP_OK:
            _check_quant(st)
        return y


load_library()
