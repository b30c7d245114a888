"""ctypes binding of libshadowkv.so (include/shadowkv.h).

Argument marshalling only: tensors become raw pointers, streams become
cudaStream_t handles, status codes become exceptions.  Every computation runs
in the library's CUDA kernels; there is no Python or CPU fallback, and the
binding raises if the library has not been built.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading
from typing import Optional

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libshadowkv.so")

DTYPE_F32, DTYPE_BF16 = 0, 1
GROUP_MAX, GROUP_SUM = 0, 1
OPT_CACHE, OPT_TIMING, OPT_SPLIT_TOKENS, OPT_CUDA_CORES, OPT_REBUILD_IN_ATTENTION = 0, 1, 2, 3, 4

FIELDS = {
    "A": 0, "BT": 1, "L": 2, "MIN_COS": 3, "OUTLIER_IDS": 4, "K_OUT": 5, "V_OUT": 6,
    "K_LOC": 7, "V_LOC": 8, "SEL": 9, "SEL_SLOT": 10, "HITS": 11, "LOGITS": 12,
    "K_SPARSE": 13, "SLOT_CHUNK": 14, "SLOT_V": 15, "V_CPU": 16, "SVD_BASIS": 17,
}
_INT_FIELDS = {"OUTLIER_IDS", "SEL", "SEL_SLOT", "HITS", "SLOT_CHUNK"}
_F32_FIELDS = {"MIN_COS", "LOGITS", "SVD_BASIS"}

STATUS = {0: "OK", 1: "INVALID_ARG", 2: "OOM", 3: "CUDA", 4: "DEVICE_CHECK", 5: "TIMEOUT",
          6: "STATE", 7: "UNSUPPORTED"}


class ShadowKVError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{STATUS.get(code, code)}: {msg}")
        self.code = code


class Params(ctypes.Structure):
    _fields_ = [("b", ctypes.c_int), ("h_q", ctypes.c_int), ("h_kv", ctypes.c_int),
                ("d", ctypes.c_int), ("s", ctypes.c_int), ("c", ctypes.c_int),
                ("r", ctypes.c_int), ("k", ctypes.c_int), ("o", ctypes.c_int),
                ("w", ctypes.c_int), ("max_new", ctypes.c_int), ("rope_theta", ctypes.c_float),
                ("dtype", ctypes.c_int), ("group_reduce", ctypes.c_int),
                ("svd_iters", ctypes.c_int), ("reserved", ctypes.c_int),
                ("seed", ctypes.c_ulonglong)]


class StateIn(ctypes.Structure):
    _fields_ = [("A", ctypes.c_void_p), ("B", ctypes.c_void_p), ("L", ctypes.c_void_p),
                ("outlier_ids", ctypes.c_void_p), ("K_out", ctypes.c_void_p),
                ("V_out", ctypes.c_void_p), ("K_loc", ctypes.c_void_p),
                ("V_loc", ctypes.c_void_p), ("V", ctypes.c_void_p), ("v_on_host", ctypes.c_int)]


class Rows(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("sb", ctypes.c_longlong), ("sh", ctypes.c_longlong),
                ("ss", ctypes.c_longlong)]


class NormRopeParams(ctypes.Structure):
    _fields_ = [("b", ctypes.c_int), ("s", ctypes.c_int), ("h_q", ctypes.c_int), ("h_kv", ctypes.c_int),
                ("d", ctypes.c_int), ("rot", ctypes.c_int), ("dtype", ctypes.c_int), ("norm", ctypes.c_int),
                ("pos_per_token", ctypes.c_int), ("eps", ctypes.c_float), ("theta", ctypes.c_float)]


class CacheDesc(ctypes.Structure):
    _fields_ = [("b", ctypes.c_int), ("h_kv", ctypes.c_int), ("d", ctypes.c_int), ("block", ctypes.c_int),
                ("max_blocks", ctypes.c_int), ("n_pool", ctypes.c_int), ("k_codes", ctypes.c_void_p),
                ("v_codes", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("table", ctypes.c_void_p), ("n_tok", ctypes.c_void_p), ("weight", ctypes.c_void_p),
                ("status", ctypes.c_void_p)]


class VerifyParams(ctypes.Structure):
    _fields_ = [("b", ctypes.c_int), ("s", ctypes.c_int), ("vocab", ctypes.c_int), ("dtype", ctypes.c_int),
                ("temperature", ctypes.c_double), ("logits_sb", ctypes.c_longlong), ("logits_ss", ctypes.c_longlong),
                ("probs_sb", ctypes.c_longlong), ("probs_ss", ctypes.c_longlong)]


class Layout(ctypes.Structure):
    _fields_ = [("kv_records", ctypes.c_int), ("a_tiled", ctypes.c_int), ("tc_score", ctypes.c_int),
                ("tc_rebuild", ctypes.c_int), ("tc_attention", ctypes.c_int),
                ("fetch_in_rebuild", ctypes.c_int), ("fetch_in_attention", ctypes.c_int),
                ("rebuild_in_attention", ctypes.c_int)]


class Stats(ctypes.Structure):
    _fields_ = [("steps", ctypes.c_longlong), ("hits", ctypes.c_longlong),
                ("misses", ctypes.c_longlong), ("link_bytes", ctypes.c_longlong),
                ("launches", ctypes.c_longlong)]


_lib = None


def lib() -> ctypes.CDLL:
    """Loads libshadowkv.so (built in-tree by sparse_rank_kv_gb300.build)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with `python -m sparse_rank_kv_gb300.build` "
                "(the ShadowKV path has no fallback)")
        L = ctypes.CDLL(LIB_PATH)
        P, V, I, S = ctypes.POINTER, ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        sig = {
            "shadowkv_validate_params": (I, [P(Params)]),
            "shadowkv_footprint": (I, [P(Params), P(S), P(S)]),
            "shadowkv_prefill": (I, [P(Params), V, V, I, V, P(V)]),
            "shadowkv_load_state": (I, [P(Params), P(StateIn), V, P(V)]),
            "shadowkv_decode_step": (I, [V, V, V, V, V, V]),
            "shadowkv_decode_step_host": (I, [V, V, V, V, V, V]),
            "shadowkv_free": (None, [V]),
            "shadowkv_rewind": (I, [V, V]),
            "shadowkv_last_error": (ctypes.c_char_p, []),
            "shadowkv_set_option": (I, [V, I, ctypes.c_longlong]),
            "shadowkv_get_stats": (I, [V, P(Stats)]),
            "shadowkv_check": (I, [V]),
            "shadowkv_get_layout": (I, [V, P(Layout)]),
            "shadowkv_num_kernels": (I, []),
            "shadowkv_kernel_name": (ctypes.c_char_p, [I]),
            "shadowkv_kernel_times": (I, [V, P(ctypes.c_double), P(ctypes.c_longlong), I]),
            "shadowkv_reset_timers": (I, [V]),
            "shadowkv_field_bytes": (I, [V, I, P(S)]),
            "shadowkv_export": (I, [V, I, V, S]),
            "shadowkv_attention_noalloc": (I, [P(Params), V, V, V, I, V, V]),
            "shadowkv_qk_norm_rope": (I, [P(NormRopeParams), P(Rows), P(Rows), V, V, V, P(Rows), P(Rows), V]),
            "shadowkv_cache_validate": (I, [P(CacheDesc)]),
            "shadowkv_cache_append": (I, [P(CacheDesc), I, P(Rows), P(Rows), I, V, V]),
            "shadowkv_cache_attend_workspace": (S, [P(CacheDesc), I]),
            "shadowkv_cache_attend": (I, [P(CacheDesc), I, I, P(Rows), ctypes.c_float, I, ctypes.c_float,
                                          P(Rows), V, V, S, V]),
            "shadowkv_cache_attend_tokens_workspace": (S, [P(CacheDesc), I, I]),
            "shadowkv_cache_attend_tokens": (I, [P(CacheDesc), I, I, I, P(Rows), V, I, ctypes.c_float, P(Rows), V, V, S, V]),
            "shadowkv_cache_evict": (I, [P(CacheDesc), P(CacheDesc), I, I, I, V, V]),
            "shadowkv_cache_share": (I, [P(CacheDesc), V, I, V, V, V]),
            "shadowkv_cache_reserve_workspace": (S, [P(CacheDesc), I]),
            "shadowkv_cache_reserve": (I, [P(CacheDesc), V, I, V, V, V, S, V]),
            "shadowkv_cache_truncate": (I, [P(CacheDesc), V, V, V]),
            "shadowkv_cache_compact_workspace": (S, [P(CacheDesc)]),
            "shadowkv_cache_compact": (I, [P(CacheDesc), V, P(CacheDesc), V, V, S, V]),
            "shadowkv_cache_check": (I, [P(CacheDesc)]),
            "shadowkv_verify_workspace": (S, [P(VerifyParams)]),
            "shadowkv_verify_drafts": (I, [P(VerifyParams)] + [V] * 10 + [S, V]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _check(code: int):
    if code != 0:
        raise ShadowKVError(code, lib().shadowkv_last_error().decode())


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to the library must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def make_params(cfg=None, **kw) -> Params:
    """Params from a synth.Config (or keyword fields)."""
    if cfg is not None:
        base = dict(b=cfg.b, h_q=cfg.h_q, h_kv=cfg.h_kv, d=cfg.d, s=cfg.s, c=cfg.c, r=cfg.r,
                    k=cfg.k, o=cfg.o, w=cfg.w, max_new=cfg.max_new, rope_theta=cfg.theta,
                    dtype=DTYPE_BF16 if cfg.dtype == "bf16" else DTYPE_F32)
        base.update(kw)
        kw = base
    p = Params()
    for name, _ in Params._fields_:
        setattr(p, name, kw.get(name, 0))
    return p


def validate_params(p: Params) -> None:
    _check(lib().shadowkv_validate_params(ctypes.byref(p)))


def footprint(p: Params):
    dev, host = ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().shadowkv_footprint(ctypes.byref(p), ctypes.byref(dev), ctypes.byref(host)))
    return dev.value, host.value


def num_kernels() -> int:
    return lib().shadowkv_num_kernels()


def kernel_names():
    return [lib().shadowkv_kernel_name(i).decode() for i in range(num_kernels())]


class Context:
    """Owns a shadowkv_ctx (freed by close() or garbage collection)."""

    def __init__(self, handle: ctypes.c_void_p, params: Params):
        self._h = handle
        self.params = params

    @property
    def handle(self):
        return self._h

    def close(self):
        if self._h:
            lib().shadowkv_free(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def decode_step(self, q, k_new, v_new, out, stream=None):
        _check(lib().shadowkv_decode_step(self._h, _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(out),
                                          _stream(stream)))

    def decode_step_host(self, q, k_new, v_new, out, stream=None):
        """decode_step on host tensors (pinned for asynchronous copies)."""
        _check(lib().shadowkv_decode_step_host(self._h, _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(out),
                                               _stream(stream)))

    def prepared_step(self, q, k_new, v_new, out, stream=None, host=False):
        """A callable that makes the decode_step call (decode_step_host with
        host=True) on these fixed buffers, with the arguments marshalled once
        (a decode loop that reuses its buffers saves that work on every step)."""
        fn = lib().shadowkv_decode_step_host if host else lib().shadowkv_decode_step
        args = (self._h, _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(out), _stream(stream))

        def step():
            rc = fn(*args)
            if rc:
                _check(rc)
        return step

    def rewind(self, stream=None):
        _check(lib().shadowkv_rewind(self._h, _stream(stream)))

    def set_option(self, option: int, value: int):
        _check(lib().shadowkv_set_option(self._h, option, value))

    def stats(self) -> Stats:
        st = Stats()
        _check(lib().shadowkv_get_stats(self._h, ctypes.byref(st)))
        return st

    def check(self):
        _check(lib().shadowkv_check(self._h))

    def layout(self) -> dict:
        lay = Layout()
        _check(lib().shadowkv_get_layout(self._h, ctypes.byref(lay)))
        return {name: bool(getattr(lay, name)) for name, _ in Layout._fields_}

    def kernel_times(self):
        n = num_kernels()
        ms = (ctypes.c_double * n)()
        cnt = (ctypes.c_longlong * n)()
        _check(lib().shadowkv_kernel_times(self._h, ms, cnt, n))
        return {name: (ms[i], cnt[i]) for i, name in enumerate(kernel_names())}

    def reset_timers(self):
        _check(lib().shadowkv_reset_timers(self._h))

    def field_bytes(self, field: str) -> int:
        nb = ctypes.c_size_t()
        _check(lib().shadowkv_field_bytes(self._h, FIELDS[field], ctypes.byref(nb)))
        return nb.value

    def export(self, field: str) -> torch.Tensor:
        """A field copied to a flat CPU tensor (int32, float32, or the context dtype)."""
        nb = self.field_bytes(field)
        if field in _INT_FIELDS:
            dt = torch.int32
        elif field in _F32_FIELDS or self.params.dtype == DTYPE_F32:
            dt = torch.float32
        else:
            dt = torch.bfloat16
        out = torch.empty(nb // torch.tensor([], dtype=dt).element_size(), dtype=dt)
        _check(lib().shadowkv_export(self._h, FIELDS[field], ctypes.c_void_p(out.data_ptr()), nb))
        return out


def prefill(p: Params, k_pre: torch.Tensor, v: torch.Tensor, stream=None) -> Context:
    """Algorithm 1 on device keys k_pre and values v (device or host tensor)."""
    h = ctypes.c_void_p()
    _check(lib().shadowkv_prefill(ctypes.byref(p), _ptr(k_pre), _ptr(v), int(not v.is_cuda),
                                  _stream(stream), ctypes.byref(h)))
    return Context(h, p)


def attention_noalloc(p: Params, q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, out: torch.Tensor,
                      stream=None) -> None:
    """softmax(q K^T / sqrt(d)) V over K, V (b, h_kv, n_tokens, d) on the device,
    with the library's static scratch instead of any allocation."""
    _check(lib().shadowkv_attention_noalloc(ctypes.byref(p), _ptr(q), _ptr(K), _ptr(V),
                                            int(K.shape[2]), _ptr(out), _stream(stream)))


def load_state(p: Params, st: dict, stream=None) -> Context:
    """A context from a given compressed state (keys as in synth.make_state)."""
    s = StateIn(A=_ptr(st["A"]), B=_ptr(st["B"]), L=_ptr(st["L"]),
                outlier_ids=_ptr(st["outlier_ids"]), K_out=_ptr(st["K_out"]),
                V_out=_ptr(st["V_out"]), K_loc=_ptr(st["K_loc"]), V_loc=_ptr(st["V_loc"]),
                V=_ptr(st["v"]), v_on_host=int(not st["v"].is_cuda))
    h = ctypes.c_void_p()
    _check(lib().shadowkv_load_state(ctypes.byref(p), ctypes.byref(s), _stream(stream),
                                     ctypes.byref(h)))
    return Context(h, p)


# ------------------------------------------------------ dense decode path
_DTYPES = {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16}


# The packed forms of Rows and NormRopeParams: the calls of a decode step are
# made every few microseconds, and a ctypes structure takes one to fill.
_PACK_ROWS = struct.Struct("Pqqq").pack
_PACK_NORM_ROPE = struct.Struct("9i2f").pack
_step = None


def _step_calls():
    """The per-step entry points, taking packed structures and raw pointers."""
    global _step
    if _step is None:
        L = lib()
        V, I, S, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
        C = ctypes.POINTER(CacheDesc)
        fns = {}
        for name, args in (("qk_norm_rope", [V] * 9), ("cache_append", [C, I, V, V, I, V, V]),
                           ("cache_attend", [C, I, I, V, F, I, F, V, V, V, S, V]),
                           ("cache_attend_tokens", [C, I, I, I, V, V, I, F, V, V, V, S, V]),
                           ("cache_evict", [C, C, I, I, I, V, V]), ("cache_share", [C, V, I, V, V, V]),
                           ("cache_reserve", [C, V, I, V, V, V, S, V]), ("cache_truncate", [C, V, V, V]),
                           ("cache_compact", [C, V, C, V, V, S, V])):
            fn = L["shadowkv_" + name]      # a function object of its own, beside lib()'s
            fn.restype, fn.argtypes = I, args
            fns[name] = fn
        _step = fns
    return _step


def _rows(t: torch.Tensor, name: str, shape, dtype, device) -> bytes:
    """A b x h x s x d (or b x h x d) tensor as strided rows (a packed Rows)."""
    if t.dtype is dtype and t.shape == shape and t.device == device:
        st = t.stride()
        if st[-1] == 1 or shape[-1] <= 1:
            return _PACK_ROWS(t.data_ptr(), st[0], st[1], st[2] if len(st) == 4 else 0)
        raise ValueError(f"{name}: the last dimension must be contiguous")
    raise ValueError(f"{name} is {t.dtype} {tuple(t.shape)} on {t.device}, expected {dtype} {tuple(shape)} on "
                     f"{device} (shape, type and device)")


def _dense(t: Optional[torch.Tensor], name: str, shape, dtype, device):
    """Data pointer of a contiguous tensor of a given shape, or None."""
    if t is None:
        return None
    if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}, got "
                     f"{t.dtype} {tuple(t.shape)} on {t.device}")


def _dtype(t: torch.Tensor, name: str) -> int:
    dt = _DTYPES.get(t.dtype)
    if dt is None:
        raise ValueError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    return dt


def _torch_fn(name: str, public):
    """torch's own short cut of that name where this build has it, else the public function."""
    return getattr(torch._C, name, None) or public


_current_device = _torch_fn("_cuda_getDevice", torch.cuda.current_device)
_current_stream = _torch_fn("_cuda_getCurrentRawStream", lambda i: torch.cuda.current_stream(i).cuda_stream)
_capturing = _torch_fn("_cuda_isCurrentStreamCapturing", torch.cuda.is_current_stream_capturing)


def _handle(stream) -> int:
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _call(fn, t, stream, *args) -> None:
    """fn(*args, cudaStream_t) with tensor t's device current; stream None:
    torch's current stream of that device."""
    if not t.is_cuda:
        raise ValueError(f"tensors must be on a CUDA device, got {t.device}")
    i = t.get_device()
    st = _current_stream(i) if stream is None else _handle(stream)
    if i == _current_device():
        rc = fn(*args, st)
    else:
        with torch.cuda.device(i):
            rc = fn(*args, st)
    if rc:
        _check(rc)


def _on_stream(stream, device):
    """A context in which `stream`, torch's or a raw cudaStream_t, is torch's current stream."""
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(_handle(stream), device)
    return torch.cuda.stream(stream)


def qk_norm_rope(q: Optional[torch.Tensor], k: Optional[torch.Tensor], q_weight: Optional[torch.Tensor] = None,
                 k_weight: Optional[torch.Tensor] = None, *, eps: float = 1e-6, norm: bool = True,
                 theta: float = 1e4, rot: Optional[int] = None, pos: Optional[torch.Tensor] = None,
                 q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None, stream=None):
    """Norm of every query and key head and its rotation to the token's position.

    q (b, h_q, s, d) and k (b, h_kv, s, d), float32 or bfloat16, d contiguous, the
    other strides (and the outputs') multiples of 4 elements; either may be None.  The weights have d elements.  pos: int32, (b,)
    first positions or (b, s), or None for 0..s-1.  rot: rotated dimensions
    (default d; 0: none).  The outputs are made like the inputs, contiguous,
    unless given; returns (q_out, k_out)."""
    x = q if q is not None else k
    if x is None:
        raise ValueError("q and k are both None")
    if (stream is not None and x.is_cuda and (q is not None and q_out is None or k is not None and k_out is None)
            and _handle(stream) != _current_stream(x.get_device())):
        # the outputs are allocated on the stream that writes them
        with _on_stream(stream, x.device):
            return qk_norm_rope(q, k, q_weight, k_weight, eps=eps, norm=norm, theta=theta, rot=rot, pos=pos,
                                q_out=q_out, k_out=k_out)
    if x.dim() != 4 or (k is not None and k.dim() != 4):
        raise ValueError("q and k must be (b, h, s, d)")
    (b, _, s, d), dev, dtype = x.shape, x.device, x.dtype
    dt = _dtype(x, "q" if q is not None else "k")
    hq = hk = 0
    rq = rk = oq = ok = wq = wk = None
    if q is not None:
        shape = q.shape
        hq = shape[1]
        if q_out is None:
            q_out = torch.empty(shape, dtype=dtype, device=dev)
        rq, oq = _rows(q, "q", shape, dtype, dev), _rows(q_out, "q_out", shape, dtype, dev)
        if q_weight is not None:
            wq = _dense(q_weight, "q_weight", (d,), dtype, dev)
    elif q_weight is not None or q_out is not None:
        raise ValueError("q is None, its weight or output is not")
    if k is not None:
        hk = k.shape[1]
        shape = (b, hk, s, d)
        if k_out is None:
            k_out = torch.empty(shape, dtype=dtype, device=dev)
        rk, ok = _rows(k, "k", shape, dtype, dev), _rows(k_out, "k_out", shape, dtype, dev)
        if k_weight is not None:
            wk = _dense(k_weight, "k_weight", (d,), dtype, dev)
    elif k_weight is not None or k_out is not None:
        raise ValueError("k is None, its weight or output is not")
    per_token, pp = False, None
    if pos is not None:
        per_token = pos.dim() == 2
        pp = _dense(pos, "pos", (b, s) if per_token else (b,), torch.int32, dev)
    p = _PACK_NORM_ROPE(b, s, hq, hk, d, d if rot is None else rot, dt, norm, per_token, eps, theta)
    _call((_step or _step_calls())["qk_norm_rope"], x, stream, p, rq, rk, wq, wk, pp, oq, ok)
    return q_out, k_out


def _stacked(t: torch.Tensor, name: str, shape, dtype, device):
    """(pointer, stride of sequences, stride of positions) of a b x s x n tensor, its n elements adjacent."""
    if t.dtype is dtype and t.shape == shape and t.device == device:
        st = t.stride()
        if st[2] == 1 or shape[2] <= 1:
            return t.data_ptr(), st[0], st[1]
        raise ValueError(f"{name}: the last dimension must be contiguous")
    raise ValueError(f"{name} is {t.dtype} {tuple(t.shape)} on {t.device}, expected {dtype} {tuple(shape)} on "
                     f"{device} (shape, type and device)")


def verify_drafts(logits: torch.Tensor, drafts: torch.Tensor, probs: Optional[torch.Tensor], accept: torch.Tensor,
                  sample: torch.Tensor, *, lens: Optional[torch.Tensor] = None, temperature=1.0,
                  tokens: Optional[torch.Tensor] = None, accepted: Optional[torch.Tensor] = None, stream=None):
    """How many drafted tokens stand, and the token that follows them, from given random
    numbers (speculative sampling; shadowkv_verify_drafts).

    logits (b, s + 1, vocab) float32 or bfloat16, the target's after 0..s drafts; drafts (b, s) int32;
    probs (b, s, vocab) float32, what the drafts were sampled from, or None for
    drafts that were looked up (the last dimension of both contiguous, the others of any stride); accept (b, s)
    and sample (b,) float32 in [0, 1); lens (b,) int32: drafts of each sequence; temperature: a number or (b,)
    float32, 0: greedy.  Returns tokens (b, s + 1) int32 (the drafts that stand, the
    next token, then -1) and accepted (b,) int32."""
    if not logits.is_cuda:
        raise ValueError(f"tensors must be on a CUDA device, got {logits.device}")
    dev = logits.device
    if stream is not None and _handle(stream) != _current_stream(dev.index):
        # the outputs and the workspace are allocated on the stream that uses them
        with _on_stream(stream, dev):
            return verify_drafts(logits, drafts, probs, accept, sample, lens=lens, temperature=temperature, tokens=tokens,
                                 accepted=accepted)
    if logits.dim() != 3 or drafts.dim() != 2 or logits.shape[1] < 1:
        raise ValueError("logits must be (b, s + 1, vocab) and drafts (b, s)")
    b, s, v = logits.shape[0], logits.shape[1] - 1, logits.shape[2]
    dt = _dtype(logits, "logits")
    lp, lb, ls = _stacked(logits, "logits", (b, s + 1, v), logits.dtype, dev)
    pp, pb, ps = (None, 0, 0) if probs is None else _stacked(probs, "probs", (b, s, v), torch.float32, dev)
    dp, ap = _dense(drafts, "drafts", (b, s), torch.int32, dev), _dense(accept, "accept", (b, s), torch.float32, dev)
    sp, np_ = _dense(sample, "sample", (b,), torch.float32, dev), _dense(lens, "lens", (b,), torch.int32, dev)
    tp, t = None, 0.0
    if isinstance(temperature, torch.Tensor):
        tp = _dense(temperature, "temperature", (b,), torch.float32, dev)
    else:
        t = float(temperature)
    if tokens is None:
        tokens = torch.empty((b, s + 1), dtype=torch.int32, device=dev)
    if accepted is None:
        accepted = torch.empty(b, dtype=torch.int32, device=dev)
    to, ao = _dense(tokens, "tokens", (b, s + 1), torch.int32, dev), _dense(accepted, "accepted", (b,), torch.int32, dev)
    p = VerifyParams(b, s, v, dt, t, lb, ls, pb, ps)
    nb = lib().shadowkv_verify_workspace(p)
    if nb == 0:
        _check(1)
    work = torch.empty(nb, dtype=torch.uint8, device=dev)
    _call(lib().shadowkv_verify_drafts, logits, None, p, lp, dp, pp, ap, sp, np_, tp, to, ao, work.data_ptr(), nb)
    return tokens, accepted


class BlockCache:
    """A dense key/value cache in e4m3 with a scale per block of tokens and head
    (shadowkv_cache), on tensors it only names:

      k_codes (n_pool, block/8, d/16, 8, 16), v_codes (n_pool, block/16, d, 16)
                                    8-bit (float8_e4m3fn or uint8)
      k_scale, v_scale (n_pool,)    float32
      table (b, h_kv, max_blocks)   int32: the pool block of each pair's blocks
      n_tok (b, h_kv)               int32: tokens held
      weight (b, h_kv, max_blocks)  float32: attention weight gathered per block, or None
      refs (n_pool,)                int32: the table entries that name each pool block, for a pool
                                    that sequences share (its tables hold -1 for no block), or None

    Copies and checkpoints are copies of these tensors.  The calls use the memory
    the tensors had at the start, so the attributes cannot be given other tensors:
    copy into them, or make another cache.  Calls on one cache
    must be ordered on one stream (or by events), from any threads."""

    _MEMORY = frozenset(("k_codes", "v_codes", "k_scale", "v_scale", "table", "n_tok", "weight", "refs", "status"))

    def __setattr__(self, name, value):
        if name in self._MEMORY and self.__dict__.get(name, value) is not value:
            raise AttributeError(f"{name} names the cache's memory: copy into it, or make another BlockCache")
        super().__setattr__(name, value)

    def __init__(self, k_codes, v_codes, k_scale, v_scale, table, n_tok, weight=None, refs=None):
        if k_codes.dim() != 5 or v_codes.dim() != 4 or table.dim() != 3:
            raise ValueError("k_codes must have 5 dimensions, v_codes 4 and table 3")
        n_pool, b8, d16, _, _ = k_codes.shape
        block, d = 8 * b8, 16 * d16
        b, h, mb = table.shape
        dev = table.device
        for name, t, shape in (("k_codes", k_codes, (n_pool, b8, d16, 8, 16)),
                               ("v_codes", v_codes, (n_pool, block // 16, d, 16))):
            if t.element_size() != 1:
                raise ValueError(f"{name} must hold 8-bit codes, got {t.dtype}")
            _dense(t, name, shape, t.dtype, dev)
        for name, t, shape, dt in (("k_scale", k_scale, (n_pool,), torch.float32),
                                   ("v_scale", v_scale, (n_pool,), torch.float32),
                                   ("table", table, (b, h, mb), torch.int32), ("n_tok", n_tok, (b, h), torch.int32),
                                   ("weight", weight, (b, h, mb), torch.float32),
                                   ("refs", refs, (n_pool,), torch.int32)):
            _dense(t, name, shape, dt, dev)
        self.k_codes, self.v_codes, self.k_scale, self.v_scale = k_codes, v_codes, k_scale, v_scale
        self.table, self.n_tok, self.weight, self.refs = table, n_tok, weight, refs
        self.b, self.h_kv, self.d, self.block, self.max_blocks, self.device = b, h, d, block, mb, dev
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self._desc = CacheDesc(b, h, d, block, mb, n_pool, k_codes.data_ptr(), v_codes.data_ptr(),
                               k_scale.data_ptr(), v_scale.data_ptr(), table.data_ptr(), n_tok.data_ptr(),
                               weight.data_ptr() if weight is not None else None, self.status.data_ptr())
        self._work, self._work_lock = {}, threading.Lock()
        _check(lib().shadowkv_cache_validate(self._desc))

    @classmethod
    def empty(cls, b: int, h_kv: int, d: int, max_blocks: int, block: int = 64, device="cuda"):
        """A cache without tokens, every pair with max_blocks pool blocks of its own."""
        dev = torch.device(device)
        n = b * h_kv * max_blocks
        z = lambda *shape, dtype=torch.float32: torch.zeros(*shape, dtype=dtype, device=dev)  # noqa: E731
        return cls(z(n, block // 8, d // 16, 8, 16, dtype=torch.uint8), z(n, block // 16, d, 16, dtype=torch.uint8),
                   z(n), z(n), torch.arange(n, dtype=torch.int32, device=dev).view(b, h_kv, max_blocks),
                   z(b, h_kv, dtype=torch.int32), z(b, h_kv, max_blocks))

    @classmethod
    def pooled(cls, b: int, h_kv: int, d: int, max_blocks: int, n_pool: int, block: int = 64, device="cuda"):
        """A cache without tokens over a pool of n_pool free blocks that its sequences share."""
        dev = torch.device(device)
        z = lambda *shape, dtype=torch.float32: torch.zeros(*shape, dtype=dtype, device=dev)  # noqa: E731
        return cls(z(n_pool, block // 8, d // 16, 8, 16, dtype=torch.uint8),
                   z(n_pool, block // 16, d, 16, dtype=torch.uint8), z(n_pool), z(n_pool),
                   torch.full((b, h_kv, max_blocks), -1, dtype=torch.int32, device=dev), z(b, h_kv, dtype=torch.int32),
                   z(b, h_kv, max_blocks), z(n_pool, dtype=torch.int32))

    def fork(self) -> "BlockCache":
        """A cache with tables, counts and weights of its own over the same pool.
        Blocks the two share must not be appended to.  (Not for a pool with reference
        counts: share() forks its sequences.)"""
        if self.refs is not None:
            raise ValueError("the pool's references count one cache's tables: fork sequences with share()")
        return BlockCache(self.k_codes, self.v_codes, self.k_scale, self.v_scale, self.table.clone(),
                          self.n_tok.clone(), None if self.weight is None else self.weight.clone())

    def append(self, k: torch.Tensor, v: torch.Tensor, lens: Optional[torch.Tensor] = None, stream=None) -> None:
        """Appends s tokens to every pair: k, v (b, h_kv, s, d), d contiguous, the
        other strides multiples of 16 bytes; lens (b,) int32: tokens of each sequence (default all s)."""
        if k.dim() != 4:
            raise ValueError("k and v must be (b, h_kv, s, d)")
        s = k.shape[2]
        dt = _dtype(k, "k")
        shape = (self.b, self.h_kv, s, self.d)
        rk, rv = _rows(k, "k", shape, k.dtype, self.device), _rows(v, "v", shape, k.dtype, self.device)
        lp = _dense(lens, "lens", (self.b,), torch.int32, self.device)
        _call((_step or _step_calls())["cache_append"], self.n_tok, stream, self._desc, dt, rk, rv, s, lp)

    def attend(self, q: torch.Tensor, *, scale: Optional[float] = None, decay: Optional[float] = None,
               out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """softmax(scale q K^T) V over the tokens held; q (b, h_q, d), scale 1/sqrt(d)
        by default.  decay: gather block weights, weight = decay weight + this
        call's (None: weights stay as they are).  lse (b, h_q) float32 receives the log sums.
        The workspace comes from torch's allocator and is kept per stream (threads
        that share a stream share it: their calls run one after the other there); a call
        under capture takes one of its own from the graph's memory, so that
        graphs share none."""
        if q.dim() != 3:
            raise ValueError("q must be (b, h_q, d)")
        dev, hq, dtype = self.device, q.shape[1], q.dtype
        dt = _dtype(q, "q")
        shape = (self.b, hq, self.d)
        rq = _rows(q, "q", shape, dtype, dev)
        lp = None if lse is None else _dense(lse, "lse", (self.b, hq), torch.float32, dev)
        if dev.type != "cuda":
            raise ValueError(f"tensors must be on a CUDA device, got {dev}")
        if stream is not None:
            # the output and the workspace are allocated on the stream that uses them
            with _on_stream(stream, dev):
                return self.attend(q, scale=scale, decay=decay, out=out, lse=lse)
        i = dev.index
        if _current_device() != i:
            with torch.cuda.device(dev):
                return self.attend(q, scale=scale, decay=decay, out=out, lse=lse)
        if out is None:
            out = torch.empty(shape, dtype=dtype, device=dev)
        ro = _rows(out, "out", shape, dtype, dev)
        st = _current_stream(i)
        _, ptr, nb = self._workspace(hq, st)
        rc = (_step or _step_calls())["cache_attend"](
            self._desc, dt, hq, rq, self.d ** -0.5 if scale is None else scale, decay is not None,
            0.0 if decay is None else decay, ro, lp, ptr, nb, st)
        if rc:
            _check(rc)
        return out

    def _workspace(self, hq: int, st: int):
        """(tensor, pointer, bytes) of attend's workspace on the current stream st."""
        capturing = _capturing()
        have = None if capturing else self._work.get((hq, st))
        if have is None:
            nb = lib().shadowkv_cache_attend_workspace(self._desc, hq)
            if nb == 0:
                _check(7)
            t = torch.empty(nb, dtype=torch.uint8, device=self.device)
            have = (t, t.data_ptr(), nb)
            if not capturing:
                with self._work_lock:
                    if len(self._work) >= 8:
                        self._work.pop(next(iter(self._work)))
                    self._work[(hq, st)] = have
        return have

    def attend_tokens(self, q: torch.Tensor, *, lens: Optional[torch.Tensor] = None, causal: bool = True,
                      scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                      lse: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """softmax(scale q K^T) V of several tokens per sequence; q (b, h_q, s, d), the last dimension
        contiguous, scale 1/sqrt(d) by default.  causal: the queries are the last tokens held (append
        them first), and each sees the tokens up to its own; else every query sees every token (an encoder's
        states).  lens (b,) int32: queries of each sequence (default s); rows past them are left as they
        were (zeros in an output made here).  lse (b, h_q, s) float32 receives the log sums.  The workspace
        comes from torch's allocator, for each call."""
        if q.dim() != 4:
            raise ValueError("q must be (b, h_q, s, d)")
        dev, dtype = self.device, q.dtype
        dt = _dtype(q, "q")
        hq, s = q.shape[1], q.shape[2]
        shape = (self.b, hq, s, self.d)
        rq = _rows(q, "q", shape, dtype, dev)
        lp = _dense(lens, "lens", (self.b,), torch.int32, dev)
        sp = _dense(lse, "lse", (self.b, hq, s), torch.float32, dev)
        if dev.type != "cuda":
            raise ValueError(f"tensors must be on a CUDA device, got {dev}")
        if stream is not None and _handle(stream) != _current_stream(dev.index):
            # the output and the workspace are allocated on the stream that uses them
            with _on_stream(stream, dev):
                return self.attend_tokens(q, lens=lens, causal=causal, scale=scale, out=out, lse=lse)
        if _current_device() != dev.index:      # the workspace's size goes by the device
            with torch.cuda.device(dev):
                return self.attend_tokens(q, lens=lens, causal=causal, scale=scale, out=out, lse=lse)
        if out is None:
            out = (torch.empty if lens is None else torch.zeros)(shape, dtype=dtype, device=dev)
        ro = _rows(out, "out", shape, dtype, dev)
        work = self._scratch(lib().shadowkv_cache_attend_tokens_workspace(self._desc, hq, s))
        _call((_step or _step_calls())["cache_attend_tokens"], q, None, self._desc, dt, hq, s, rq, lp, bool(causal),
              self.d ** -0.5 if scale is None else scale, ro, sp, work.data_ptr(), work.numel())
        return out

    def evict(self, keep: int, *, sink: int = 0, recent: int = 1, into: Optional["BlockCache"] = None,
              kept: Optional[torch.Tensor] = None, stream=None) -> None:
        """Keeps at most `keep` blocks of every pair: the first `sink`, the last
        `recent` and those of largest weight.  into: a cache of the same sizes
        that takes the table, counts and weights (default: in place).  kept (b, h_kv, keep) int32
        receives the old index of each block still held, then -1."""
        kp = _dense(kept, "kept", (self.b, self.h_kv, keep), torch.int32, self.device)
        if into is not None and into is not self and (self.refs is not None or into.refs is not None):
            raise ValueError("the pool's references count one cache's tables: evict in place")
        dst = None if into is None else into._desc
        if into is not None and into.device != self.device:
            raise ValueError(f"into is on {into.device}, expected {self.device}")
        _call((_step or _step_calls())["cache_evict"], self.n_tok, stream, self._desc, dst, keep, sink, recent, kp)

    def _counts(self) -> torch.Tensor:
        if self.refs is None:
            raise ValueError("the cache's pool keeps no reference counts (refs)")
        return self.refs

    def share(self, src: torch.Tensor, dst: torch.Tensor, stream=None) -> None:
        """Forks: sequence dst[k] becomes a copy of sequence src[k] that names the same
        blocks; src, dst (n,) int32.  A dst that is any source, or named twice,
        is left out and recorded (check())."""
        refs, n = self._counts(), src.numel()
        sp, dp = _dense(src, "src", (n,), torch.int32, self.device), _dense(dst, "dst", (n,), torch.int32, self.device)
        _call((_step or _step_calls())["cache_share"], self.n_tok, stream, self._desc, refs.data_ptr(), n, sp, dp)

    def reserve(self, s: int, lens: Optional[torch.Tensor] = None, granted: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
        """Room for an append of s tokens to every sequence (lens (b,) int32: of each): the blocks it
        writes to, and partly filled ones in any case, become the pairs' own, free ones or copies.  Returns granted (b,) int32: lens
        where the pool had the blocks, else 0, to append with."""
        refs = self._counts()
        if s >= 1 << 31:    # (it goes on as 32 bits)
            raise ValueError(f"s must be below 2^31, got {s}")
        lp = _dense(lens, "lens", (self.b,), torch.int32, self.device)
        if self.device.type != "cuda":
            raise ValueError(f"tensors must be on a CUDA device, got {self.device}")
        if stream is not None and _handle(stream) != _current_stream(self.device.index):
            # the output and the workspace are allocated on the stream that uses them
            with _on_stream(stream, self.device):
                return self.reserve(s, lens, granted)
        if granted is None:
            granted = torch.empty(self.b, dtype=torch.int32, device=self.device)
        gp = _dense(granted, "granted", (self.b,), torch.int32, self.device)
        work = self._scratch(lib().shadowkv_cache_reserve_workspace(self._desc, s))
        _call((_step or _step_calls())["cache_reserve"], self.n_tok, None, self._desc, refs.data_ptr(), s, lp, gp,
              work.data_ptr(), work.numel())
        return granted

    def truncate(self, drop: Optional[torch.Tensor] = None, stream=None) -> None:
        """Takes drop[i] tokens (drop (b,) int32, default none) off the end of every sequence i; blocks past the
        tokens go back to a shared pool.  A block that keeps some of its tokens keeps the scales and the
        weight that the others gave it; share() to a spare sequence before their append, and back, leaves no trace."""
        dp = _dense(drop, "drop", (self.b,), torch.int32, self.device)
        _call((_step or _step_calls())["cache_truncate"], self.n_tok, stream, self._desc,
              None if self.refs is None else self.refs.data_ptr(), dp)

    def compact(self, into: "BlockCache", stream=None) -> None:
        """Moves the cache to `into`, a cache of the same sizes over a pool of another size:
        the blocks in use become its blocks 0, 1, ...; self stays as it is."""
        refs, to = self._counts(), into._counts()
        if into.device != self.device:
            raise ValueError(f"into is on {into.device}, expected {self.device}")
        if self.device.type != "cuda":
            raise ValueError(f"tensors must be on a CUDA device, got {self.device}")
        if stream is not None and _handle(stream) != _current_stream(self.device.index):
            with _on_stream(stream, self.device):   # for the workspace
                return self.compact(into)
        work = self._scratch(lib().shadowkv_cache_compact_workspace(self._desc))
        _call((_step or _step_calls())["cache_compact"], self.n_tok, None, self._desc, refs.data_ptr(), into._desc,
              to.data_ptr(), work.data_ptr(), work.numel())

    def _scratch(self, nb: int) -> torch.Tensor:
        """A workspace from torch's allocator, for one call on the current stream."""
        if nb == 0:
            _check(7)
        return torch.empty(nb, dtype=torch.uint8, device=self.device)

    def reset(self) -> None:
        """Drops every token (on torch's current stream)."""
        if self.refs is not None:
            self.truncate(torch.full((self.b,), 2**31 - 1, dtype=torch.int32, device=self.device))
            return
        self.n_tok.zero_()

    def check(self) -> None:
        """Waits for the device; raises if a call met a bad block id, length or count."""
        with torch.cuda.device(self.device):
            _check(lib().shadowkv_cache_check(self._desc))
