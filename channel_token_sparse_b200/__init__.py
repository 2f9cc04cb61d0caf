"""B200-native Double Sparsity decode attention.

Thin ctypes binding over ``libds.so`` (C ABI declared in ``include/ds.h``).
This module only marshals arguments: every step runs in the library's CUDA
kernels. PyTorch supplies device memory and the current stream.

There is no fallback: importing works without a GPU (so the ABI can be
inspected), but calling an entry point needs ``libds.so`` (``build()``) and a
CUDA device, and raises otherwise.

Layouts (see include/ds.h): q [B, Hq, D]; k, v [B, Hkv, S_cap, D];
idx [Hkv, C] int32; label [B, Hkv, S_cap, C] (dtype of k) or, 4-bit,
[B, Hkv, S_cap, C/2] uint8 with fp16 lscale / lzero [B, Hkv, S_cap].
"""

from __future__ import annotations

import ctypes as C
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libds.so")

DS_OK, DS_ERR_INVALID_ARG, DS_ERR_UNSUPPORTED, DS_ERR_CUDA, DS_ERR_WORKSPACE, DS_ERR_TIMEOUT = range(6)
DS_F32, DS_BF16, DS_F16, DS_INT4, DS_E4M3 = range(5)
DS_ROPE_HALF, DS_ROPE_INTERLEAVED = range(2)
DS_FALLBACK_PER_ENTRY, DS_FALLBACK_BATCH = range(2)
DS_CRIT_LEANK_RATIO, DS_CRIT_Q_OUTLIER, DS_CRIT_K_OUTLIER, DS_CRIT_QK_OUTLIER, DS_CRIT_QK_CHUNKED = range(5)

# every C-ABI entry point: name -> (restype, argtypes)
_vp, _i, _f, _sz, _ll = C.c_void_p, C.c_int, C.c_float, C.c_size_t, C.c_longlong
SIGNATURES = {
    "ds_status_string": (C.c_char_p, [_i]),
    "ds_last_error": (C.c_char_p, []),
    "ds_calibrate_workspace_size": (_i, [_i, _i, _i, _i, _i, _i, C.POINTER(_sz)]),
    "ds_calibrate_channels": (_i, [_vp, _vp, _i, _i, _i, _i, _i, _i, _i, _i, _vp, _vp, _vp, _sz, _vp]),
    "ds_calibrate_channels_noalloc": (_i, [_vp, _vp, _i, _i, _i, _i, _i, _i, _i, _i, _vp, _vp, _vp]),
    "ds_decode_step_kv": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _vp, _i, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i,
                               _i, _f, _vp, _i, _vp, _vp, _vp]),
    "ds_build_label_cache_paged": (_i, [_vp, _i, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _i, _i, _vp, _i, _vp,
                                        _vp, _vp]),
    "ds_decode_step_paged": (_i, [_vp, _vp, _vp, _i, _vp, _i, _vp, _vp, _vp, _vp, _i, _i, _i, _vp, _i, _i, _i,
                                  _i, _i, _i, _i, _i, _i, _i, _f, _vp, _i, _vp, _vp, _vp]),
    "ds_calibrate_channels_criterion": (_i, [_vp, _vp, _i, _i, _i, _i, _i, _i, _i, _i, _i, _i, _vp, _vp,
                                             _vp, _sz, _vp]),
    "ds_build_label_cache": (_i, [_vp, _i, _vp, _i, _i, _i, _i, _i, _i, _vp, _i, _vp, _vp, _vp]),
    "ds_append_label": (_i, [_vp, _i, _vp, _i, _i, _i, _i, _i, _i, _vp, _i, _vp, _vp, _vp]),
    "ds_sparse_decode": (_i, [_vp, _vp, _vp, _i, _vp, _i, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _i,
                              _f, _vp, _i, _vp, _vp, _vp]),
    "ds_decode_step": (_i, [_vp, _vp, _vp, _i, _vp, _i, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _i,
                            _f, _vp, _i, _vp, _vp, _vp]),
    "ds_decode_step_varlen": (_i, [_vp, _vp, _vp, _i, _vp, _i, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i,
                                   _i, _i, _i, _f, _vp, _i, _vp, _vp, _vp]),
    "ds_sparse_decode_plan": (_i, [_i, _i, _i, _i, _i, _i, _i, _i, _i, C.POINTER(_i), C.POINTER(_i),
                                   C.POINTER(_i)]),
    "ds_sparse_decode_set_cluster": (None, [_i]),
    "ds_sparse_decode_tune": (_i, [C.c_char_p, _i]),
    "ds_check_device": (_i, [_vp]),
    "ds_selftest_bounded_wait": (_i, [_i, _vp]),
    "ds_sparse_decode_workspace": (_i, [_i, _i, _i, _i, _i, _i, _i, C.POINTER(_sz)]),
    "ds_write_kv": (_i, [_vp, _ll, _ll, _vp, _ll, _ll, _vp, _ll, _ll, _i, _vp, _vp, _f, _vp, _i, _i, _vp, _vp, _vp,
                         _i, _i, _i, _i, _i, _i, _vp, _vp, _vp, _i, _vp, _vp, _vp]),
    "ds_write_kv_paged": (_i, [_vp, _ll, _ll, _vp, _ll, _ll, _vp, _ll, _ll, _i, _vp, _vp, _f, _vp, _i, _i, _vp, _vp,
                               _vp, _i, _i, _i, _i, _i, _vp, _vp, _vp, _i, _vp, _vp, _vp, _i, _i, _i, _vp]),
    "ds_read_kv": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, _vp, _i, _i, _vp]),
    "ds_read_kv_paged": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _vp, _i, _i, _i, _i, _vp, _vp, _i, _i, _vp]),
    "ds_tree_decode_workspace_size": (_i, [_i, _i, _i, _i, _i, _i, _i, C.POINTER(_sz)]),
    "ds_tree_decode": (_i, [_vp, _vp, _vp, _i, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _f, _vp, _i, _vp,
                            _sz, _vp]),
    "ds_tree_decode_paged": (_i, [_vp, _vp, _vp, _i, _vp, _vp, _vp, _vp, _i, _i, _i, _vp, _vp, _i, _i, _i, _i, _i, _i,
                                  _f, _vp, _i, _vp, _sz, _vp]),
    "ds_dense_decode": (_i, [_vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _f, _vp, _i, _vp]),
}

_lib = None


class DSError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{status_string(status) if _lib else status}: {msg}")
        self.status = status


def build(force: bool = False) -> str:
    """Compile libds.so for sm_100a (nvcc) if it is missing or stale."""
    from . import buildlib as _b
    return _b.build(force=force)


def lib():
    """The loaded libds.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: run channel_token_sparse_b200.build() first")
        _lib = C.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(_lib, name)
            fn.restype = res
            fn.argtypes = args
    return _lib


def status_string(st: int) -> str:
    return lib().ds_status_string(st).decode()


def last_error() -> str:
    return lib().ds_last_error().decode()


def _check(st: int):
    if st != DS_OK:
        raise DSError(st, last_error())


# ------------------------------------------------------------------ helpers

def _torch():
    import torch
    return torch


def _ptr(t):
    return None if t is None else C.c_void_p(t.data_ptr())


_mapped = {}  # host address of a pinned tensor -> its device-mapped address


def _ptr_kv(t):
    """Device address of a tensor the kernels may read (or write) over the
    host link: a CUDA tensor, or a pinned host tensor mapped into the
    device's address space (DS-Offload keeps K/V there; a decode step may also
    take its new rows and query from there and write its output there)."""
    if t is None:
        return None
    if t.is_cuda:
        return C.c_void_p(t.data_ptr())
    if not t.is_pinned():
        raise ValueError("a tensor in host memory must be pinned")
    hp = t.data_ptr()
    dp = _mapped.get(hp)
    if dp is None:
        from cuda.bindings import runtime as rt
        err, dp = rt.cudaHostGetDevicePointer(hp, 0)
        if err != rt.cudaError_t.cudaSuccess:
            raise ValueError(f"pinned host tensor is not mapped for the device: {err}")
        dp = int(dp)
        if len(_mapped) > 4096:
            _mapped.clear()
        _mapped[hp] = dp
    return C.c_void_p(dp)


def _need_cuda_or_pinned(*ts):
    for t in ts:
        if not (t.is_cuda or t.is_pinned()):
            raise ValueError("key/value caches must be CUDA tensors or pinned host tensors")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")


def _stream(stream=None):
    torch = _torch()
    s = torch.cuda.current_stream() if stream is None else stream
    return C.c_void_p(s.cuda_stream)


def _kv_dtype(t) -> int:
    torch = _torch()
    if t.dtype == torch.float32:
        return DS_F32
    if t.dtype == torch.bfloat16:
        return DS_BF16
    raise TypeError(f"unsupported k/v dtype {t.dtype}")


def _need_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("tensors must be CUDA tensors")
        if t is not None and not t.is_contiguous():
            raise ValueError("tensors must be contiguous")


def set_cluster(n: int) -> None:
    """Force CTAs per (b, kv head) cluster (1..16, power of two); 0 = automatic."""
    lib().ds_sparse_decode_set_cluster(int(n))


def check_device(stream=None) -> None:
    """Raise DSError(DS_ERR_TIMEOUT) if a kernel gave up a bounded wait since
    the last check (synchronises the stream)."""
    _check(lib().ds_check_device(_stream(stream)))


def tune(name: str, value: int) -> None:
    """Set a decode tuning knob ("scan_prefetch", "i4_ring");
    a negative value restores its default."""
    _check(lib().ds_sparse_decode_tune(name.encode(), int(value)))


def plan(b, hq, hkv, s, d, c, topk, kv_dtype=DS_BF16, label_dtype=DS_BF16):
    """(cluster size, tokens per CTA, shared memory bytes) of ds_sparse_decode."""
    n, ch, sm = C.c_int(), C.c_int(), C.c_int()
    _check(lib().ds_sparse_decode_plan(b, hq, hkv, s, d, c, topk, kv_dtype, label_dtype,
                                       C.byref(n), C.byref(ch), C.byref(sm)))
    return n.value, ch.value, sm.value


def sparse_decode_workspace(b, hq, hkv, s, d, c, topk) -> int:
    """Device scratch bytes ds_sparse_decode needs for a shape (0: on chip)."""
    out = C.c_size_t()
    _check(lib().ds_sparse_decode_workspace(b, hq, hkv, s, d, c, topk, C.byref(out)))
    return out.value


# -------------------------------------------------------------- entry points

def calibrate_workspace_size(n, hq, hkv, w, s, d) -> int:
    out = C.c_size_t()
    _check(lib().ds_calibrate_workspace_size(n, hq, hkv, w, s, d, C.byref(out)))
    return out.value


def calibrate_channels(q_win, k, c: int, ratio_out=None, idx_out=None, ws=None, stream=None):
    """Heavy channels idx [Hkv, C] (and ratio r [Hkv, D]) from q_win [N, Hq, W, D],
    k [N, Hkv, S, D]. Returns (idx, ratio)."""
    torch = _torch()
    _need_cuda(q_win, k)
    n, hq, w, d = q_win.shape
    _, hkv, s, _ = k.shape
    if idx_out is None:
        idx_out = torch.empty((hkv, c), dtype=torch.int32, device=k.device)
    if ratio_out is None:
        ratio_out = torch.empty((hkv, d), dtype=torch.float32, device=k.device)
    nbytes = calibrate_workspace_size(n, hq, hkv, w, s, d)
    if ws is None:
        ws = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=k.device)
    _check(lib().ds_calibrate_channels(_ptr(q_win), _ptr(k), _kv_dtype(k), n, hq, hkv, w, s, d, c,
                                       _ptr(ratio_out), _ptr(idx_out), _ptr(ws), ws.numel(),
                                       _stream(stream)))
    return idx_out, ratio_out


def calibrate_channels_criterion(q_win, k, c: int, criterion: int, chunk: int = 0, score_out=None,
                                 idx_out=None, ws=None, stream=None):
    """Heavy channels ranked by one of the DS_CRIT_* criteria. Returns (idx, score)."""
    torch = _torch()
    _need_cuda(q_win, k)
    n, hq, w, d = q_win.shape
    _, hkv, s, _ = k.shape
    if idx_out is None:
        idx_out = torch.empty((hkv, c), dtype=torch.int32, device=k.device)
    if score_out is None:
        score_out = torch.empty((hkv, d), dtype=torch.float32, device=k.device)
    nbytes = calibrate_workspace_size(n, hq, hkv, w, s, d)
    if ws is None:
        ws = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=k.device)
    _check(lib().ds_calibrate_channels_criterion(_ptr(q_win), _ptr(k), _kv_dtype(k), n, hq, hkv, w, s, d,
                                                 c, int(criterion), int(chunk), _ptr(score_out),
                                                 _ptr(idx_out), _ptr(ws), ws.numel(), _stream(stream)))
    return idx_out, score_out


def calibrate_channels_noalloc(q_win, k, c: int, ratio_out, idx_out, stream=None):
    """ds_calibrate_channels with the library's fixed scratch instead of a
    workspace (for callers that cannot allocate device memory); the outputs
    must be provided."""
    _need_cuda(q_win, k, ratio_out, idx_out)
    n, hq, w, d = q_win.shape
    _, hkv, s, _ = k.shape
    _check(lib().ds_calibrate_channels_noalloc(_ptr(q_win), _ptr(k), _kv_dtype(k), n, hq, hkv, w, s, d, c,
                                               _ptr(ratio_out), _ptr(idx_out), _stream(stream)))
    return idx_out, ratio_out


def _label_args(label, lscale, lzero, kdt):
    torch = _torch()
    if label.dtype == torch.uint8:
        if lscale is None or lzero is None:
            raise ValueError("4-bit label needs lscale and lzero")
        return DS_INT4
    return kdt


def build_label_cache(k, idx, s: int, label, lscale=None, lzero=None, stream=None):
    """Fill label rows [0, s) from the key cache k [B, Hkv, S_cap, D] (device,
    or pinned host memory)."""
    _need_cuda_or_pinned(k)
    _need_cuda(idx, label, lscale, lzero)
    b, hkv, s_cap, d = k.shape
    c = idx.shape[1]
    kdt = _kv_dtype(k)
    _check(lib().ds_build_label_cache(_ptr_kv(k), kdt, _ptr(idx), b, hkv, s, s_cap, d, c, _ptr(label),
                                      _label_args(label, lscale, lzero, kdt), _ptr(lscale),
                                      _ptr(lzero), _stream(stream)))


def append_label(k, idx, pos: int, label, lscale=None, lzero=None, stream=None):
    """Fill label row `pos` from k[:, :, pos]."""
    _need_cuda_or_pinned(k)
    _need_cuda(idx, label, lscale, lzero)
    b, hkv, s_cap, d = k.shape
    c = idx.shape[1]
    kdt = _kv_dtype(k)
    _check(lib().ds_append_label(_ptr_kv(k), kdt, _ptr(idx), b, hkv, pos, s_cap, d, c, _ptr(label),
                                 _label_args(label, lscale, lzero, kdt), _ptr(lscale), _ptr(lzero),
                                 _stream(stream)))


def new_label_cache(k, c: int, int4: bool = False):
    """Allocate (uninitialised) label storage matching a key cache (torch)."""
    torch = _torch()
    b, hkv, s_cap, d = k.shape
    if int4:
        return (torch.empty((b, hkv, s_cap, c // 2), dtype=torch.uint8, device=k.device),
                torch.empty((b, hkv, s_cap), dtype=torch.int16, device=k.device),
                torch.empty((b, hkv, s_cap), dtype=torch.int16, device=k.device))
    return torch.empty((b, hkv, s_cap, c), dtype=k.dtype, device=k.device), None, None


def sparse_decode(q, k, v, label, idx, s: int, topk: int, lscale=None, lzero=None, out=None,
                  out_dtype=None, sm_scale: float = 0.0, sel_out=None, score_out=None, stream=None):
    """One Double Sparsity decode step; returns out [B, Hq, D]."""
    torch = _torch()
    _need_cuda_or_pinned(k, v)
    _need_cuda(q, label, idx, lscale, lzero, out, sel_out, score_out)
    b, hq, d = q.shape
    _, hkv, s_cap, _ = k.shape
    c = idx.shape[1]
    kdt = _kv_dtype(k)
    if out is None:
        out = torch.empty((b, hq, d), dtype=out_dtype or torch.float32, device=q.device)
    odt = DS_F32 if out.dtype == torch.float32 else DS_BF16
    _check(lib().ds_sparse_decode(_ptr(q), _ptr_kv(k), _ptr_kv(v), kdt, _ptr(label),
                                  _label_args(label, lscale, lzero, kdt), _ptr(lscale), _ptr(lzero),
                                  _ptr(idx), b, hq, hkv, s, s_cap, d, c, topk, float(sm_scale),
                                  _ptr(out), odt, _ptr(sel_out), _ptr(score_out), _stream(stream)))
    return out


def decode_step(q, k, v, label, idx, s: int, topk: int, lscale=None, lzero=None, out=None,
                out_dtype=None, sm_scale: float = 0.0, sel_out=None, score_out=None, stream=None):
    """append_label(pos = s - 1) followed by sparse_decode, in one launch;
    returns out [B, Hq, D]."""
    torch = _torch()
    _need_cuda_or_pinned(k, v)
    _need_cuda(q, label, idx, lscale, lzero, out, sel_out, score_out)
    b, hq, d = q.shape
    _, hkv, s_cap, _ = k.shape
    c = idx.shape[1]
    kdt = _kv_dtype(k)
    if out is None:
        out = torch.empty((b, hq, d), dtype=out_dtype or torch.float32, device=q.device)
    odt = DS_F32 if out.dtype == torch.float32 else DS_BF16
    _check(lib().ds_decode_step(_ptr(q), _ptr_kv(k), _ptr_kv(v), kdt, _ptr(label),
                                _label_args(label, lscale, lzero, kdt), _ptr(lscale), _ptr(lzero),
                                _ptr(idx), b, hq, hkv, s, s_cap, d, c, topk, float(sm_scale),
                                _ptr(out), odt, _ptr(sel_out), _ptr(score_out), _stream(stream)))
    return out


def decode_step_kv(q, k_new, v_new, k, v, label, idx, s: int, topk: int, lscale=None, lzero=None, out=None,
                   out_dtype=None, sm_scale: float = 0.0, sel_out=None, score_out=None, stream=None):
    """decode_step that first writes the new token's rows k_new, v_new
    [B, Hkv, D] into k, v at position s - 1 (in the same launch); returns
    out [B, Hq, D]. q, k_new, v_new and out may be pinned host tensors: the
    kernel then reads the step's inputs and writes its output over the host
    link itself, so a step from host buffers is this one call."""
    torch = _torch()
    _need_cuda_or_pinned(k, v, q, k_new, v_new)
    if out is not None:
        _need_cuda_or_pinned(out)
    _need_cuda(label, idx, lscale, lzero, sel_out, score_out)
    b, hq, d = q.shape
    _, hkv, s_cap, _ = k.shape
    c = idx.shape[1]
    kdt = _kv_dtype(k)
    if k_new.dtype != k.dtype or v_new.dtype != v.dtype:
        raise TypeError("k_new / v_new must have the caches' dtype")
    if out is None:
        out = torch.empty((b, hq, d), dtype=out_dtype or torch.float32, device=label.device)
    odt = DS_F32 if out.dtype == torch.float32 else DS_BF16
    _check(lib().ds_decode_step_kv(_ptr_kv(q), _ptr_kv(k_new), _ptr_kv(v_new), _ptr_kv(k), _ptr_kv(v), kdt,
                                   _ptr(label), _label_args(label, lscale, lzero, kdt), _ptr(lscale), _ptr(lzero),
                                   _ptr(idx), b, hq, hkv, s, s_cap, d, c, topk, float(sm_scale),
                                   _ptr_kv(out), odt, _ptr(sel_out), _ptr(score_out), _stream(stream)))
    return out


class PreparedDecodeStepKV:
    """decode_step_kv with every argument checked and converted once.

    A serving loop decodes token after token into the same caches, label
    cache and (pinned host or device) buffers; only their contents and the
    token count change. Preparing the call keeps the per-step host cost to
    one C-ABI call: ``step()`` enqueues one step (ds_decode_step_kv) on the
    stream that was current at preparation (or `stream`), and
    ``step.set_length(s)`` moves to another token count."""

    _S_ARG = 14  # position of `s` in the ds_decode_step_kv argument list

    def __init__(self, q, k_new, v_new, k, v, label, idx, s: int, topk: int, lscale=None, lzero=None,
                 out=None, out_dtype=None, sm_scale: float = 0.0, stream=None):
        torch = _torch()
        _need_cuda_or_pinned(k, v, q, k_new, v_new)
        _need_cuda(label, idx, lscale, lzero)
        b, hq, d = q.shape
        _, hkv, s_cap, _ = k.shape
        c = idx.shape[1]
        kdt = _kv_dtype(k)
        if k_new.dtype != k.dtype or v_new.dtype != v.dtype:
            raise TypeError("k_new / v_new must have the caches' dtype")
        if out is None:
            out = torch.empty((b, hq, d), dtype=out_dtype or torch.float32, device=label.device)
        _need_cuda_or_pinned(out)
        odt = DS_F32 if out.dtype == torch.float32 else DS_BF16
        self.out = out
        self._keep = (q, k_new, v_new, k, v, label, idx, lscale, lzero, out)  # keep the memory alive
        self._args = [_ptr_kv(q), _ptr_kv(k_new), _ptr_kv(v_new), _ptr_kv(k), _ptr_kv(v), kdt, _ptr(label),
                      _label_args(label, lscale, lzero, kdt), _ptr(lscale), _ptr(lzero), _ptr(idx), b, hq, hkv,
                      int(s), s_cap, d, c, int(topk), float(sm_scale), _ptr_kv(out), odt, None, None,
                      _stream(stream)]
        assert self._args[self._S_ARG - 1] == hkv and self._args[self._S_ARG + 1] == s_cap  # layout check
        self._fn = lib().ds_decode_step_kv

    def set_length(self, s: int) -> None:
        self._args[self._S_ARG] = int(s)

    def __call__(self):
        st = self._fn(*self._args)
        if st != DS_OK:
            raise DSError(st, last_error())
        return self.out


def decode_step_varlen(q, k, v, label, idx, seq_lens, s_max: int, topk: int, lscale=None, lzero=None, out=None,
                       out_dtype=None, sm_scale: float = 0.0, sel_out=None, score_out=None,
                       sparse_threshold: int = 0, fallback: int = DS_FALLBACK_PER_ENTRY, stream=None):
    """decode_step with a per-batch-entry token count seq_lens [B] (int32,
    device) and the short-entry fallback rule; returns out [B, Hq, D]."""
    torch = _torch()
    _need_cuda_or_pinned(k, v)
    _need_cuda(q, label, idx, seq_lens, lscale, lzero, out, sel_out, score_out)
    b, hq, d = q.shape
    _, hkv, s_cap, _ = k.shape
    c = idx.shape[1]
    kdt = _kv_dtype(k)
    if out is None:
        out = torch.empty((b, hq, d), dtype=out_dtype or torch.float32, device=q.device)
    odt = DS_F32 if out.dtype == torch.float32 else DS_BF16
    _check(lib().ds_decode_step_varlen(_ptr(q), _ptr_kv(k), _ptr_kv(v), kdt, _ptr(label),
                                       _label_args(label, lscale, lzero, kdt), _ptr(lscale), _ptr(lzero),
                                       _ptr(idx), _ptr(seq_lens), int(sparse_threshold), int(fallback),
                                       b, hq, hkv, s_max, s_cap, d, c, topk,
                                       float(sm_scale), _ptr(out), odt, _ptr(sel_out), _ptr(score_out),
                                       _stream(stream)))
    return out


def build_label_cache_paged(k_pool, idx, block_table, s: int, label, lscale=None, lzero=None, stream=None):
    """Fill label rows [0, s) (label [B, Hkv, S_cap, ...]) from a paged key
    pool k_pool [num_blocks, Hkv, page, D] through block_table [B, max_blocks]."""
    _need_cuda_or_pinned(k_pool)
    _need_cuda(idx, block_table, label, lscale, lzero)
    num_blocks, hkv, page, d = k_pool.shape
    b, max_blocks = block_table.shape
    s_cap = label.shape[2]
    c = idx.shape[1]
    kdt = _kv_dtype(k_pool)
    _check(lib().ds_build_label_cache_paged(_ptr_kv(k_pool), kdt, _ptr(idx), _ptr(block_table), max_blocks, page,
                                            num_blocks, b, hkv, s, s_cap, d, c, _ptr(label),
                                            _label_args(label, lscale, lzero, kdt), _ptr(lscale), _ptr(lzero),
                                            _stream(stream)))


def decode_step_paged(q, k_pool, v_pool, label, idx, block_table, s_max: int, topk: int, seq_lens=None,
                      lscale=None, lzero=None, out=None, out_dtype=None, sm_scale: float = 0.0, sel_out=None,
                      score_out=None, sparse_threshold: int = 0, fallback: int = DS_FALLBACK_PER_ENTRY,
                      stream=None):
    """decode_step(_varlen) over paged pools k_pool/v_pool [num_blocks, Hkv,
    page, D] with block_table [B, max_blocks]; returns out [B, Hq, D]."""
    torch = _torch()
    _need_cuda_or_pinned(k_pool, v_pool)
    _need_cuda(q, label, idx, block_table, seq_lens, lscale, lzero, out, sel_out, score_out)
    b, hq, d = q.shape
    num_blocks, hkv, page, _ = k_pool.shape
    max_blocks = block_table.shape[1]
    s_cap = label.shape[2]
    c = idx.shape[1]
    kdt = _kv_dtype(k_pool)
    if out is None:
        out = torch.empty((b, hq, d), dtype=out_dtype or torch.float32, device=q.device)
    odt = DS_F32 if out.dtype == torch.float32 else DS_BF16
    _check(lib().ds_decode_step_paged(_ptr(q), _ptr_kv(k_pool), _ptr_kv(v_pool), kdt, _ptr(label),
                                      _label_args(label, lscale, lzero, kdt), _ptr(lscale), _ptr(lzero),
                                      _ptr(idx), _ptr(block_table), max_blocks, page, num_blocks, _ptr(seq_lens),
                                      int(sparse_threshold), int(fallback), b, hq, hkv, s_max, s_cap, d, c, topk,
                                      float(sm_scale), _ptr(out), odt, _ptr(sel_out), _ptr(score_out),
                                      _stream(stream)))
    return out


def dense_decode(q, k, v, s: int, out=None, out_dtype=None, sm_scale: float = 0.0, stream=None):
    """Dense decode attention over tokens [0, s) (measurement baseline)."""
    torch = _torch()
    _need_cuda_or_pinned(k, v)
    _need_cuda(q, out)
    b, hq, d = q.shape
    _, hkv, s_cap, _ = k.shape
    if out is None:
        out = torch.empty((b, hq, d), dtype=out_dtype or torch.float32, device=q.device)
    odt = DS_F32 if out.dtype == torch.float32 else DS_BF16
    _check(lib().ds_dense_decode(_ptr(q), _ptr_kv(k), _ptr_kv(v), _kv_dtype(k), b, hq, hkv, s, s_cap, d,
                                 float(sm_scale), _ptr(out), odt, _stream(stream)))
    return out


# ------------------------------------------- writing and reading caches, trees

def _cache_dtype(t) -> int:
    return DS_E4M3 if t.dtype == _torch().float8_e4m3fn else _kv_dtype(t)


def _int32(name, t, *shape):
    """A contiguous int32 tensor of the given shape, or None."""
    if t is not None and (t.dtype != _torch().int32 or tuple(t.shape) != shape):
        raise ValueError(f"{name} must be int32 of shape {shape}, got {t.dtype} {tuple(t.shape)}")


def _scales(dt, k, v, k_scale, v_scale):
    if dt != DS_E4M3:
        if k_scale is not None or v_scale is not None:
            raise ValueError("scales belong to 8-bit caches")
        return
    torch = _torch()
    for c, sc in ((k, k_scale), (v, v_scale)):
        if c is not None and (sc is None or sc.dtype != torch.float32 or sc.shape != c.shape[:-1]):
            raise ValueError("an 8-bit cache needs a float32 scale of its shape without the last dimension")


def _same_caches(k, v):
    if v is not None and (k.dtype != v.dtype or k.shape != v.shape):
        raise ValueError("the key and value caches must have one dtype and shape")
    if k.dim() != 4:
        raise ValueError("a cache has four dimensions")


def _on_one_device(*ts):
    """The device of all given CUDA tensors."""
    dev = None
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("tensors must be CUDA tensors")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"tensors on {dev} and {t.device}")
    return dev


class _Prepared:
    """A C-ABI call with its arguments checked and converted once. Calling it
    enqueues the call on `stream`, or on the stream that is current on the
    tensors' device at that time, and returns the outputs.

    A handle may be called on one stream after another and dropped at any time:
    its tensors' memory is not given out again before what it enqueued is done.
    Its calls share its outputs and workspace, so two of them must not run at
    the same time: one that follows on another stream waits for the one before
    (an event), and streams that run side by side have a handle each. A graph
    that captured a call needs the handle for as long as it is replayed."""

    def _bind(self, fn, args, dev, stream, keep, result, once=False):
        self._fn, self._args, self._dev, self._stream = fn, args, dev, stream
        self._keep = keep  # keeps the memory alive
        self._result = result
        # streams that the tensors' memory waits for when it is freed: the one it belongs to
        # (a handle that is called right away and dropped does not look it up: the call does)
        self._streams = set()
        if stream is None:
            self._streams = None if once else {_torch().cuda.current_stream(dev).cuda_stream}

    def _record(self, stream):
        """The allocator hears of a stream that the tensors were not made on."""
        torch = _torch()
        with torch.cuda.stream(stream):
            if torch.cuda.is_current_stream_capturing():
                return  # nothing runs now, and replays are the graph's owner's to order
        for x in _tensors(self._keep, self._result):
            x.record_stream(stream)
        self._streams.add(stream.cuda_stream)

    def __call__(self):
        torch = _torch()
        dev = self._dev
        stream = torch.cuda.current_stream(dev) if self._stream is None else self._stream
        s = stream.cuda_stream
        if self._streams is None:
            self._streams = {s}
        elif s not in self._streams:
            self._record(stream)
        if torch.cuda.current_device() != dev.index:
            with torch.cuda.device(dev):
                st = self._fn(*self._args, s)
        else:
            st = self._fn(*self._args, s)
        if st != DS_OK:
            raise DSError(st, last_error())
        return self._result


def _tensors(*xs):
    """The tensors among xs and in their tuples."""
    for x in xs:
        if isinstance(x, tuple):
            yield from _tensors(*x)
        elif x is not None:
            yield x


def _alloc(shape, dtype, dev, stream):
    """torch.empty in the memory pool of the stream that will use it."""
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def new_kv_cache(shape, dtype, device="cuda"):
    """Zeroed caches k, v of `shape` ([B, Hkv, S_cap, D], or a pool
    [num_blocks, Hkv, page, D]) and, for torch.float8_e4m3fn, their scales:
    (k, v, k_scale, v_scale)."""
    torch = _torch()
    k, v = (torch.zeros(shape, dtype=torch.uint8, device=device).view(dtype) if dtype == torch.float8_e4m3fn
            else torch.zeros(shape, dtype=dtype, device=device) for _ in range(2))
    if dtype != torch.float8_e4m3fn:
        return k, v, None, None
    return k, v, *(torch.zeros(tuple(shape)[:-1], dtype=torch.float32, device=device) for _ in range(2))


class PreparedWriteKV(_Prepared):
    """write_kv bound once; calling it enqueues the write and returns q_out."""

    def __init__(self, q, k, v, k_cache, v_cache, starts=None, positions=None, lens=None, q_weight=None,
                 k_weight=None, eps: float = 1e-6, inv_freq=None, rope: int = DS_ROPE_HALF, k_scale=None,
                 v_scale=None, block_table=None, q_out=None, stream=None, _once=False):
        torch = _torch()
        dev = _on_one_device(k, v, q, k_cache, v_cache, starts, positions, lens, q_weight, k_weight, inv_freq,
                             k_scale, v_scale, block_table, q_out)
        for t in (k_cache, v_cache, starts, positions, lens, q_weight, k_weight, inv_freq, k_scale, v_scale,
                  block_table, q_out):
            if t is not None and not t.is_contiguous():
                raise ValueError("all tensors but q, k and v must be contiguous")
        for t in (k, v) if q is None else (k, v, q):
            if t.dim() != 4 or t.dtype != k.dtype or t.shape[:2] != k.shape[:2] or t.shape[3] != k.shape[3]:
                raise ValueError("q, k, v must be [B, T, heads, D] of one dtype")
            if t.numel() and (t.stride(3) != 1 or (t.shape[2] > 1 and t.stride(2) != t.shape[3])):
                raise ValueError("the heads of a token of q, k, v must be contiguous")
        if k.shape != v.shape:
            raise ValueError("k and v must have one shape")
        dt, cdt = _kv_dtype(k), _cache_dtype(k_cache)
        _same_caches(k_cache, v_cache)
        _scales(cdt, k_cache, v_cache, k_scale, v_scale)
        b, t, hkv, d = k.shape
        if k_cache.shape[1] != hkv or k_cache.shape[3] != d:
            raise ValueError("the caches' heads or head size differ from k's")
        _int32("starts", starts, b)
        _int32("lens", lens, b)
        _int32("positions", positions, b, t)
        for w in (q_weight, k_weight):
            if w is not None and (w.dtype != k.dtype or tuple(w.shape) != (d,)):
                raise ValueError("a norm weight must be [D] of q's dtype")
        rot = 0
        if inv_freq is not None:
            if inv_freq.dtype != torch.float32 or inv_freq.dim() != 1:
                raise ValueError("inv_freq must be a float32 vector")
            rot = 2 * inv_freq.shape[0]
        hq = 0
        if q is not None:
            hq = q.shape[2]
            if q_out is None:
                q_out = _alloc((b, t, hq, d), q.dtype, dev, stream)
            elif tuple(q_out.shape) != (b, t, hq, d) or q_out.dtype != q.dtype:
                raise ValueError("q_out must have q's shape and dtype")
        elif q_out is not None or q_weight is not None:
            raise ValueError("q_out and q_weight need q")

        def strided(x):  # (a dimension of size 1 may have any stride: it is never taken)
            return (None, 0, 0) if x is None else (x.data_ptr(), x.stride(0) if x.shape[0] > 1 else 0,
                                                   x.stride(1) if x.shape[1] > 1 else 0)

        def ptr(x):
            return None if x is None else x.data_ptr()

        args = [*strided(q), *strided(k), *strided(v), dt, ptr(q_weight), ptr(k_weight), float(eps), ptr(inv_freq), rot,
                int(rope), ptr(positions), ptr(starts), ptr(lens), b, t, hq, hkv]
        tail = [d, ptr(q_out), ptr(k_cache), ptr(v_cache), cdt, ptr(k_scale), ptr(v_scale)]
        if block_table is None:
            if k_cache.shape[0] != b:
                raise ValueError("the caches' batch differs from k's")
            fn, args = lib().ds_write_kv, args + [k_cache.shape[2]] + tail
        else:
            _int32("block_table", block_table, b, *block_table.shape[1:2])
            fn = lib().ds_write_kv_paged
            args = args + tail + [ptr(block_table), block_table.shape[1], k_cache.shape[2], k_cache.shape[0]]
        self.q_out = q_out
        self._bind(fn, args, dev, stream, (q, k, v, k_cache, v_cache, starts, positions, lens, q_weight, k_weight,
                                           inv_freq, k_scale, v_scale, block_table), q_out, _once)


def write_kv(q, k, v, k_cache, v_cache, **kw):
    """Write the keys and values of T new tokens an entry, k and v [B, T, Hkv,
    D] as the projections left them, into the caches at rows starts[b] + i,
    with the per-head norm (k_weight), the rotation (inv_freq, positions) and
    the 8-bit quantisation (k_scale, v_scale) in the same pass; q [B, T, Hq, D]
    (or None) gets its norm and rotation into q_out, which is returned. q, k
    and v may be views of one fused projection. Caches [B, Hkv, S_cap, D], or
    pools with block_table. Arguments as PreparedWriteKV's; see ds_write_kv."""
    return PreparedWriteKV(q, k, v, k_cache, v_cache, _once=True, **kw)()


def read_kv(k, v, k_scale, v_scale, s: int, seq_lens=None, block_table=None, dtype=None, k_out=None, v_out=None,
            stream=None):
    """Rows [0, s) of an 8-bit cache (k, v torch.float8_e4m3fn, dense or pools
    with block_table) as dtype (bf16 by default) rows: (k_out, v_out), each
    [B, Hkv, s, D] unless given (then [B, Hkv, >= s, D]). v, v_scale None: the
    keys alone. Rows past seq_lens[b] are not written."""
    torch = _torch()
    dev = _on_one_device(k, v, k_scale, v_scale, seq_lens, block_table, k_out, v_out)
    for t in (k, v, k_scale, v_scale, seq_lens, block_table, k_out, v_out):
        if t is not None and not t.is_contiguous():
            raise ValueError("tensors must be contiguous")
    if _cache_dtype(k) != DS_E4M3:
        raise TypeError("read_kv reads float8_e4m3fn caches")
    _same_caches(k, v)
    _scales(DS_E4M3, k, v, k_scale, v_scale)
    b = k.shape[0] if block_table is None else block_table.shape[0]
    hkv, d = k.shape[1], k.shape[3]
    _int32("seq_lens", seq_lens, b)
    if k_out is None:
        k_out = _alloc((b, hkv, s, d), dtype or torch.bfloat16, dev, stream)
    if v is None:
        if v_out is not None or v_scale is not None:
            raise ValueError("v_out and v_scale need v")
    elif v_out is None:
        v_out = _alloc(k_out.shape, k_out.dtype, dev, stream)
    for o in (k_out,) if v is None else (k_out, v_out):
        if o.dim() != 4 or o.shape[0] != b or o.shape[1] != hkv or o.shape[3] != d or o.shape != k_out.shape:
            raise ValueError("k_out and v_out must be [B, Hkv, S, D]")
        if o.dtype != k_out.dtype or (dtype is not None and o.dtype != dtype):
            raise ValueError("k_out and v_out must have one dtype")

    def ptr(x):
        return None if x is None else x.data_ptr()

    tail = [ptr(k_out), ptr(v_out), _kv_dtype(k_out), k_out.shape[2]]
    call = _Prepared()
    if block_table is None:
        fn, args = lib().ds_read_kv, [ptr(k), ptr(v), ptr(k_scale), ptr(v_scale), ptr(seq_lens), b, hkv, int(s),
                                      k.shape[2], d, *tail]
    else:
        _int32("block_table", block_table, b, *block_table.shape[1:2])
        fn = lib().ds_read_kv_paged
        args = [ptr(k), ptr(v), ptr(k_scale), ptr(v_scale), ptr(block_table), block_table.shape[1], k.shape[2],
                k.shape[0], ptr(seq_lens), b, hkv, int(s), d, *tail]
    call._bind(fn, args, dev, stream, (k, v, k_scale, v_scale, seq_lens, block_table), (k_out, v_out), True)
    return call()


def tree_mask(parents):
    """The mask of drafted trees from their parents [B, T] (int tensor: the
    index of each node's parent, which is a smaller one, or -1 for the prefix):
    node i sees itself and its ancestors. int32 [B, T, ceil(T / 32)] on
    parents' device. Worked out on the host, a node at a time: reads parents
    back where they are on the GPU, and cannot be captured in a graph."""
    torch = _torch()
    b, t = parents.shape
    p = parents.to("cpu", torch.int64)
    if bool((p >= torch.arange(t)).any()) or bool((p < -1).any()):
        raise ValueError("a parent must be -1 or an earlier node")
    sees = torch.zeros((b, t, t), dtype=torch.bool)
    for i in range(t):
        has = (p[:, i] >= 0)[:, None]
        sees[:, i] = sees[torch.arange(b), p[:, i].clamp_min(0)] & has
        sees[:, i, i] = True
    words = (t + 31) // 32
    bits = torch.zeros((b, t, words * 32), dtype=torch.int64)
    bits[:, :, :t] = sees.long()
    bits = (bits.view(b, t, words, 32) << torch.arange(32)).sum(-1)
    return torch.where(bits >= 1 << 31, bits - (1 << 32), bits).to(torch.int32).to(parents.device)


def tree_decode_workspace(b, t, hq, hkv, s, d, kv_dtype=DS_BF16) -> int:
    """Device scratch bytes tree_decode needs for a shape."""
    out = C.c_size_t()
    _check(lib().ds_tree_decode_workspace_size(b, t, hq, hkv, s, d, kv_dtype, C.byref(out)))
    return out.value


class PreparedTreeDecode(_Prepared):
    """tree_decode bound once, with its output and workspace; calling it
    enqueues the attention and returns out. Two calls of one handle must not
    run at the same time: they share both. set_length(s) moves to another prefix
    length, up to the one it was made with."""

    _S_ARG = {False: 13, True: 17}

    def __init__(self, q, k, v, s: int, mask=None, seq_lens=None, node_lens=None, k_scale=None, v_scale=None,
                 block_table=None, out=None, out_dtype=None, sm_scale: float = 0.0, ws=None, stream=None, _once=False):
        torch = _torch()
        dev = _on_one_device(q, k, v, mask, seq_lens, node_lens, k_scale, v_scale, block_table, out, ws)
        for t in (q, k, v, mask, seq_lens, node_lens, k_scale, v_scale, block_table, out, ws):
            if t is not None and not t.is_contiguous():
                raise ValueError("tensors must be contiguous")
        if q.dim() != 4:
            raise ValueError("q must be [B, T, Hq, D]")
        b, t, hq, d = q.shape
        kdt = _cache_dtype(k)
        _same_caches(k, v)
        _scales(kdt, k, v, k_scale, v_scale)
        if _kv_dtype(q) != (DS_F32 if kdt == DS_F32 else DS_BF16):
            raise TypeError("q must be float32 with a float32 cache, else bfloat16")
        if k.shape[3] != d:
            raise ValueError("the caches' head size differs from q's")
        hkv = k.shape[1]
        _int32("mask", mask, b, t, (t + 31) // 32)
        _int32("seq_lens", seq_lens, b)
        _int32("node_lens", node_lens, b)
        need = tree_decode_workspace(b, t, hq, hkv, s, d, kdt)
        if out is None:
            out = _alloc((b, t, hq, d), out_dtype or torch.float32, dev, stream)
        elif out.shape != q.shape or (out_dtype is not None and out.dtype != out_dtype):
            raise ValueError("out must have q's shape (and out_dtype)")
        if ws is None:
            ws = _alloc((need,), torch.uint8, dev, stream)

        def ptr(x):
            return None if x is None else x.data_ptr()

        head = [ptr(q), ptr(k), ptr(v), kdt, ptr(k_scale), ptr(v_scale), ptr(mask)]
        tail = [d, float(sm_scale), ptr(out), _kv_dtype(out), ptr(ws), ws.numel() * ws.element_size()]
        if block_table is None:
            if k.shape[0] != b:
                raise ValueError("the caches' batch differs from q's")
            fn = lib().ds_tree_decode
            args = head + [ptr(seq_lens), ptr(node_lens), b, t, hq, hkv, int(s), k.shape[2]] + tail
        else:
            _int32("block_table", block_table, b, *block_table.shape[1:2])
            fn = lib().ds_tree_decode_paged
            args = head + [ptr(block_table), block_table.shape[1], k.shape[2], k.shape[0], ptr(seq_lens),
                           ptr(node_lens), b, t, hq, hkv, int(s)] + tail
        self.out, self._s_at, self._s_max = out, self._S_ARG[block_table is not None], int(s)
        self._bind(fn, args, dev, stream, (q, k, v, mask, seq_lens, node_lens, k_scale, v_scale, block_table, ws), out, _once)

    def set_length(self, s: int) -> None:
        if not 0 <= s <= self._s_max:
            raise ValueError(f"prefix length {s} outside [0, {self._s_max}]")
        self._args[self._s_at] = int(s)


def tree_decode(q, k, v, s: int, **kw):
    """Attention of the T drafted tokens q [B, T, Hq, D] over caches k, v
    [B, Hkv, S_cap, D] that hold a prefix of s tokens (seq_lens[b], at most s)
    and, in the T rows behind it, the drafted tokens' own keys and values;
    mask as tree_mask makes it (None: a chain). float8_e4m3fn caches need
    k_scale and v_scale; a row that holds a NaN code needs the scale NaN, as
    write_kv leaves it (a conversion of out-of-range values by torch does not). Returns out [B, T, Hq, D]. Arguments as
    PreparedTreeDecode's; see ds_tree_decode."""
    return PreparedTreeDecode(q, k, v, s, _once=True, **kw)()


def tree_decode_paged(q, k_pool, v_pool, block_table, s: int, **kw):
    """tree_decode over pools [num_blocks, Hkv, page, D] with block_table
    [B, max_blocks]."""
    return PreparedTreeDecode(q, k_pool, v_pool, s, block_table=block_table, _once=True, **kw)()
