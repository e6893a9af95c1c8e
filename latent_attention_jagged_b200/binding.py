"""ctypes binding of libllatte.so: the same entry points as include/llatte.h,
with argument marshalling from torch tensors (device memory and streams only;
every step of the forward runs in the library's kernels).
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Optional, Sequence

import numpy as np
import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libllatte.so")
MAX_LAYERS = 16
STEPS = ("plan", "gather", "ctx_bias", "kv", "q", "attn", "o", "ffn1", "ffn2", "readout", "ffn",
         "summary", "attn_export")

LLATTE_OK, LLATTE_ERR_ARG, LLATTE_ERR_UNSUPPORTED, LLATTE_ERR_CUDA, LLATTE_ERR_OOM, \
    LLATTE_ERR_DEVICE = 0, -1, -2, -3, -4, -5
LLATTE_BF16, LLATTE_FP32 = 0, 1
DEV_BAD_OFFSETS, DEV_TOO_LONG, DEV_TOO_MANY_ROWS, DEV_TIMEOUT, DEV_BAD_ID = 1, 2, 4, 8, 16


class LlatteError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {error_string(code)} ({code})")


class llatte_dims(ctypes.Structure):
    _fields_ = [("d", ctypes.c_int32), ("heads", ctypes.c_int32), ("d_head", ctypes.c_int32),
                ("rank", ctypes.c_int32), ("d_ctx", ctypes.c_int32), ("n_q", ctypes.c_int32),
                ("n_layers", ctypes.c_int32), ("keep", ctypes.c_int32 * MAX_LAYERS),
                ("d_out", ctypes.c_int32), ("ffn_mult", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("kv_norm", ctypes.c_int32), ("eps", ctypes.c_float),
                ("max_batch", ctypes.c_int32), ("max_len", ctypes.c_int64),
                ("max_total", ctypes.c_int64), ("n_sum", ctypes.c_int32),
                ("sum_rank", ctypes.c_int32), ("d_seq", ctypes.c_int32),
                ("q_rank", ctypes.c_int32), ("d_time", ctypes.c_int32),
                ("attn_form", ctypes.c_int32)]


LAYER_KEYS = ("W_dkv", "g_kv", "W_q", "W_uk", "W_uv", "W_o", "g1", "W1", "W2", "g2",
              "W_dq", "g_q", "W_uq")


class llatte_layer_w(ctypes.Structure):
    _fields_ = [(k, ctypes.c_void_p) for k in LAYER_KEYS]


SUMMARY_KEYS = ("W_down", "W_up")


class llatte_summary_w(ctypes.Structure):
    _fields_ = [(k, ctypes.c_void_p) for k in SUMMARY_KEYS]


class llatte_batch(ctypes.Structure):
    _fields_ = [("values", ctypes.c_void_p), ("offsets", ctypes.c_void_p), ("B", ctypes.c_int32),
                ("context", ctypes.c_void_p), ("cand", ctypes.c_void_p),
                ("event_age", ctypes.c_void_p)]


class llatte_tok_dims(ctypes.Structure):
    _fields_ = [("n_fields", ctypes.c_int32), ("rows", ctypes.c_int64 * 8),
                ("width", ctypes.c_int32 * 8), ("d_hid", ctypes.c_int32), ("d", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("max_events", ctypes.c_int64)]


class llatte_tok_w(ctypes.Structure):
    _fields_ = [("tables", ctypes.c_void_p * 8), ("W_a1", ctypes.c_void_p),
                ("W_a2", ctypes.c_void_p)]


class llatte_attn_export(ctypes.Structure):
    _fields_ = [("layer", ctypes.c_int32), ("n_k", ctypes.c_int32), ("n_hours", ctypes.c_int32),
                ("event_age", ctypes.c_void_p), ("recent", ctypes.c_void_p),
                ("topk", ctypes.c_void_p), ("hours", ctypes.c_void_p)]


class llatte_cache_dims(ctypes.Structure):
    _fields_ = [("heads", ctypes.c_int32), ("rank", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("n_pages", ctypes.c_int32),
                ("max_batch", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("max_rows", ctypes.c_int64)]


class llatte_cache_view(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("table_stride", ctypes.c_int32),
                ("lengths", ctypes.c_void_p), ("B", ctypes.c_int32)]


class llatte_cache_attn(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("q_offsets", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("n_cand", ctypes.c_int32), ("scale", ctypes.c_float), ("window", ctypes.c_int32),
                ("n_sink", ctypes.c_int32), ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p),
                ("accumulate", ctypes.c_int32)]


class llatte_cache_evict_args(ctypes.Structure):
    _fields_ = [("budget", ctypes.c_int32), ("n_sink", ctypes.c_int32),
                ("n_recent", ctypes.c_int32), ("dst_table", ctypes.c_void_p),
                ("dst_stride", ctypes.c_int32), ("new_lengths", ctypes.c_void_p),
                ("kept", ctypes.c_void_p)]


class llatte_forward_cache(ctypes.Structure):
    _fields_ = [("caches", ctypes.POINTER(ctypes.c_void_p)),
                ("views", ctypes.POINTER(llatte_cache_view)), ("window", ctypes.c_int32),
                ("n_sink", ctypes.c_int32), ("accumulate", ctypes.c_int32)]


EXPORTS = ("llatte_create", "llatte_forward", "llatte_plan_export", "llatte_get_status",
           "llatte_workspace_bytes", "llatte_error_string", "llatte_destroy",
           "llatte_set_profiling", "llatte_profile_reset", "llatte_profile_step",
           "llatte_plan_static", "llatte_exp2_eval", "llatte_forward_export",
           "llatte_forward_batch", "llatte_attn_form_mask", "llatte_tokenizer_create",
           "llatte_tokenize", "llatte_tokenizer_get_status", "llatte_tokenizer_uses_tensor_cores",
           "llatte_tokenizer_destroy", "llatte_inject_timeout", "llatte_cache_workspace_bytes",
           "llatte_cache_create", "llatte_cache_append", "llatte_cache_attend",
           "llatte_cache_evict", "llatte_cache_get_status", "llatte_cache_uses_tensor_cores",
           "llatte_cache_destroy", "llatte_forward_cached", "llatte_cache_inject_timeout")
TOK_MAX_FIELDS = 8
PLAN_STATIC_MAX_BATCH = 4096

_lib = None


def load_library(path: Optional[str] = None) -> ctypes.CDLL:
    """Open libllatte.so (raises if it has not been built: there is no fallback)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"{p} is missing: build it with "
                           "`python -m latent_attention_jagged_b200.build`")
    lib = ctypes.CDLL(p)
    P, I32, I64, VP = ctypes.POINTER, ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p
    lib.llatte_create.argtypes = [P(VP), P(llatte_dims), P(llatte_layer_w), VP,
                                  P(llatte_summary_w), ctypes.c_int]
    lib.llatte_create.restype = ctypes.c_int
    lib.llatte_forward.argtypes = [VP, VP, VP, I32, VP, VP, VP, VP]
    lib.llatte_forward.restype = ctypes.c_int
    lib.llatte_forward_export.argtypes = [VP, VP, VP, I32, VP, VP, VP, P(llatte_attn_export), VP]
    lib.llatte_forward_export.restype = ctypes.c_int
    lib.llatte_forward_batch.argtypes = [VP, P(llatte_batch), VP, P(llatte_attn_export), VP]
    lib.llatte_forward_batch.restype = ctypes.c_int
    lib.llatte_plan_export.argtypes = [VP, VP, VP]
    lib.llatte_plan_export.restype = ctypes.c_int
    lib.llatte_get_status.argtypes = [VP, P(I32)]
    lib.llatte_get_status.restype = ctypes.c_int
    lib.llatte_workspace_bytes.argtypes = [P(llatte_dims)]
    lib.llatte_workspace_bytes.restype = ctypes.c_size_t
    lib.llatte_error_string.argtypes = [ctypes.c_int]
    lib.llatte_error_string.restype = ctypes.c_char_p
    lib.llatte_destroy.argtypes = [VP]
    lib.llatte_destroy.restype = None
    lib.llatte_set_profiling.argtypes = [VP, ctypes.c_int]
    lib.llatte_set_profiling.restype = ctypes.c_int
    lib.llatte_profile_reset.argtypes = [VP]
    lib.llatte_profile_reset.restype = ctypes.c_int
    lib.llatte_profile_step.argtypes = [VP, ctypes.c_int, P(ctypes.c_char_p),
                                        P(ctypes.c_double), P(I64), P(I64)]
    lib.llatte_profile_step.restype = ctypes.c_int
    lib.llatte_plan_static.argtypes = [P(llatte_dims), VP, I32, VP, VP, VP]
    lib.llatte_plan_static.restype = ctypes.c_int
    lib.llatte_exp2_eval.argtypes = [VP, VP, VP, I64, VP]
    lib.llatte_exp2_eval.restype = ctypes.c_int
    lib.llatte_attn_form_mask.argtypes = [VP, P(ctypes.c_uint32)]
    lib.llatte_attn_form_mask.restype = ctypes.c_int
    lib.llatte_inject_timeout.argtypes = [VP, ctypes.c_int]
    lib.llatte_inject_timeout.restype = ctypes.c_int
    lib.llatte_tokenizer_create.argtypes = [P(VP), P(llatte_tok_dims), P(llatte_tok_w),
                                            ctypes.c_int]
    lib.llatte_tokenizer_create.restype = ctypes.c_int
    lib.llatte_tokenize.argtypes = [VP, VP, I64, VP, VP]
    lib.llatte_tokenize.restype = ctypes.c_int
    lib.llatte_tokenizer_get_status.argtypes = [VP, P(I32)]
    lib.llatte_tokenizer_get_status.restype = ctypes.c_int
    lib.llatte_tokenizer_uses_tensor_cores.argtypes = [VP]
    lib.llatte_tokenizer_uses_tensor_cores.restype = ctypes.c_int
    lib.llatte_tokenizer_destroy.argtypes = [VP]
    lib.llatte_tokenizer_destroy.restype = None
    lib.llatte_cache_workspace_bytes.argtypes = [P(llatte_cache_dims)]
    lib.llatte_cache_workspace_bytes.restype = ctypes.c_size_t
    lib.llatte_cache_create.argtypes = [P(VP), P(llatte_cache_dims), VP, VP]
    lib.llatte_cache_create.restype = ctypes.c_int
    lib.llatte_cache_append.argtypes = [VP, P(llatte_cache_view), VP, I64, VP, VP,
                                        ctypes.c_float, VP]
    lib.llatte_cache_append.restype = ctypes.c_int
    lib.llatte_cache_attend.argtypes = [VP, P(llatte_cache_view), P(llatte_cache_attn), VP]
    lib.llatte_cache_attend.restype = ctypes.c_int
    lib.llatte_cache_evict.argtypes = [VP, P(llatte_cache_view), P(llatte_cache_evict_args), VP]
    lib.llatte_cache_evict.restype = ctypes.c_int
    lib.llatte_cache_get_status.argtypes = [VP, P(I32)]
    lib.llatte_cache_get_status.restype = ctypes.c_int
    lib.llatte_cache_uses_tensor_cores.argtypes = [VP]
    lib.llatte_cache_uses_tensor_cores.restype = ctypes.c_int
    lib.llatte_cache_inject_timeout.argtypes = [VP, ctypes.c_int]
    lib.llatte_cache_inject_timeout.restype = ctypes.c_int
    lib.llatte_cache_destroy.argtypes = [VP]
    lib.llatte_cache_destroy.restype = None
    lib.llatte_forward_cached.argtypes = [VP, P(llatte_batch), P(llatte_forward_cache), VP, VP]
    lib.llatte_forward_cached.restype = ctypes.c_int
    if path is None:
        _lib = lib
    return lib


def error_string(code: int) -> str:
    try:
        return load_library().llatte_error_string(code).decode()
    except Exception:
        return "unknown"


def make_dims(dims, max_batch: int, max_len: int, max_total: int = 0) -> llatte_dims:
    """Fill the C struct from any object with the Dims attributes."""
    if len(dims.keep) > MAX_LAYERS:
        raise ValueError(f"at most {MAX_LAYERS} layers")
    c = llatte_dims()
    c.d, c.heads, c.d_head, c.rank = dims.d, dims.heads, dims.d_head, dims.rank
    c.d_ctx, c.n_q, c.n_layers = dims.d_ctx, dims.n_q, len(dims.keep)
    for i, k in enumerate(dims.keep):
        c.keep[i] = int(k)
    c.d_out, c.ffn_mult = dims.d_out, dims.ffn_mult
    c.dtype = {"bf16": LLATTE_BF16, "fp32": LLATTE_FP32}[dims.dtype]
    c.kv_norm, c.eps = dims.kv_norm, float(dims.eps)
    c.max_batch, c.max_len, c.max_total = int(max_batch), int(max_len), int(max_total)
    c.n_sum = int(getattr(dims, "n_sum", 0))
    c.sum_rank = int(getattr(dims, "sum_rank", 0))
    c.d_seq = int(getattr(dims, "d_seq", 0))
    c.q_rank = int(getattr(dims, "q_rank", 0))
    c.d_time = int(getattr(dims, "d_time", 0))
    c.attn_form = int(getattr(dims, "attn_form", 0))
    return c


def torch_dtype(dims) -> torch.dtype:
    return {"bf16": torch.bfloat16, "fp32": torch.float32}[dims.dtype]


def _host(a, dt: torch.dtype) -> torch.Tensor:
    t = a if isinstance(a, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(a))
    return t.detach().to(device="cpu", dtype=dt).contiguous()


def _ptr(t: Optional[torch.Tensor]):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _stream_ptr(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


# Address of a device's current stream; torch.cuda.current_stream builds an object
# around it first.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _int32(**numbers):
    """Refuses what a C int32 field would cut off without an error."""
    for name, n in numbers.items():
        if not -0x80000000 <= n <= 0x7fffffff:
            raise ValueError(f"{name} = {n} does not fit 32 bits")


def _made(make, stream, device):
    """make(), a tensor for a call on `stream` (None: the current stream; else a torch
    stream or its address).  It comes from that stream's memory, whose earlier uses the
    call follows in order; memory of the current stream may still be written by work that
    the call does not wait for.  The caller reads it on the current stream."""
    if stream is None:
        return make()
    ptr, here = _stream_ptr(stream).value or 0, torch.cuda.current_stream(device)
    if ptr == here.cuda_stream:
        return make()
    if not isinstance(stream, torch.cuda.Stream):
        # (ExternalStream takes 0 for "any stream")
        stream = (torch.cuda.ExternalStream(ptr, device=device) if ptr
                  else torch.cuda.default_stream(device))
    with torch.cuda.stream(stream):
        t = make()
    t.record_stream(here)
    return t


class Llatte:
    """A forward handle: weights (non-absorbed, pages' layout) are copied and
    absorbed at construction; `forward` runs the whole sequence module."""

    def __init__(self, dims, layers: Sequence[dict], W_e=None, max_batch: int = 1,
                 max_len: int = 0, max_total: int = 0, lib_path: Optional[str] = None,
                 summaries: Optional[Sequence[dict]] = None):
        self.lib = load_library(lib_path)
        self.dims = dims
        self.cdims = make_dims(dims, max_batch, max_len, max_total)
        self.dt = torch_dtype(dims)
        if len(layers) != len(dims.keep):
            raise ValueError("one weight dict per layer is required")
        keep_alive = []
        arr = (llatte_layer_w * len(layers))()
        for i, w in enumerate(layers):
            for k in LAYER_KEYS:
                if w.get(k) is None:         # W_q or the low-rank query's matrices
                    continue
                t = _host(w[k], self.dt)
                keep_alive.append(t)
                setattr(arr[i], k, t.data_ptr())
        we = None
        if dims.d_out:
            we = _host(W_e, self.dt)
            keep_alive.append(we)
        n_sum = int(getattr(dims, "n_sum", 0))
        sarr = None
        if n_sum:
            if summaries is None or len(summaries) != n_sum:
                raise ValueError(f"{n_sum} summary weight dicts are required")
            sarr = (llatte_summary_w * n_sum)()
            for i, w in enumerate(summaries):
                for k in SUMMARY_KEYS:
                    t = _host(w[k], self.dt)
                    keep_alive.append(t)
                    setattr(sarr[i], k, t.data_ptr())
        h = ctypes.c_void_p()
        rc = self.lib.llatte_create(ctypes.byref(h), ctypes.byref(self.cdims), arr,
                                    _ptr(we), sarr, 0)
        if rc != LLATTE_OK:
            raise LlatteError(rc, "llatte_create")
        self.h = h
        self.last_B = 0

    def per_head_layers(self) -> int:
        """Bit l set: layer l runs MLA in its per-head form on this handle."""
        m = ctypes.c_uint32(0)
        rc = self.lib.llatte_attn_form_mask(self.h, ctypes.byref(m))
        if rc != LLATTE_OK:
            raise LlatteError(rc, "llatte_attn_form_mask")
        return int(m.value)

    def inject_timeout(self, enable: bool = True):
        """Failure-detection aid: the forward calls that follow make a bounded
        wait of the per-head attention run out on purpose (status bit
        DEV_TIMEOUT, output unspecified) until switched off again."""
        rc = self.lib.llatte_inject_timeout(self.h, 1 if enable else 0)
        if rc != LLATTE_OK:
            raise LlatteError(rc, "llatte_inject_timeout")

    def workspace_bytes(self) -> int:
        return int(self.lib.llatte_workspace_bytes(ctypes.byref(self.cdims)))

    def out_shape(self, B: int):
        d = self.dims
        if getattr(d, "n_sum", 0):
            return (B, d.n_sum, d.d_seq)
        return (B, d.d_out) if d.d_out else (B, d.n_q, d.d)

    def _check_inputs(self, values, offsets, context, cand, event_age):
        d = self.dims
        B = int(offsets.numel()) - 1
        if B < 0:
            raise ValueError("offsets needs B+1 entries")
        for name, t, dt in (("values", values, self.dt), ("offsets", offsets, torch.int64),
                            ("context", context, self.dt), ("cand", cand, self.dt),
                            ("event_age", event_age, torch.float32)):
            if t is None:
                continue
            if not t.is_cuda or t.dtype != dt or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous CUDA {dt} tensor")
        if values.dim() != 2 or values.shape[1] != d.d:
            raise ValueError(f"values must be [rows, {d.d}]")
        if d.d_ctx and (context is None or tuple(context.shape) != (B, d.d_ctx)):
            raise ValueError(f"context must be [{B}, {d.d_ctx}]")
        if d.n_q and (cand is None or tuple(cand.shape) != (B, d.n_q, d.d)):
            raise ValueError(f"cand must be [{B}, {d.n_q}, {d.d}]")
        if getattr(d, "d_time", 0) and (event_age is None or event_age.dim() != 1 or
                                        event_age.shape[0] < values.shape[0]):
            raise ValueError("event_age [rows] (hours before the request) is required")
        return B

    def _out(self, out, B, device, stream=None):
        if out is None:
            return _made(lambda: torch.empty(self.out_shape(B), dtype=torch.float32,
                                             device=device), stream, device)
        if (tuple(out.shape) != self.out_shape(B) or out.dtype != torch.float32
                or not out.is_contiguous()):
            raise ValueError(f"out must be a contiguous float32 {self.out_shape(B)} tensor")
        return out

    def _run(self, values, offsets, context, cand, event_age, out, ex, stream, B):
        if ex is None and event_age is None:
            rc = self.lib.llatte_forward(self.h, _ptr(values), _ptr(offsets), B, _ptr(context),
                                         _ptr(cand), _ptr(out), _stream_ptr(stream))
            what = "llatte_forward"
        else:
            b = llatte_batch(values=values.data_ptr(), offsets=offsets.data_ptr(), B=B,
                             context=context.data_ptr() if context is not None else None,
                             cand=cand.data_ptr() if cand is not None else None,
                             event_age=event_age.data_ptr() if event_age is not None else None)
            rc = self.lib.llatte_forward_batch(self.h, ctypes.byref(b), _ptr(out),
                                               ctypes.byref(ex) if ex is not None else None,
                                               _stream_ptr(stream))
            what = "llatte_forward_batch"
        if rc != LLATTE_OK:
            raise LlatteError(rc, what)
        self.last_B = B

    def forward(self, values: torch.Tensor, offsets: torch.Tensor, context=None, cand=None,
                out: Optional[torch.Tensor] = None, stream=None, event_age=None) -> torch.Tensor:
        """One forward pass.  event_age (float32 [rows], hours before the
        request of every history event) is required when dims.d_time > 0."""
        B = self._check_inputs(values, offsets, context, cand, event_age)
        out = self._out(out, B, values.device, stream)
        if not getattr(self.dims, "d_time", 0):
            event_age = None
        self._run(values, offsets, context, cand, event_age, out, None, stream, B)
        return out

    def forward_export(self, values: torch.Tensor, offsets: torch.Tensor, context=None,
                       cand=None, layer: int = 0, n_k: int = 8, event_age=None,
                       n_hours: int = 0, out: Optional[torch.Tensor] = None, stream=None):
        """Forward plus the attention statistics of `layer`'s query tokens:
        returns (out, recent [B, n_q, h, n_k], topk [B, n_q, h, n_k],
        hours [B, n_q, h, n_hours] or None).  event_age serves both the hour
        bins and, when dims.d_time > 0, the timestamp code."""
        d = self.dims
        B = self._check_inputs(values, offsets, context, cand, event_age)
        dev = values.device
        if n_hours and event_age is None:
            raise ValueError("event_age is required for hour bins")

        def made(n):
            return _made(lambda: torch.empty((B, d.n_q, d.heads, n), dtype=torch.float32,
                                             device=dev), stream, dev)
        recent, topk = made(n_k), made(n_k)
        hours = made(n_hours) if n_hours else None
        ex = llatte_attn_export(layer=layer, n_k=n_k, n_hours=n_hours,
                                event_age=event_age.data_ptr() if n_hours else None,
                                recent=recent.data_ptr(), topk=topk.data_ptr(),
                                hours=hours.data_ptr() if hours is not None else None)
        out = self._out(out, B, dev, stream)
        self._run(values, offsets, context, cand,
                  event_age if getattr(d, "d_time", 0) else None, out, ex, stream, B)
        return out, recent, topk, hours

    def query_rows(self) -> int:
        """Most query rows of a call: the max_rows a cache of forward_cached needs."""
        c = self.cdims
        rows = int(c.max_total) or int(c.max_batch) * int(c.max_len)
        return min(rows, int(c.max_batch) * int(c.keep[0])) + int(c.max_batch) * int(c.n_q)

    def forward_cached(self, values: torch.Tensor, offsets: torch.Tensor,
                       caches: Sequence["LatentCache"], tables, lengths: torch.Tensor,
                       context=None, cand=None, window: int = 0, n_sink: int = 0,
                       accumulate: bool = False, out: Optional[torch.Tensor] = None,
                       stream=None) -> torch.Tensor:
        """A forward pass whose `values` are only the new events of every user: layer l
        appends their latents to caches[l] and attends over it.  tables: one page
        table, or one per layer; lengths: cached events, the new ones included.
        Every layer must keep every cached event: no cache may hold (max_pages, or the
        table's width) more pages than min(keep) events take, and a user with more
        than min(keep) events is left out (see llatte_forward_cached)."""
        if getattr(self.dims, "d_time", 0):      # the code of an event changes with the request
            raise LlatteError(LLATTE_ERR_UNSUPPORTED, "llatte_forward_cached")
        _int32(window=window, n_sink=n_sink)
        B = self._check_inputs(values, offsets, context, cand, None)
        n = len(self.dims.keep)
        if len(caches) != n:
            raise ValueError("one cache per layer is required")
        if isinstance(tables, torch.Tensor):
            tables = [tables] * n
        if len(tables) != n:
            raise ValueError("one page table, or one per layer, is required")
        handles = (ctypes.c_void_p * n)(*[c.h for c in caches])
        views = (llatte_cache_view * n)(*[c._view(t, lengths)[0] for c, t in zip(caches, tables)])
        if any(v.B != B for v in views):
            raise ValueError(f"tables and lengths must have {B} users")
        out = self._out(out, B, values.device, stream)
        b = llatte_batch(values=values.data_ptr(), offsets=offsets.data_ptr(), B=B,
                         context=context.data_ptr() if context is not None else None,
                         cand=cand.data_ptr() if cand is not None else None, event_age=None)
        fc = llatte_forward_cache(handles, views, int(window), int(n_sink), 1 if accumulate else 0)
        rc = self.lib.llatte_forward_cached(self.h, ctypes.byref(b), ctypes.byref(fc), _ptr(out),
                                            _stream_ptr(stream))
        if rc != LLATTE_OK:
            raise LlatteError(rc, "llatte_forward_cached")
        self.last_B = B
        return out

    def plan_export(self, stream=None) -> torch.Tensor:
        L, B = len(self.dims.keep), self.last_B
        dst = torch.empty((L, 2, B + 1), dtype=torch.int64, device="cuda")
        rc = self.lib.llatte_plan_export(self.h, _ptr(dst), _stream_ptr(stream))
        if rc != LLATTE_OK:
            raise LlatteError(rc, "llatte_plan_export")
        return dst

    def status(self) -> int:
        v = ctypes.c_int32(0)
        rc = self.lib.llatte_get_status(self.h, ctypes.byref(v))
        if rc not in (LLATTE_OK, LLATTE_ERR_DEVICE):
            raise LlatteError(rc, "llatte_get_status")
        return int(v.value)

    def set_profiling(self, on: bool = True):
        self.lib.llatte_set_profiling(self.h, 1 if on else 0)

    def profile_reset(self):
        self.lib.llatte_profile_reset(self.h)

    def profile(self) -> dict:
        res = {}
        for i in range(len(STEPS)):
            name = ctypes.c_char_p()
            ms = ctypes.c_double()
            nl = ctypes.c_int64()
            nc = ctypes.c_int64()
            rc = self.lib.llatte_profile_step(self.h, i, ctypes.byref(name), ctypes.byref(ms),
                                              ctypes.byref(nl), ctypes.byref(nc))
            if rc != LLATTE_OK:
                raise LlatteError(rc, "llatte_profile_step")
            res[name.value.decode()] = {"ms": ms.value, "launches": nl.value, "calls": nc.value}
        return res

    def close(self):
        if getattr(self, "h", None):
            self.lib.llatte_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def plan_static(dims, offsets: torch.Tensor, max_batch: int, max_len: int, max_total: int = 0,
                stream=None, out: Optional[torch.Tensor] = None,
                status: Optional[torch.Tensor] = None):
    """Pyramid plan of one batch through llatte_plan_static, the entry point
    that allocates no device memory (its scratch is a fixed array inside the
    library).  Pass `out` / `status` to reuse caller-owned buffers.  Returns
    (plan [n_layers, 2, B+1] int64, status int32 tensor)."""
    lib = load_library()
    cd = make_dims(dims, max_batch, max_len, max_total)
    B = int(offsets.numel()) - 1
    if not offsets.is_cuda or offsets.dtype != torch.int64 or not offsets.is_contiguous():
        raise ValueError("offsets must be a contiguous CUDA int64 tensor")
    if out is None:
        out = torch.empty((len(dims.keep), 2, B + 1), dtype=torch.int64, device=offsets.device)
    if status is None:
        status = torch.empty(1, dtype=torch.int32, device=offsets.device)
    if tuple(out.shape) != (len(dims.keep), 2, B + 1) or out.dtype != torch.int64:
        raise ValueError("out must be int64 [n_layers, 2, B+1]")
    rc = lib.llatte_plan_static(ctypes.byref(cd), _ptr(offsets), B, _ptr(out), _ptr(status),
                                _stream_ptr(stream))
    if rc != LLATTE_OK:
        raise LlatteError(rc, "llatte_plan_static")
    return out, status


def exp2_eval(x: torch.Tensor, with_hw: bool = True, stream=None):
    """2^x through the softmax's FMA-pipe exponential (and, with `with_hw`,
    through the hardware ex2.approx) for a contiguous CUDA float32 tensor."""
    lib = load_library()
    if not x.is_cuda or x.dtype != torch.float32 or not x.is_contiguous():
        raise ValueError("x must be a contiguous CUDA float32 tensor")
    y = torch.empty_like(x)
    y_hw = torch.empty_like(x) if with_hw else None
    rc = lib.llatte_exp2_eval(_ptr(x), _ptr(y), _ptr(y_hw), x.numel(), _stream_ptr(stream))
    if rc != LLATTE_OK:
        raise LlatteError(rc, "llatte_exp2_eval")
    return (y, y_hw) if with_hw else y


class Tokenizer:
    """Action tokenizer MLP_act: x_t = W_a2 SiLU(W_a1 [E_1(id_t1); ...; E_F(id_tF)]).

    `tables` are CUDA tensors [rows_f, width_f] in the storage dtype that the
    tokenizer references (not copied): they must stay alive and unchanged.
    W_a1 [d_hid, D_in] and W_a2 [d, d_hid] are copied."""

    def __init__(self, tables, W_a1, W_a2, dtype: str = "bf16", max_events: int = 1 << 20):
        self.lib = load_library()
        self.dt = {"bf16": torch.bfloat16, "fp32": torch.float32}[dtype]
        if not 1 <= len(tables) <= TOK_MAX_FIELDS:
            raise ValueError(f"1 .. {TOK_MAX_FIELDS} tables")
        self.tables = []
        for t in tables:
            if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype == self.dt
                    and t.dim() == 2 and t.is_contiguous()):
                raise ValueError("tables must be contiguous 2-D CUDA tensors of the storage dtype")
            self.tables.append(t)
        w1, w2 = _host(W_a1, self.dt), _host(W_a2, self.dt)
        c = llatte_tok_dims()
        c.n_fields = len(tables)
        for f, t in enumerate(tables):
            c.rows[f], c.width[f] = int(t.shape[0]), int(t.shape[1])
        c.d_hid, c.d = int(w1.shape[0]), int(w2.shape[0])
        if w1.shape[1] != sum(int(t.shape[1]) for t in tables) or w2.shape[1] != c.d_hid:
            raise ValueError("W_a1 must be [d_hid, sum of widths], W_a2 [d, d_hid]")
        c.dtype = LLATTE_BF16 if dtype == "bf16" else LLATTE_FP32
        c.max_events = int(max_events)
        self.cdims = c
        self.d = c.d
        w = llatte_tok_w()
        for f, t in enumerate(tables):
            w.tables[f] = t.data_ptr()
        w.W_a1, w.W_a2 = w1.data_ptr(), w2.data_ptr()
        h = ctypes.c_void_p()
        rc = self.lib.llatte_tokenizer_create(ctypes.byref(h), ctypes.byref(c), ctypes.byref(w), 0)
        if rc != LLATTE_OK:
            raise LlatteError(rc, "llatte_tokenizer_create")
        self.h = h

    def uses_tensor_cores(self) -> bool:
        return self.lib.llatte_tokenizer_uses_tensor_cores(self.h) == 1

    def __call__(self, ids: torch.Tensor, out: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
        """Tokens [n, d] of ids (int32 CUDA [n, n_fields])."""
        if (not ids.is_cuda or ids.dtype != torch.int32 or ids.dim() != 2
                or ids.shape[1] != self.cdims.n_fields or not ids.is_contiguous()):
            raise ValueError("ids must be a contiguous CUDA int32 [n, n_fields] tensor")
        n = int(ids.shape[0])
        if out is None:
            out = torch.empty((n, self.d), dtype=self.dt, device=ids.device)
        elif (tuple(out.shape) != (n, self.d) or out.dtype != self.dt or not out.is_contiguous()):
            raise ValueError(f"out must be a contiguous {self.dt} [{n}, {self.d}] tensor")
        rc = self.lib.llatte_tokenize(self.h, _ptr(ids), n, _ptr(out), _stream_ptr(stream))
        if rc != LLATTE_OK:
            raise LlatteError(rc, "llatte_tokenize")
        return out

    def status(self) -> int:
        v = ctypes.c_int32(0)
        rc = self.lib.llatte_tokenizer_get_status(self.h, ctypes.byref(v))
        if rc not in (LLATTE_OK, LLATTE_ERR_DEVICE):
            raise LlatteError(rc, "llatte_tokenizer_get_status")
        return int(v.value)

    def close(self):
        if getattr(self, "h", None):
            self.lib.llatte_tokenizer_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class LatentCache:
    """Paged cache of users' latent K = V rows, and attention over it.

    pool [n_pages, page_size, rank] (bfloat16 or float32) and mass (float32
    [n_pages, page_size], the attention weight every event has collected) are
    CUDA tensors that the cache references (not copied).  Every call takes the
    page table (int32 [B, pages]) and the lengths (int32 [B], the call's new
    events included) of its users; event t of user u lies in row t % page_size
    of page table[u, t // page_size]."""

    def __init__(self, pool: torch.Tensor, heads: int, mass: Optional[torch.Tensor] = None,
                 max_batch: int = 1, max_rows: int = 1, max_pages: int = 1):
        self.lib = load_library()
        if (not isinstance(pool, torch.Tensor) or not pool.is_cuda or pool.dim() != 3
                or pool.dtype not in (torch.bfloat16, torch.float32) or not pool.is_contiguous()):
            raise ValueError("pool must be a contiguous CUDA bfloat16 or float32 "
                             "[n_pages, page_size, rank] tensor")
        if mass is not None and (tuple(mass.shape) != tuple(pool.shape[:2])
                                 or mass.dtype != torch.float32 or mass.device != pool.device
                                 or not mass.is_contiguous()):
            raise ValueError("mass must be a contiguous float32 [n_pages, page_size] tensor on "
                             "the pool's device")
        self.pool, self.mass, self.heads = pool, mass, int(heads)
        self.n_pages, self.page_size, self.rank = (int(n) for n in pool.shape)
        self.device, self.dt, self.index = pool.device, pool.dtype, pool.get_device()
        _int32(heads=self.heads, max_batch=max_batch, max_pages=max_pages)
        if not -1 << 63 <= max_rows < 1 << 63:
            raise ValueError(f"max_rows = {max_rows} does not fit 64 bits")
        c = llatte_cache_dims()
        c.heads, c.rank, c.page_size, c.n_pages = self.heads, self.rank, self.page_size, self.n_pages
        c.dtype = LLATTE_BF16 if self.dt == torch.bfloat16 else LLATTE_FP32
        c.max_batch, c.max_pages, c.max_rows = int(max_batch), int(max_pages), int(max_rows)
        self.cdims = c
        h = ctypes.c_void_p()
        with torch.cuda.device(self.device):
            rc = self.lib.llatte_cache_create(ctypes.byref(h), ctypes.byref(c), _ptr(pool),
                                              _ptr(mass))
        if rc != LLATTE_OK:
            raise LlatteError(rc, "llatte_cache_create")
        self.h = h

    def workspace_bytes(self) -> int:
        return int(self.lib.llatte_cache_workspace_bytes(ctypes.byref(self.cdims)))

    def uses_tensor_cores(self) -> bool:
        return self.lib.llatte_cache_uses_tensor_cores(self.h) == 1

    # A call is a few microseconds of device time at its smallest, so its checks are
    # kept to one pass over each tensor; _refuse words the error.
    def _fits(self, t, dtype, dims):
        return (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == self.index
                and t.dim() == dims and t.is_contiguous())

    def _refuse(self, name, dtype, shape):
        raise ValueError(f"{name} must be a contiguous {dtype} [{shape}] tensor on {self.device}")

    def _view(self, table, lengths):
        if not self._fits(lengths, torch.int32, 1):
            self._refuse("lengths", torch.int32, "*")
        B = lengths.shape[0]
        if not self._fits(table, torch.int32, 2) or table.shape[0] != B:
            self._refuse("table", torch.int32, f"{B}, *")
        return llatte_cache_view(table.data_ptr(), table.shape[1], lengths.data_ptr(), B), B

    def _on(self, stream):
        return _raw_stream(self.index) if stream is None else _stream_ptr(stream)

    def append(self, x: torch.Tensor, offsets: torch.Tensor, table: torch.Tensor,
               lengths: torch.Tensor, gain: Optional[torch.Tensor] = None, eps: float = 1e-6,
               stream=None):
        """Rows x[offsets[u]:offsets[u + 1]] become user u's newest events (lengths
        counts them already); with `gain` each is RMS-normalised first.  Their masses
        are set to 0, also where the same rows are appended again."""
        v, B = self._view(table, lengths)
        if not self._fits(x, self.dt, 2) or x.shape[1] != self.rank:
            self._refuse("x", self.dt, f"*, {self.rank}")
        if not self._fits(offsets, torch.int64, 1) or offsets.shape[0] != B + 1:
            self._refuse("offsets", torch.int64, B + 1)
        if gain is not None and (not self._fits(gain, self.dt, 1) or gain.shape[0] != self.rank):
            self._refuse("gain", self.dt, self.rank)
        rc = self.lib.llatte_cache_append(
            self.h, ctypes.byref(v), x.data_ptr(), x.shape[0], offsets.data_ptr(),
            None if gain is None else gain.data_ptr(), eps, self._on(stream))
        if rc != LLATTE_OK:
            raise LlatteError(rc, "llatte_cache_append")

    def attend(self, q: torch.Tensor, q_offsets: torch.Tensor, table: torch.Tensor,
               lengths: torch.Tensor, n_cand: int = 0, scale: float = 1.0, window: int = 0,
               n_sink: int = 0, out: Optional[torch.Tensor] = None,
               lse: Optional[torch.Tensor] = None, accumulate: bool = False,
               stream=None) -> torch.Tensor:
        """Attention of the query rows q [rows, heads, rank] over the cache.  User u's
        rows are q_offsets[u] .. q_offsets[u + 1] - 1: its newest events (already
        appended), then its last n_cand rows, query tokens that see every event.
        `window` > 0 limits a row to that many events back from its position and
        the first n_sink.  `lse` (float32 [rows, heads]) receives the log of the
        softmax denominators; `accumulate` adds all weights to `mass`."""
        _int32(n_cand=n_cand, window=window, n_sink=n_sink)
        v, B = self._view(table, lengths)
        if not self._fits(q, self.dt, 3) or q.shape[1:] != (self.heads, self.rank):
            self._refuse("q", self.dt, f"*, {self.heads}, {self.rank}")
        rows = q.shape[0]
        if not self._fits(q_offsets, torch.int64, 1) or q_offsets.shape[0] != B + 1:
            self._refuse("q_offsets", torch.int64, B + 1)
        if out is None:
            out = _made(lambda: torch.empty_like(q), stream, self.device)
        elif not self._fits(out, self.dt, 3) or out.shape != q.shape:
            self._refuse("out", self.dt, f"{rows}, {self.heads}, {self.rank}")
        if lse is not None and (not self._fits(lse, torch.float32, 2)
                                or lse.shape != (rows, self.heads)):
            self._refuse("lse", torch.float32, f"{rows}, {self.heads}")
        a = llatte_cache_attn(q.data_ptr(), q_offsets.data_ptr(), rows, n_cand, scale, window,
                              n_sink, out.data_ptr(), None if lse is None else lse.data_ptr(),
                              1 if accumulate else 0)
        rc = self.lib.llatte_cache_attend(self.h, ctypes.byref(v), ctypes.byref(a),
                                          self._on(stream))
        if rc != LLATTE_OK:
            raise LlatteError(rc, "llatte_cache_attend")
        return out

    def evict(self, table: torch.Tensor, lengths: torch.Tensor, budget: int, n_sink: int = 0,
              n_recent: int = 0, dst_table: Optional[torch.Tensor] = None,
              new_lengths: Optional[torch.Tensor] = None, kept: Optional[torch.Tensor] = None,
              stream=None) -> torch.Tensor:
        """Keep at most `budget` events per user: the first n_sink, the last n_recent
        and the heaviest of the others by `mass`, packed in order into the pages
        of dst_table, which `table` may not name (default: in place, into the user's
        own first pages).  Returns the new
        lengths; `kept` (int32 [B, budget]) receives the old slots.  A user left out
        (see the status) keeps what new_lengths held, by default the length given."""
        _int32(budget=budget, n_sink=n_sink, n_recent=n_recent)
        v, B = self._view(table, lengths)
        if new_lengths is None:              # a user left out keeps its length
            new_lengths = _made(lambda: lengths.clone(), stream, self.device)
        elif not self._fits(new_lengths, torch.int32, 1) or new_lengths.shape[0] != B:
            self._refuse("new_lengths", torch.int32, B)
        if dst_table is not None and (not self._fits(dst_table, torch.int32, 2)
                                      or dst_table.shape[0] != B):
            self._refuse("dst_table", torch.int32, f"{B}, *")
        if kept is not None and (not self._fits(kept, torch.int32, 2)
                                 or kept.shape != (B, budget)):
            self._refuse("kept", torch.int32, f"{B}, {budget}")
        a = llatte_cache_evict_args(
            budget, n_sink, n_recent, None if dst_table is None else dst_table.data_ptr(),
            0 if dst_table is None else dst_table.shape[1], new_lengths.data_ptr(),
            None if kept is None else kept.data_ptr())
        rc = self.lib.llatte_cache_evict(self.h, ctypes.byref(v), ctypes.byref(a),
                                         self._on(stream))
        if rc != LLATTE_OK:
            raise LlatteError(rc, "llatte_cache_evict")
        return new_lengths

    def inject_timeout(self, enable: bool = True):
        """Failure-detection aid: the attention calls that follow make a bounded wait run
        out on purpose (status bit DEV_TIMEOUT, outputs and accumulated masses
        unspecified) until switched off again."""
        rc = self.lib.llatte_cache_inject_timeout(self.h, 1 if enable else 0)
        if rc != LLATTE_OK:
            raise LlatteError(rc, "llatte_cache_inject_timeout")

    def status(self) -> int:
        v = ctypes.c_int32(0)
        rc = self.lib.llatte_cache_get_status(self.h, ctypes.byref(v))
        if rc not in (LLATTE_OK, LLATTE_ERR_DEVICE):
            raise LlatteError(rc, "llatte_cache_get_status")
        return int(v.value)

    def close(self):
        if getattr(self, "h", None):
            self.lib.llatte_cache_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
