"""The paged 8-bit cache and prompt attention (``include/kvq.h``): the calls of
a serving loop over a changing set of requests.

A step::

    plan = cache.reserve(lens, new_tokens, table, free_pages, free_count, max_tokens)
    for layer in range(num_layers):
        cache.write(layer, k, v, plan.cu_tokens, plan.slots, plan.lens)
        o = prompt_attention(q, k, v, plan.cu_tokens, scale)     # prompts, or
        o = cache.decode(layer, q, table, plan.lens, scale)      # one token per request
    cache.release(done, plan.lens, table, free_pages, free_count)

Lengths, tables, slots and the free list are int32 tensors on the cache's
device; no call copies them to the host, so a step can be captured into a CUDA
graph and replayed.
"""
from __future__ import annotations

import ctypes
from collections import namedtuple

import torch

PAGE_INT8 = 0
PAGE_E4M3 = 1
_DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}

_P = ctypes.c_void_p
_I = ctypes.c_int32
_L = ctypes.c_int64


class PagedConfig(ctypes.Structure):
    _fields_ = [(n, _I) for n in ("num_layers", "max_requests", "num_kv_heads", "head_dim", "page_tokens",
                                  "num_pages", "max_pages", "code", "dtype")]


class PagedLayout(ctypes.Structure):
    _fields_ = [(n, _L) for n in ("pages_bytes", "scales_bytes", "tails_bytes")] + [
        (n, _P) for n in ("pages", "scales", "tails")]


SIGNATURES = {
    "kvq_paged_cache_bytes": [ctypes.POINTER(PagedConfig), ctypes.POINTER(ctypes.c_size_t)],
    "kvq_paged_cache_create": [ctypes.POINTER(PagedConfig), _P, ctypes.c_size_t, _P, ctypes.POINTER(_P)],
    "kvq_paged_cache_destroy": [_P],
    "kvq_paged_cache_get_layout": [_P, _I, ctypes.POINTER(PagedLayout)],
    "kvq_paged_cache_status": [_P, _P, ctypes.POINTER(ctypes.c_uint32)],
    "kvq_paged_reserve": [_P, _I] + [_P] * 5 + [_I] + [_P] * 6,
    "kvq_paged_release": [_P, _I] + [_P] * 6,
    "kvq_paged_write": [_P, _I, _I, _P, _P, _L, _L, _I, _P, _P, _P, _P],
    "kvq_paged_decode_workspace_bytes": [_P, _I, ctypes.POINTER(ctypes.c_size_t)],
    "kvq_paged_decode_attention": [_P, _I, _I, _P, _L, _I, _P, _P, ctypes.c_float, _P, _I, _P, ctypes.c_size_t, _P],
    "kvq_prompt_attention": [_P, _P, _P, _L, _L, _L, _I, _I, _P, _I, _I, _I, _I, ctypes.c_float, _P, _P, _P],
}

#: What reserve() planned: prefix sums of the new tokens, the slot and the
#: position of each packed token, the lengths and the free count after the step.
StepPlan = namedtuple("StepPlan", "cu_tokens slots positions lens free_count")


def _kvq():
    from . import lib, check, _stream_ptr
    return lib(), check, _stream_ptr


def _empty(shape, dtype, device, stream):
    """A new tensor for a kernel on ``stream``: allocated there, so that its
    memory is not reused from or given back to another stream's work."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _ints(t, name, shape, device):
    if not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or t.device != device:
        raise TypeError("%s must be an int32 tensor on %s" % (name, device))
    if tuple(t.shape) != shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), shape))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _rows(t, name, dtype, device, heads=None, dim=None):
    """(pointer, token stride) of packed rows [token][head][channel]: the
    tokens may lie apart (a slice of a fused projection), a row may not."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.device != device:
        raise TypeError("%s must be a %s tensor on %s" % (name, dtype, device))
    if t.dim() != 3 or (heads is not None and t.shape[1] != heads) or (dim is not None and t.shape[2] != dim):
        raise ValueError("%s has shape %s, expected [tokens][%s][%s]" % (name, tuple(t.shape), heads, dim))
    _, h, d = t.shape
    st, sh, sd = t.stride()
    if (sd != 1 and d > 1) or (sh != d and h > 1):
        raise ValueError("the rows of %s must be contiguous" % name)
    if t.shape[0] <= 1:  # its stride is not read
        st = h * d
    return t.data_ptr(), st


class PagedKVCache:
    """A paged 8-bit KV cache in one torch-owned device buffer, driven through
    the C ABI. ``dtype`` is the type of K, V and Q."""

    def __init__(self, num_layers, max_requests, num_kv_heads, head_dim, page_tokens, num_pages, max_pages,
                 code=PAGE_INT8, dtype=torch.float16, device=None, stream=None):
        lib, check, stream_ptr = _kvq()
        if dtype not in (torch.float16, torch.bfloat16):
            raise TypeError("dtype must be torch.float16 or torch.bfloat16")
        self.cfg = PagedConfig(num_layers, max_requests, num_kv_heads, head_dim, page_tokens, num_pages, max_pages,
                               code, _DTYPES[dtype])
        self.dtype = dtype
        n = ctypes.c_size_t()
        check(lib.kvq_paged_cache_bytes(ctypes.byref(self.cfg), ctypes.byref(n)))
        self.nbytes = n.value
        self.buffer = torch.empty(self.nbytes, dtype=torch.uint8, device=device if device is not None else "cuda")
        self.device = self.buffer.device
        h = _P()
        check(lib.kvq_paged_cache_create(ctypes.byref(self.cfg), self.buffer.data_ptr(), self.nbytes,
                                         stream_ptr(stream), ctypes.byref(h)))
        self.handle = h
        self._ws = {}

    # -- hot path -----------------------------------------------------------
    def reserve(self, lens, new_tokens, table, free_pages, free_count, max_tokens, lens_out=None,
                free_count_out=None, plan=None, stream=None):
        """Plans a step (kvq_paged_reserve): new table entries in place, the
        rest as a StepPlan. ``plan``: an earlier step's StepPlan whose tensors
        are written again (for captured steps); lens_out / free_count_out may
        be ``lens`` / ``free_count``."""
        lib, check, stream_ptr = _kvq()
        c, dev = self.cfg, self.device
        r = lens.shape[0]
        if plan is None:
            # one allocation, cut up
            cu, slots, positions, lo, fo = _empty(2 * r + 2 + 2 * max_tokens, torch.int32, dev, stream).split(
                [r + 1, max_tokens, max_tokens, r, 1])
            plan = StepPlan(cu, slots, positions, lens_out if lens_out is not None else lo,
                            free_count_out if free_count_out is not None else fo)
        elif lens_out is not None or free_count_out is not None:
            raise ValueError("plan already names the outputs")
        check(lib.kvq_paged_reserve(
            self.handle, r, _ints(lens, "lens", (r,), dev), _ints(new_tokens, "new_tokens", (r,), dev),
            _ints(table, "table", (r, c.max_pages), dev), _ints(free_pages, "free_pages", (c.num_pages,), dev),
            _ints(free_count, "free_count", (1,), dev), max_tokens, _ints(plan.cu_tokens, "cu_tokens", (r + 1,), dev),
            _ints(plan.slots, "slots", (max_tokens,), dev), _ints(plan.positions, "positions", (max_tokens,), dev),
            _ints(plan.lens, "lens_out", (r,), dev), _ints(plan.free_count, "free_count_out", (1,), dev),
            stream_ptr(stream)))
        return plan

    def release(self, done, lens, table, free_pages, free_count, stream=None):
        """Ends the requests with done != 0 (kvq_paged_release), in place."""
        lib, check, stream_ptr = _kvq()
        c, dev = self.cfg, self.device
        r = lens.shape[0]
        check(lib.kvq_paged_release(
            self.handle, r, _ints(done, "done", (r,), dev), _ints(lens, "lens", (r,), dev),
            _ints(table, "table", (r, c.max_pages), dev), _ints(free_pages, "free_pages", (c.num_pages,), dev),
            _ints(free_count, "free_count", (1,), dev), stream_ptr(stream)))

    def write(self, layer, k, v, cu_tokens, slots, lens, stream=None):
        """Writes the step's packed tokens (kvq_paged_write). ``lens``: the
        lengths after the step."""
        lib, check, stream_ptr = _kvq()
        c, dev = self.cfg, self.device
        r = lens.shape[0]
        kp, ks = _rows(k, "k", self.dtype, dev, c.num_kv_heads, c.head_dim)
        vp, vs = _rows(v, "v", self.dtype, dev, c.num_kv_heads, c.head_dim)
        t = k.shape[0]
        if v.shape[0] != t:
            raise ValueError("k and v hold %d and %d tokens" % (t, v.shape[0]))
        check(lib.kvq_paged_write(self.handle, layer, r, kp, vp, ks, vs, t,
                                  _ints(cu_tokens, "cu_tokens", (r + 1,), dev), _ints(slots, "slots", (t,), dev),
                                  _ints(lens, "lens", (r,), dev), stream_ptr(stream)))

    def workspace_bytes(self, num_q_heads):
        lib, check, _ = _kvq()
        n = ctypes.c_size_t()
        check(lib.kvq_paged_decode_workspace_bytes(self.handle, num_q_heads, ctypes.byref(n)))
        return n.value

    def workspace(self, num_q_heads):
        """The cache's own workspace for decode(): calls that overlap on the
        GPU need one each (``workspace=``)."""
        ws = self._ws.get(num_q_heads)
        if ws is None:
            ws = torch.empty(self.workspace_bytes(num_q_heads), dtype=torch.uint8, device=self.device)
            self._ws[num_q_heads] = ws
        return ws

    def decode(self, layer, q, table, lens, softmax_scale, out=None, out_dtype=None, workspace=None, stream=None):
        """Attention of one query token per request (kvq_paged_decode_attention):
        q [requests][H_q][D] -> out [requests][H_q][D], zeros where lens is 0."""
        lib, check, stream_ptr = _kvq()
        c, dev = self.cfg, self.device
        qp, qs = _rows(q, "q", self.dtype, dev, dim=c.head_dim)
        r, hq, d = q.shape
        if out is None:
            out = _empty((r, hq, d), out_dtype or self.dtype, dev, stream)
        elif tuple(out.shape) != (r, hq, d) or out.device != dev or not out.is_contiguous() or out.dtype not in _DTYPES:
            raise ValueError("out must be a contiguous tensor of shape %s on %s" % ((r, hq, d), dev))
        ws = self.workspace(hq) if workspace is None else workspace
        check(lib.kvq_paged_decode_attention(
            self.handle, layer, r, qp, qs, hq, _ints(table, "table", (r, c.max_pages), dev),
            _ints(lens, "lens", (r,), dev), softmax_scale, out.data_ptr(), _DTYPES[out.dtype], ws.data_ptr(),
            ws.numel() * ws.element_size(), stream_ptr(stream)))
        return out

    # -- inspection ---------------------------------------------------------
    def _view(self, layer, name, shape, dtype):
        lib, check, _ = _kvq()
        lo = PagedLayout()
        check(lib.kvq_paged_cache_get_layout(self.handle, layer, ctypes.byref(lo)))
        off = getattr(lo, name) - self.buffer.data_ptr()
        return self.buffer[off:off + getattr(lo, name + "_bytes")].view(dtype).view(shape)

    def pages(self, layer):
        """Codes [page][kv head][K, V][token][channel]: int8, or uint8 bits of
        torch.float8_e4m3fn."""
        c = self.cfg
        return self._view(layer, "pages", (c.num_pages, c.num_kv_heads, 2, c.page_tokens, c.head_dim),
                          torch.int8 if c.code == PAGE_INT8 else torch.uint8)

    def scales(self, layer):
        """fp32 [page][kv head][K, V]."""
        c = self.cfg
        return self._view(layer, "scales", (c.num_pages, c.num_kv_heads, 2), torch.float32)

    def tails(self, layer):
        """Rows of the open pages [request][kv head][K, V][token][channel]."""
        c = self.cfg
        return self._view(layer, "tails", (c.max_requests, c.num_kv_heads, 2, c.page_tokens, c.head_dim), self.dtype)

    def status(self, stream=None):
        """Synchronizes and clears the status word; raises KVQError if it was set."""
        lib, check, stream_ptr = _kvq()
        w = ctypes.c_uint32()
        check(lib.kvq_paged_cache_status(self.handle, stream_ptr(stream), ctypes.byref(w)))
        return w.value

    def close(self):
        if getattr(self, "handle", None):
            _kvq()[0].kvq_paged_cache_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def prompt_attention(q, k, v, cu_tokens, softmax_scale, out=None, status=None, stream=None):
    """Causal attention over packed prompts (kvq_prompt_attention): q
    [tokens][H_q][D], k and v [tokens][H_kv][D] in fp16 or bf16, cu_tokens
    int32 [sequences + 1]. Rows of ``out`` outside every sequence are left as
    they are (uninitialised where ``out`` is not given)."""
    lib, check, stream_ptr = _kvq()
    if not isinstance(q, torch.Tensor) or q.dtype not in (torch.float16, torch.bfloat16) or not q.is_cuda:
        raise TypeError("q must be a CUDA float16 or bfloat16 tensor")
    dev = q.device
    qp, qs = _rows(q, "q", q.dtype, dev)
    t, hq, d = q.shape
    kp, ks = _rows(k, "k", q.dtype, dev, dim=d)
    vp, vs = _rows(v, "v", q.dtype, dev, heads=k.shape[1], dim=d)
    if k.shape[0] != t or v.shape[0] != t:
        raise ValueError("q, k and v hold %d, %d and %d tokens" % (t, k.shape[0], v.shape[0]))
    if out is None:
        out = _empty((t, hq, d), q.dtype, dev, stream)
    elif tuple(out.shape) != (t, hq, d) or out.dtype != q.dtype or out.device != dev or not out.is_contiguous():
        raise ValueError("out must be a contiguous %s tensor of shape %s on %s" % (q.dtype, (t, hq, d), dev))
    seqs = cu_tokens.shape[0] - 1
    check(lib.kvq_prompt_attention(
        qp, kp, vp, qs, ks, vs, t, seqs, _ints(cu_tokens, "cu_tokens", (seqs + 1,), dev), hq, k.shape[1], d,
        _DTYPES[q.dtype], softmax_scale, out.data_ptr(),
        None if status is None else _ints(status, "status", (1,), dev), stream_ptr(stream)))
    return out
