"""The paged 8-bit cache and prompt attention (``include/kvq.h``): the calls of
a serving loop over a changing set of requests.

A step::

    plan = cache.reserve(lens, new_tokens, table, free_pages, free_count, max_tokens)
    for layer in range(num_layers):
        q, k = norm_rotate(q, k, plan.positions, rotation, q_weight, k_weight)           # where the model has it
        cache.write(layer, k, v, plan.cu_tokens, plan.slots, plan.lens)
        o = prompt_attention(q, k, v, plan.cu_tokens, scale, status=cache.status_word)   # whole prompts, or
        o = cache.decode(layer, q, table, plan.lens, scale)                              # one token per request, or
        o = cache.attend(layer, q, plan.cu_tokens, table, plan.lens, scale)              # any number of each
    cache.release(done, plan.lens, table, free_pages, plan.free_count)
    cache.status()                                               # whether a call found something amiss

Requests may branch: ``cache.fork(src, dst, plan.lens, table, free_pages,
plan.free_count, shared)`` makes requests ``dst`` of requests ``src``, on the same complete
pages, and ``release(..., shared=shared)`` gives a page back with its last holder.

Rejected drafts are taken back by a smaller length, no further than the start of the request's
open page (kvq.h has the rule); where drafts may complete a page, a fork takes them.

Lengths, tables, slots and the free list are int32 tensors on the cache's
device; no call copies them to the host, so a step can be captured into a CUDA
graph and replayed.
"""
from __future__ import annotations

import ctypes
import math
from collections import namedtuple
from fractions import Fraction

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
    "kvq_paged_release_shared": [_P, _I] + [_P] * 7,
    "kvq_paged_fork": [_P, _I, _I] + [_P] * 8,
    "kvq_paged_write": [_P, _I, _I, _P, _P, _L, _L, _I, _P, _P, _P, _P],
    "kvq_paged_decode_workspace_bytes": [_P, _I, ctypes.POINTER(ctypes.c_size_t)],
    "kvq_paged_decode_attention": [_P, _I, _I, _P, _L, _I, _P, _P, ctypes.c_float, _P, _I, _P, ctypes.c_size_t, _P],
    "kvq_paged_attention_workspace_bytes": [_P, _I, ctypes.POINTER(ctypes.c_size_t)],
    "kvq_paged_attention": [_P, _I, _I, _P, _L, _I, _I, _P, _P, _P, ctypes.c_float, _P, _P, ctypes.c_size_t, _P],
    "kvq_norm_rotate": [_P, _P, _L, _L] + [_I] * 5 + [_P, _P, _I, _I, ctypes.c_float, _P, _P, ctypes.c_float, _P, _P,
                                                      _L, _L, _P],
    "kvq_prompt_attention": [_P, _P, _P, _L, _L, _L, _I, _I, _P, _I, _I, _I, _I, ctypes.c_float, _P, _P, _P],
}

_TWO_PI = 2 * Fraction("3.14159265358979323846264338327950288419716939937510")

#: What reserve() planned: prefix sums of the new tokens, the slot and the
#: position of each packed token, the lengths and the free count after the step.
StepPlan = namedtuple("StepPlan", "cu_tokens slots positions lens free_count")


_lib = None
_Tensor, _int32 = torch.Tensor, torch.int32
_current_stream = torch._C._cuda_getCurrentRawStream
_capturing = torch.cuda.is_current_stream_capturing


def _bind():
    """The library's entry points and the error check, looked up once: the calls
    below are made per layer and step, where the host's time counts."""
    global _lib, _check
    from . import check, lib
    _lib, _check = lib(), check
    return _lib


def _raw_stream(stream, device):
    if stream is not None:
        return stream.cuda_stream
    return _current_stream(device.index)


def _empty(shape, dtype, device, stream):
    """A new tensor for a kernel on ``stream``: allocated there, so that its
    memory is not reused from or given back to another stream's work."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _captured(stream):
    """Whether a graph is being captured on the stream that a call goes to."""
    if stream is None:
        return _capturing()
    with torch.cuda.stream(stream):
        return _capturing()


def _ints(t, name, shape, device):
    """Pointer of an int32 tensor of the given shape."""
    if not isinstance(t, _Tensor) or t.dtype is not _int32 or t.device != device:
        raise TypeError("%s must be an int32 tensor on %s" % (name, device))
    if t.shape != shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), shape))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _rows(t, name, dtype, device, heads=None, dim=None):
    """(pointer, token stride) of packed rows [token][head][channel]: the
    tokens may lie apart (a slice of a fused projection), a row may not."""
    if not isinstance(t, _Tensor) or t.dtype is not dtype or t.device != device:
        raise TypeError("%s must be a %s tensor on %s" % (name, dtype, device))
    shape = t.shape
    if len(shape) != 3 or (heads is not None and shape[1] != heads) or (dim is not None and shape[2] != dim):
        raise ValueError("%s has shape %s, expected [tokens][%s][%s]" % (name, tuple(shape), heads, dim))
    n, h, d = shape
    st, sh, sd = t.stride()
    if (sd != 1 and d > 1) or (sh != d and h > 1):
        raise ValueError("the rows of %s must be contiguous" % name)
    return t.data_ptr(), st if n > 1 else h * d  # of one token the stride is not read


class PagedKVCache:
    """A paged 8-bit KV cache in one torch-owned device buffer, driven through
    the C ABI. ``dtype`` is the type of K, V and Q. The buffer is allocated and
    zeroed on ``stream`` (default: the current one): calls on other streams are
    ordered after that by the caller, and done before the cache is dropped."""

    def __init__(self, num_layers, max_requests, num_kv_heads, head_dim, page_tokens, num_pages, max_pages,
                 code=PAGE_INT8, dtype=torch.float16, device=None, stream=None):
        lib = _lib or _bind()
        if dtype not in (torch.float16, torch.bfloat16):
            raise TypeError("dtype must be torch.float16 or torch.bfloat16")
        self.cfg = PagedConfig(num_layers, max_requests, num_kv_heads, head_dim, page_tokens, num_pages, max_pages,
                               code, _DTYPES[dtype])
        self.dtype = dtype
        n = ctypes.c_size_t()
        _check(lib.kvq_paged_cache_bytes(ctypes.byref(self.cfg), ctypes.byref(n)))
        self.nbytes = n.value
        self.buffer = _empty(self.nbytes, torch.uint8, device if device is not None else "cuda", stream)
        self.device = self.buffer.device
        h = _P()
        _check(lib.kvq_paged_cache_create(ctypes.byref(self.cfg), self.buffer.data_ptr(), self.nbytes,
                                          _raw_stream(stream, self.device), ctypes.byref(h)))
        self.handle = h
        #: The device word that status() reads, int32 [1]: given to prompt_attention
        #: as ``status``, it collects that call's bits too.
        self.status_word = self.buffer[:4].view(_int32)
        self._ws_bytes, self._ws = {}, {}
        self._views = {}
        self._table_pages, self._all_pages = max_pages, num_pages
        self._heads, self._dim = num_kv_heads, head_dim

    # -- hot path -----------------------------------------------------------
    def reserve(self, lens, new_tokens, table, free_pages, free_count, max_tokens, lens_out=None,
                free_count_out=None, plan=None, stream=None):
        """Plans a step (kvq_paged_reserve): new table entries in place, the
        rest as a StepPlan. ``plan``: an earlier step's StepPlan whose tensors
        are written again (for captured steps); lens_out / free_count_out may
        be ``lens`` / ``free_count``."""
        lib = _lib or _bind()
        dev = self.device
        r = lens.shape[0]
        table_p = _ints(table, "table", (r, self._table_pages), dev)
        if plan is None:
            # one allocation, cut up; what is cut here needs no check
            t = max_tokens
            if t < 0:
                raise ValueError("max_tokens must be >= 0")
            buf = _empty(2 * r + 2 + 2 * t, _int32, dev, stream)
            slots, positions, cu, lo, fo = buf.split_with_sizes([t, t, r + 1, r, 1])
            slots_p = buf.data_ptr()
            positions_p = slots_p + 4 * t
            cu_p = positions_p + 4 * t
            lo_p = cu_p + 4 * (r + 1)
            fo_p = lo_p + 4 * r
            if lens_out is not None:
                lo, lo_p = lens_out, _ints(lens_out, "lens_out", (r,), dev)
            if free_count_out is not None:
                fo, fo_p = free_count_out, _ints(free_count_out, "free_count_out", (1,), dev)
            plan = StepPlan(cu, slots, positions, lo, fo)
        elif lens_out is not None or free_count_out is not None:
            raise ValueError("plan already names the outputs")
        else:
            cu_p = _ints(plan.cu_tokens, "cu_tokens", (r + 1,), dev)
            slots_p = _ints(plan.slots, "slots", (max_tokens,), dev)
            positions_p = _ints(plan.positions, "positions", (max_tokens,), dev)
            lo_p = _ints(plan.lens, "lens_out", (r,), dev)
            fo_p = _ints(plan.free_count, "free_count_out", (1,), dev)
        _check(lib.kvq_paged_reserve(
            self.handle, r, _ints(lens, "lens", (r,), dev), _ints(new_tokens, "new_tokens", (r,), dev), table_p,
            _ints(free_pages, "free_pages", (self._all_pages,), dev), _ints(free_count, "free_count", (1,), dev),
            max_tokens, cu_p, slots_p, positions_p, lo_p, fo_p, _raw_stream(stream, dev)))
        return plan

    def release(self, done, lens, table, free_pages, free_count, stream=None, shared=None):
        """Ends the requests with done != 0, in place (kvq_paged_release; with
        ``shared``, as fork() keeps it, kvq_paged_release_shared)."""
        lib = _lib or _bind()
        dev = self.device
        r = lens.shape[0]
        args = (self.handle, r, _ints(done, "done", (r,), dev), _ints(lens, "lens", (r,), dev),
                _ints(table, "table", (r, self._table_pages), dev), _ints(free_pages, "free_pages", (self._all_pages,), dev),
                _ints(free_count, "free_count", (1,), dev))
        raw = _raw_stream(stream, dev)
        if shared is None:
            _check(lib.kvq_paged_release(*args, raw))
        else:
            _check(lib.kvq_paged_release_shared(*args, _ints(shared, "shared", (self._all_pages,), dev), raw))

    def fork(self, src, dst, lens, table, free_pages, free_count, shared, stream=None):
        """Request dst[i], which is empty, becomes a copy of request src[i] on the
        same complete pages, in place (kvq_paged_fork); pairs with src[i] < 0 are left
        out. ``shared``: int32 [pages], zeros where nothing is shared yet; requests that
        share pages end by release(..., shared=shared)."""
        lib = _lib or _bind()
        dev = self.device
        r, n = lens.shape[0], src.shape[0]
        _check(lib.kvq_paged_fork(
            self.handle, r, n, _ints(src, "src", (n,), dev), _ints(dst, "dst", (n,), dev), _ints(lens, "lens", (r,), dev),
            _ints(table, "table", (r, self._table_pages), dev), _ints(free_pages, "free_pages", (self._all_pages,), dev),
            _ints(free_count, "free_count", (1,), dev), _ints(shared, "shared", (self._all_pages,), dev),
            _raw_stream(stream, dev)))

    def write(self, layer, k, v, cu_tokens, slots, lens, stream=None):
        """Writes the step's packed tokens (kvq_paged_write). ``lens``: the
        lengths after the step."""
        lib = _lib or _bind()
        dev = self.device
        r = lens.shape[0]
        kp, ks = _rows(k, "k", self.dtype, dev, self._heads, self._dim)
        vp, vs = _rows(v, "v", self.dtype, dev, self._heads, self._dim)
        t = k.shape[0]
        if v.shape[0] != t:
            raise ValueError("k and v hold %d and %d tokens" % (t, v.shape[0]))
        _check(lib.kvq_paged_write(self.handle, layer, r, kp, vp, ks, vs, t,
                                  _ints(cu_tokens, "cu_tokens", (r + 1,), dev), _ints(slots, "slots", (t,), dev),
                                  _ints(lens, "lens", (r,), dev), _raw_stream(stream, dev)))

    def workspace_bytes(self, num_q_heads, attend=False):
        """Bytes of a workspace of decode(), or of attend()."""
        n = self._ws_bytes.get((num_q_heads, attend))
        if n is None:
            size = ctypes.c_size_t()
            f = _lib.kvq_paged_attention_workspace_bytes if attend else _lib.kvq_paged_decode_workspace_bytes
            _check(f(self.handle, num_q_heads, ctypes.byref(size)))
            n = self._ws_bytes[num_q_heads, attend] = size.value
        return n

    def _workspace(self, hq, raw, stream, attend=False):
        if _captured(stream):
            return _empty(self.workspace_bytes(hq, attend), torch.uint8, self.device, stream)
        ws = self._ws.get((hq, attend, raw))
        if ws is None:
            ws = self._ws[hq, attend, raw] = _empty(self.workspace_bytes(hq, attend), torch.uint8, self.device, stream)
        return ws

    def decode(self, layer, q, table, lens, softmax_scale, out=None, out_dtype=None, workspace=None, stream=None):
        """Attention of one query token per request (kvq_paged_decode_attention):
        q [requests][H_q][D] -> out [requests][H_q][D], zeros where lens is 0.
        Without ``workspace`` the cache keeps one for each stream, and a captured
        call takes one of its own from the graph's memory pool: neither streams nor
        graphs share it (but graphs that share a pool, which replay in turn)."""
        lib = _lib or _bind()
        dev = self.device
        qp, qs = _rows(q, "q", self.dtype, dev, dim=self._dim)
        r, hq, d = q.shape
        if out is None:
            out = _empty((r, hq, d), out_dtype or self.dtype, dev, stream)
        elif tuple(out.shape) != (r, hq, d) or out.device != dev or not out.is_contiguous() or out.dtype not in _DTYPES:
            raise ValueError("out must be a contiguous tensor of shape %s on %s" % ((r, hq, d), dev))
        raw = _raw_stream(stream, dev)
        if workspace is None:
            ws = self._workspace(hq, raw, stream)
        else:
            ws = workspace
            if not isinstance(ws, _Tensor) or ws.device != dev or not ws.is_contiguous():
                raise TypeError("workspace must be a contiguous tensor on %s" % dev)
        _check(lib.kvq_paged_decode_attention(
            self.handle, layer, r, qp, qs, hq, _ints(table, "table", (r, self._table_pages), dev),
            _ints(lens, "lens", (r,), dev), softmax_scale, out.data_ptr(), _DTYPES[out.dtype], ws.data_ptr(), ws.nbytes,
            raw))
        return out

    def attend(self, layer, q, cu_tokens, table, lens, softmax_scale, out=None, workspace=None, stream=None):
        """Attention of a step's packed new tokens, any number of each request, over
        all that the cache holds of it with them, causally (kvq_paged_attention; call
        after write()): q [tokens][H_q][D] -> out [tokens][H_q][D]. cu_tokens, lens: as
        reserve() planned the step. ``out`` must not overlap q; its rows outside every request are
        left as they are (uninitialised where ``out`` is not given). ``workspace``: as in decode()."""
        lib = _lib or _bind()
        dev = self.device
        qp, qs = _rows(q, "q", self.dtype, dev, dim=self._dim)
        t, hq, d = q.shape
        r = lens.shape[0]
        if out is None:
            out = _empty((t, hq, d), self.dtype, dev, stream)
        elif tuple(out.shape) != (t, hq, d) or out.device != dev or not out.is_contiguous() or out.dtype != self.dtype:
            raise ValueError("out must be a contiguous %s tensor of shape %s on %s" % (self.dtype, (t, hq, d), dev))
        raw = _raw_stream(stream, dev)
        if workspace is None:
            ws = self._workspace(hq, raw, stream, True)
        else:
            ws = workspace
            if not isinstance(ws, _Tensor) or ws.device != dev or not ws.is_contiguous():
                raise TypeError("workspace must be a contiguous tensor on %s" % dev)
        _check(lib.kvq_paged_attention(
            self.handle, layer, r, qp, qs, t, hq, _ints(cu_tokens, "cu_tokens", (r + 1,), dev),
            _ints(table, "table", (r, self._table_pages), dev), _ints(lens, "lens", (r,), dev), softmax_scale,
            out.data_ptr(), ws.data_ptr(), ws.nbytes, raw))
        return out

    # -- inspection ---------------------------------------------------------
    def _view(self, layer, name):
        view = self._views.get((layer, name))
        if view is None:
            c, lo = self.cfg, PagedLayout()
            _check(_lib.kvq_paged_cache_get_layout(self.handle, layer, ctypes.byref(lo)))
            shape, dtype = {
                "pages": ((c.num_pages, c.num_kv_heads, 2, c.page_tokens, c.head_dim),
                          torch.int8 if c.code == PAGE_INT8 else torch.uint8),
                "scales": ((c.num_pages, c.num_kv_heads, 2), torch.float32),
                "tails": ((c.max_requests, c.num_kv_heads, 2, c.page_tokens, c.head_dim), self.dtype)}[name]
            off = getattr(lo, name) - self.buffer.data_ptr()
            view = self.buffer[off:off + getattr(lo, name + "_bytes")].view(dtype).view(shape)
            self._views[layer, name] = view
        return view

    def pages(self, layer):
        """Codes [page][kv head][K, V][token][channel]: int8, or uint8 bits of
        torch.float8_e4m3fn."""
        return self._view(layer, "pages")

    def scales(self, layer):
        """fp32 [page][kv head][K, V]."""
        return self._view(layer, "scales")

    def tails(self, layer):
        """Rows of the open pages [request][kv head][K, V][token][channel]."""
        return self._view(layer, "tails")

    def status(self, stream=None):
        """Synchronizes the stream and clears the status word; raises KVQError if
        it was set. Work on other streams is done before, by the caller."""
        lib = _lib or _bind()
        w = ctypes.c_uint32()
        _check(lib.kvq_paged_cache_status(self.handle, _raw_stream(stream, self.device), ctypes.byref(w)))
        return w.value

    def close(self):
        if getattr(self, "handle", None):
            _lib.kvq_paged_cache_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Rotation:
    """Rotation by position, for norm_rotate: pair j of a row's first
    ``2 * len(inv_freq)`` channels is turned by position * inv_freq[j] radians. Pairs are
    channels (j, j + len(inv_freq)), or neighbours where ``interleaved``; the rotated
    channels are multiplied by ``magnitude``. len(inv_freq) is a multiple of 4."""

    def __init__(self, inv_freq, interleaved=False, magnitude=1.0, device=None):
        freq = [float(f) for f in inv_freq]
        if len(freq) % 4 != 0:
            raise ValueError("inv_freq has %d frequencies, a multiple of 4 is needed" % len(freq))
        if not all(math.isfinite(f) for f in freq):
            raise ValueError("inv_freq must be finite")
        self.dim, self.interleaved, self.magnitude = 2 * len(freq), bool(interleaved), float(magnitude)
        # turns a position as a 64-bit fraction; a negative frequency turns back
        turns = [round(Fraction(f) / _TWO_PI * 2 ** 64) % 2 ** 64 for f in freq]
        signed = [t - 2 ** 64 if t >= 2 ** 63 else t for t in turns]
        #: The turns' bits, int64 on the device.
        self.turns = torch.tensor(signed, dtype=torch.int64, device=device if device is not None else "cuda")

    @classmethod
    def standard(cls, dim, theta=10000.0, **kw):
        """theta^(-2 j / dim) for the pairs of ``dim`` channels."""
        return cls([theta ** (-2.0 * j / dim) for j in range(dim // 2)], **kw)


def _head_rows(x, out, name, stream):
    """Pointer, stride and heads of rows, and the same of their output."""
    if not isinstance(x, _Tensor) or x.dtype not in (torch.float16, torch.bfloat16) or not x.is_cuda:
        raise TypeError("%s must be a CUDA float16 or bfloat16 tensor" % name)
    p, s = _rows(x, name, x.dtype, x.device)
    t, h, d = x.shape
    if out is None:
        out = _empty((t, h, d), x.dtype, x.device, stream)
    op, os = _rows(out, name + "_out", x.dtype, x.device, heads=h, dim=d)
    if out.shape[0] != t:
        raise ValueError("%s_out holds %d tokens, expected %d" % (name, out.shape[0], t))
    return out, p, s, h, op, os


def _weight(w, name, d, device):
    if w is None:
        return None
    if not isinstance(w, _Tensor) or w.dtype is not torch.float32 or w.device != device:
        raise TypeError("%s must be a float32 tensor on %s" % (name, device))
    if w.shape != (d,) or not w.is_contiguous():
        raise ValueError("%s must be a contiguous tensor of shape (%d,)" % (name, d))
    return w.data_ptr()


def norm_rotate(q, k, positions, rotation, q_weight=None, k_weight=None, eps=1e-6, q_out=None, k_out=None, stream=None):
    """Norm of each head and rotation by position in one pass (kvq_norm_rotate): q
    [tokens][H_q][D], k [tokens][H_k][D] in fp16 or bf16, positions int32 [tokens]
    (reserve()'s), rotation a Rotation. Without a weight (fp32 [D]) there is no norm.
    Returns (q, k) rotated: new tensors, or ``q_out`` / ``k_out``, which may be q and k
    themselves. Rows of tokens with a negative position are left as they are there."""
    lib = _lib or _bind()
    q_out, qp, qs, hq, qop, qos = _head_rows(q, q_out, "q", stream)
    k_out, kp, ks, hk, kop, kos = _head_rows(k, k_out, "k", stream)
    t, _, d = q.shape
    dev = q.device
    if k.dtype is not q.dtype or k.device != dev:
        raise TypeError("q and k must have the same type and device")
    if k.shape[0] != t or k.shape[2] != d:
        raise ValueError("q has shape %s, k %s" % (tuple(q.shape), tuple(k.shape)))
    turns = rotation.turns
    if turns.device != dev:
        raise TypeError("the rotation must be on %s" % dev)
    _check(lib.kvq_norm_rotate(
        qp, kp, qs, ks, t, hq, hk, d, _DTYPES[q.dtype], _ints(positions, "positions", (t,), dev), turns.data_ptr(),
        rotation.dim, rotation.interleaved, rotation.magnitude, _weight(q_weight, "q_weight", d, dev),
        _weight(k_weight, "k_weight", d, dev), eps, qop, kop, qos, kos, _raw_stream(stream, dev)))
    return q_out, k_out


def prompt_attention(q, k, v, cu_tokens, softmax_scale, out=None, status=None, stream=None):
    """Causal attention over packed prompts on their own keys and values, not
    on what the cache holds of them before (kvq_prompt_attention): q
    [tokens][H_q][D], k and v [tokens][H_kv][D] in fp16 or bf16, cu_tokens
    int32 [sequences + 1]. Rows of ``out`` outside every sequence are left as
    they are (uninitialised where ``out`` is not given). ``status``: int32 [1],
    such as ``PagedKVCache.status_word``, which a range of cu_tokens outside the
    tokens or a wait that gave up sets; without it they go unseen."""
    lib = _lib or _bind()
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
    _check(lib.kvq_prompt_attention(
        qp, kp, vp, qs, ks, vs, t, seqs, _ints(cu_tokens, "cu_tokens", (seqs + 1,), dev), hq, k.shape[1], d,
        _DTYPES[q.dtype], softmax_scale, out.data_ptr(),
        None if status is None else _ints(status, "status", (1,), dev), _raw_stream(stream, dev)))
    return out
