"""Paged serving over the C ABI: K and V in pages, rotary positions, chunk attention.

One step of a server is ``paged_plan`` (pages, slots and positions of the new
rows, from request lengths on the device), then per layer ``paged_append``
(rotate q and k, write k and v to their slots) and ``paged_attention``.  Nothing
is read back, so a step can be captured into a CUDA graph and replayed.  Pages hold
16-bit rows or, with half the memory, codes of 8 bits with a scale for each page of a
KV head (``PagedKvCache(dtype=torch.float8_e4m3fn)``); ``paged_read`` gives rows back.
A call goes to the current stream, or to `stream`, where what it returns is to be
had.  What it reads has to be there on that stream, and to stay until it is read
(Tensor.record_stream), as with any stream of torch's.
``rope`` alone rotates rows for the contiguous caches (``kv_append``,
``rswa_ring_write`` and ``rswa_record_prefill`` take rotated rows).

As in the rest of the binding, every computation runs in libkvd.so; this module
allocates buffers, marshals pointers and raises on a non-OK status.
"""

from __future__ import annotations

import ctypes as C
import functools
import math
import struct

import torch

from . import _abi
from .api import _empty

_I32, _F32 = torch.int32, torch.float32
_DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
_E4M3 = torch.float8_e4m3fn
_PAGES = {torch.float16: 1, torch.bfloat16: 2, _E4M3: 3}
_LAYOUTS = {"interleaved": 0, "half": 1}
_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3, "bands": 4}

# A step makes four calls a layer, so what the binding costs a call counts: the
# structs of the ABI are packed as bytes, checks read each attribute once, and
# the current device and stream are asked for without building objects.
_pack_rows = struct.Struct("Pqq").pack          # kvd_rows
_pack_config = struct.Struct("iiii8d").pack     # kvd_rope_config
_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
# A workspace of one call is taken from torch's allocator by pointer and given
# back once the launches are in: it is bound to the call's stream, so the next
# taker on that stream comes after them.  (A tensor in its place costs some 4 us.)
_take = getattr(torch._C, "_cuda_cudaCachingAllocator_raw_alloc", None)
_give = getattr(torch._C, "_cuda_cudaCachingAllocator_raw_delete", None)


def _stream(index, stream):
    if stream is not None:
        return stream.cuda_stream
    return _raw_stream(index) if _raw_stream is not None else torch.cuda.current_stream().cuda_stream


def _i32(t, name, numel, device):
    """A contiguous int32 tensor of so many numbers on the device; its pointer."""
    if not (t.dtype is _I32 and t.device == device and t.is_contiguous()):
        raise ValueError("%s must be a contiguous int32 tensor on %s" % (name, device))
    if numel is not None and t.numel() != numel:
        raise ValueError("%s must hold %d numbers, has %d" % (name, numel, t.numel()))
    return t.data_ptr()


def _rows(t, name, shape, device):
    """kvd_rows of a [tokens, heads, head_dim] view (head_dim contiguous)."""
    stride = t.stride()
    if t.shape != shape or t.device != device or (stride[2] != 1 and shape[2] > 1):
        raise ValueError("%s must be %s on %s with head_dim contiguous" % (name, list(shape), device))
    return _pack_rows(t.data_ptr(), stride[0], stride[1])


def _cuda(device):
    """The index of a CUDA device."""
    if device.type != "cuda":
        raise ValueError("the paged calls take CUDA tensors, got one on %s" % device)
    return device.index if device.index is not None else _device()


class RopeTable:
    """Frequencies of rotary positions (host memory; see kvd_rope_config).

    layout: 'interleaved' (channels 2i, 2i+1) or 'half' (i, i + rot_dim/2).
    scaling: 'none', 'linear', 'ntk', 'yarn' or 'bands', with `factor` and, for
    the last two, the trained length `original_len` and their band limits.
    attention_factor multiplies cos and sin (None: 1, for yarn 0.1 ln(factor) + 1).
    """

    __slots__ = ("rot_dim", "layout", "scaling", "R")

    def __init__(self, rot_dim: int, layout: str = "half", scaling: str = "none", base: float = 10000.0,
                 factor: float = 1.0, original_len: float = 0.0, beta_fast: float = 32.0, beta_slow: float = 1.0,
                 low_freq_factor: float = 1.0, high_freq_factor: float = 4.0, attention_factor: float | None = None):
        if layout not in _LAYOUTS:
            raise ValueError("layout must be one of %s" % ", ".join(sorted(_LAYOUTS)))
        if scaling not in _SCALINGS:
            raise ValueError("scaling must be one of %s" % ", ".join(sorted(_SCALINGS)))
        self.rot_dim, self.layout, self.scaling = int(rot_dim), layout, scaling
        self.R = _abi.kvd_rope()
        st = _abi.lib().kvd_rope_init(self.R, _pack_config(
            self.rot_dim, _LAYOUTS[layout], _SCALINGS[scaling], 0, base, factor, original_len, beta_fast, beta_slow,
            low_freq_factor, high_freq_factor, 0.0 if attention_factor is None else attention_factor))
        if st:
            _abi.check("kvd_rope_init", st)


def rope(q: torch.Tensor | None, k: torch.Tensor | None, positions: torch.Tensor, table: RopeTable,
         q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None, stream=None):
    """Rotate q [tokens, n_q, hd] and k [tokens, n_kv, hd] (either may be None) by
    positions (int32 [tokens]); returns (q_out, k_out).  float32, float16 or
    bfloat16; views with head_dim contiguous are taken as they are; q_out=q and
    k_out=k rotate in place.  Rows with a negative position are left as they
    were in the outputs (whatever the memory held in outputs allocated here)."""
    some = q if q is not None else k
    if some is None:
        raise ValueError("rope needs q or k")
    dev, dtype = some.device, some.dtype
    index = _cuda(dev)
    if _device() != index:
        with torch.cuda.device(dev):
            return rope(q, k, positions, table, q_out, k_out, stream)
    if dtype not in _DTYPES:
        raise ValueError("rope takes float32, float16 or bfloat16")
    if some.dim() != 3:
        raise ValueError("rope takes [tokens, heads, head_dim]")
    tokens, _, hd = some.shape
    pos = _i32(positions, "positions", tokens, dev)
    qi = qo = ki = ko = None
    n_q = n_k = 0
    if q is not None:
        n_q = q.shape[1]
        qi = _rows(q, "q", (tokens, n_q, hd), dev)
        if q_out is None:
            q_out = torch.empty_like(q) if stream is None else _empty([q.shape], dtype, dev, stream)[0]
        elif q_out.dtype is not dtype:
            raise ValueError("q_out must have q's dtype")
        qo = _rows(q_out, "q_out", (tokens, n_q, hd), dev)
    elif q_out is not None:
        raise ValueError("q_out without q")
    if k is not None:
        if k.dtype is not dtype or k.dim() != 3:
            raise ValueError("q and k must have one dtype and be [tokens, heads, head_dim]")
        n_k = k.shape[1]
        ki = _rows(k, "k", (tokens, n_k, hd), dev)
        if k_out is None:
            k_out = torch.empty_like(k) if stream is None else _empty([k.shape], dtype, dev, stream)[0]
        elif k_out.dtype is not dtype:
            raise ValueError("k_out must have k's dtype")
        ko = _rows(k_out, "k_out", (tokens, n_k, hd), dev)
    elif k_out is not None:
        raise ValueError("k_out without k")
    st = _abi.lib().kvd_rope_apply(table.R, qi, qo, n_q, ki, ko, n_k, hd, _DTYPES[dtype], pos, tokens, _stream(index, stream))
    if st:
        _abi.check("kvd_rope_apply", st)
    return q_out, k_out


class PagedKvCache:
    """One layer's pages plus the request state that layers share.

    Requests 0 .. n_seq - 1 are the places of a batch; each holds seq_len[b] rows
    in the pages block_table[b].  Layers of one model share block_table, seq_len
    and the free pages: build the first layer's cache, then ``layer_like`` it.
    dtype: torch.bfloat16, torch.float16 or torch.float8_e4m3fn.  Pages of 8 bits
    hold codes; k_scale and v_scale (float32 [n_pages, n_kv], else None) have one
    scale for each page of a KV head, and a row is its codes times that.
    """

    __slots__ = ("k", "v", "k_scale", "v_scale", "block_table", "seq_len", "free_pages", "n_free", "error", "page_size",
                 "n_pages", "n_kv", "head_dim", "n_seq", "max_pages", "dtype", "device", "index")

    def __init__(self, n_pages: int, page_size: int, n_kv: int, head_dim: int, n_seq: int, max_pages: int,
                 dtype=torch.bfloat16, device="cuda"):
        dev = torch.device(device)
        shape = (int(n_pages), int(n_kv), int(page_size), int(head_dim))
        scales = [torch.ones(shape[:2], dtype=_F32, device=dev) for _ in range(2)] if dtype is _E4M3 else (None, None)
        self._bind(torch.empty(shape, dtype=dtype, device=dev), torch.empty(shape, dtype=dtype, device=dev),
                   torch.full((int(n_seq), int(max_pages)), -1, dtype=torch.int32, device=dev),
                   torch.zeros(int(n_seq), dtype=torch.int32, device=dev),
                   # the stack's top is its last entry: page 0 is taken first
                   torch.arange(int(n_pages) - 1, -1, -1, dtype=torch.int32, device=dev),
                   torch.full((1,), int(n_pages), dtype=torch.int32, device=dev),
                   torch.zeros(1, dtype=torch.int32, device=dev), None, *scales)

    @classmethod
    def of(cls, k, v, block_table, seq_len, free_pages=None, n_free=None, error=None, page_size=None, k_scale=None,
           v_scale=None):
        """Bind to buffers that a program already has.  k and v may be None for a
        cache that is only planned on (page_size then says the pages' rows);
        without free_pages and n_free it cannot be planned on.  Pages of 8 bits
        come with their scales."""
        self = cls.__new__(cls)
        self._bind(k, v, block_table, seq_len, free_pages, n_free, error, page_size, k_scale, v_scale)
        return self

    def layer_like(self) -> "PagedKvCache":
        """Another layer's pages with this one's tables, lengths and free pages."""
        scales = [None if s is None else torch.ones_like(s) for s in (self.k_scale, self.v_scale)]
        return PagedKvCache.of(torch.empty_like(self.k), torch.empty_like(self.v), self.block_table, self.seq_len,
                               self.free_pages, self.n_free, self.error, None, *scales)

    def _bind(self, k, v, block_table, seq_len, free_pages, n_free, error, page_size, k_scale, v_scale):
        dev = block_table.device
        self.index = _cuda(dev)
        if block_table.dim() != 2:
            raise ValueError("block_table must be [n_seq, max_pages]")
        n, self.max_pages = block_table.shape
        self.n_seq, self.device = n, dev
        _i32(block_table, "block_table", None, dev)
        _i32(seq_len, "seq_len", n, dev)
        if k is not None:
            dtype, shape = k.dtype, k.shape
            if v is None or v.dtype is not dtype or v.shape != shape or dtype not in _PAGES:
                raise ValueError("k and v must have one shape and be float16, bfloat16 or float8_e4m3fn")
            if not (len(shape) == 4 and k.device == dev and v.device == dev and k.is_contiguous() and v.is_contiguous()):
                raise ValueError("k and v must be contiguous pages [n_pages, n_kv, page_size, head_dim] on %s" % dev)
            self.n_pages, self.n_kv, self.page_size, self.head_dim = shape
            if page_size is not None and page_size != self.page_size:
                raise ValueError("page_size is not that of the pages")
            self.dtype = dtype
            if dtype is _E4M3:
                for s, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
                    if s is None or not (s.dtype is _F32 and s.shape == shape[:2] and s.device == dev and s.is_contiguous()):
                        raise ValueError("pages of 8 bits need %s, contiguous float32 [n_pages, n_kv] on %s" % (name, dev))
        else:
            if page_size is None or free_pages is None or v is not None:
                raise ValueError("a cache without k and v needs page_size and free_pages")
            self.n_pages, self.n_kv, self.page_size, self.head_dim, self.dtype = free_pages.numel(), 0, int(page_size), 0, None
        if (k_scale is not None or v_scale is not None) and self.dtype is not _E4M3:
            raise ValueError("scales belong to pages of 8 bits")
        if free_pages is not None:
            if n_free is None:
                raise ValueError("free_pages without n_free")
            _i32(free_pages, "free_pages", self.n_pages, dev)
            _i32(n_free, "n_free", 1, dev)
        if error is None:
            error = torch.zeros(1, dtype=_I32, device=dev)
        _i32(error, "error", 1, dev)
        self.k, self.v, self.block_table, self.seq_len = k, v, block_table, seq_len
        self.k_scale, self.v_scale = k_scale, v_scale
        self.free_pages, self.n_free, self.error = free_pages, n_free, error

    def device_error(self, clear: bool = True) -> int:
        """The error word, once every stream of the device has done what it was given:
        bit 0 a bounded wait gave up, bit 1 metadata out of range, bit 2 a plan did
        not fit."""
        w = C.c_uint32(0)
        with torch.cuda.device(self.device):
            torch.cuda.synchronize()  # the copy below waits for no non-blocking stream
            st = _abi.lib().kv_paged_device_error(self.error.data_ptr(), int(clear), C.byref(w))
        if st not in (_abi.OK, _abi.EDEVICE):
            _abi.check("kv_paged_device_error", st)
        return int(w.value)


class PagedPlan:
    """Where a step's new rows go (device int32): request b's are rows cu_new[b] ..
    cu_new[b+1] - 1 of the packed batch, at `positions`, in `slots`; seq_len and
    n_free are the state after the step."""

    __slots__ = ("cu_new", "seq_len", "n_free", "positions", "slots")

    def __init__(self, cu_new, seq_len, n_free=None, positions=None, slots=None):
        self.cu_new, self.seq_len, self.n_free, self.positions, self.slots = cu_new, seq_len, n_free, positions, slots


def paged_plan(cache: PagedKvCache, new_len: torch.Tensor, n_tokens: int, keep_len: torch.Tensor | None = None,
               advance: bool = True, plan: PagedPlan | None = None, stream=None) -> PagedPlan:
    """Shorten requests to keep_len (int32 [n_seq]; None keeps all rows, 0 drops a
    request), grow them by new_len (int32 [n_seq]), take and give back pages, and
    lay out up to n_tokens new rows (places behind the last are -1).

    advance: the cache's seq_len and n_free move on.  With advance=False they
    stay (the plan holds the new ones), and the step may be planned again.
    plan: buffers of an earlier plan to fill again, as a captured graph needs.
    A step that does not fit changes nothing and sets the error word's bit 2."""
    free = cache.free_pages
    if free is None:
        raise ValueError("the cache has no free pages to plan with")
    dev, n, index = cache.device, cache.n_seq, cache.index
    if _device() != index:
        with torch.cuda.device(dev):
            return paged_plan(cache, new_len, n_tokens, keep_len, advance, plan, stream)
    new = _i32(new_len, "new_len", n, dev)
    keep = None if keep_len is None else _i32(keep_len, "keep_len", n, dev)
    n_tokens = int(n_tokens)
    if plan is None:
        if n_tokens < 0:
            raise ValueError("n_tokens must not be negative")
        if stream is None:
            empty = torch.empty
            plan = PagedPlan(empty(n + 1, dtype=_I32, device=dev), cache.seq_len if advance else empty(n, dtype=_I32, device=dev),
                             cache.n_free if advance else empty(1, dtype=_I32, device=dev),
                             empty(n_tokens, dtype=_I32, device=dev), empty(n_tokens, dtype=_I32, device=dev))
        else:
            cu, lens, height, pos, slots = _empty((n + 1, n, 1, n_tokens, n_tokens), _I32, dev, stream)
            if advance:
                lens, height = cache.seq_len, cache.n_free
                lens.record_stream(stream)
                height.record_stream(stream)
            plan = PagedPlan(cu, lens, height, pos, slots)
        cu, pos, slots = plan.cu_new.data_ptr(), plan.positions.data_ptr(), plan.slots.data_ptr()
    else:
        cu = _i32(plan.cu_new, "plan.cu_new", n + 1, dev)
        pos = _i32(plan.positions, "plan.positions", n_tokens, dev)
        slots = _i32(plan.slots, "plan.slots", n_tokens, dev)
        if advance:
            plan.seq_len, plan.n_free = cache.seq_len, cache.n_free
        lens, height = _i32(plan.seq_len, "plan.seq_len", n, dev), _i32(plan.n_free, "plan.n_free", 1, dev)
        if not advance and (lens == cache.seq_len.data_ptr() or height == cache.n_free.data_ptr()):
            raise ValueError("plan holds the cache's own state: pass advance=True, or a plan made with advance=False")
    st = _abi.lib().kv_paged_plan(
        cache.seq_len.data_ptr(), keep, new, n, cache.n_pages, cache.page_size, cache.block_table.data_ptr(),
        cache.max_pages, free.data_ptr(), cache.n_free.data_ptr(), plan.seq_len.data_ptr(), plan.n_free.data_ptr(), cu, pos,
        slots, n_tokens, cache.error.data_ptr(), _stream(index, stream))
    if st:
        _abi.check("kv_paged_plan", st)
    return plan


def paged_append(cache: PagedKvCache, plan: PagedPlan, k: torch.Tensor, v: torch.Tensor, q: torch.Tensor | None = None,
                 q_out: torch.Tensor | None = None, rope: RopeTable | None = None, stream=None) -> torch.Tensor | None:
    """Write the new rows k, v [tokens, n_kv, hd] to the plan's slots, k rotated by
    `rope` (None: as they are), and return q [tokens, n_q, hd] rotated in the
    pages' dtype (rows without a position are left as they were).
    Inputs are float32 or the pages' dtype, all of one.

    Pages of 8 bits take float32, float16 or bfloat16: every block's scale grows to
    what its rows need, and the codes before them move with it.  q comes in the
    inputs' dtype, for float32 in q_out's (without one: bfloat16).  The rows of one
    page have to stand together and in order, as a plan lays them."""
    if cache.k is None:
        raise ValueError("the cache has no pages")
    if plan.positions is None or plan.slots is None:
        raise ValueError("the plan has no positions and slots")
    dev, hd, n_kv, index = cache.device, cache.head_dim, cache.n_kv, cache.index
    if _device() != index:
        with torch.cuda.device(dev):
            return paged_append(cache, plan, k, v, q, q_out, rope, stream)
    tokens, dtype = k.shape[0], k.dtype
    pos = _i32(plan.positions, "plan.positions", tokens, dev)
    slots = _i32(plan.slots, "plan.slots", tokens, dev)
    if dtype not in _DTYPES or v.dtype is not dtype:
        raise ValueError("q, k and v must have one dtype: float32 or the pages'")
    coded = cache.k_scale is not None
    q_dtype = cache.dtype
    if coded:
        q_dtype = dtype if dtype is not _F32 else torch.bfloat16 if q_out is None else q_out.dtype
    shape = (tokens, n_kv, hd)
    if k.dim() != 3 or v.dim() != 3:
        raise ValueError("k and v must be [tokens, n_kv, head_dim]")
    ki, vi = _rows(k, "k", shape, dev), _rows(v, "v", shape, dev)
    qi = qo = None
    n_q = 0
    if q is not None:
        if q.dim() != 3 or q.dtype is not dtype:
            raise ValueError("q must be [tokens, n_q, head_dim] of k's dtype")
        n_q = q.shape[1]
        shape = (tokens, n_q, hd)
        qi = _rows(q, "q", shape, dev)
        if q_out is None:
            q_out = torch.empty(shape, dtype=q_dtype, device=dev) if stream is None else _empty([shape], q_dtype, dev, stream)[0]
        elif q_out.dtype is not q_dtype or (coded and q_dtype is not torch.bfloat16 and q_dtype is not torch.float16):
            raise ValueError("q_out must have the inputs' dtype, for float32 float16 or bfloat16" if coded else "q_out must have the pages' dtype")
        qo = _rows(q_out, "q_out", shape, dev)
    elif q_out is not None:
        raise ValueError("q_out without q")
    if coded:
        st = _abi.lib().kv_paged_append_q8(
            None if rope is None else rope.R, qi, qo, n_q, ki, vi, n_kv, hd, _DTYPES[dtype], _DTYPES.get(q_dtype, -1), pos, slots,
            tokens, cache.k.data_ptr(), cache.v.data_ptr(), cache.k_scale.data_ptr(), cache.v_scale.data_ptr(), cache.n_pages,
            cache.page_size, cache.error.data_ptr(), _stream(index, stream))
        if st:
            _abi.check("kv_paged_append_q8", st)
        return q_out
    st = _abi.lib().kv_paged_append(
        None if rope is None else rope.R, qi, qo, n_q, ki, vi, n_kv, hd, _DTYPES[dtype], _DTYPES[cache.dtype], pos, slots,
        tokens, cache.k.data_ptr(), cache.v.data_ptr(), cache.n_pages, cache.page_size, cache.error.data_ptr(),
        _stream(index, stream))
    if st:
        _abi.check("kv_paged_append", st)
    return q_out


def paged_read(cache: PagedKvCache, cu_rows: torch.Tensor, n_rows: int, start: torch.Tensor | None = None,
               dtype: torch.dtype = torch.bfloat16, k_out: torch.Tensor | None = None, v_out: torch.Tensor | None = None,
               stream=None):
    """Rows of requests read back from their pages: rows start[b] (int32 [n_seq];
    None: 0) and on of every request b, as many as cu_rows (int32 [n_seq + 1]) says,
    packed; returns (k, v) [n_rows, n_kv, hd] of `dtype` (float32, float16 or
    bfloat16; k_out and v_out given: theirs).  Pages of any dtype.  Rows behind
    cu_rows' last are left as they were; a row that its request does not hold reads
    as zeros and sets the error word's bit 1."""
    if cache.k is None:
        raise ValueError("the cache has no pages")
    dev, index = cache.device, cache.index
    if _device() != index:
        with torch.cuda.device(dev):
            return paged_read(cache, cu_rows, n_rows, start, dtype, k_out, v_out, stream)
    n_rows = int(n_rows)
    if n_rows < 0:
        raise ValueError("n_rows must not be negative")
    cu = _i32(cu_rows, "cu_rows", cache.n_seq + 1, dev)
    first = None if start is None else _i32(start, "start", cache.n_seq, dev)
    shape = (n_rows, cache.n_kv, cache.head_dim)
    given = k_out if k_out is not None else v_out
    if given is not None:
        dtype = given.dtype
    if dtype not in _DTYPES:
        raise ValueError("paged_read gives float32, float16 or bfloat16")
    outs = []
    for o, name in ((k_out, "k_out"), (v_out, "v_out")):
        if o is None:
            o = torch.empty(shape, dtype=dtype, device=dev) if stream is None else _empty([shape], dtype, dev, stream)[0]
        elif o.dim() != 3 or o.dtype is not dtype:
            raise ValueError("k_out and v_out must have one dtype and be [n_rows, n_kv, head_dim]")
        outs.append((o, _rows(o, name, shape, dev)))
    (k_out, ko), (v_out, vo) = outs
    ks, vs = cache.k_scale, cache.v_scale
    st = _abi.lib().kv_paged_read(
        cache.k.data_ptr(), cache.v.data_ptr(), None if ks is None else ks.data_ptr(), None if vs is None else vs.data_ptr(),
        _PAGES[cache.dtype], cache.n_pages, cache.page_size, cache.n_kv, cache.head_dim, cache.block_table.data_ptr(),
        cache.max_pages, cache.seq_len.data_ptr(), first, cu, cache.n_seq, ko, vo, _DTYPES[dtype], n_rows,
        cache.error.data_ptr(), _stream(index, stream))
    if st:
        _abi.check("kv_paged_read", st)
    return k_out, v_out


@functools.lru_cache(maxsize=4096)
def paged_attention_workspace(n_tokens: int, n_q: int, n_kv: int, head_dim: int, dtype: torch.dtype | None = None) -> int:
    """Bytes of workspace that paged_attention needs for up to n_tokens new rows
    (dtype: the pages', where they may be of 8 bits)."""
    n = C.c_int64(0)
    _abi.call("paged_attention_q8_workspace_bytes" if dtype is _E4M3 else "paged_attention_workspace_bytes", int(n_tokens), int(n_q),
              int(n_kv), int(head_dim), C.byref(n))
    return int(n.value)


def paged_attention(q: torch.Tensor, cache: PagedKvCache, plan: PagedPlan, out: torch.Tensor | None = None,
                    scale: float | None = None, window: int = 0, softcap: float = 0.0, sinks: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Causal attention of the step's new rows q [tokens, n_q, hd] (appended already)
    over all rows their requests hold; out has q's shape and dtype (rows behind
    the last new one are left as they were).  q has the pages' dtype; over pages of
    8 bits it is float16 or bfloat16.  Rows that a request holds have to be finite: a NaN
    in one may reach all new rows of its request, those that do not see it too (pages of
    8 bits keep a NaN that is appended).
    window, softcap and sinks as in decode_attention."""
    k = cache.k
    if k is None:
        raise ValueError("the cache has no pages")
    dev, hd, n_kv, index, dtype = cache.device, cache.head_dim, cache.n_kv, cache.index, cache.dtype
    if _device() != index:
        with torch.cuda.device(dev):
            return paged_attention(q, cache, plan, out, scale, window, softcap, sinks, workspace, stream)
    shape = q.shape
    coded = dtype is _E4M3
    if coded:
        dtype = q.dtype if q.dtype is torch.bfloat16 or q.dtype is torch.float16 else None
    if len(shape) != 3 or shape[2] != hd or q.dtype is not dtype:
        raise ValueError("q must be [tokens, n_q, head_dim] in the pages' dtype (over pages of 8 bits float16 or bfloat16)")
    tokens, n_q, _ = shape
    cu = _i32(plan.cu_new, "plan.cu_new", cache.n_seq + 1, dev)
    lens = _i32(plan.seq_len, "plan.seq_len", cache.n_seq, dev)
    if sinks is not None:
        if not (sinks.dtype is _F32 and sinks.device == dev and sinks.is_contiguous() and sinks.numel() == n_q):
            raise ValueError("sinks must be contiguous float32 [n_q] on %s" % dev)
        sinks = sinks.data_ptr()
    qi = _rows(q, "q", shape, dev)
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=dev) if stream is None else _empty([shape], dtype, dev, stream)[0]
    elif out.dtype is not dtype:
        raise ValueError("out must have q's dtype")
    oi = _rows(out, "out", shape, dev)
    on = _stream(index, stream)
    taken = None
    if workspace is None:
        size = paged_attention_workspace(tokens, n_q, n_kv, hd, cache.dtype)
        if _take is not None and _give is not None:
            ws = taken = _take(size, on)
        else:
            workspace = torch.empty(size, dtype=torch.uint8, device=dev) if stream is None else _empty([size], torch.uint8, dev, stream)[0]
            ws = workspace.data_ptr()
    else:
        size = workspace.numel() * workspace.element_size()
        if workspace.device != dev or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on %s" % dev)
        ws = workspace.data_ptr()
    try:
        if coded:
            st = _abi.lib().paged_attention_q8(
                qi, oi, tokens, n_q, n_kv, hd, _DTYPES[dtype], k.data_ptr(), cache.v.data_ptr(), cache.k_scale.data_ptr(),
                cache.v_scale.data_ptr(), cache.n_pages, cache.page_size, cache.block_table.data_ptr(), cache.max_pages, cu, lens,
                cache.n_seq, 1.0 / math.sqrt(hd) if scale is None else scale, window, softcap, sinks, ws, size,
                cache.error.data_ptr(), on)
        else:
            st = _abi.lib().paged_attention(
                qi, oi, tokens, n_q, n_kv, hd, _DTYPES[dtype], k.data_ptr(), cache.v.data_ptr(), cache.n_pages, cache.page_size,
                cache.block_table.data_ptr(), cache.max_pages, cu, lens, cache.n_seq, 1.0 / math.sqrt(hd) if scale is None else scale,
                window, softcap, sinks, ws, size, cache.error.data_ptr(), on)
    finally:
        if taken is not None:
            _give(taken)
    if st:
        _abi.check("paged_attention_q8" if coded else "paged_attention", st)
    return out
