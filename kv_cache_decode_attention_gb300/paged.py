"""Paged serving over the C ABI: K and V in pages, rotary positions, chunk attention.

One step of a server is ``paged_plan`` (pages, slots and positions of the new
rows, from request lengths on the device), then per layer ``paged_append``
(rotate q and k, write k and v to their slots) and ``paged_attention``.  Nothing
is read back, so a step can be captured into a CUDA graph and replayed.
``rope`` alone rotates rows for the contiguous caches (``kv_append``,
``rswa_ring_write`` and ``rswa_record_prefill`` take rotated rows).

As in the rest of the binding, every computation runs in libkvd.so; this module
allocates buffers, marshals pointers and raises on a non-OK status.
"""

from __future__ import annotations

import ctypes as C
import math

import torch

from . import _abi
from .api import _ptr, _stream

_DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
_LAYOUTS = {"interleaved": 0, "half": 1}
_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3, "bands": 4}


def _i32(t, name, numel=None, device=None):
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype == torch.int32 and t.is_contiguous()):
        raise ValueError("%s must be a contiguous int32 CUDA tensor" % name)
    if numel is not None and t.numel() != numel:
        raise ValueError("%s must hold %d numbers, has %d" % (name, numel, t.numel()))
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, not on %s" % (name, t.device, device))
    return t


def _rows(t, name, heads_dim, device):
    """kvd_rows of a [tokens, heads, head_dim] view (head_dim contiguous)."""
    if not (t.is_cuda and t.device == device):
        raise ValueError("%s must be a CUDA tensor on %s" % (name, device))
    if t.dim() != 3 or (heads_dim is not None and t.shape[2] != heads_dim) or (t.shape[2] > 1 and t.stride(2) != 1):
        raise ValueError("%s must be [tokens, heads, head_dim] with head_dim contiguous" % name)
    return _abi.kvd_rows(t.data_ptr(), t.stride(0), t.stride(1))


class _on:
    """Makes `device` current for the launches inside (nothing to do when it is)."""

    __slots__ = ("device", "before")

    def __init__(self, device):
        self.device = device.index

    def __enter__(self):
        self.before = torch.cuda.current_device()
        if self.device is not None and self.before != self.device:
            torch.cuda.set_device(self.device)

    def __exit__(self, *a):
        if self.device is not None and self.before != self.device:
            torch.cuda.set_device(self.before)


def _own(t, stream):
    """A tensor allocated here and used on a stream of the caller's choice."""
    if stream is not None:
        t.record_stream(stream)
    return t


class RopeTable:
    """Frequencies of rotary positions (host memory; see kvd_rope_config).

    layout: 'interleaved' (channels 2i, 2i+1) or 'half' (i, i + rot_dim/2).
    scaling: 'none', 'linear', 'ntk', 'yarn' or 'bands', with `factor` and, for
    the last two, the trained length `original_len` and their band limits.
    attention_factor multiplies cos and sin (None: 1, for yarn 0.1 ln(factor) + 1).
    """

    __slots__ = ("rot_dim", "layout", "scaling", "R", "_ref")

    def __init__(self, rot_dim: int, layout: str = "half", scaling: str = "none", base: float = 10000.0,
                 factor: float = 1.0, original_len: float = 0.0, beta_fast: float = 32.0, beta_slow: float = 1.0,
                 low_freq_factor: float = 1.0, high_freq_factor: float = 4.0, attention_factor: float | None = None):
        if layout not in _LAYOUTS:
            raise ValueError("layout must be one of %s" % ", ".join(sorted(_LAYOUTS)))
        if scaling not in _SCALINGS:
            raise ValueError("scaling must be one of %s" % ", ".join(sorted(_SCALINGS)))
        self.rot_dim, self.layout, self.scaling = int(rot_dim), layout, scaling
        cfg = _abi.kvd_rope_config(self.rot_dim, _LAYOUTS[layout], _SCALINGS[scaling], 0, base, factor, original_len,
                                   beta_fast, beta_slow, low_freq_factor, high_freq_factor,
                                   0.0 if attention_factor is None else attention_factor)
        self.R = _abi.kvd_rope()
        self._ref = C.byref(self.R)
        _abi.call("kvd_rope_init", self._ref, C.byref(cfg))


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
    dev, tokens, hd = some.device, some.shape[0], some.shape[-1]
    if some.dtype not in _DTYPES:
        raise ValueError("rope takes float32, float16 or bfloat16")
    if not some.is_cuda:
        raise ValueError("rope takes CUDA tensors")
    _i32(positions, "positions", tokens, dev)
    args = []
    outs = []
    with _on(dev):
        for t, o, name in ((q, q_out, "q"), (k, k_out, "k")):
            if t is None:
                if o is not None:
                    raise ValueError("%s_out without %s" % (name, name))
                args += [None, None, 0]
                outs.append(None)
                continue
            if t.dtype != some.dtype or t.shape[0] != tokens:
                raise ValueError("q and k must have one dtype and as many tokens")
            if o is None:
                o = _own(torch.empty(t.shape, dtype=t.dtype, device=dev), stream)
            elif o.dtype != t.dtype or o.shape != t.shape:
                raise ValueError("%s_out must have the shape and dtype of %s" % (name, name))
            args += [_rows(t, name, hd, dev), _rows(o, name + "_out", hd, dev), t.shape[1]]
            outs.append(o)
        _abi.call("kvd_rope_apply", table._ref, *args, hd, _DTYPES[some.dtype], positions.data_ptr(), tokens,
                  _stream(stream))
    return outs[0], outs[1]


class PagedKvCache:
    """One layer's pages plus the request state that layers share.

    Requests 0 .. n_seq - 1 are the places of a batch; each holds seq_len[b] rows
    in the pages block_table[b].  Layers of one model share block_table, seq_len
    and the free pages: build the first layer's cache, then ``layer_like`` it.
    dtype: torch.bfloat16 or torch.float16.
    """

    __slots__ = ("k", "v", "block_table", "seq_len", "free_pages", "n_free", "error", "page_size", "n_pages", "n_kv",
                 "head_dim", "n_seq", "max_pages", "dtype", "device")

    def __init__(self, n_pages: int, page_size: int, n_kv: int, head_dim: int, n_seq: int, max_pages: int,
                 dtype=torch.bfloat16, device="cuda"):
        dev = torch.device(device)
        shape = (int(n_pages), int(n_kv), int(page_size), int(head_dim))
        self._bind(torch.empty(shape, dtype=dtype, device=dev), torch.empty(shape, dtype=dtype, device=dev),
                   torch.full((int(n_seq), int(max_pages)), -1, dtype=torch.int32, device=dev),
                   torch.zeros(int(n_seq), dtype=torch.int32, device=dev),
                   # the stack's top is its last entry: page 0 is taken first
                   torch.arange(int(n_pages) - 1, -1, -1, dtype=torch.int32, device=dev),
                   torch.full((1,), int(n_pages), dtype=torch.int32, device=dev),
                   torch.zeros(1, dtype=torch.int32, device=dev), None)

    @classmethod
    def of(cls, k, v, block_table, seq_len, free_pages=None, n_free=None, error=None, page_size=None):
        """Bind to buffers that a program already has.  k and v may be None for a
        cache that is only planned on (page_size then says the pages' rows);
        without free_pages and n_free it cannot be planned on."""
        self = cls.__new__(cls)
        self._bind(k, v, block_table, seq_len, free_pages, n_free, error, page_size)
        return self

    def layer_like(self) -> "PagedKvCache":
        """Another layer's pages with this one's tables, lengths and free pages."""
        return PagedKvCache.of(torch.empty_like(self.k), torch.empty_like(self.v), self.block_table, self.seq_len,
                               self.free_pages, self.n_free, self.error)

    def _bind(self, k, v, block_table, seq_len, free_pages, n_free, error, page_size):
        if block_table.dim() != 2:
            raise ValueError("block_table must be [n_seq, max_pages]")
        dev = block_table.device
        self.n_seq, self.max_pages = block_table.shape
        _i32(block_table, "block_table")
        _i32(seq_len, "seq_len", self.n_seq, dev)
        if k is not None:
            for t, name in ((k, "k"), (v, "v")):
                if not (t is not None and t.is_cuda and t.device == dev and t.dim() == 4 and t.is_contiguous()):
                    raise ValueError("%s must be contiguous pages [n_pages, n_kv, page_size, head_dim] on %s" % (name, dev))
            if k.shape != v.shape or k.dtype != v.dtype or k.dtype not in (torch.float16, torch.bfloat16):
                raise ValueError("k and v must have one shape and be float16 or bfloat16")
            self.n_pages, self.n_kv, self.page_size, self.head_dim = k.shape
            if page_size is not None and page_size != self.page_size:
                raise ValueError("page_size is not that of the pages")
            self.dtype = k.dtype
        else:
            if page_size is None or free_pages is None or v is not None:
                raise ValueError("a cache without k and v needs page_size and free_pages")
            self.n_pages, self.n_kv, self.page_size, self.head_dim, self.dtype = free_pages.numel(), 0, int(page_size), 0, None
        if free_pages is not None:
            _i32(free_pages, "free_pages", self.n_pages, dev)
            _i32(n_free, "n_free", 1, dev)
        if error is None:
            error = torch.zeros(1, dtype=torch.int32, device=dev)
        _i32(error, "error", 1, dev)
        self.k, self.v, self.block_table, self.seq_len = k, v, block_table, seq_len
        self.free_pages, self.n_free, self.error, self.device = free_pages, n_free, error, dev

    def device_error(self, clear: bool = True) -> int:
        """The error word (synchronises): bit 0 a bounded wait gave up, bit 1
        metadata out of range, bit 2 a plan did not fit."""
        w = C.c_uint32(0)
        with _on(self.device):
            st = _abi.lib().kv_paged_device_error(_ptr(self.error), int(clear), C.byref(w))
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
    if cache.free_pages is None:
        raise ValueError("the cache has no free pages to plan with")
    dev, n = cache.device, cache.n_seq
    _i32(new_len, "new_len", n, dev)
    if keep_len is not None:
        _i32(keep_len, "keep_len", n, dev)
    n_tokens = int(n_tokens)
    with _on(dev):
        if plan is None:
            if n_tokens < 0:
                raise ValueError("n_tokens must not be negative")
            # one allocation, cut into the step's arrays
            sizes = [n + 1, n_tokens, n_tokens] + ([] if advance else [n, 1])
            parts = _own(torch.empty(sum(sizes), dtype=torch.int32, device=dev), stream).split(sizes)
            plan = PagedPlan(parts[0], cache.seq_len if advance else parts[3], cache.n_free if advance else parts[4],
                             parts[1], parts[2])
        else:
            _i32(plan.cu_new, "plan.cu_new", n + 1, dev)
            _i32(plan.positions, "plan.positions", n_tokens, dev)
            _i32(plan.slots, "plan.slots", n_tokens, dev)
            if advance:
                plan.seq_len, plan.n_free = cache.seq_len, cache.n_free
            _i32(plan.seq_len, "plan.seq_len", n, dev)
            _i32(plan.n_free, "plan.n_free", 1, dev)
            if not advance and (plan.seq_len is cache.seq_len or plan.n_free is cache.n_free):
                raise ValueError("plan holds the cache's own state: pass advance=True, or a plan made with advance=False")
        _abi.call("kv_paged_plan", cache.seq_len.data_ptr(), None if keep_len is None else keep_len.data_ptr(),
                  new_len.data_ptr(), n, cache.n_pages, cache.page_size, cache.block_table.data_ptr(), cache.max_pages,
                  cache.free_pages.data_ptr(), cache.n_free.data_ptr(), plan.seq_len.data_ptr(), plan.n_free.data_ptr(),
                  plan.cu_new.data_ptr(), plan.positions.data_ptr(), plan.slots.data_ptr(), n_tokens,
                  cache.error.data_ptr(), _stream(stream))
    return plan


def paged_append(cache: PagedKvCache, plan: PagedPlan, k: torch.Tensor, v: torch.Tensor, q: torch.Tensor | None = None,
                 q_out: torch.Tensor | None = None, rope: RopeTable | None = None, stream=None) -> torch.Tensor | None:
    """Write the new rows k, v [tokens, n_kv, hd] to the plan's slots, k rotated by
    `rope` (None: as they are), and return q [tokens, n_q, hd] rotated in the
    pages' dtype (rows without a position are left as they were).
    Inputs are float32 or the pages' dtype, all of one."""
    if cache.k is None:
        raise ValueError("the cache has no pages")
    if plan.positions is None or plan.slots is None:
        raise ValueError("the plan has no positions and slots")
    dev, hd, tokens = cache.device, cache.head_dim, k.shape[0]
    _i32(plan.positions, "plan.positions", tokens, dev)
    _i32(plan.slots, "plan.slots", tokens, dev)
    if k.dtype not in _DTYPES or v.dtype != k.dtype or (q is not None and q.dtype != k.dtype):
        raise ValueError("q, k and v must have one dtype")
    if k.shape != (tokens, cache.n_kv, hd) or v.shape != k.shape:
        raise ValueError("k and v must be [tokens, n_kv, head_dim]")
    with _on(dev):
        args = [None, None, 0]
        if q is not None:
            if q.dim() != 3 or q.shape[0] != tokens:
                raise ValueError("q must be [tokens, n_q, head_dim]")
            if q_out is None:
                q_out = _own(torch.empty(q.shape, dtype=cache.dtype, device=dev), stream)
            elif q_out.dtype != cache.dtype or q_out.shape != q.shape:
                raise ValueError("q_out must have q's shape and the pages' dtype")
            args = [_rows(q, "q", hd, dev), _rows(q_out, "q_out", hd, dev), q.shape[1]]
        elif q_out is not None:
            raise ValueError("q_out without q")
        _abi.call("kv_paged_append", None if rope is None else rope._ref, *args, _rows(k, "k", hd, dev), _rows(v, "v", hd, dev),
                  cache.n_kv, hd, _DTYPES[k.dtype], _DTYPES[cache.dtype], plan.positions.data_ptr(), plan.slots.data_ptr(),
                  tokens, cache.k.data_ptr(), cache.v.data_ptr(), cache.n_pages, cache.page_size, cache.error.data_ptr(),
                  _stream(stream))
    return q_out


def paged_attention_workspace(n_tokens: int, n_q: int, n_kv: int, head_dim: int) -> int:
    """Bytes of workspace that paged_attention needs for up to n_tokens new rows."""
    n = C.c_int64(0)
    _abi.call("paged_attention_workspace_bytes", int(n_tokens), int(n_q), int(n_kv), int(head_dim), C.byref(n))
    return int(n.value)


def paged_attention(q: torch.Tensor, cache: PagedKvCache, plan: PagedPlan, out: torch.Tensor | None = None,
                    scale: float | None = None, window: int = 0, softcap: float = 0.0, sinks: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Causal attention of the step's new rows q [tokens, n_q, hd] (appended already)
    over all rows their requests hold; out has q's shape and dtype (rows behind
    the last new one are left as they were).
    window, softcap and sinks as in decode_attention."""
    if cache.k is None:
        raise ValueError("the cache has no pages")
    dev, hd, n_kv = cache.device, cache.head_dim, cache.n_kv
    if q.dim() != 3 or q.shape[2] != hd or q.dtype != cache.dtype:
        raise ValueError("q must be [tokens, n_q, head_dim] in the pages' dtype")
    tokens, n_q = q.shape[0], q.shape[1]
    _i32(plan.cu_new, "plan.cu_new", cache.n_seq + 1, dev)
    _i32(plan.seq_len, "plan.seq_len", cache.n_seq, dev)
    if sinks is not None and not (sinks.is_cuda and sinks.dtype == torch.float32 and sinks.is_contiguous() and
                                  sinks.numel() == n_q and sinks.device == dev):
        raise ValueError("sinks must be contiguous float32 [n_q] on %s" % dev)
    with _on(dev):
        if out is None:
            out = _own(torch.empty(q.shape, dtype=q.dtype, device=dev), stream)
        elif out.dtype != q.dtype or out.shape != q.shape:
            raise ValueError("out must have q's shape and dtype")
        if workspace is None:
            workspace = _own(torch.empty(paged_attention_workspace(tokens, n_q, n_kv, hd), dtype=torch.uint8, device=dev), stream)
        elif not (workspace.is_cuda and workspace.device == dev and workspace.is_contiguous()):
            raise ValueError("workspace must be a contiguous CUDA tensor on %s" % dev)
        _abi.call("paged_attention", _rows(q, "q", hd, dev), _rows(out, "out", hd, dev), tokens, n_q, n_kv, hd,
                  _DTYPES[q.dtype], cache.k.data_ptr(), cache.v.data_ptr(), cache.n_pages, cache.page_size,
                  cache.block_table.data_ptr(), cache.max_pages, plan.cu_new.data_ptr(), plan.seq_len.data_ptr(), cache.n_seq,
                  1.0 / math.sqrt(hd) if scale is None else scale, window, softcap, None if sinks is None else sinks.data_ptr(),
                  workspace.data_ptr(), workspace.numel() * workspace.element_size(), cache.error.data_ptr(), _stream(stream))
    return out
