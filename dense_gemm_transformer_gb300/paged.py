"""Generation on a paged cache: rotary positions, attention of new tokens, and the cache's pages.

Argument marshalling only, like the rest of the binding, here by a native
module (csrc/binding.cpp): it checks the tensors and calls the C ABI
(include/gemm.h, "Generation on a paged cache"), which also holds the
operators' exact meaning.  Calls run on the current stream or on `stream` (a
torch stream or a raw handle), whose memory new outputs then come from.  One
step of generation:

    freqs, amplitude = dg.rotary_frequencies(128, base=10000.0, device="cuda")   # once
    positions, slots, info = dg.cache_grow(table, lens, refs, page_size, seqs, counts, tokens)
    q = dg.rotary_append(q, k, v, positions, slots, k_pages, v_pages, freqs, amplitude=amplitude)
    o = dg.paged_attention(q, k_pages, v_pages, table, lens, cu_q=cu, max_q=max_q)

PagedCache holds the tensors of a cache and makes these calls on them.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import math
import os

from . import _build

_native = None   # _build/_binding.so, loaded by the first call
_defaults = {}   # the package's default handles by device, from then on

_vp, _i64, _desc = ctypes.c_void_p, ctypes.c_int64, ctypes.c_char_p
FUNCTIONS = {  # in the order in which the native module takes them
    "gemm_rotary": [_vp, _desc, _vp],
    "gemm_paged_attention": [_vp, _desc, _vp],
    "gemm_cache_grow": [_vp, _desc, _i64, _vp, _vp, _i64, _vp, _vp, _vp, _vp],
    "gemm_cache_shrink": [_vp, _desc, _i64, _vp, _vp, _vp],
    "gemm_cache_fork": [_vp, _desc, _i64, _vp, _vp, _vp, _vp, _vp],
    "gemm_cache_compact": [_vp, _desc, _vp, _vp],
    "gemm_cache_copy": [_vp, _desc, _i64, _vp, _vp, _vp],
}


def declare(lib):
    """The argument types of the library's functions that the native module calls."""
    for name, args in FUNCTIONS.items():
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = args, ctypes.c_int


def _load(lib):
    """The native module, calling the functions of `lib`."""
    global _native, _defaults
    import torch  # noqa: F401  the module uses its libraries
    from . import GemmError, _default
    path = _build.BINDING_PATH
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with __graft_entry__.build()")
    loader = importlib.machinery.ExtensionFileLoader("_binding", path)
    module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_binding", loader))
    loader.exec_module(module)
    module.bind(GemmError, tuple(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in FUNCTIONS))
    _native, _defaults = module, _default
    return module


def rotary_frequencies(rotary_dim, base=10000.0, scaling=None, factor=1.0, original_length=None, beta_fast=32.0,
                       beta_slow=1.0, device="cpu"):
    """(frequencies, amplitude) for rotary and rotary_append: rotary_dim / 2
    float64 radians a position, base^(-2 i / rotary_dim), and the factor on
    the rotated elements.

    scaling None: as they are.  "linear": positions divided by `factor`.
    "ntk": the base raised so that the slowest pair slows down by `factor`
    and the fastest keeps its frequency.  "yarn": pairs that turn more than
    beta_fast times in original_length positions keep their frequency, those
    that turn less than beta_slow times slow down by `factor`, linearly
    between; amplitude 0.1 ln(factor) + 1."""
    import torch
    if rotary_dim < 2 or rotary_dim % 2:
        raise ValueError("rotary_dim must be even and at least 2")
    if not (base > 0 and factor >= 1):
        raise ValueError("base must be positive and factor at least 1")
    i = torch.arange(rotary_dim // 2, dtype=torch.float64) * 2 / rotary_dim
    amplitude = 1.0
    if scaling == "ntk" and rotary_dim > 2:
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    f = float(base) ** -i
    if scaling == "linear":
        f = f / factor
    elif scaling == "yarn":
        if not original_length or beta_fast <= beta_slow:
            raise ValueError("yarn needs original_length, and beta_fast above beta_slow")
        turns = original_length * f / (2 * math.pi)
        keep = ((turns - beta_slow) / (beta_fast - beta_slow)).clamp(0, 1)
        f = f / factor * (1 - keep) + f * keep
        amplitude = 0.1 * math.log(factor) + 1.0
    elif scaling not in (None, "ntk"):
        raise ValueError(f"unknown scaling {scaling!r}")
    return f.to(device), amplitude


class PagedOps:
    """The methods of a library handle (Gemm) that work on a paged cache."""

    def rotary(self, q, k, positions, freqs, amplitude=1.0, interleaved=False, inverse=False, q_out=None, k_out=None,
               stream=None):
        """Rotary positions through gemm_rotary.  q: [tokens, heads, head_dim],
        k: [tokens, kv_heads, head_dim] or None, float32, bfloat16 or float16
        with any strides but a unit last one; positions: int32 or int64
        [tokens]; freqs: float64 [rotary_dim / 2] on the device
        (rotary_frequencies), rotary_dim <= head_dim.  inverse: the transposed
        rotation, which takes the outputs' gradients to the inputs'.  Returns
        (q_out, k_out), new tensors of the inputs' type unless given (in place
        with q_out=q, k_out=k)."""
        return (_native or _load(self._lib)).rotary(
            self._h and self._h.value, q, k, positions, freqs, amplitude, interleaved, inverse, q_out, k_out, stream)

    def rotary_append(self, q, k, v, positions, slots, k_pages, v_pages, freqs=None, amplitude=1.0, interleaved=False,
                      q_out=None, stream=None):
        """Rotates q and k (rotary) and writes k and v, converted to the pools'
        type, into the slots of a paged cache.  k_pages, v_pages: [pages,
        page_size, kv_heads, head_dim], any strides but a unit last one;
        slots: int64 [tokens], page * page_size + slot, negative to write
        nothing.  freqs None: no rotation (positions may be None).  Returns
        the queries in the pools' type (q_out, new unless given)."""
        return (_native or _load(self._lib)).rotary_append(
            self._h and self._h.value, q, k, v, positions, slots, k_pages, v_pages, freqs, amplitude, interleaved,
            q_out, stream)

    def paged_attention(self, q, k_pages, v_pages, table, kv_lens, cu_q=None, max_q=None, max_kv=0, scale=None,
                        softcap=0.0, window=0, out=None, return_lse=False, stream=None):
        """Attention of new tokens over a paged cache through
        gemm_paged_attention.  q: [tokens, heads, 64 or 128] bfloat16 or
        float16; k_pages, v_pages: [pages, page_size, kv_heads, head_dim] of
        q's type; table: int32 [sequences, width] (rows of any stride);
        kv_lens: int32 [sequences], with the new tokens; cu_q: int32
        [sequences + 1], the first new token of each sequence, with max_q the
        most new tokens of one (None: one new token each); max_kv: an upper
        bound on kv_lens where one is known.  scale defaults to
        1 / sqrt(head_dim).  Returns out, or (out, lse) with return_lse: lse
        float32 [tokens, heads]."""
        return (_native or _load(self._lib)).paged_attention(
            self._h and self._h.value, q, k_pages, v_pages, table, kv_lens, cu_q, max_q, max_kv, scale, softcap, window,
            out, return_lse, stream)

    def cache_grow(self, table, lens, refs, page_size, seqs, counts, tokens, stream=None, pools=None):
        """Room for counts[i] more tokens of sequence seqs[i] (gemm_cache_grow):
        table int32 [sequences, width], lens int32 [sequences] and refs int32
        [pages] are updated in place; seqs (distinct) and counts are int32 on
        the device, tokens the sum of counts.  pools (as in cache_fork): where
        the new tokens would go to a page that another sequence holds too, the
        sequence gets a copy of it.  Returns (positions, slots, info): int64
        [tokens] each, and int32 [3]: pages taken, pages missing, sequences
        without room in their row or, without pools, on such a page; where one
        of the last two is not 0 nothing has been changed and every slot is -1."""
        return (_native or _load(self._lib)).cache_grow(
            self._h and self._h.value, table, lens, refs, page_size, seqs, counts, tokens, stream, pools)

    def cache_shrink(self, table, lens, refs, page_size, seqs, counts=None, stream=None):
        """Takes the last counts[i] tokens of sequence seqs[i] back, all of them
        without counts (gemm_cache_shrink); pages that no sequence holds any
        more become free.  table, lens and refs are updated in place."""
        (_native or _load(self._lib)).cache_shrink(
            self._h and self._h.value, table, lens, refs, page_size, seqs, counts, stream)

    def cache_fork(self, pools, table, lens, refs, page_size, parents, children, stream=None):
        """Makes the empty sequences children (distinct) copies of parents
        (gemm_cache_fork): full pages are shared, a last page that is not full
        is copied in every pool.  pools: tensors whose pages (dimension -4 of
        [..., pages, page_size, kv_heads, head_dim], or dimension -2 of [...,
        pages, elements]) are contiguous.  Returns (copied, info): int32 [n],
        the page each child's last tokens were copied to or -1, and int32 [3]:
        pages copied, pages missing, children that are not empty."""
        return (_native or _load(self._lib)).cache_fork(
            self._h and self._h.value, pools, table, lens, refs, page_size, parents, children, stream)

    def cache_compact(self, pools, table, refs, stream=None):
        """Moves the pages in use to the front of every pool
        (gemm_cache_compact); table and refs follow.  Returns info, int32 [2]:
        pages moved, pages in use."""
        return (_native or _load(self._lib)).cache_compact(
            self._h and self._h.value, pools, table, refs, stream)

    def cache_copy(self, pools, src, dst, stream=None):
        """Copies page src[i] to page dst[i] of every pool (gemm_cache_copy):
        int32 vectors on the device; no page both a source and a destination."""
        (_native or _load(self._lib)).cache_copy(self._h and self._h.value, pools, src, dst, stream)


class PagedCache:
    """The tensors of a paged cache for `layers` layers, and the calls on them.

    k, v: [layers, pages, page_size, kv_heads, head_dim]; table, lens, refs:
    the sequences (see the C ABI).  No call waits for the device; the counts
    in the returned infos say whether there was room."""

    def __init__(self, layers, pages, page_size, kv_heads, head_dim, sequences, width, dtype=None, device="cuda"):
        import torch
        dtype = torch.bfloat16 if dtype is None else dtype
        self.page_size = page_size
        self.k = torch.empty((layers, pages, page_size, kv_heads, head_dim), dtype=dtype, device=device)
        self.v = torch.empty_like(self.k)
        # pages of other than whole 16 bytes cannot be copied: fork refuses them, so none is ever shared
        self._copied = page_size * kv_heads * head_dim * self.k.element_size() % 16 == 0
        self.table = torch.full((sequences, width), -1, dtype=torch.int32, device=device)
        self.lens = torch.zeros(sequences, dtype=torch.int32, device=device)
        self.refs = torch.zeros(pages, dtype=torch.int32, device=device)

    def grow(self, seqs, counts, tokens):
        """cache_grow over every layer: (positions, slots, info) of the new tokens."""
        return cache_grow(self.table, self.lens, self.refs, self.page_size, seqs, counts, tokens,
                          pools=(self.k, self.v) if self._copied else None)

    def shrink(self, seqs, counts=None):
        """cache_shrink: takes tokens back, all of them without counts."""
        cache_shrink(self.table, self.lens, self.refs, self.page_size, seqs, counts)

    def fork(self, parents, children):
        """cache_fork over every layer: (copied, info)."""
        return cache_fork((self.k, self.v), self.table, self.lens, self.refs, self.page_size, parents, children)

    def compact(self):
        """cache_compact over every layer: info."""
        return cache_compact((self.k, self.v), self.table, self.refs)

    def append(self, layer, q, k, v, positions, slots, freqs=None, **kwargs):
        """rotary_append into one layer's pools."""
        return rotary_append(q, k, v, positions, slots, self.k[layer], self.v[layer], freqs, **kwargs)

    def attention(self, layer, q, seqs=None, **kwargs):
        """paged_attention over one layer's pools, of the sequences seqs (an
        index tensor; None: all, in order).  With a stream (a torch stream or
        a raw handle), all of it runs there."""
        stream = kwargs.pop("stream", None)
        if stream is not None:
            import torch
            with torch.cuda.stream(_torch_stream(stream)):
                return self.attention(layer, q, seqs, **kwargs)
        table = self.table if seqs is None else self.table.index_select(0, seqs)
        lens = self.lens if seqs is None else self.lens.index_select(0, seqs)
        return paged_attention(q, self.k[layer], self.v[layer], table, lens, **kwargs)


def _torch_stream(stream):
    """A torch stream for a stream as the calls take it."""
    import torch
    if not isinstance(stream, int):
        return stream
    return torch.cuda.default_stream() if stream in (0, 1) else torch.cuda.ExternalStream(stream)


def _handle():
    handle = _defaults.get(_native.device()) if _native else None
    if handle is None:
        from . import default_handle
        handle = default_handle()
    return handle


# With the current device's default handle.  In full, not through the methods
# or *args: a Python call with a dozen arguments more is 1 us, and a small call
# 5-8.
def rotary(q, k, positions, freqs, amplitude=1.0, interleaved=False, inverse=False, q_out=None, k_out=None,
           stream=None):
    """PagedOps.rotary with the current device's default handle."""
    h = _handle()
    return (_native or _load(h._lib)).rotary(
        h._h and h._h.value, q, k, positions, freqs, amplitude, interleaved, inverse, q_out, k_out, stream)


def rotary_append(q, k, v, positions, slots, k_pages, v_pages, freqs=None, amplitude=1.0, interleaved=False,
                  q_out=None, stream=None):
    """PagedOps.rotary_append with the current device's default handle."""
    h = _handle()
    return (_native or _load(h._lib)).rotary_append(
        h._h and h._h.value, q, k, v, positions, slots, k_pages, v_pages, freqs, amplitude, interleaved, q_out,
        stream)


def paged_attention(q, k_pages, v_pages, table, kv_lens, cu_q=None, max_q=None, max_kv=0, scale=None, softcap=0.0,
                    window=0, out=None, return_lse=False, stream=None):
    """PagedOps.paged_attention with the current device's default handle."""
    h = _handle()
    return (_native or _load(h._lib)).paged_attention(
        h._h and h._h.value, q, k_pages, v_pages, table, kv_lens, cu_q, max_q, max_kv, scale, softcap, window, out,
        return_lse, stream)


def cache_grow(table, lens, refs, page_size, seqs, counts, tokens, stream=None, pools=None):
    """PagedOps.cache_grow with the current device's default handle."""
    h = _handle()
    return (_native or _load(h._lib)).cache_grow(
        h._h and h._h.value, table, lens, refs, page_size, seqs, counts, tokens, stream, pools)


def cache_shrink(table, lens, refs, page_size, seqs, counts=None, stream=None):
    """PagedOps.cache_shrink with the current device's default handle."""
    h = _handle()
    (_native or _load(h._lib)).cache_shrink(h._h and h._h.value, table, lens, refs, page_size, seqs, counts, stream)


def cache_fork(pools, table, lens, refs, page_size, parents, children, stream=None):
    """PagedOps.cache_fork with the current device's default handle."""
    h = _handle()
    return (_native or _load(h._lib)).cache_fork(
        h._h and h._h.value, pools, table, lens, refs, page_size, parents, children, stream)


def cache_compact(pools, table, refs, stream=None):
    """PagedOps.cache_compact with the current device's default handle."""
    h = _handle()
    return (_native or _load(h._lib)).cache_compact(h._h and h._h.value, pools, table, refs, stream)


def cache_copy(pools, src, dst, stream=None):
    """PagedOps.cache_copy with the current device's default handle."""
    h = _handle()
    (_native or _load(h._lib)).cache_copy(h._h and h._h.value, pools, src, dst, stream)
