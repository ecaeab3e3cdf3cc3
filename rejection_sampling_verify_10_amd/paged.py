"""A paged key/value cache: pages handed out on the GPU, rows written, attention behind shared prefixes.

The binding of ``spec_page_step``, ``spec_paged_append``, ``spec_paged_plan`` and ``spec_paged_attention``
(``include/spec_verify.h`` states what every argument means).  One :class:`PagePool` serves all layers, a
:class:`PagedCache` is one layer's pages.  With ``lengths`` [T] the committed slots of the pool's table rows (batch rows
first, then rows that hold prefixes), a speculative step of N new tokens for B batch rows is

    granted, slots = page_step(pool, lengths, N, counts=counts)                 # rows that got pages
    plan = paged_plan(cache, pool.tables, lengths, N, q_heads, B=B, counts=granted[:B], prefix_row=prefix_row)
    for each layer:
        paged_append(cache, k, v, slots[:B])
        out, lse = paged_attention(q, cache, plan, mask=mask)
    ...                                                                         # LM head, verify_*: path, accept_len
    paged_append(cache, k, v, slots[:B], path=path, accept_len=accept_len)      # a tree's accepted rows, every layer
    lengths[:B] += accept_len + 1                                               # -1: a malformed row adds none

A chain's accepted rows are in place already.  Pages past the new lengths stay with their sequence until the next
``page_step``, which gives back what the next window does not need.
"""

from __future__ import annotations

import ctypes
import math
from typing import Optional, Tuple

import torch

from . import lib
from .kvq import _CODES, _DIMS, _call, _optional, _overlaps, _Rows, _scratch, _tensor

_PAGE_SIZES = tuple(1 << i for i in range(4, 11))


class _CacheArgs(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("k", "v")] +
                [(n, ctypes.c_int32) for n in ("pages", "page_size", "heads", "head_dim")] +
                [(n, ctypes.c_int64) for n in ("page_stride", "slot_stride", "head_stride")])


class PagePool:
    """The pages of a cache's sequences, over the caller's int32 tensors on one GPU.

    tables [T, width] (rows may be strided): pages of each row's slots, in order; held [T]: how many of them it has;
    ring [pages]: the free pages, ``free`` of them from entry ``head`` on (mod pages); state [2]: (head, free).
    page_size is a power of two from 16 to 1024.
    """

    def __init__(self, tables: torch.Tensor, held: torch.Tensor, ring: torch.Tensor, state: torch.Tensor, page_size: int):
        if tables.dim() != 2 or tables.shape[0] < 1 or tables.shape[1] < 1:
            raise ValueError("tables must be [T, width]")
        if not tables.is_cuda:
            raise ValueError("tables must be a GPU tensor")
        if tables.dtype != torch.int32:
            raise TypeError(f"tables must be torch.int32, got {tables.dtype}")
        T, width = tables.shape
        if (width > 1 and tables.stride(1) != 1) or (T > 1 and tables.stride(0) < width):
            raise ValueError("the rows of tables must be contiguous and not overlap")
        if page_size not in _PAGE_SIZES:
            raise ValueError(f"page_size must be one of {_PAGE_SIZES}, got {page_size}")
        if ring.dim() != 1 or ring.shape[0] < 1:
            raise ValueError("ring must be [pages]")
        dev = tables.device
        _tensor(held, "held", torch.int32, (T,), dev)
        _tensor(ring, "ring", torch.int32, ring.shape, dev)
        _tensor(state, "state", torch.int32, (2,), dev)
        self.tables, self.held, self.ring, self.state = tables, held, ring, state
        self.T, self.width, self.pages, self.page_size, self.device = T, width, ring.shape[0], int(page_size), dev
        self._workspace = torch.zeros(512, dtype=torch.uint8, device=dev)
        self._wp = (self._workspace.data_ptr() + 255) // 256 * 256
        self._sizes = (tables.data_ptr(), tables.stride(0) if T > 1 else width, T, width, self.page_size, self.pages)
        self._lists = (held.data_ptr(), state.data_ptr())
        self._ring = ring.data_ptr()


def new_page_pool(T: int, width: int, pages: int, page_size: int, device) -> PagePool:
    """A pool whose pages are all free: T table rows of up to ``width`` pages each."""
    i32 = dict(dtype=torch.int32, device=device)
    state = torch.zeros(2, **i32)
    state[1] = pages
    return PagePool(torch.full((T, width), -1, **i32), torch.zeros(T, **i32), torch.arange(pages, **i32), state, page_size)


def page_step(pool: PagePool, lengths: torch.Tensor, N: int, *, counts: Optional[torch.Tensor] = None,
              out_held: Optional[torch.Tensor] = None, out_state: Optional[torch.Tensor] = None
              ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Pages for up to N new tokens a row, behind ``lengths`` [T] int32 (``spec_page_step``).

    counts [T] int32, N by default; a row with a negative length has ended and gives its pages back.  The pool changes
    in place (held and state go to ``out_held`` and ``out_state`` instead, if given; tables and ring always in place).
    Returns granted [T] (counts, 0 for ended rows, -1 for rows that were not served) and slots [T, N], int32.  Calls on
    one pool must not overlap.
    """
    N = int(N)
    if not 1 <= N <= 65536:
        raise ValueError(f"N must lie in [1, 65536], got {N}")
    dev, T = pool.device, pool.T
    held, state = pool._lists
    granted, slots = lengths.new_empty((T,)), lengths.new_empty((T, N))
    _call(lib().spec_page_step, "spec_page_step", dev, *pool._sizes, held, state, pool._ring,
          _tensor(lengths, "lengths", torch.int32, (T,), dev), _optional(counts, "counts", torch.int32, (T,), dev), N,
          held if out_held is None else _tensor(out_held, "out_held", torch.int32, (T,), dev),
          state if out_state is None else _tensor(out_state, "out_state", torch.int32, (2,), dev),
          granted.data_ptr(), slots.data_ptr(), pool._wp, 256)
    return granted, slots


class PagedCache:
    """One layer's pages over the caller's tensors: k_pages, v_pages [pages, page_size, heads, D] bf16 on one GPU.

    The first three dimensions may be strided in any order (K and V alike), the last is contiguous; no two rows may
    share memory.  D is 64, 128 or 256, page_size a power of two from 16 to 1024.
    """

    def __init__(self, k_pages: torch.Tensor, v_pages: torch.Tensor):
        if k_pages.dim() != 4 or 0 in k_pages.shape:
            raise ValueError("k_pages must be [pages, page_size, heads, D]")
        pages, size, H, D = k_pages.shape
        if D not in _DIMS:
            raise ValueError(f"head_dim must be one of {_DIMS}, got {D}")
        if size not in _PAGE_SIZES:
            raise ValueError(f"page_size must be one of {_PAGE_SIZES}, got {size}")
        for t, name in ((k_pages, "k_pages"), (v_pages, "v_pages")):
            if not t.is_cuda or t.device != k_pages.device:
                raise ValueError(f"{name} must be a tensor on the cache's GPU")
            if t.dtype != torch.bfloat16:
                raise TypeError(f"{name} must be bfloat16, got {t.dtype}")
            if t.shape != k_pages.shape:
                raise ValueError(f"{name} must have shape {tuple(k_pages.shape)}, got {tuple(t.shape)}")
            if t.stride(3) != 1:
                raise ValueError(f"the rows of {name} must be contiguous")
            if _overlaps(t):
                raise ValueError(f"the rows of {name} must not share memory")
        if k_pages.stride() != v_pages.stride():
            raise ValueError("K and V must have the same strides")
        self.k_pages, self.v_pages = k_pages, v_pages
        self.pages, self.page_size, self.heads, self.head_dim = pages, size, H, D
        self.device = k_pages.device
        self._args = _CacheArgs(k_pages.data_ptr(), v_pages.data_ptr(), pages, size, H, D, *k_pages.stride()[:3])
        self._ref = ctypes.addressof(self._args)
        self._needs = {}                        # workspace bytes of the calls made so far, by their sizes


def new_paged_cache(pages: int, page_size: int, heads: int, head_dim: int, device) -> PagedCache:
    """One layer's empty pages; contents are undefined until appended."""
    shape = (pages, page_size, heads, head_dim)
    return PagedCache(*(torch.empty(shape, dtype=torch.bfloat16, device=device) for _ in range(2)))


def _rows(t: torch.Tensor, name: str, cache: PagedCache) -> _Rows:
    """The strided rows [B, N, heads, D] of a call."""
    shape = t.shape
    if len(shape) != 4 or 0 in shape or shape[3] != cache.head_dim:
        raise ValueError(f"{name} must be [B, N, heads, {cache.head_dim}], got {tuple(shape)}")
    if t.dtype not in _CODES:
        raise TypeError(f"{name} must be bfloat16 or float32, got {t.dtype}")
    if t.get_device() != cache.device.index:
        raise ValueError(f"{name} must be on {cache.device}, got {t.device}")
    s = t.stride()
    if s[3] != 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    # the stride of a dimension of one element never counts
    return _Rows(t.data_ptr(), s[0] if shape[0] > 1 else 0, s[1] if shape[1] > 1 else 0, s[2] if shape[2] > 1 else 0)


def paged_append(cache: PagedCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, *,
                 path: Optional[torch.Tensor] = None, accept_len: Optional[torch.Tensor] = None) -> None:
    """K and V rows k, v [B, N, heads, D] (bf16 or f32, strided) into ``slots`` [B, N] int32 (``spec_paged_append``).

    With ``path`` [B, D+1] and ``accept_len`` [B] int32 of a verification, row path[b][i] goes to slots[b][i] for i <=
    accept_len[b]: a tree's accepted rows into place.  Negative slots, and slots outside the pool, get nothing.
    """
    ra, rb = _rows(k, "k", cache), _rows(v, "v", cache)
    B, N = k.shape[:2]
    if k.shape[2] != cache.heads or v.shape != k.shape or v.dtype != k.dtype:
        raise ValueError(f"k and v must both be [{B}, {N}, {cache.heads}, {cache.head_dim}] of one type")
    dev = cache.device
    if slots.dim() != 2 or slots.shape[0] != B or slots.shape[1] < 1 or (path is None and slots.shape[1] != N):
        raise ValueError(f"slots must be [{B}, {N}], got {tuple(slots.shape)}")
    if slots.dtype != torch.int32:
        raise TypeError(f"slots must be torch.int32, got {slots.dtype}")
    if slots.get_device() != dev.index:
        raise ValueError(f"slots must be on {dev}, got {slots.device}")
    if (slots.shape[1] > 1 and slots.stride(1) != 1) or (B > 1 and slots.stride(0) < slots.shape[1]):
        raise ValueError("the rows of slots must be contiguous and not overlap")
    n, pp, ap = N, None, None
    if (path is None) != (accept_len is None):
        raise ValueError("path and accept_len come together")
    if path is not None:
        if path.dim() != 2 or path.shape[1] < 1:
            raise ValueError("path must be [B, D+1]")
        pp = _tensor(path, "path", torch.int32, (B, path.shape[1]), dev)
        ap = _tensor(accept_len, "accept_len", torch.int32, (B,), dev)
        n = min(path.shape[1], slots.shape[1])
    _call(lib().spec_paged_append, "spec_paged_append", dev, cache._ref, ctypes.addressof(ra), ctypes.addressof(rb),
          _CODES[k.dtype], B, n, N, slots.data_ptr(), slots.stride(0) if B > 1 else n, pp, 0 if path is None else path.shape[1], ap)


class PagedPlan:
    """How one step's attention is cut up (:func:`paged_plan`): sizes, the tables, and the plan on the GPU."""

    def __init__(self, B, N, q_heads, heads, head_dim, tables, page_size, with_prefix):
        self.B, self.N, self.q_heads, self.heads, self.head_dim, self.with_prefix = B, N, q_heads, heads, head_dim, with_prefix
        self.tables, self.width, self.page_size = tables, tables.shape[1], page_size
        self.bytes = int(lib().spec_paged_plan_bytes(B, N, q_heads, heads, head_dim, with_prefix))
        self._buffer = torch.empty(self.bytes + 256, dtype=torch.uint8, device=tables.device)
        self._ptr = (self._buffer.data_ptr() + 255) // 256 * 256


def paged_plan(cache: PagedCache, tables: torch.Tensor, lengths: torch.Tensor, N: int, q_heads: int, *,
               B: Optional[int] = None, counts: Optional[torch.Tensor] = None, prefix_row: Optional[torch.Tensor] = None,
               out: Optional[PagedPlan] = None) -> PagedPlan:
    """The plan of a step's attention, made once for all layers (``spec_paged_plan``).

    tables [T, width] int32 and lengths [T] int32: a pool's tables and the committed slots of their rows.  The first B
    rows (all by default) are the batch's, with counts [B] new tokens each (N by default).  prefix_row [B] int32: the
    table row whose slots come before batch row b's own, negative for none; neighbouring rows with the same one share
    the reading of it.  Without it a large batch's rows are not split over the GPU: where some are much longer than the
    rest, give -1 for all.  ``out``: a plan of the same sizes and tables to make anew (as a captured graph does).
    """
    if tables.dim() != 2 or 0 in tables.shape:
        raise ValueError("tables must be [T, width]")
    T, width = tables.shape
    B, N, q_heads, dev = T if B is None else int(B), int(N), int(q_heads), cache.device
    if not 1 <= B <= T:
        raise ValueError(f"B must lie in [1, {T}], got {B}")
    if N < 1:
        raise ValueError(f"N must be at least 1, got {N}")
    if q_heads < 1 or q_heads % cache.heads:
        raise ValueError(f"q_heads must be a multiple of {cache.heads}, got {q_heads}")
    if tables.dtype != torch.int32:
        raise TypeError(f"tables must be torch.int32, got {tables.dtype}")
    if tables.get_device() != dev.index:
        raise ValueError(f"tables must be on {dev}, got {tables.device}")
    if (width > 1 and tables.stride(1) != 1) or (T > 1 and tables.stride(0) < width):
        raise ValueError("the rows of tables must be contiguous and not overlap")
    with_prefix = prefix_row is not None
    if out is None:
        out = PagedPlan(B, N, q_heads, cache.heads, cache.head_dim, tables, cache.page_size, with_prefix)
    elif ((out.B, out.N, out.q_heads, out.heads, out.head_dim, out.with_prefix, out.page_size) !=
          (B, N, q_heads, cache.heads, cache.head_dim, with_prefix, cache.page_size) or out.tables is not tables):
        raise ValueError("out must be a plan of the same sizes and tables")
    _call(lib().spec_paged_plan, "spec_paged_plan", dev, B, N, q_heads, cache.heads, cache.head_dim, T, width, cache.page_size,
          _tensor(lengths, "lengths", torch.int32, (T,), dev), _optional(counts, "counts", torch.int32, (B,), dev),
          _optional(prefix_row, "prefix_row", torch.int32, (B,), dev), out._ptr, out.bytes)
    return out


def paged_attention_workspace_bytes(plan: PagedPlan, head_dim: int) -> int:
    """Bytes of :func:`paged_attention`'s workspace (give a tensor of 256 more)."""
    return int(lib().spec_paged_attention_workspace_bytes(plan.B, plan.N, plan.q_heads, plan.heads, head_dim,
                                                          plan.with_prefix))


def paged_attention(q: torch.Tensor, cache: PagedCache, plan: PagedPlan, *, mask: Optional[torch.Tensor] = None,
                    scale: Optional[float] = None, out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None,
                    workspace: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Softmax attention of the step's queries over prefix, cache and draft (``spec_paged_attention``).

    q [B, N, q_heads, D] bf16 or f32 (strided); the new tokens' rows are in their slots already (:func:`paged_append`).
    mask: None (token n sees new tokens 0..n) or an ancestor mask, [B, N, N] or [N, N] uint8, N <= 64 (what
    :func:`tree_rerank` gives).  scale defaults to D ** -0.5.  Returns (out, of q's type and shape, lse [B, N, q_heads]
    f32); tokens n >= counts[b] and batch rows out of range give zeros and -inf.  With bf16 queries the probabilities round
    to bf16 before they meet V where more than 32 query rows of a head see the same slots (a shared prefix's, a large
    window's); ``q.float()`` avoids that, for a float32 output and twice the time.
    """
    rq = _rows(q, "q", cache)
    B, N, Hq, D = q.shape
    dev = cache.device
    if (B, N, Hq, cache.heads, D, cache.page_size) != (plan.B, plan.N, plan.q_heads, plan.heads, plan.head_dim, plan.page_size):
        raise ValueError("q and cache must have the plan's sizes")
    if plan.tables.get_device() != dev.index:
        raise ValueError(f"the plan must be on {dev}, got {plan.tables.device}")
    mp, mb = None, 0
    if mask is not None:
        rows = mask.dim() == 3
        mp, mb = _tensor(mask, "mask", torch.uint8, (B, N, N) if rows else (N, N), dev), N * N if rows else 0
    if out is None:
        o = torch.empty_like(q, memory_format=torch.contiguous_format)
        lse = torch.empty((B, N, Hq), dtype=torch.float32, device=dev)
    else:
        o, lse = out
        _tensor(o, "out", q.dtype, (B, N, Hq, D), dev)
        _tensor(lse, "out lse", torch.float32, (B, N, Hq), dev)
    sizes = (B, N, Hq, plan.with_prefix)
    need = cache._needs.get(sizes)
    if need is None:
        need = cache._needs[sizes] = paged_attention_workspace_bytes(plan, D)
    wp, _ws = _scratch(need, dev, workspace)
    tables = plan.tables
    _call(lib().spec_paged_attention, "spec_paged_attention", dev, ctypes.addressof(rq), _CODES[q.dtype], B, N, Hq, cache._ref,
          tables.data_ptr(), tables.stride(0) if tables.shape[0] > 1 else plan.width, plan.width, plan._ptr, plan.bytes,
          plan.with_prefix, mp, mb, 1.0 / math.sqrt(D) if scale is None else float(scale), o.data_ptr(), lse.data_ptr(), wp, need)
    return o, lse
