"""A key/value cache held in four bits: append, read back, attend, commit, score and evict.

The binding of the ``spec_kvq_*`` calls of ``include/spec_verify.h`` (which states the row format and what
every argument means).  One :class:`KVQCache` is one layer's cache; a speculative step is

    kvq_append(cache, k, v, prefix)                          # the draft's N rows
    out, lse = kvq_attention(q, cache, prefix, mask=mask)    # in every layer
    ...                                                      # LM head, verify_tree_*: path, accept_len
    lengths = kvq_commit(cache, prefix, path, accept_len, N)
    kvq_score(q, lse, cache, prefix, accept_len, scores, positions, seen, path=path)
    seen = seen + accept_len + 1                             # once a step; a malformed row (accept_len -1) adds none
    prefix, _ = kvq_evict(cache, scores, positions, lengths, seen, keep, sink=4, recent=64)

``prefix`` holds the rows in the cache, ``seen`` the tokens that the sequences have had, evicted ones too: score
numbers the step's rows from ``seen`` as it was before the step, evict counts ``recent`` back from it after the step.
A chain's accepted rows (verify_chain) are in place already: no commit and no path, lengths = prefix + accept_len + 1.
"""

from __future__ import annotations

import ctypes
import math
from typing import Optional, Tuple

import torch

from . import SPEC_BF16, SPEC_F32, SpecError, _check, _stream, lib

_DIMS = (64, 128, 256)
# the handle of a device's current stream, without the Stream object around it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or _stream
_CODES = {torch.bfloat16: SPEC_BF16, torch.float32: SPEC_F32}


class _CacheArgs(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("k_codes", "k_scales", "v_codes", "v_scales")] +
                [(n, ctypes.c_int32) for n in ("B", "heads", "capacity", "head_dim")] +
                [(n, ctypes.c_int64) for n in ("code_batch", "code_head", "code_pos",
                                               "scale_batch", "scale_head", "scale_pos")])


class _Rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p)] + [(n, ctypes.c_int64) for n in ("batch", "pos", "head")]


class KVQCache:
    """One layer's four-bit cache over the caller's tensors.

    k_codes, v_codes [B, heads, capacity, D/2] and k_scales, v_scales [B, heads, capacity, D/32], all uint8 on
    one GPU.  The first three dimensions may be strided in any order (K and V alike), the last is contiguous;
    no two rows may share memory.  D (``head_dim``) is 64, 128 or 256.
    """

    def __init__(self, k_codes: torch.Tensor, k_scales: torch.Tensor, v_codes: torch.Tensor, v_scales: torch.Tensor):
        if k_codes.dim() != 4:
            raise ValueError("k_codes must be [B, heads, capacity, D/2]")
        B, H, S, half = k_codes.shape
        D = 2 * half
        if D not in _DIMS:
            raise ValueError(f"head_dim must be one of {_DIMS}, got {D}")
        if B < 1 or H < 1 or S < 1:
            raise ValueError("a cache needs at least one batch row, head and position")
        for t, name, last in ((k_codes, "k_codes", half), (v_codes, "v_codes", half),
                              (k_scales, "k_scales", D // 32), (v_scales, "v_scales", D // 32)):
            if not t.is_cuda or t.device != k_codes.device:
                raise ValueError(f"{name} must be a tensor on the cache's GPU")
            if t.dtype != torch.uint8:
                raise TypeError(f"{name} must be uint8, got {t.dtype}")
            if tuple(t.shape) != (B, H, S, last):
                raise ValueError(f"{name} must have shape {(B, H, S, last)}, got {tuple(t.shape)}")
            if t.stride(3) != 1:
                raise ValueError(f"the rows of {name} must be contiguous")
            if _overlaps(t):
                raise ValueError(f"the rows of {name} must not share memory")
        if k_codes.stride() != v_codes.stride() or k_scales.stride() != v_scales.stride():
            raise ValueError("K and V must have the same strides")
        self.k_codes, self.k_scales, self.v_codes, self.v_scales = k_codes, k_scales, v_codes, v_scales
        self.B, self.heads, self.capacity, self.head_dim = B, H, S, D
        self.device = k_codes.device
        self._args = _CacheArgs(k_codes.data_ptr(), k_scales.data_ptr(), v_codes.data_ptr(), v_scales.data_ptr(),
                                B, H, S, D, *k_codes.stride()[:3], *k_scales.stride()[:3])
        self._ref = ctypes.addressof(self._args)
        self._needs = {}                # workspace bytes of the calls made so far, by their sizes

    def _need(self, fn, *sizes) -> int:
        n = self._needs.get(sizes)
        if n is None:
            n = self._needs[sizes] = int(fn())
        return n


def _overlaps(t: torch.Tensor) -> bool:
    """Whether two rows of a strided tensor may share bytes (dimensions nested by stride are taken as apart)."""
    reach = t.shape[3]
    for stride, size in sorted((t.stride(d), t.shape[d]) for d in range(3) if t.shape[d] > 1):
        if stride < reach:
            return True
        reach += stride * (size - 1)
    return False


def new_kvq_cache(B: int, heads: int, capacity: int, head_dim: int, device) -> KVQCache:
    """An empty cache, [B, heads, capacity] rows; contents are undefined until appended."""
    if head_dim not in _DIMS:
        raise ValueError(f"head_dim must be one of {_DIMS}, got {head_dim}")
    codes = [torch.empty((B, heads, capacity, head_dim // 2), dtype=torch.uint8, device=device) for _ in range(2)]
    scales = [torch.empty((B, heads, capacity, head_dim // 32), dtype=torch.uint8, device=device) for _ in range(2)]
    return KVQCache(codes[0], scales[0], codes[1], scales[1])


def _tensor(t: torch.Tensor, name: str, dtype, shape, device) -> int:
    """Checks a contiguous tensor of the call and returns its address."""
    if t.dtype is dtype and t.get_device() == device.index and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != device.index:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _optional(t: Optional[torch.Tensor], name: str, dtype, shape, device):
    return None if t is None else _tensor(t, name, dtype, shape, device)


def _rows(t: torch.Tensor, name: str, cache: KVQCache) -> _Rows:
    """The strided rows [B, N, heads, D] of a call."""
    shape = t.shape
    if len(shape) != 4 or shape[0] != cache.B or shape[3] != cache.head_dim or shape[1] < 1 or shape[2] < 1:
        raise ValueError(f"{name} must be [{cache.B}, N, heads, {cache.head_dim}], got {tuple(shape)}")
    if t.dtype not in _CODES:
        raise TypeError(f"{name} must be bfloat16 or float32, got {t.dtype}")
    if t.get_device() != cache.device.index:
        raise ValueError(f"{name} must be on {cache.device}, got {t.device}")
    s = t.stride()
    if s[3] != 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    # the stride of a dimension of one element never counts
    return _Rows(t.data_ptr(), s[0] if shape[0] > 1 else 0, s[1] if shape[1] > 1 else 0, s[2] if shape[2] > 1 else 0)


def _call(fn, what: str, device: torch.device, *args) -> None:
    """One library call on the device's current stream, with that device current."""
    if torch.cuda.current_device() == device.index:
        rc = fn(*args, _raw_stream(device.index))
    else:
        with torch.cuda.device(device):
            rc = fn(*args, _raw_stream(device.index))
    if rc:
        _check(rc, what)


def _scratch(need: int, device: torch.device, given: Optional[torch.Tensor]) -> Tuple[Optional[int], object]:
    """A 256-byte aligned workspace (its contents do not matter): the given one, or a fresh one."""
    if need == 0:
        return None, None
    if given is None:
        given = torch.empty(need + 256, dtype=torch.uint8, device=device)
    elif given.dtype != torch.uint8 or given.device != device or not given.is_contiguous():
        raise ValueError(f"workspace must be a contiguous uint8 tensor on {device}")
    elif given.numel() < need + 256:
        raise ValueError(f"workspace needs {need + 256} bytes, got {given.numel()}")
    return (given.data_ptr() + 255) // 256 * 256, given


def kvq_append(cache: KVQCache, k: torch.Tensor, v: torch.Tensor, prefix: torch.Tensor, *,
               counts: Optional[torch.Tensor] = None) -> None:
    """Quantise k, v [B, N, heads, D] (bf16 or f32, strided) into slots prefix[b] .. prefix[b] + counts[b] - 1
    (``spec_kvq_append``).  prefix [B] int32; counts [B] int32, N by default.  Batch rows whose rows do not fit
    (or whose prefix is negative) are left as they were."""
    ra, rb = _rows(k, "k", cache), _rows(v, "v", cache)
    N = k.shape[1]
    if k.shape[2] != cache.heads or v.shape != k.shape or v.dtype != k.dtype:
        raise ValueError(f"k and v must both be [{cache.B}, {N}, {cache.heads}, {cache.head_dim}] of one type")
    dev, row = cache.device, (cache.B,)
    _call(lib().spec_kvq_append, "spec_kvq_append", dev, cache._ref, ctypes.addressof(ra), ctypes.addressof(rb),
          _CODES[k.dtype], N, _tensor(prefix, "prefix", torch.int32, row, dev),
          _optional(counts, "counts", torch.int32, row, dev))


def kvq_read(cache: KVQCache, prefix: torch.Tensor, N: int, *, counts: Optional[torch.Tensor] = None,
             dtype: torch.dtype = torch.bfloat16) -> Tuple[torch.Tensor, torch.Tensor]:
    """The values of slots prefix[b] .. prefix[b] + counts[b] - 1 (``spec_kvq_read``): (k, v) [B, N, heads, D] of
    ``dtype`` (bf16 or f32; exact in both), zeros past counts[b] and for batch rows out of range."""
    if dtype not in _CODES:
        raise TypeError(f"dtype must be bfloat16 or float32, got {dtype}")
    if N < 1:
        raise ValueError(f"N must be at least 1, got {N}")
    dev, row = cache.device, (cache.B,)
    shape = (cache.B, int(N), cache.heads, cache.head_dim)
    k = torch.empty(shape, dtype=dtype, device=dev)
    v = torch.empty_like(k)
    _call(lib().spec_kvq_read, "spec_kvq_read", dev, cache._ref, _CODES[dtype], int(N),
          _tensor(prefix, "prefix", torch.int32, row, dev), _optional(counts, "counts", torch.int32, row, dev),
          k.data_ptr(), v.data_ptr())
    return k, v


def kvq_attention_workspace_bytes(cache: KVQCache, N: int, q_heads: int, dtype: torch.dtype = torch.bfloat16) -> int:
    """Bytes of :func:`kvq_attention`'s workspace (give a tensor of 256 more)."""
    return int(lib().spec_kvq_attention_workspace_bytes(cache.B, N, q_heads, cache.heads, cache.head_dim,
                                                        cache.capacity, _CODES[dtype]))


def kvq_attention(q: torch.Tensor, cache: KVQCache, prefix: torch.Tensor, *, mask: Optional[torch.Tensor] = None,
                  counts: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                  out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None, workspace: Optional[torch.Tensor] = None
                  ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Softmax attention of the step's queries over cache and draft (``spec_kvq_attention``).

    q [B, N, q_heads, D] bf16 or f32 (strided); the new tokens' K and V rows are in slots prefix[b] + n already
    (:func:`kvq_append`).  mask: None (token n sees new tokens 0..n) or an ancestor mask, [B, N, N] or [N, N]
    uint8 (what :func:`tree_rerank` gives).  scale defaults to D ** -0.5.  Returns (out, of q's type and shape,
    lse [B, N, q_heads] f32); tokens n >= counts[b] and batch rows out of range give zeros and -inf.
    """
    rq = _rows(q, "q", cache)
    B, N, Hq, D = q.shape
    if Hq % cache.heads:
        raise ValueError(f"q_heads must be a multiple of {cache.heads}, got {Hq}")
    dev, row = cache.device, (B,)
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
    code = _CODES[q.dtype]
    need = cache._need(lambda: kvq_attention_workspace_bytes(cache, N, Hq, q.dtype), N, Hq, code)
    wp, _ws = _scratch(need, dev, workspace)
    _call(lib().spec_kvq_attention, "spec_kvq_attention", dev, ctypes.addressof(rq), code, Hq, N, cache._ref,
          _tensor(prefix, "prefix", torch.int32, row, dev), _optional(counts, "counts", torch.int32, row, dev),
          mp, mb, 1.0 / math.sqrt(D) if scale is None else float(scale), o.data_ptr(), lse.data_ptr(), wp, need)
    return o, lse


def kvq_commit(cache: KVQCache, prefix: torch.Tensor, path: torch.Tensor, accept_len: torch.Tensor,
               N: int) -> torch.Tensor:
    """The accepted paths' rows into place in the cache's four arrays (``spec_kv_commit`` on each); returns the new
    lengths [B] int32, -1 for malformed rows.  prefix and accept_len [B], path [B, D+1] int32."""
    dev, row = cache.device, (cache.B,)
    if path.dim() != 2 or path.shape[1] < 1:
        raise ValueError("path must be [B, D+1]")
    lists = (_tensor(prefix, "prefix", torch.int32, row, dev),
             _tensor(path, "path", torch.int32, (cache.B, path.shape[1]), dev), path.shape[1], int(N),
             _tensor(accept_len, "accept_len", torch.int32, row, dev))
    new_len = torch.empty(row, dtype=torch.int32, device=dev)
    for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales):
        batch, head, pos = t.stride()[:3]
        if cache.capacity == 1:                              # the stride of a dimension of one element never counts
            pos = t.shape[3]
        _call(lib().spec_kv_commit, "spec_kv_commit", dev, t.data_ptr(), cache.heads, head, cache.B, batch, pos,
              t.shape[3], cache.capacity, *lists, new_len.data_ptr())
    return new_len


def kvq_score_workspace_bytes(cache: KVQCache, N: int, q_heads: int, path_len: int = 0,
                              dtype: torch.dtype = torch.bfloat16) -> int:
    """Bytes of :func:`kvq_score`'s workspace (give a tensor of 256 more); path_len: path.shape[1], 0 without one."""
    return int(lib().spec_kvq_score_workspace_bytes(cache.B, N, q_heads, cache.heads, cache.head_dim, cache.capacity,
                                                    path_len, _CODES[dtype]))


def kvq_score(q: torch.Tensor, lse: torch.Tensor, cache: KVQCache, prefix: torch.Tensor, accept_len: torch.Tensor,
              scores: torch.Tensor, positions: torch.Tensor, seen: torch.Tensor, *,
              path: Optional[torch.Tensor] = None, scale: Optional[float] = None,
              workspace: Optional[torch.Tensor] = None) -> None:
    """Add the accepted queries' attention weights onto ``scores``, in place (``spec_kvq_score``).

    After :func:`kvq_commit`: q and lse [B, N, q_heads] as :func:`kvq_attention` took and gave them, prefix [B] the
    lengths BEFORE the step, path [B, D+1] and accept_len [B] the verification's (path None: tokens 0 ..
    accept_len[b]).  scores [B, heads, capacity] f32 and positions [B, heads, capacity] int32: the slots the step
    added start at their weight and at position seen[b] + i; seen [B] int32 counts the sequence's tokens before the
    step and is left as it is (add accept_len + 1 before :func:`kvq_evict` and the next step).
    """
    rq = _rows(q, "q", cache)
    B, N, Hq, D = q.shape
    if Hq % cache.heads:
        raise ValueError(f"q_heads must be a multiple of {cache.heads}, got {Hq}")
    dev, row, slots = cache.device, (B,), (B, cache.heads, cache.capacity)
    pp, stride = None, N
    if path is not None:
        if path.dim() != 2 or path.shape[1] < 1:
            raise ValueError("path must be [B, D+1]")
        stride = path.shape[1]
        pp = _tensor(path, "path", torch.int32, (B, stride), dev)
    width = 0 if path is None else stride
    need = cache._need(lambda: kvq_score_workspace_bytes(cache, N, Hq, width, q.dtype), N, Hq, width, q.dtype)
    wp, _ws = _scratch(need, dev, workspace)
    _call(lib().spec_kvq_score, "spec_kvq_score", dev, ctypes.addressof(rq), _CODES[q.dtype], Hq, N,
          _tensor(lse, "lse", torch.float32, (B, N, Hq), dev), cache._ref,
          _tensor(prefix, "prefix", torch.int32, row, dev), pp, stride,
          _tensor(accept_len, "accept_len", torch.int32, row, dev),
          1.0 / math.sqrt(D) if scale is None else float(scale), _tensor(scores, "scores", torch.float32, slots, dev),
          _tensor(positions, "positions", torch.int32, slots, dev), _tensor(seen, "seen", torch.int32, row, dev), wp, need)


def kvq_evict_workspace_bytes(cache: KVQCache, keep: int) -> int:
    """Bytes of :func:`kvq_evict`'s workspace (give a tensor of 256 more)."""
    return int(lib().spec_kvq_evict_workspace_bytes(cache.B, cache.heads, cache.capacity, keep))


def kvq_evict(cache: KVQCache, scores: torch.Tensor, positions: torch.Tensor, lengths: torch.Tensor,
              seen: torch.Tensor, keep: int, *, sink: int = 0, recent: int = 0,
              out_scores: Optional[torch.Tensor] = None, out_positions: Optional[torch.Tensor] = None,
              workspace: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Cut every head to its ``keep`` best rows, in place (``spec_kvq_evict``).

    Kept first are rows with positions below ``sink`` or at seen[b] - recent and later, then those of largest
    score; seen [B] int32 counts the sequence's tokens with this step's.  scores, positions [B, heads, capacity] are moved along in place, or written to ``out_scores`` and
    ``out_positions``.  Returns (new lengths [B], the slot each kept row came from [B, heads, keep]) int32.
    """
    dev, row, slots = cache.device, (cache.B,), (cache.B, cache.heads, cache.capacity)
    keep = int(keep)
    if not 1 <= keep <= cache.capacity:
        raise ValueError(f"keep must lie in [1, {cache.capacity}]")
    for n, name in ((sink, "sink"), (recent, "recent")):
        if not 0 <= n < 2 ** 31:
            raise ValueError(f"{name} must lie in [0, 2^31)")
    out_scores = scores if out_scores is None else out_scores
    out_positions = positions if out_positions is None else out_positions
    new_len = torch.empty(row, dtype=torch.int32, device=dev)
    source = torch.empty((cache.B, cache.heads, keep), dtype=torch.int32, device=dev)
    need = cache._need(lambda: kvq_evict_workspace_bytes(cache, keep), keep)
    wp, _ws = _scratch(need, dev, workspace)
    _call(lib().spec_kvq_evict, "spec_kvq_evict", dev, cache._ref,
          _tensor(scores, "scores", torch.float32, slots, dev),
          _tensor(positions, "positions", torch.int32, slots, dev),
          _tensor(lengths, "lengths", torch.int32, row, dev), _tensor(seen, "seen", torch.int32, row, dev), keep,
          int(sink), int(recent), _tensor(out_scores, "out_scores", torch.float32, slots, dev),
          _tensor(out_positions, "out_positions", torch.int32, slots, dev), new_len.data_ptr(), source.data_ptr(),
          wp, need)
    return new_len, source
