"""Serving operators: rotation of queries and keys at given positions, a paged
key-value cache in 8 bits, the attention over it, and the causal attention of
packed prompts.

A prompt and the steps after it, for a model with H query heads and Hkv key
heads of d columns (T packed tokens, sequence b in rows starts[b] to
starts[b + 1]):

    cos, sin = rope_tables(d, max_positions)
    cache = paged_cache(pages, page_tokens, Hkv, d)
    # the prompts: attention over the prompt itself, and its keys and values kept
    q, k_turned = rope_at(q, k, positions, cos, sin)
    o, _ = prompt_attn(q, k_turned, v, starts)
    cache_append(cache, k, v, starts, cached, table, cos, sin)   # cached = 0
    # one more token (or a few) of each sequence
    q, _ = rope_at(q, None, positions, cos, sin)
    cache_append(cache, k, v, starts, cached, table, cos, sin)
    o, _ = cache_attn(q.view(B, n, H, d), cache, cached + n, table)

All arithmetic of the operators runs in the CUDA library behind the C ABI
(include/attn_jvp.h); this module checks tensors and passes pointers, strides
and the current stream. Positions, lengths and page numbers live on the
device; one that is out of range is not used, and sync_status() then returns 7.
"""
from __future__ import annotations

import functools
import math
import struct
from typing import NamedTuple, Optional, Tuple

import torch

from . import _abi

_TYPES = {torch.bfloat16: _abi.DTYPE_BF16, torch.float32: _abi.DTYPE_F32,
          torch.float16: _abi.DTYPE_F16}
_LAYOUTS = {"interleaved": _abi.ROPE_INTERLEAVED, "half": _abi.ROPE_HALF}
_F8 = torch.float8_e4m3fn
_pack3 = struct.Struct("@3q").pack
# by value: the same numbers give the same (never changed) argument
_strides = functools.lru_cache(maxsize=4096)(_abi.Strides)
_NO_STRIDES = _abi.Strides(0, 0)


class PagedCache(NamedTuple):
    """Keys and values in pages: e4m3 codes k, v [pages, Hkv, page_tokens, d]
    and fp32 scales k_scale, v_scale [pages, Hkv]; a code c stands for c times
    its page's and head's scale. Views with other strides (tokens before heads,
    k and v interleaved by page) work as long as the d codes are adjacent, the
    strides are multiples of 16 and k and v have the same ones."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor


def paged_cache(pages: int, page_tokens: int, kv_heads: int, d: int, device="cuda") -> PagedCache:
    """An empty cache; page_tokens is 16, 32, 64 or 128, d 64 or 128."""
    if page_tokens not in (16, 32, 64, 128) or d not in (64, 128):
        raise ValueError("page_tokens is 16, 32, 64 or 128 and d is 64 or 128")
    if pages < 1 or kv_heads < 1:
        raise ValueError("pages and kv_heads must be positive")
    codes = [torch.zeros(pages, kv_heads, page_tokens, d, dtype=torch.uint8,
                         device=device).view(torch.float8_e4m3fn) for _ in range(2)]
    scales = [torch.ones(pages, kv_heads, dtype=torch.float32, device=device) for _ in range(2)]
    return PagedCache(*codes, *scales)


def rope_tables(rot: int, n_positions: int, base: float = 10000.0, scaling: Optional[str] = None,
                factor: float = 1.0, original_positions: Optional[int] = None,
                fast_turns: float = 32.0, slow_turns: float = 1.0,
                magnitude: Optional[float] = None,
                device="cuda") -> Tuple[torch.Tensor, torch.Tensor]:
    """cos and sin tables, fp32 [n_positions, rot/2], of the angles
    position * base^(-2i/rot), formed in 64 bits (the angle of a far position
    needs more than 32). `scaling` stretches them by `factor` for contexts
    longer than the original one:

      "linear"   every frequency divided by factor;
      "base"     base * factor^(rot / (rot - 2)): the lowest frequency divided
                 by factor, the highest kept;
      "by_parts" frequencies with at least fast_turns turns over
                 original_positions kept, those with at most slow_turns divided
                 by factor, a linear ramp over their index between; both tables
                 times `magnitude`, by default 0.1 ln(factor) + 1.
    """
    if rot < 16 or rot % 16:
        raise ValueError("rot must be a positive multiple of 16")
    if n_positions < 1 or not base > 1.0 or not factor >= 1.0:
        raise ValueError("n_positions >= 1, base > 1 and factor >= 1 are needed")
    i = torch.arange(0, rot, 2, dtype=torch.float64, device=device)
    if scaling == "base":
        base = base * factor ** (rot / (rot - 2))
    freq = base ** (-i / rot)
    scale = 1.0 if magnitude is None else magnitude
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "by_parts":
        if original_positions is None or original_positions < 1 or not fast_turns > slow_turns > 0:
            raise ValueError("by_parts needs original_positions and fast_turns > slow_turns > 0")

        def index(turns):  # of the frequency with that many turns over the original positions
            return rot * math.log(original_positions / (turns * 2 * math.pi)) / (2 * math.log(base))

        low = max(math.floor(index(fast_turns)), 0)
        high = min(math.ceil(index(slow_turns)), rot - 1)
        ramp = ((i / 2 - low) / max(high - low, 1e-3)).clamp(0, 1)
        freq = freq * (1 - ramp) + freq / factor * ramp
        if magnitude is None:
            scale = 0.1 * math.log(factor) + 1.0
    elif scaling not in (None, "base"):
        raise ValueError("scaling is None, 'linear', 'base' or 'by_parts'")
    angle = torch.arange(n_positions, dtype=torch.float64, device=device)[:, None] * freq
    return (angle.cos() * scale).float(), (angle.sin() * scale).float()


def _rows(t: torch.Tensor, what: str, like: Optional[torch.Tensor] = None) -> _abi.Strides:
    """Strides of a [T, heads, d] CUDA tensor whose d elements are adjacent."""
    st = t.stride()
    if len(st) != 3:
        raise ValueError(f"{what} must be [T, heads, d]")
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    if like is not None:
        a, b = t.shape, like.shape
        if a[0] != b[0] or a[2] != b[2] or t.dtype != like.dtype or t.device != like.device:
            raise ValueError(f"{what} must share tokens, head dim, dtype and device with the others")
    if st[2] != 1:
        raise ValueError(f"the last dimension of {what} must be contiguous")
    return _strides(st[0], st[1])


def _int32(t: torch.Tensor, what: str, device: torch.device, *shape) -> int:
    if t.dtype != torch.int32 or t.device != device or t.shape != shape or \
            (t.dim() == 1 and not t.is_contiguous()):
        raise ValueError(f"{what} must be a contiguous int32 {list(shape)} tensor on the inputs' device")
    return t.data_ptr()


def _table(t: torch.Tensor, B: int, device: torch.device) -> int:
    if t.dim() != 2 or t.dtype != torch.int32 or t.device != device or t.shape[0] != B or \
            t.shape[1] < 1 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError("page_table must be int32 [B, pages] with contiguous rows on the inputs' device")
    return t.data_ptr()


def _rope(cos: torch.Tensor, sin: torch.Tensor, layout: str, device: torch.device) -> bytes:
    for t in (cos, sin):
        if t.dim() != 2 or t.shape != cos.shape or t.dtype != torch.float32 or \
                t.device != device or not t.is_contiguous():
            raise ValueError("cos and sin must be contiguous fp32 [positions, rot/2] on the inputs' device")
    if layout not in _LAYOUTS:
        raise ValueError("layout is 'interleaved' or 'half'")
    n, half = cos.shape
    return _abi.pack_rope_tables(cos.data_ptr(), sin.data_ptr(), n, 2 * half, _LAYOUTS[layout])


def _cache(cache: PagedCache, device: torch.device) -> bytes:
    k, v, ks, vs = cache
    st, ss = k.stride(), ks.stride()
    if k.dim() != 4 or k.dtype != _F8 or v.dtype != _F8 or v.shape != k.shape or \
            v.stride() != st or st[3] != 1 or k.device != device or v.device != device:
        raise ValueError("cache k and v must be float8_e4m3fn [pages, Hkv, page_tokens, d] of the "
                         "same strides, d contiguous, on the inputs' device")
    if ks.shape != k.shape[:2] or vs.shape != ks.shape or ks.dtype != torch.float32 or \
            vs.dtype != torch.float32 or vs.stride() != ss or \
            ks.device != device or vs.device != device:
        raise ValueError("cache scales must be fp32 [pages, Hkv] of the same strides on the inputs' device")
    return _abi.pack_cache(k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), k.shape[0],
                           k.shape[2], st[0], st[1], st[2], ss[0], ss[1])


def _dtype(t: torch.Tensor, types=_TYPES) -> int:
    code = types.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return code


def _call(fn, name: str, device: torch.device, *args) -> None:
    """fn(*args, stream) on the tensors' device and its current stream."""
    # the stream's handle without an object around it: a few microseconds less
    stream = torch._C._cuda_getCurrentRawStream(device.index)
    if device.index == torch.cuda.current_device():
        rc = fn(*args, stream)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, stream)
    if rc != _abi.OK:
        _abi.check(rc, name)


def rope_at(q: torch.Tensor, k: Optional[torch.Tensor], positions: torch.Tensor,
            cos: torch.Tensor, sin: torch.Tensor, layout: str = "interleaved",
            transpose: bool = False, out=None):
    """Rotary embedding of q [T, H, d] and k [T, Hkv, d] (or None) at positions
    [T] (int32 or int64) by the tables' rows, on the first rot columns of each
    head: pairs (2i, 2i + 1) ("interleaved") or (i, i + rot/2) ("half").
    Returns (q_out, k_out). `transpose` applies the transposed matrix: given
    gradients of the rotated tensors, those of q and k. `out` may give the two
    outputs, the inputs themselves for an in-place rotation."""
    sq = _rows(q, "q")
    sk = _rows(k, "k", q) if k is not None else _NO_STRIDES
    T, H, d = q.shape
    if positions.shape != (T,) or positions.dtype not in (torch.int32, torch.int64) or \
            positions.device != q.device or not positions.is_contiguous():
        raise ValueError("positions must be contiguous int32 or int64 [T] on the inputs' device")
    tables = _rope(cos, sin, layout, q.device)
    if out is None:
        qo = torch.empty((T, H, d), dtype=q.dtype, device=q.device)
        so = _strides(H * d, d)
        ko, sko = None, _NO_STRIDES
        if k is not None:
            ko, sko = torch.empty(k.shape, dtype=q.dtype, device=q.device), _strides(k.shape[1] * d, d)
    else:
        qo, ko = out
        if qo.shape != q.shape or (k is None) != (ko is None) or \
                (k is not None and ko.shape != k.shape):
            raise ValueError("out must give tensors of q's and k's shapes")
        so = _rows(qo, "out", q)
        sko = _rows(ko, "out", q) if ko is not None else _NO_STRIDES
    shape = _abi.pack_tokens(T, H, k.shape[1] if k is not None else 0, d, _dtype(q), 0.0)
    _call(_abi.load().attn_jvp_rope_at, "attn_jvp_rope_at", q.device, shape, q.data_ptr(), sq,
          k.data_ptr() if k is not None else None, sk, positions.data_ptr(),
          positions.element_size(), tables, int(transpose), qo.data_ptr(), so,
          ko.data_ptr() if ko is not None else None, sko)
    return qo, ko


def cache_append(cache: PagedCache, k: torch.Tensor, v: torch.Tensor, starts: torch.Tensor,
                 cached: torch.Tensor, page_table: torch.Tensor,
                 cos: Optional[torch.Tensor] = None, sin: Optional[torch.Tensor] = None,
                 layout: str = "interleaved") -> None:
    """Append the packed tokens k, v [T, Hkv, d] to the cache: rows starts[b] to
    starts[b + 1] (starts [B + 1], int32) become tokens cached[b] on (cached [B],
    int32) of sequence b, in the pages page_table[b] (int32 [B, W]). With cos and
    sin the keys are rotated by their position in the sequence on the way. Each
    page and head keeps one power-of-two scale, the smallest that its tokens fit
    under; it grows (and the page is rounded to it) when later tokens need it."""
    sk, sv = _rows(k, "k"), _rows(v, "v", k)
    if v.shape != k.shape:
        raise ValueError("k and v must have the same shape")
    if cache.k.dim() != 4 or cache.k.shape[1] != k.shape[1] or cache.k.shape[3] != k.shape[2]:
        raise ValueError("the cache must have the heads and head dim of k and v")
    T, heads, d = k.shape
    B = cached.shape[0] if cached.dim() == 1 else -1
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin go together")
    tables = _rope(cos, sin, layout, k.device) if cos is not None else None
    desc = _cache(cache, k.device)
    shape = _abi.pack_tokens(T, heads, heads, d, _dtype(k), 0.0)
    _call(_abi.load().attn_jvp_cache_append, "attn_jvp_cache_append", k.device, shape,
          k.data_ptr(), sk, v.data_ptr(), sv, desc, B,
          _int32(starts, "starts", k.device, B + 1), _int32(cached, "cached", k.device, B),
          _table(page_table, B, k.device), page_table.shape[1], page_table.stride(0),
          tables)


_ATTN_TYPES = {torch.bfloat16: _abi.DTYPE_BF16, torch.float16: _abi.DTYPE_F16}


def _scale(scale: Optional[float]) -> float:
    if scale is None:
        return 0.0
    if not (scale > 0 and math.isfinite(scale)):
        raise ValueError("scale must be positive and finite")
    return float(scale)


def cache_attn(q: torch.Tensor, cache: PagedCache, seq_lens: torch.Tensor,
               page_table: torch.Tensor, causal: bool = True, scale: Optional[float] = None,
               max_len: int = 0, out=None):
    """Attention of the newest n tokens of each of B sequences, q [B, n, H, d]
    (bf16 or fp16), over the cache: seq_lens [B] (int32) tokens each, the new
    ones included, in the pages page_table[b]. causal: query i sees the keys up
    to its own token; else every query sees all seq_lens[b] keys (a chunk with
    full attention inside it). Returns O [B, n, H, d] and LSE [B, H, n] (fp32);
    a row without keys gets 0 and -inf. `max_len`, an upper bound of the lengths
    known on the host, helps to split the work when the table is much wider."""
    if q.dim() != 4 or not q.is_cuda:
        raise ValueError("q must be a CUDA tensor [B, n, H, d]")
    B, n, H, d = q.shape
    st = q.stride()
    if st[3] != 1:
        raise ValueError("the last dimension of q must be contiguous")
    Hkv = cache.k.shape[1] if cache.k.dim() == 4 else 0
    if Hkv < 1 or cache.k.shape[3] != d or H % Hkv:
        raise ValueError("the cache must have q's head dim and a number of heads that divides q's")
    desc = _cache(cache, q.device)
    lens_at, table_at = _int32(seq_lens, "seq_lens", q.device, B), _table(page_table, B, q.device)
    if out is None:
        o = torch.empty((B, n, H, d), dtype=q.dtype, device=q.device)
        lse = torch.empty((B, H, n), dtype=torch.float32, device=q.device)
    else:
        o, lse = out
        _check_out(o, lse, q, (B, n, H, d), (B, H, n))
    shape = _abi.pack_shape(B, n, H, d, _dtype(q, _ATTN_TYPES), _scale(scale))
    most = page_table.shape[1] * cache.k.shape[2]
    if 0 < max_len < most:
        most = max_len
    size = _workspace_bytes(q.device.index, B, n, H, d, Hkv, most)
    work = torch.empty(size, dtype=torch.uint8, device=q.device) if size else None
    _call(_abi.load().attn_jvp_cache_attn, "attn_jvp_cache_attn", q.device, shape, Hkv,
          q.data_ptr(), _pack3(st[0], st[1], st[2]), desc,
          lens_at, table_at, page_table.shape[1], page_table.stride(0), max_len, int(causal),
          work.data_ptr() if size else None, size, o.data_ptr(), lse.data_ptr())
    return o, lse


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(device: int, B: int, n: int, H: int, d: int, Hkv: int, most: int) -> int:
    with torch.cuda.device(device):
        size = _abi.load().attn_jvp_cache_attn_workspace_bytes(
            _abi.pack_shape(B, n, H, d, _abi.DTYPE_BF16, 0.0), Hkv, most)
    if size < 0:
        raise ValueError("bad shape, or no usable device")
    return size


def _check_out(o, lse, q, o_shape, lse_shape):
    if o.shape != o_shape or o.dtype != q.dtype or o.device != q.device or not o.is_contiguous() or \
            lse.shape != lse_shape or lse.dtype != torch.float32 or lse.device != q.device or \
            not lse.is_contiguous():
        raise ValueError(f"out must be contiguous: o {list(o_shape)} of q's type, "
                         f"lse fp32 {list(lse_shape)}, on q's device")


def prompt_attn(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, starts: torch.Tensor,
                scale: Optional[float] = None, out=None):
    """Causal attention inside each packed sequence: q [T, H, d], k and v
    [T, Hkv, d] (bf16 or fp16, H a multiple of Hkv), sequence b in rows
    starts[b] to starts[b + 1] (starts [B + 1], int32). Returns O [T, H, d] and
    LSE [H, T] (fp32). Rows outside the sequences are left as they were in
    `out` (and undefined without it)."""
    sq, sk, sv = _rows(q, "q"), _rows(k, "k", q), _rows(v, "v", q)
    T, H, d = q.shape
    if v.shape != k.shape or k.shape[1] < 1 or H % k.shape[1]:
        raise ValueError("k and v must have the same number of heads, which divides q's")
    if starts.dim() != 1 or starts.shape[0] < 1:
        raise ValueError("starts must be [B + 1]")
    B = starts.shape[0] - 1
    if out is None:
        o = torch.empty((T, H, d), dtype=q.dtype, device=q.device)
        lse = torch.empty((H, T), dtype=torch.float32, device=q.device)
    else:
        o, lse = out
        _check_out(o, lse, q, (T, H, d), (H, T))
    shape = _abi.pack_tokens(T, H, k.shape[1], d, _dtype(q, _ATTN_TYPES), _scale(scale))
    _call(_abi.load().attn_jvp_prompt_attn, "attn_jvp_prompt_attn", q.device, shape, q.data_ptr(),
          sq, k.data_ptr(), sk, v.data_ptr(), sv, B,
          _int32(starts, "starts", q.device, B + 1), o.data_ptr(), lse.data_ptr())
    return o, lse
