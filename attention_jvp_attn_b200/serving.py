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
(include/attn_jvp.h); a binding in C++ (csrc/serve_binding.cpp) checks tensors
and passes pointers, strides and the current stream. Positions, lengths and page numbers live on the
device; one that is out of range is not used, and sync_status() then returns 7.

As the package's other functions, none of these is registered with autograd: results carry
no graph, whatever the inputs require. The gradient of rope_at is rope_at(..., transpose=True).
Sums, maxima and LSE of the attentions are in 32 bits, probabilities in 16 (prompt_attn:
the inputs' type; cache_attn: fp16, the page's value scale included).
"""
from __future__ import annotations

import math
import threading
from typing import NamedTuple, Optional, Tuple

import torch

from . import _abi

_bound = None
_lock = threading.Lock()


def _native():
    """The binding (csrc/serve_binding.cpp), set to the library that is loaded."""
    global _bound
    lib = _abi.load()
    if _bound is None or _bound[0] is not lib:
        with _lock:
            try:
                from . import _serving, build
            except ImportError as e:
                raise RuntimeError("binding of the serving operators not built or not loadable "
                                   f"(run `python -m attention_jvp_attn_b200.build`): {e}") from e
            if _serving.built_for != build.binding_built_for():
                raise RuntimeError(f"binding of the serving operators built for {_serving.built_for!r}, this is "
                                   f"{build.binding_built_for()!r} (run `python -m attention_jvp_attn_b200.build`)")
            _serving.bind(_abi.check, *(_abi.address(lib, f) for f in (
                "attn_jvp_rope_at", "attn_jvp_cache_append", "attn_jvp_cache_attn",
                "attn_jvp_cache_attn_workspace_bytes", "attn_jvp_prompt_attn")))
            _bound = lib, _serving
    return _bound[1]


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

    "base" is the published NTK-aware change of base, "by_parts" the published YaRN
    method. So that tables agree with those of other programs two of its conventions
    are kept: the ramp's upper index is bounded by rot - 1 (indices end at rot/2 - 1),
    and its width is at least 1e-3.
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


def rope_at(q: torch.Tensor, k: Optional[torch.Tensor], positions: torch.Tensor,
            cos: torch.Tensor, sin: torch.Tensor, layout: str = "interleaved",
            transpose: bool = False, out=None):
    """Rotary embedding of q [T, H, d] and k [T, Hkv, d] (or None) at positions
    [T] (int32 or int64) by the tables' rows, on the first rot columns of each
    head: pairs (2i, 2i + 1) ("interleaved") or (i, i + rot/2) ("half").
    Returns (q_out, k_out). `transpose` applies the transposed matrix: given
    gradients of the rotated tensors, those of q and k. `out` may give the two
    outputs, the inputs themselves for an in-place rotation."""
    return _native().rope_at(q, k, positions, cos, sin, layout, transpose, out)


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
    _native().cache_append(cache, k, v, starts, cached, page_table, cos, sin, layout)


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
    return _native().cache_attn(q, cache, seq_lens, page_table, causal, scale, max_len, out)


def prompt_attn(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, starts: torch.Tensor,
                scale: Optional[float] = None, out=None):
    """Causal attention inside each packed sequence: q [T, H, d], k and v
    [T, Hkv, d] (bf16 or fp16, H a multiple of Hkv), sequence b in rows
    starts[b] to starts[b + 1] (starts [B + 1], int32). Returns O [T, H, d] and
    LSE [H, T] (fp32). Rows outside the sequences are left as they were in
    `out` (and undefined without it)."""
    return _native().prompt_attn(q, k, v, starts, scale, out)
