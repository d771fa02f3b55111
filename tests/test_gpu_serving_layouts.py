"""The serving operators over the layouts that strides allow: heads before tokens,
caches in any order of pages, heads and tokens, and many query heads per key head."""
import numpy as np
import pytest
import torch

import attention_jvp_attn_b200 as aj
from oracle import serving_oracle as orc
from test_gpu_serving import F8, check_attn, f64, filled, ints, ok, randn, rng, stale, tables
from test_gpu_serving_use import same

pytestmark = pytest.mark.gpu


def heads_first(x):
    """The same [T, heads, d] values, stored as [heads, T, d]."""
    return x.transpose(0, 1).contiguous().transpose(0, 1)


@pytest.mark.parametrize("T,H,Hkv,d,dtype", [(1, 2, 1, 64, torch.float16), (300, 4, 2, 128, torch.bfloat16),
                                             (1100, 40, 8, 64, torch.bfloat16)])
def test_prompt_heads_before_tokens(T, H, Hkv, d, dtype):
    g = rng(T + H)
    q, k, v = (randn(g, T, h, d, dtype=dtype) for h in (H, Hkv, Hkv))
    starts = ints([0, T // 3, T])
    want = aj.prompt_attn(q, k, v, starts)
    for given in ((heads_first(q), heads_first(k), heads_first(v)), (q, heads_first(k), v), (heads_first(q), k, heads_first(v))):
        got = aj.prompt_attn(*given, starts)
        ok()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rope_and_append_heads_before_tokens(dtype):
    g = rng(4)
    q, k, v = (randn(g, 50, h, 128, dtype=dtype) for h in (6, 2, 2))
    cos, sin = aj.rope_tables(96, 200)
    pos = torch.arange(50, device="cuda")
    want = aj.rope_at(q, k, pos, cos, sin, layout="half")
    out = (heads_first(torch.zeros_like(q)), torch.zeros_like(k))
    got = aj.rope_at(heads_first(q), heads_first(k), pos, cos, sin, layout="half", out=out)
    ok()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    a, b = (aj.paged_cache(4, 32, 2, 128) for _ in range(2))
    for cache, kv in ((a, (k, v)), (b, (heads_first(k), v))):
        aj.cache_append(cache, *kv, ints([0, 20, 50]), ints([40, 3]), ints([[3, 2], [1, 0]]), cos, sin)
    ok()
    assert all(same(x, y) for x, y in zip(a, b))


ORDERS = [(1, 0, 2), (2, 0, 1), (0, 2, 1), (2, 1, 0), (1, 2, 0)]  # of pages, heads and tokens in memory


@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("d,page", [(64, 128), (128, 16)])
def test_cache_in_any_order(order, d, page):
    g = rng(d + sum(i * o for i, o in enumerate(order)))
    base = filled(g, 40, 3, page, d)

    def ordered(t):
        x = t.view(torch.uint8)
        back = [order.index(i) for i in range(3)]
        return x.permute(*order, 3).contiguous().permute(*back, 3).view(F8)

    turned = aj.PagedCache(ordered(base.k), ordered(base.v), *(s.t().contiguous().t() for s in (base.k_scale, base.v_scale)))
    assert turned.k.stride() != base.k.stride() and same(turned.k.contiguous(), base.k)
    lens = [300, 150]
    table = tables(g, 40, lens, page)
    k, v = randn(g, 60, 3, d), randn(g, 60, 3, d)
    for c in (base, turned):
        aj.cache_append(c, k, v, ints([0, 1, 60]), ints([299, 91]), table)
    ok()
    assert same(turned.k.contiguous(), base.k) and same(turned.v.contiguous(), base.v)
    assert torch.equal(turned.k_scale, base.k_scale) and torch.equal(turned.v_scale, base.v_scale)
    for n, H in ((1, 3), (3, 12), (30, 6), (150, 3)):
        q = randn(g, 2, n, H, d)
        # the queries too: heads before tokens
        turned_q = q.transpose(1, 2).contiguous().transpose(1, 2)
        a, b = aj.cache_attn(q, base, ints(lens), table), aj.cache_attn(turned_q, turned, ints(lens), table)
        ok()
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("n,H,Hkv,d,dtype", [(1, 17, 1, 64, torch.bfloat16), (1, 64, 2, 128, torch.float16),
                                             (1, 128, 1, 64, torch.bfloat16), (1, 300, 1, 128, torch.bfloat16),
                                             (3, 129, 1, 64, torch.float16)])
def test_many_query_heads_per_key_head(n, H, Hkv, d, dtype):
    """Single tokens whose key head has more than 16 query heads, up to several row tiles."""
    g = rng(n + H)
    lens = [700, 1, 0, 129]
    pages = sum(max(1, -(-m // 32)) for m in lens) + 2
    cache = filled(g, pages, Hkv, 32, d)
    table = tables(g, pages, lens, 32)
    stale(cache, table, lens, 32)
    q = randn(g, 4, n, H, d, dtype=dtype)
    scale = 0.8 / np.sqrt(d)
    ref = orc.cache_attn(f64(q), f64(cache.k), f64(cache.v), f64(cache.k_scale), f64(cache.v_scale), lens,
                         table.cpu().numpy(), True, scale)
    lost = 4 * max(lens) * 448 * 2.0 ** -7 * 2.0 ** -32 * np.moveaxis(ref[4], -1, 1)[..., None]
    o, lse = aj.cache_attn(q, cache, ints(lens), table, scale=scale)
    ok()
    check_attn(o, lse, q, ref, scale, 2.0 ** -11, lost)
