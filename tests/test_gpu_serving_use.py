"""The serving operators as they are used: a prompt and decode steps after one
another, captured in graphs, on several streams at once, with values that must
not reach masked rows, with data out of range, and in caches beyond 4 GB."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import attention_jvp_attn_b200 as aj
from oracle import serving_oracle as orc
from test_gpu_serving import F8, check_attn, f64, filled, ints, ok, pool, randn, rng, stale, tables

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


def same(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("layout,d,page", [("half", 64, 16), ("interleaved", 128, 64)])
def test_prompt_then_steps(layout, d, page):
    """Packed prompts, then single tokens and a run of three, each step's cache and
    attention against the oracle on the cache as it then is, and against attention
    over the keys before they were rounded (e4m3 keeps 2^-4 of each)."""
    g = rng(d)
    H, Hkv, lens = 4, 2, [5, 130, 0]
    B = len(lens)
    cos, sin = aj.rope_tables(d // 2, 400)
    cache = aj.paged_cache(40, page, Hkv, d)
    table = tables(g, 40, [m + 40 for m in lens], page)
    starts = ints([0, 5, 135, 135])
    T = 135
    qkv = randn(g, T, H + 2 * Hkv, d)
    q, k, v = qkv.split([H, Hkv, Hkv], 1)
    pos = torch.cat([torch.arange(m) for m in lens]).cuda()
    qr, kr = aj.rope_at(q, k, pos, cos, sin, layout=layout)
    o, lse = aj.prompt_attn(qr, kr, v, starts)
    ok()
    scale = 1 / np.sqrt(d)
    check_attn(o, lse, q, orc.prompt_attn(f64(qr), f64(kr), f64(v), [0, 5, 135, 135], scale), scale, 2.0 ** -8)
    keys = [f64(kr)[0:5], f64(kr)[5:135], np.zeros((0, Hkv, d))]
    vals = [f64(v)[0:5], f64(v)[5:135], np.zeros((0, Hkv, d))]
    cached = ints([0, 0, 0])
    aj.cache_append(cache, k, v, starts, cached, table, cos, sin, layout=layout)
    have = list(lens)
    for n in (1, 1, 3, 1):
        qkv = randn(g, B * n, H + 2 * Hkv, d)
        q, k, v = qkv.split([H, Hkv, Hkv], 1)
        pos = torch.cat([m + torch.arange(n) for m in have]).cuda()
        qr, kr = aj.rope_at(q, k, pos, cos, sin, layout=layout)
        aj.cache_append(cache, k, v, ints([n * b for b in range(B + 1)]), ints(have), table, cos, sin, layout=layout)
        have = [m + n for m in have]
        qb = qr.view(B, n, H, d)
        o, lse = aj.cache_attn(qb, cache, ints(have), table)
        ok()
        ref = orc.cache_attn(f64(qb), f64(cache.k), f64(cache.v), f64(cache.k_scale), f64(cache.v_scale), have,
                             table.cpu().numpy(), True, scale)
        check_attn(o, lse, qb, ref, scale, 2.0 ** -11, 200 * 448 * 2.0 ** -5 * 2.0 ** -25)
        for b in range(B):
            keys[b] = np.concatenate([keys[b], f64(kr)[b * n:(b + 1) * n]])
            vals[b] = np.concatenate([vals[b], f64(v)[b * n:(b + 1) * n]])
            seen = have[b] - n + 1 + np.arange(n)
            for h in range(H):
                full, *_ , pv, qk, pm = orc.softmax_rows(f64(qb)[b, :, h], keys[b][:, h // 2], vals[b][:, h // 2], scale, seen)
                # scores off by at most 2^-4 A, each probability by e^(2 * 2^-4 A) - 1, each value by 2^-4
                off = np.expm1(2 * (2.0 ** -4 + 2.0 ** -8) * qk)[:, None] * pv * 1.07 + 2.0 ** -4 * pv + 2.0 ** -6
                assert (np.abs(f64(o)[b, :, h] - full) <= off + 2.0 ** -7 * np.abs(full)).all()


# ------------------------------------------------------------------ values that must not reach a row
@pytest.mark.parametrize("d,dtype", [(64, torch.bfloat16), (128, torch.float16), (128, torch.bfloat16)])
def test_prompt_nonfinite_rows(d, dtype):
    """Infinities and NaN in k and v of some rows: rows before them (and other
    sequences) come out bit for bit as without them, rows that see them as the
    formula says."""
    g = rng(d + 1)
    lens = [300, 70, 200]
    starts = np.concatenate([[0], np.cumsum(lens)])
    q, k, v = (randn(g, 570, h, d, dtype=dtype) for h in (4, 2, 2))
    clean = aj.prompt_attn(q, k, v, ints(starts))
    v2, k2 = v.clone(), k.clone()
    for row, col, val in ((129, 3, INF), (200, 5, NAN), (299, 0, -INF), (299, 7, NAN), (330, 9, -INF)):
        v2[row, :, col] = val
    v2[131, 1, 3] = -INF  # meets the +inf of row 129 in head 1 of the keys: NaN from row 131 on
    o, lse = aj.prompt_attn(q, k, v2, ints(starts))
    ok()
    assert torch.equal(lse, clean[1])
    want = clean[0].float().clone()
    want[129:300, :, 3] = INF
    want[131:300, 2:, 3] = NAN
    want[200:300, :, 5] = NAN
    want[299:300, :, 0] = -INF
    want[299:300, :, 7] = NAN
    want[330:370, :, 9] = -INF
    bad = ~torch.isfinite(want)
    assert torch.equal(o.float()[~bad], want[~bad])
    assert (torch.isnan(o) == torch.isnan(want)).all()
    assert torch.equal(o.float()[bad & ~torch.isnan(want)], want[bad & ~torch.isnan(want)])
    k2[250] = NAN  # every row of the sequence from it on is NaN; the others unchanged
    o, lse = aj.prompt_attn(q, k2, v, ints(starts))
    ok()
    keep = torch.ones(570, dtype=torch.bool, device="cuda")
    keep[250:300] = False
    assert torch.equal(o[keep], clean[0][keep]) and torch.equal(lse[:, keep], clean[1][:, keep])
    assert torch.isnan(o[~keep]).all()


@pytest.mark.parametrize("n,H,lens", [(3, 2, [40, 33]), (5, 8, [70, 6]), (150, 2, [400, 150]), (40, 16, [300, 41])])
def test_cache_nan_values(n, H, lens):
    """NaN codes among the newest tokens reach only the rows that see them."""
    g = rng(n)
    cache = filled(g, 40, 2, 16, 64)
    table = tables(g, 40, lens, 16)
    q = randn(g, 2, n, H, 64)
    clean = aj.cache_attn(q, cache, ints(lens), table)
    raw = cache.v.view(torch.uint8)
    want = clean[0].float().clone()
    for b, back, col in ((0, 2, 5), (1, 1, 63), (0, n, 0)):  # the token `back` before the end
        j = lens[b] - back
        raw[table[b, j // 16].item(), :, j % 16, col] = 0xFF if back == 1 else 0x7F
        want[b, max(0, j - (lens[b] - n)):, :, col] = NAN
    o, lse = aj.cache_attn(q, cache, ints(lens), table)
    ok()
    assert (torch.isnan(o) == torch.isnan(want)).all() and torch.equal(lse, clean[1])
    # bit for bit, but that the slow path's other columns are the same products
    assert torch.equal(o.float()[~torch.isnan(want)], want[~torch.isnan(want)])
    full = aj.cache_attn(q, cache, ints(lens), table, causal=False)[0]
    ok()
    assert torch.isnan(full[0, :, :, 5]).all() and torch.isnan(full[1, :, :, 63]).all()


def test_cache_far_earlier_nan():
    """A NaN value that every row sees."""
    g = rng(2)
    for n, H in ((1, 4), (100, 4)):
        cache = filled(g, 40, 2, 64, 128)
        table = tables(g, 40, [700], 64)
        cache.v.view(torch.uint8)[table[0, 1].item(), :, 3, 17] = 0x7F
        o, _ = aj.cache_attn(randn(g, 1, n, H, 128), cache, ints([700]), table)
        ok()
        assert torch.isnan(o[..., 17]).all() and torch.isfinite(o[..., :17]).all() and torch.isfinite(o[..., 18:]).all()


# ------------------------------------------------------------------ scales and layouts
@pytest.mark.parametrize("n,H", [(1, 4), (70, 4)])
def test_cache_scales_of_any_size(n, H):
    """Scales that are no powers of two and differ by 2^20 from page to page."""
    g = rng(31 + n)
    cache = filled(g, 60, 2, 16, 64)
    for s in (cache.k_scale, cache.v_scale):
        s.mul_(torch.exp(torch.rand(s.shape, generator=g, device="cuda")))
    cache.v_scale.mul_(torch.exp2(torch.randint(-10, 11, (60, 2), generator=g, device="cuda").float()))
    lens = [500, 290]
    table = tables(g, 60, lens, 16)
    q = randn(g, 2, n, H, 64)
    ref = orc.cache_attn(f64(q), f64(cache.k), f64(cache.v), f64(cache.k_scale), f64(cache.v_scale), lens,
                         table.cpu().numpy(), True, 0.125)
    o, lse = aj.cache_attn(q, cache, ints(lens), table)
    ok()
    # a probability times its value scale is rounded to fp16 with an absolute error of
    # at most 2^-25 of the largest such product so far: over the tokens, times codes up to 448
    most = ref[4].max() * f64(cache.v_scale).max()
    check_attn(o, lse, q, ref, 0.125, 2.0 ** -11, 500 * 448 * 2.0 ** -25 * most)


def test_cache_views_of_one_pool():
    """k and v interleaved by page in one pool, table rows with a stride, scales of one tensor."""
    g = rng(12)
    base = filled(g, 30, 2, 32, 128)
    both = torch.stack([base.k.view(torch.uint8), base.v.view(torch.uint8)], 1)  # [pages, 2, heads, page, d]
    scales = torch.stack([base.k_scale, base.v_scale], -1)                         # [pages, heads, 2]
    view = aj.PagedCache(both[:, 0].view(F8), both[:, 1].view(F8), scales[..., 0], scales[..., 1])
    lens = [100, 333]
    table = tables(g, 30, lens, 32)
    wide = torch.zeros(2, 40, dtype=torch.int32, device="cuda")
    wide[:, 7:7 + table.shape[1]] = table
    part = wide[:, 7:7 + table.shape[1]]
    for n, H in ((2, 4), (60, 4)):
        q = randn(g, 2, n, H, 128)
        a, b = aj.cache_attn(q, base, ints(lens), table), aj.cache_attn(q, view, ints(lens), part)
        ok()
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    k, v = randn(g, 9, 2, 128), randn(g, 9, 2, 128)
    for c, t in ((base, table), (view, part)):
        aj.cache_append(c, k, v, ints([0, 4, 9]), ints([92, 300]), t)
    ok()
    assert same(base.k, view.k.contiguous()) and same(base.v, view.v.contiguous())
    assert torch.equal(base.k_scale, view.k_scale) and torch.equal(base.v_scale, view.v_scale)


def test_shared_prefix_pages():
    """Two sequences whose tables name the same pages."""
    g = rng(13)
    cache = filled(g, 10, 1, 16, 64)
    table = ints([[3, 1, 7], [3, 1, 2]])
    q = randn(g, 1, 1, 2, 64).expand(2, 1, 2, 64)  # a stride of 0 over the sequences
    o, lse = aj.cache_attn(q, cache, ints([32, 32]), table)
    ok()
    assert torch.equal(o[0], o[1]) and torch.equal(lse[0], lse[1])


# ------------------------------------------------------------------ data out of range
@pytest.mark.parametrize("n,H,width", [(1, 4, 4), (40, 4, 4), (1, 4, 300)])
def test_cache_attn_bad_indices(n, H, width):
    g = rng(n + width)
    cache = filled(g, 20, 2, 16, 64)
    table = torch.zeros(3, width, dtype=torch.int32, device="cuda")
    table[:, :4] = ints([[1, 2, 3, 4], [5, 6, 7, 8], [9, 10, 11, 12]])
    q = randn(g, 3, n, H, 64)
    good = aj.cache_attn(q, cache, ints([60, 64, 50]), table)
    assert aj.sync_status() == 0
    for bad in (-1, 16 * width + 1, 2 ** 31 - 1):
        o, lse = aj.cache_attn(q, cache, ints([60, bad, 50]), table)
        assert aj.sync_status() == 7
        assert (o[1] == 0).all() and torch.isneginf(lse[1]).all()
        for b in (0, 2):
            assert torch.allclose(o[b].float(), good[0][b].float(), rtol=2.0 ** -7, atol=2.0 ** -7)
    for page in (20, -5, 2 ** 31 - 1):  # the tokens of a bad page count as hidden
        t = table.clone()
        t[1, 1] = page
        o, lse = aj.cache_attn(q, cache, ints([60, 64, 50]), t, causal=False)
        assert aj.sync_status() == 7
        t2 = table.clone()
        t2[1, :3] = ints([5, 7, 8])
        want = aj.cache_attn(q, cache, ints([60, 48, 50]), t2, causal=False)
        assert aj.sync_status() == 0
        assert torch.allclose(o.float(), want[0].float(), rtol=2.0 ** -7, atol=2.0 ** -7)
        assert torch.allclose(lse, want[1], rtol=1e-5, atol=1e-5)


@pytest.mark.parametrize("d,dtype", [(64, torch.float16), (128, torch.bfloat16)])
def test_prompt_blocks_of_one_and_two_row_tiles(d, dtype):
    """Many heads take blocks of two row tiles, few heads blocks of one; both against
    the oracle over sequences that end inside, at and behind tiles, and with values
    that are not finite in their last rows, which earlier rows must not meet."""
    g = rng(d + 3)
    lens = [300, 1, 257, 128, 0, 129, 511]
    starts = np.concatenate([[0], np.cumsum(lens)])
    T, H, few = int(starts[-1]), 64, 4  # 64 heads: more than 800 pairs of row tiles
    q, k, v = randn(g, T, H, d, dtype=dtype), randn(g, T, 2, d, dtype=dtype), randn(g, T, 2, d, dtype=dtype)
    u = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -11
    scale = 0.7 / np.sqrt(d)
    ref = orc.prompt_attn(f64(q[:, 30:34]), f64(k), f64(v), starts, scale)  # two heads of each key head
    qf = q[:, 30:34].contiguous()
    outs = {}
    for bad in (False, True):
        if bad:
            v = v.clone()
            for e in starts[1:]:
                v[e - 1, :, 3] = NAN
                v[max(e - 2, 0), :, 5] = INF
        many = aj.prompt_attn(q, k, v, ints(starts), scale=scale)
        one = aj.prompt_attn(qf, k, v, ints(starts), scale=scale)
        ok()
        outs[bad] = (many[0][:, 30:34], many[1][30:34]), one
    for o, lse in outs[False]:
        check_attn(o, lse, qf, ref, scale, u)
    for (o, lse), (good, same_lse) in zip(outs[True], outs[False]):
        met = torch.zeros(T, d, dtype=torch.bool, device="cuda")
        for a, e in zip(starts, starts[1:]):
            met[a:e] = (~torch.isfinite(v[a:e, 0])).cumsum(0) > 0
        assert torch.equal(lse, same_lse)
        keep = ~met[:, None].expand_as(o)
        assert torch.equal(o[keep], good[keep])
        assert not torch.isfinite(o[~keep]).any()


def test_prompt_bad_starts():
    g = rng(6)
    q, k, v = (randn(g, 50, h, 64) for h in (2, 1, 1))
    good = aj.prompt_attn(q, k, v, ints([0, 20, 50]))
    assert aj.sync_status() == 0
    for starts in ([0, 20, 51], [-1, 20, 50], [0, 20, 2 ** 31 - 1]):
        o, lse = aj.prompt_attn(q, k, v, ints(starts))
        assert aj.sync_status() == 7
        assert torch.equal(o, good[0]) and torch.equal(lse, good[1])
    aj.prompt_attn(q, k, v, ints([0, 40, 10, 50]))  # backwards: reported, whatever comes out
    assert aj.sync_status() == 7
    out = (torch.full_like(q, 3.0), torch.full((2, 50), 4.0, device="cuda"))
    aj.prompt_attn(q, k, v, ints([7]), out=out)     # no sequence
    aj.prompt_attn(q, k, v, ints([9, 9, 9]), out=out)
    ok()
    assert (out[0] == 3).all() and (out[1] == 4).all()


def test_empty_calls():
    g = rng(7)
    q = randn(g, 0, 2, 64)
    cos, sin = aj.rope_tables(64, 4)
    qo, ko = aj.rope_at(q, q[:, :1], torch.zeros(0, dtype=torch.int64, device="cuda"), cos, sin)
    assert qo.shape == (0, 2, 64) and ko.shape == (0, 1, 64)
    assert aj.prompt_attn(q, q[:, :1], q[:, :1], ints([0, 0]))[0].shape == (0, 2, 64)
    cache = filled(g, 3, 1, 16, 64)
    before = cache.k.clone()
    aj.cache_append(cache, q[:, :1], q[:, :1], ints([0, 0]), ints([5]), ints([[0]]))
    assert aj.cache_attn(randn(g, 0, 1, 2, 64), cache, ints([]), torch.zeros(0, 1, dtype=torch.int32, device="cuda"))[0].numel() == 0
    assert aj.cache_attn(randn(g, 2, 0, 2, 64), cache, ints([1, 1]), ints([[0], [1]]))[1].shape == (2, 2, 0)
    ok()
    assert same(before, cache.k)


# ------------------------------------------------------------------ refusals
def test_forms_of_out_and_scale():
    """`out` is any pair and comes back as it was given; a scale is a number that 32 bits hold."""
    g = rng(12)
    q, k = randn(g, 3, 2, 64), randn(g, 3, 1, 64)
    cos, sin = aj.rope_tables(64, 8)
    at = ints([0, 5, 7])
    want = aj.rope_at(q, k, at, cos, sin)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    got = aj.rope_at(q, k, at, cos, sin, out=[qo, ko])
    assert got[0] is qo and got[1] is ko and torch.equal(qo, want[0]) and torch.equal(ko, want[1])
    only = aj.rope_at(q, None, at.long(), cos, sin)
    assert only[1] is None and torch.equal(only[0], want[0])
    got = aj.rope_at(q, None, at, cos, sin, out=(qo, None))
    assert got[0] is qo and got[1] is None
    for out in ((qo,), (qo, ko, qo), (qo, None), (ko, qo), (qo[:2], ko), (qo.float(), ko), 3):
        with pytest.raises((ValueError, TypeError)):
            aj.rope_at(q, k, at, cos, sin, out=out)
    starts = ints([0, 3])
    o, lse = aj.prompt_attn(q, k, k, starts, scale=1)
    mine = torch.empty_like(o), torch.empty_like(lse)
    got = aj.prompt_attn(q, k, k, starts, scale=np.float64(1.0), out=mine)
    assert got[0] is mine[0] and got[1] is mine[1] and torch.equal(mine[0], o) and torch.equal(mine[1], lse)
    for scale in (0.0, -1.0, float("nan"), float("inf"), 1e-60, 1e60, "1"):
        with pytest.raises((ValueError, TypeError)):
            aj.prompt_attn(q, k, k, starts, scale=scale)
    with pytest.raises(TypeError):
        aj.prompt_attn(q.float(), k.float(), k.float(), starts)
    ok()


def test_wrong_arguments_are_refused():
    """Calls that need tensors on the GPU to be refused; nothing is launched."""
    g = rng(8)
    cache = filled(g, 4, 2, 16, 64)
    q, lens, table = randn(g, 2, 1, 4, 64), ints([5, 6]), ints([[0], [1]])
    flat = aj.PagedCache(cache.k[0], cache.v[0], cache.k_scale, cache.v_scale)
    for bad in (dict(q=q[0]), dict(q=q.float()), dict(q=randn(g, 2, 1, 3, 64)), dict(q=randn(g, 2, 1, 4, 128)),
                dict(q=q.transpose(2, 3)), dict(cache=flat), dict(cache=cache._replace(k_scale=cache.k_scale[:3])),
                dict(cache=cache._replace(v=cache.v.view(torch.uint8))), dict(seq_lens=lens.long()),
                dict(seq_lens=lens[:1]), dict(seq_lens=lens.cpu()), dict(page_table=table[:, 0]),
                dict(page_table=table[:1]), dict(page_table=table.long()), dict(scale=-1.0), dict(max_len=-1),
                dict(out=(q, torch.empty(2, 4, 2, device="cuda")))):
        args = dict(q=q, cache=cache, seq_lens=lens, page_table=table) | bad
        with pytest.raises((ValueError, TypeError, RuntimeError)):
            aj.cache_attn(**args)
    k, starts, cached = randn(g, 3, 2, 64), ints([0, 1, 3]), ints([2, 2])
    for bad in (dict(cache=flat), dict(k=k[:, :1]), dict(v=k[:2]), dict(starts=starts[:2]), dict(cached=cached[:1]),
                dict(page_table=table[0]), dict(cos=torch.ones(9, 32, device="cuda")), dict(layout="other", cos=1, sin=1)):
        args = dict(cache=cache, k=k, v=k, starts=starts, cached=cached, page_table=table) | bad
        with pytest.raises((ValueError, AttributeError)):
            aj.cache_append(**args)
    with pytest.raises(ValueError):
        aj.prompt_attn(k[:, :1], k, k, starts)
    with pytest.raises(RuntimeError):  # one key head for two, by a stride of 0
        aj.prompt_attn(k, k[:, :1].expand(3, 2, 64), k, starts)
    ok()
    one = ints([0, 1])[:, None]  # a column whose own stride means nothing
    assert torch.equal(aj.cache_attn(q, cache, lens, table)[0], aj.cache_attn(q, cache, lens, one)[0])
    ok()


@pytest.mark.parametrize("n,pages", [(1, 400), (20, 4)])
def test_workspace_is_checked(n, pages):
    """The C entry with the workspace that it asks for, with less, and with none."""
    from attention_jvp_attn_b200 import _abi
    lib = _abi.load()
    g = rng(8)
    cache = filled(g, pages, 1, 16, 64)
    q = randn(g, 1, n, 1, 64)
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    lens = ints([16 * pages])
    want, _ = aj.cache_attn(q, cache, lens, table)
    o, lse = torch.full_like(want, 3.0), torch.empty(1, 1, n, device="cuda")
    shape = _abi.pack_shape(1, n, 1, 64, _abi.DTYPE_BF16, 0.0)
    size = lib.attn_jvp_cache_attn_workspace_bytes(shape, 1, 16 * pages)
    assert size > 0
    work = torch.empty(size + 16, dtype=torch.uint8, device="cuda")

    def call(at, bytes_):
        import ctypes
        desc = _abi.pack_cache(cache.k.data_ptr(), cache.v.data_ptr(), cache.k_scale.data_ptr(), cache.v_scale.data_ptr(),
                               pages, 16, *cache.k.stride()[:3], *cache.k_scale.stride())
        rc = lib.attn_jvp_cache_attn(shape, 1, q.data_ptr(), (ctypes.c_int64 * 3)(*q.stride()[:3]), desc,
                                     lens.data_ptr(), table.data_ptr(), pages, pages, 0, 1, at, bytes_,
                                     o.data_ptr(), lse.data_ptr(), torch.cuda.current_stream().cuda_stream)
        ok()
        return rc

    assert call(None, 0) == call(work.data_ptr(), size - 1) == call(None, size) == _abi.ERR_INVALID_ARGUMENT
    assert call(work.data_ptr() + 8, size) == _abi.ERR_MISALIGNED
    assert (o == 3).all()
    assert call(work.data_ptr(), size) == _abi.OK
    assert torch.equal(o, want)


# ------------------------------------------------------------------ many sequences
def test_many_sequences():
    """More sequences than a block has threads: empty, single and two-tile ones."""
    g = rng(9)
    lens = [(i * 7) % 5 if i % 400 else 300 for i in range(2000)]
    starts = np.concatenate([[0], np.cumsum(lens)])
    T = int(starts[-1])
    q, k, v = (randn(g, T, h, 64) for h in (2, 1, 1))
    o, lse = aj.prompt_attn(q, k, v, ints(starts))
    ok()
    check_attn(o, lse, q, orc.prompt_attn(f64(q), f64(k), f64(v), starts, 0.125), 0.125, 2.0 ** -8)
    pages = sum(max(1, -(-m // 16)) for m in lens)
    cache = pool(g, pages, 1, 16, 64)
    table = tables(g, pages, lens, 16)
    want = orc.append(f64(cache.k), f64(cache.k_scale), f64(k), starts, [0] * 2000, table.cpu().numpy())
    aj.cache_append(cache, k, v, ints(starts), ints([0] * 2000), table)
    ok()
    nan = np.isnan(want[0])
    assert (f64(cache.k)[~nan] == want[0][~nan]).all() and (f64(cache.k_scale) == want[1]).all()
    for n, width in ((1, table.shape[1]), (20, table.shape[1]), (1, 300)):
        wide = torch.zeros(2000, width, dtype=torch.int32, device="cuda")
        wide[:, :table.shape[1]] = table
        qn = randn(g, 2000, n, 2, 64)
        at = [0, 1, 2, 3, 400, 399, 1200, 1999]
        o, lse = aj.cache_attn(qn, cache, ints(lens), wide)
        ok()
        ref = orc.cache_attn(f64(qn[at]), f64(cache.k), f64(cache.v), f64(cache.k_scale), f64(cache.v_scale),
                             [lens[i] for i in at], table.cpu().numpy()[at], True, 0.125)
        check_attn(o[at], lse[at], qn, ref, 0.125, 2.0 ** -11, 300 * 448 * 2.0 ** -5 * 2.0 ** -25)


# ------------------------------------------------------------------ streams and graphs
def step(cache, q, k, v, pos, starts, cached, lens, table, cos, sin, B):
    qr, _ = aj.rope_at(q, None, pos, cos, sin)
    aj.cache_append(cache, k, v, starts, cached, table, cos, sin)
    return aj.cache_attn(qr.view(B, -1, *q.shape[1:]), cache, lens, table)


@pytest.mark.parametrize("n,width", [(1, 10), (1, 400), (40, 10)])
def test_decode_step_in_a_graph(n, width):
    """A step captured once and replayed while the lengths grow on the device."""
    g = rng(n + width)
    B, H, Hkv, d = 3, 4, 2, 64
    cos, sin = aj.rope_tables(d, 400)
    eager, graphed = (filled(rng(5), 60, Hkv, 16, d) for _ in range(2))
    table = torch.zeros(B, width, dtype=torch.int32, device="cuda")
    table[:, :10] = torch.arange(30, device="cuda").view(3, 10).int()
    starts = ints([0, n, 2 * n, 3 * n])
    q, k, v = (torch.empty(B * n, h, d, dtype=torch.bfloat16, device="cuda") for h in (H, Hkv, Hkv))
    cached, lens = ints([0, 5, 33]), ints([0, 5, 33])
    pos = torch.zeros(B * n, dtype=torch.int32, device="cuda")

    def advance():
        qkv = randn(g, B * n, H + 2 * Hkv, d)
        for t, x in zip((q, k, v), qkv.split([H, Hkv, Hkv], 1)):
            t.copy_(x)
        cached.copy_(lens)
        lens.add_(n)
        pos.copy_((cached[:, None] + torch.arange(n, device="cuda")).view(-1))

    advance()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(graphed, q, k, v, pos, starts, cached, lens, table, cos, sin, B)
    for _ in range(2):
        graph.replay()
        want = step(eager, q, k, v, pos, starts, cached, lens, table, cos, sin, B)
        ok()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
        assert same(eager.k, graphed.k) and same(eager.v, graphed.v) and torch.equal(eager.k_scale, graphed.k_scale)
        advance()


def test_two_graphs_at_once():
    """Two captured calls (each with a workspace of its own) replayed on two streams."""
    g = rng(21)
    cache = filled(g, 400, 2, 16, 64)
    table = torch.randperm(400, generator=g, device="cuda").int().view(1, 400)
    qs = [randn(g, 1, n, 8, 64) for n in (1, 30)]
    want = [aj.cache_attn(q, cache, ints([6000]), table) for q in qs for _ in range(2)]
    graphs, outs = [], []
    lens = ints([6000])
    for q in qs:
        for _ in range(2):
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1]):
                outs.append(aj.cache_attn(q, cache, lens, table))
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, gr in zip(streams, graphs):
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    ok()
    for w, o in zip(want, outs):
        assert torch.equal(w[0], o[0]) and torch.equal(w[1], o[1])


def test_calls_on_two_streams():
    g = rng(22)
    cache = filled(g, 300, 2, 16, 64)
    table = torch.randperm(300, generator=g, device="cuda").int().view(1, 300)
    lens = ints([4500])
    q, k, v = (randn(g, 900, h, 64) for h in (4, 2, 2))
    starts = ints([0, 500, 900])
    qa, qb = randn(g, 1, 1, 4, 64), randn(g, 1, 64, 4, 64)
    run = [lambda: aj.prompt_attn(q, k, v, starts), lambda: aj.cache_attn(qa, cache, lens, table),
           lambda: aj.cache_attn(qb, cache, lens, table)]
    want = [f() for f in run]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in run]
    got = []
    for _ in range(10):
        for s, f in zip(streams, run):
            with torch.cuda.stream(s):
                got.append(f())
    torch.cuda.synchronize()
    ok()
    for i, r in enumerate(got):
        assert torch.equal(r[0], want[i % 3][0]) and torch.equal(r[1], want[i % 3][1])


def test_first_call_inside_a_capture():
    """The library's one-off set-up may fall into a capture (a process of its own)."""
    code = """
import torch, attention_jvp_attn_b200 as aj
q = torch.randn(300, 2, 64, device="cuda").bfloat16()
s = torch.tensor([0, 300], dtype=torch.int32, device="cuda")
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    o, lse = aj.prompt_attn(q, q, q, s)
g.replay()
torch.cuda.synchronize()
w = aj.prompt_attn(q, q, q, s)
assert torch.equal(o, w[0]) and torch.equal(lse, w[1]) and aj.sync_status() == 0
print("fine")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=root)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]


# ------------------------------------------------------------------ large
def test_cache_beyond_4_gb():
    """Pages whose offset passes 32 bits, written and read."""
    pages, heads, page, d = 36000, 8, 128, 128  # 4.7e9 bytes each
    if torch.cuda.mem_get_info()[0] < 30e9:
        pytest.skip("needs 30 GB")
    k = torch.zeros(pages, heads, page, d, dtype=torch.uint8, device="cuda").view(F8)
    v = torch.zeros(pages, heads, page, d, dtype=torch.uint8, device="cuda").view(F8)
    big = aj.PagedCache(k, v, torch.ones(pages, heads, device="cuda"), torch.ones(pages, heads, device="cuda"))
    small = aj.paged_cache(4, page, heads, d)
    g = rng(1)
    x, y = randn(g, 300, heads, d), randn(g, 300, heads, d)
    far, near = ints([[35999, 17, 35000]]), ints([[0, 1, 2]])
    for c, t in ((big, far), (small, near)):
        aj.cache_append(c, x, y, ints([0, 300]), ints([0]), t)
    ok()
    for a, b in ((35999, 0), (17, 1), (35000, 2)):
        assert same(big.k[a], small.k[b]) and same(big.v[a], small.v[b])
    for n in (1, 3, 50):
        q = randn(g, 1, n, 16, d)
        a, b = aj.cache_attn(q, big, ints([300]), far), aj.cache_attn(q, small, ints([300]), near)
        ok()
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_rows_beyond_32_bits():
    """Token rows whose element offset passes 2^31: one sequence at the end of a long packed tensor."""
    T, H, d = 140000, 128, 128  # 2.3e9 elements
    if torch.cuda.mem_get_info()[0] < 30e9:
        pytest.skip("needs 30 GB")
    g = rng(3)
    x = torch.zeros(T, H, d, dtype=torch.bfloat16, device="cuda")
    x[-260:] = randn(g, 260, H, d)
    part = x[-260:].clone()
    k, v = x[:, :2], x[:, 2:4]
    o, lse = aj.prompt_attn(x, k, v, ints([T - 260, T]))
    want = aj.prompt_attn(part, part[:, :2], part[:, 2:4], ints([0, 260]))
    ok()
    assert torch.equal(o[-260:], want[0]) and torch.equal(lse[:, -260:], want[1])
    cos, sin = aj.rope_tables(d, T)
    pos = torch.arange(T, device="cuda")
    r, _ = aj.rope_at(x, None, pos, cos, sin)
    w, _ = aj.rope_at(part, None, pos[-260:].contiguous(), cos, sin)
    ok()
    assert torch.equal(r[-260:], w)
