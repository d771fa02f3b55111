"""The serving operators on the GPU against the float64 oracle.

Bounds. A product sum of d terms in fp32 is off by at most d 2^-24 of the sum of
its terms' sizes, so a score x by A d 2^-24 with A = max s sum |q||k| (plus, where
bf16 queries are scaled into fp16, 2^-25 of the row's largest |q| per column: at
most another A-like sum, bounded below by Q); the hardware's exponential adds
2^-22. So each probability, and the sum that divides it, is relatively off by at
most delta = A d 2^-24 + Q + 2^-20 (1 + max |x| 2^-3 for the fp32 rounding of the
exponent's argument, within 2^-20 for |x| <= 64, which the inputs here keep).
Then with u_p the half step of the type that holds the probabilities and u that of
the output,
    |O - ref| <= u |ref| + (u_p + 2 delta + 2^-20) sum p |v|   (+ what fp16 flushes),
    |LSE - ref| <= delta + 2^-20 (1 + |ref|).
"""
import numpy as np
import pytest
import torch

import attention_jvp_attn_b200 as aj
from oracle import serving_oracle as orc

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def rng(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype=torch.bfloat16, size=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * size).to(dtype)


def f64(t):
    return t.detach().to(torch.float32 if t.dtype == F8 else t.dtype).double().cpu().numpy()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def ok():
    assert aj.sync_status() == 0


# ------------------------------------------------------------------ rotation
def check_rope(got, x, ref, cos, sin, positions, layout, dtype):
    """The rounding of the type, and of two products in fp32, on each pair."""
    mag = np.maximum(orc.rope(np.abs(f64(x)), positions, np.abs(cos), -np.abs(sin), layout),
                     orc.rope(np.abs(f64(x)), positions, np.abs(cos), np.abs(sin), layout))
    err = np.abs(f64(got) - ref)
    assert (err <= HALF[dtype] * np.abs(ref) + 2.0 ** -22 * np.abs(mag) + 1e-30
            + (2.0 ** -25 if dtype == torch.float16 else 0)).all(), err.max()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("T,H,Hkv,d,rot", [(1, 1, 1, 64, 64), (5, 4, 2, 64, 32), (37, 32, 8, 128, 128),
                                           (130, 3, 1, 128, 96), (2, 40, 40, 128, 16), (3001, 2, 2, 64, 48)])
def test_rope_at(dtype, layout, T, H, Hkv, d, rot):
    g = rng(T + rot)
    qkv = randn(g, T, H + 2 * Hkv, d, dtype=dtype)
    q, k = qkv[:, :H], qkv[:, H:H + Hkv]
    cos, sin = aj.rope_tables(rot, 5000)
    pos = torch.randint(0, 5000, (T,), generator=g, device="cuda", dtype=torch.int64)
    for transpose in (False, True):
        for p in (pos, pos.int()):
            qo, ko = aj.rope_at(q, k, p, cos, sin, layout=layout, transpose=transpose)
            ok()
            for got, x in ((qo, q), (ko, k)):
                ref = orc.rope(f64(x), pos.cpu().numpy(), f64(cos), f64(sin), layout, transpose)
                check_rope(got, x, ref, f64(cos), f64(sin), pos.cpu().numpy(), layout, dtype)
    # in place, on the views, and without k
    want_q, want_k = aj.rope_at(q, k, pos, cos, sin, layout=layout)
    alone, none = aj.rope_at(q, None, pos, cos, sin, layout=layout)
    assert none is None and torch.equal(alone, want_q)
    v = qkv[:, H + Hkv:].clone()
    aj.rope_at(q, k, pos, cos, sin, layout=layout, out=(q, k))
    ok()
    assert torch.equal(q, want_q) and torch.equal(k, want_k) and torch.equal(qkv[:, H + Hkv:], v)


def test_rope_at_gradient_by_differences():
    """<R^T g, e> against <g, R(x + e) - R(x)> in fp32: R is linear, so they agree to rounding."""
    g = rng(3)
    x = randn(g, 9, 3, 64, dtype=torch.float32)
    w = randn(g, 9, 3, 64, dtype=torch.float32)
    e = randn(g, 9, 3, 64, dtype=torch.float32)
    cos, sin = aj.rope_tables(32, 100, scaling="by_parts", factor=4.0, original_positions=50)
    pos = torch.arange(9, device="cuda") * 11
    turn = lambda t, tr=False: aj.rope_at(t, None, pos, cos, sin, layout="half", transpose=tr)[0].double()
    left = (turn(w, True) * e.double()).sum()
    right = (w.double() * (turn(x + e) - turn(x))).sum()
    size = (w.double().abs() * (x.abs() + e.abs()).double()).sum()
    assert abs(left - right) <= 8 * 2.0 ** -24 * size


def test_rope_at_position_out_of_range():
    g = rng(4)
    q = randn(g, 6, 2, 64)
    cos, sin = aj.rope_tables(64, 10)
    pos = torch.tensor([0, 9, 10, -1, 3, 2 ** 40], device="cuda")
    out = torch.full_like(q, 7.0)
    aj.rope_at(q, None, pos, cos, sin, out=(out, None))
    assert aj.sync_status() == 7 and aj.sync_status() == 0
    good = aj.rope_at(q[[0, 1, 4]].contiguous(), None, pos[[0, 1, 4]].contiguous(), cos, sin)[0]
    assert torch.equal(out[[0, 1, 4]], good) and (out[[2, 3, 5]] == 7).all()


# ------------------------------------------------------------------ cache
def pool(g, pages, heads, page, d, layout="pages"):
    """A cache full of other sequences' leftovers, NaN codes among them."""
    def codes():
        raw = torch.randint(0, 256, (pages, heads, page, d), generator=g, device="cuda", dtype=torch.uint8)
        if layout == "tokens first":  # [pages, page, heads, d], seen as [pages, heads, page, d]
            raw = raw.transpose(1, 2).contiguous().transpose(1, 2)
        return raw.view(F8)
    scale = lambda: torch.exp2(torch.randint(-6, 4, (pages, heads), generator=g, device="cuda").float())
    return aj.PagedCache(codes(), codes(), scale(), scale())


def tables(g, pages, lens, page, width=None):
    need = [max(1, -(-n // page)) for n in lens]
    order = torch.randperm(pages, generator=g, device="cuda").int()
    table = torch.full((len(lens), width or max(need)), 2 ** 30, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    assert at <= pages
    return table


def same_codes(got, ref, exact_share=1.0):
    """Equal values, but for a share of them one step apart (a rotated key at the
    border of two codes, where fp32 and 64 bits may differ)."""
    got = f64(got)
    nan = np.isnan(ref)
    assert (np.isnan(got) == nan).all()
    off = (got != ref) & ~nan
    assert off.mean() <= 1.0 - exact_share
    if off.any():
        a, b = np.abs(got[off]), np.abs(ref[off])
        assert (np.abs(got[off] - ref[off]) <= np.maximum(2.0 ** -9, 0.125 * np.maximum(a, b))).all()


APPENDS = [  # (new per sequence, cached before, heads, d, page, rot, layout, dtype, pool layout)
    ([1], [0], 1, 64, 16, 0, "half", torch.bfloat16, "pages"),
    ([1, 1, 1, 1], [5, 15, 16, 31], 2, 64, 16, 64, "interleaved", torch.bfloat16, "pages"),
    ([0, 3, 0, 40, 1], [7, 14, 0, 0, 63], 3, 128, 16, 128, "half", torch.float16, "tokens first"),
    ([17, 200, 64], [1, 63, 64], 2, 128, 64, 64, "half", torch.float32, "pages"),
    ([129, 5], [127, 0], 2, 128, 128, 32, "interleaved", torch.bfloat16, "tokens first"),
    ([50, 1], [31, 32], 4, 64, 32, 48, "half", torch.float32, "pages"),
    ([100], [900], 1, 64, 128, 64, "interleaved", torch.float16, "pages"),
]


@pytest.mark.parametrize("new,cached,heads,d,page,rot,layout,dtype,where", APPENDS)
def test_cache_append(new, cached, heads, d, page, rot, layout, dtype, where):
    g = rng(sum(new) + page)
    lens = [a + b for a, b in zip(new, cached)]
    pages = sum(max(1, -(-n // page)) for n in lens) + 2
    cache = pool(g, pages, heads, page, d, where)
    table = tables(g, pages, lens, page)
    starts = np.concatenate([[2], 2 + np.cumsum(new)])  # two rows before, three behind
    T = int(starts[-1]) + 3
    kv = randn(g, T, 2 * heads, d, dtype=dtype, size=3.0)
    k, v = kv[:, :heads], kv[:, heads:]
    cos, sin = aj.rope_tables(rot, max(lens)) if rot else (None, None)
    place = np.zeros(T, int)
    for b, n in enumerate(cached):
        place[starts[b]:starts[b + 1]] = n + np.arange(new[b])
    turned = orc.rope(f64(k), place, f64(cos), f64(sin), layout) if rot else f64(k)
    tab = table.cpu().numpy()
    want_k = orc.append(f64(cache.k), f64(cache.k_scale), turned, starts, cached, tab)
    want_v = orc.append(f64(cache.v), f64(cache.v_scale), f64(v), starts, cached, tab)
    for _ in range(2):  # the second time changes nothing
        aj.cache_append(cache, k, v, ints(starts), ints(cached), table, cos, sin, layout=layout)
        ok()
        assert (f64(cache.k_scale) == want_k[1]).all() and (f64(cache.v_scale) == want_v[1]).all()
        same_codes(cache.k, want_k[0], 1.0 - 1e-4 if rot else 1.0)
        same_codes(cache.v, want_v[0])


def test_cache_append_growing_scale_one_by_one():
    """Tokens of growing size, one call each: earlier tokens of the page are rounded to the larger scale."""
    g = rng(8)
    cache = aj.paged_cache(3, 16, 2, 64)
    table = ints([[2, 0]])
    k = randn(g, 20, 2, 64, dtype=torch.float32) * torch.exp2(torch.arange(20, device="cuda") / 2 - 5)[:, None, None]
    v = randn(g, 20, 2, 64, dtype=torch.float32) * torch.exp2(5 - torch.arange(20, device="cuda") / 2)[:, None, None]
    want_k, want_v = [(f64(c), f64(s)) for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale))]
    for t in range(20):
        aj.cache_append(cache, k[t:t + 1], v[t:t + 1], ints([0, 1]), ints([t]), table)
        want_k = orc.append(*want_k, f64(k[t:t + 1]), [0, 1], [t], table.cpu().numpy())
        want_v = orc.append(*want_v, f64(v[t:t + 1]), [0, 1], [t], table.cpu().numpy())
    ok()
    for got, want in ((cache.k, want_k), (cache.v, want_v)):
        same_codes(got, want[0])
    assert (f64(cache.k_scale) == want_k[1]).all() and (f64(cache.v_scale) == want_v[1]).all()


def test_cache_append_special_values():
    cache = aj.paged_cache(4, 16, 1, 64)
    x = torch.zeros(6, 1, 64, device="cuda")
    x[0, 0, :4] = torch.tensor([float("inf"), float("-inf"), float("nan"), 3.0], device="cuda")
    x[2, 0, 0] = 448.0      # the largest code at scale 1
    x[3, 0, 0] = 448.0001   # needs the next scale
    x[4, 0, 0] = 1e38       # beyond the largest scale
    x[5, 0, 0] = 1e-30      # below the smallest
    for row, at in ((0, 0), (1, 1), (2, 2), (4, 3)):
        aj.cache_append(cache, x[row:row + 1], x[row:row + 1], ints([0, 1]), ints([0]), ints([[at]]))
    ok()
    k, s = f64(cache.k)[:, 0, 0], f64(cache.k_scale)[:, 0]
    assert s[0] == 2.0 ** -7 and k[0, 0] == 448 and k[0, 1] == -448 and np.isnan(k[0, 2]) and k[0, 3] == 384
    assert s[1] == 2.0 ** -32 and (k[1] == 0).all()
    assert s[2] == 1.0 and k[2, 0] == 448
    assert s[3] == 2.0 ** 32 and k[3, 0] == 448
    aj.cache_append(cache, x[3:4], x[5:6], ints([0, 1]), ints([0]), ints([[1]]))
    ok()
    assert f64(cache.k_scale)[1, 0] == 2.0 and f64(cache.k)[1, 0, 0, 0] == 224
    assert f64(cache.v_scale)[1, 0] == 2.0 ** -32 and (f64(cache.v)[1] == 0).all()


def test_cache_append_bad_indices():
    """Pages, lengths, positions and starts out of range: reported, nothing else touched."""
    g = rng(5)
    base = pool(g, 6, 2, 16, 64)
    k, v = randn(g, 8, 2, 64), randn(g, 8, 2, 64)
    cos, sin = aj.rope_tables(64, 40)

    def run(starts, cached, table, tables=(None, None)):
        cache = aj.PagedCache(*(t.clone() for t in base))
        aj.cache_append(cache, k, v, ints(starts), ints(cached), ints(table), *tables)
        return cache, aj.sync_status()

    def untouched(cache, pages):
        return all(torch.equal(a.view(torch.uint8)[pages], b.view(torch.uint8)[pages]) for a, b in zip(cache, base))

    good, st = run([0, 4, 8], [0, 0], [[1], [3]])
    assert st == 0 and untouched(good, [0, 2, 4, 5])
    for starts, cached, table, tabs in [
            ([0, 4, 8], [0, 0], [[1], [6]], (None, None)),
            ([0, 4, 8], [0, 0], [[1], [-1]], (None, None)),
            ([0, 4, 8], [0, 16], [[1], [3]], (None, None)),      # page 1 of a table of 1
            ([0, 4, 8], [0, -3], [[1], [3]], (None, None)),
            ([0, 4, 8], [0, 2 ** 31 - 5], [[1], [3]], (None, None)),
            ([0, 4, 8], [0, 37], [[1, 1, 1], [3, 3, 3]], (cos, sin))]:  # positions 37..40 of 40
        cache, st = run(starts, cached, table, tabs)
        assert st == 7, (starts, cached, table)
        assert untouched(cache, [0, 2, 3, 4, 5])
        if tabs[0] is None:
            assert torch.equal(cache.k.view(torch.uint8)[1], good.k.view(torch.uint8)[1])
    cache, st = run([0, 4, 100], [0, 0], [[1], [3]])  # rows behind the last are cut off
    assert st == 7 and torch.equal(cache.k.view(torch.uint8), good.k.view(torch.uint8))
    cache, st = run([-7, 4, 8], [0, 0], [[1], [3]])
    assert st == 7 and untouched(cache, [0, 2, 4, 5])
    cache, st = run([4, 0, 0], [0, 0], [[1], [3]])    # backwards
    assert st == 7 and untouched(cache, [0, 1, 2, 3, 4, 5])


# ------------------------------------------------------------------ attention over the cache
def filled(g, pages, heads, page, d, layout="pages", size=1.0):
    """A cache whose values are of a model's sizes; the pages' own scales differ."""
    cache = pool(g, pages, heads, page, d, layout)
    for codes, scale in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        scale.copy_(torch.exp2(torch.randint(-9, -6, scale.shape, generator=g, device="cuda").float()))
        x = torch.randn(codes.shape, generator=g, device="cuda") * size / scale[..., None, None]
        codes.view(torch.uint8).copy_(x.clamp(-448, 448).to(F8).view(torch.uint8))
    return cache


def stale(cache, table, lens, page):
    """NaN codes and absurd scales wherever no token of a sequence lies."""
    used = torch.zeros(cache.k.shape[0], page, dtype=torch.bool, device="cuda")
    for b, n in enumerate(lens):
        for j in range(-(-n // page)):
            used[table[b, j].item(), :min(page, n - j * page)] = True
    for codes, scale in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        codes.view(torch.uint8).masked_fill_(~used[:, None, :, None], 0x7F)
        scale.masked_fill_(~used.any(1)[:, None], float("nan"))


def check_attn(o, lse, q, ref, scale, u_p, flushed=0.0):
    ro, rl, pv, qk, pm = ref
    d = q.shape[-1]
    delta = qk * d * 2.0 ** -24 + 2.0 ** -20
    if q.dtype == torch.bfloat16 and u_p == 2.0 ** -11:
        # scaled into fp16: at most 2^-25 of the row's largest |q| per column, and
        # no |q| is above it, so at most d 2^-25 of s max|q| max|k| <= 8 qk here
        delta = delta + 8 * qk * 2.0 ** -25 * d
    dd = np.moveaxis(delta, -1, 1)[..., None] if o.dim() == 4 else delta.T[..., None]
    err = np.abs(f64(o) - ro)
    bound = HALF[q.dtype] * np.abs(ro) + (u_p + 2 * dd + 2.0 ** -20) * pv + flushed + 2.0 ** -25
    assert not np.isnan(f64(o)).any() and (err <= bound).all(), (err / bound).max()
    got = f64(lse)
    seen = np.isfinite(rl)
    assert (np.isneginf(got) == ~seen).all()
    assert (np.abs(got[seen] - rl[seen]) <= (delta[seen] + 2.0 ** -20 * (1 + np.abs(rl[seen])))).all()


CACHES = [  # (lens, n, H, Hkv, d, page, causal, dtype, pool layout)
    ([1], 1, 1, 1, 64, 16, True, torch.bfloat16, "pages"),
    ([0, 1, 15, 16, 17, 100], 1, 4, 2, 64, 16, True, torch.bfloat16, "pages"),
    ([33, 128, 129, 0, 2], 1, 8, 1, 128, 32, False, torch.float16, "tokens first"),
    ([5, 3, 1, 0, 64], 4, 4, 1, 128, 64, True, torch.bfloat16, "pages"),
    ([5, 3, 1, 0, 64], 4, 4, 1, 128, 64, False, torch.bfloat16, "pages"),
    ([700, 31], 3, 12, 4, 64, 128, True, torch.float16, "pages"),
    ([2000], 1, 32, 8, 128, 16, True, torch.bfloat16, "tokens first"),
    ([1999, 1500, 3], 2, 16, 2, 128, 64, True, torch.bfloat16, "pages"),
    ([300, 290], 17, 4, 4, 64, 64, True, torch.float16, "pages"),
    ([257, 400], 130, 2, 1, 128, 32, True, torch.bfloat16, "pages"),
    ([515], 300, 3, 3, 64, 64, False, torch.bfloat16, "tokens first"),
    ([640], 129, 2, 2, 128, 128, False, torch.float16, "pages"),
    ([40, 200], 200, 6, 2, 64, 16, True, torch.bfloat16, "pages"),
]


@pytest.mark.parametrize("lens,n,H,Hkv,d,page,causal,dtype,where", CACHES)
def test_cache_attn(lens, n, H, Hkv, d, page, causal, dtype, where):
    g = rng(sum(lens) + n)
    pages = sum(max(1, -(-m // page)) for m in lens) + 2
    cache = filled(g, pages, Hkv, page, d, where)
    table = tables(g, pages, lens, page, width=-(-max(lens) // page) + 3)
    stale(cache, table, lens, page)
    qkv = randn(g, len(lens), n, H + 3, d, dtype=dtype)
    q = qkv[:, :, 1:H + 1]
    scale = 0.2 / np.sqrt(d) * 4
    ref = orc.cache_attn(f64(q), f64(cache.k), f64(cache.v), f64(cache.k_scale), f64(cache.v_scale),
                         lens, table.cpu().numpy(), causal, scale)
    # fp16 flushes p below 2^-25 of the largest p b: of codes up to 448 over the keys
    flushed = max(lens) * 448 * 2.0 ** -7 * 2.0 ** -25 * np.moveaxis(ref[4], -1, 1)[..., None]
    for max_len in (0, 1, max(lens)):
        o, lse = aj.cache_attn(q, cache, ints(lens), table, causal=causal, scale=scale, max_len=max_len)
        ok()
        check_attn(o, lse, q, ref, scale, 2.0 ** -11, flushed)
    again = aj.cache_attn(q, cache, ints(lens), table, causal=causal, scale=scale, max_len=max(lens))
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


LONG = [  # tables of more than 4096 tokens: the steps of all sequences shared out over the blocks
    ([4500, 33, 0, 700], 1, 8, 2, 128, 64, True, torch.bfloat16, 4600),
    ([0, 0, 1], 1, 4, 1, 64, 16, True, torch.float16, 5000),
    ([9001], 1, 2, 1, 128, 16, True, torch.bfloat16, 9001),
    ([5000, 4999, 31], 4, 8, 2, 64, 128, True, torch.bfloat16, 6000),
    ([6000, 1], 3, 15, 3, 128, 32, False, torch.float16, 6000),
    ([(37 * i) % 100 for i in range(300)], 1, 4, 2, 64, 32, True, torch.bfloat16, 4100),
    ([20000, 5, 4096], 1, 12, 12, 64, 64, True, torch.bfloat16, 20000),
]


@pytest.mark.parametrize("lens,n,H,Hkv,d,page,causal,dtype,width", LONG)
def test_cache_attn_shared_out(lens, n, H, Hkv, d, page, causal, dtype, width):
    g = rng(sum(lens) + n)
    pages = sum(max(1, -(-m // page)) for m in lens) + 2
    cache = filled(g, pages, Hkv, page, d)
    table = tables(g, pages, lens, page, width=-(-width // page))
    stale(cache, table, lens, page)
    q = randn(g, len(lens), n, H, d, dtype=dtype)
    scale = 0.8 / np.sqrt(d)
    ref = orc.cache_attn(f64(q), f64(cache.k), f64(cache.v), f64(cache.k_scale), f64(cache.v_scale),
                         lens, table.cpu().numpy(), causal, scale)
    flushed = max(lens) * 448 * 2.0 ** -7 * 2.0 ** -25 * np.moveaxis(ref[4], -1, 1)[..., None]
    o, lse = aj.cache_attn(q, cache, ints(lens), table, causal=causal, scale=scale)
    ok()
    check_attn(o, lse, q, ref, scale, 2.0 ** -11, flushed)
    again = aj.cache_attn(q, cache, ints(lens), table, causal=causal, scale=scale)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    # the same sequences split within clusters
    short = aj.cache_attn(q, cache, ints(lens), table, causal=causal, scale=scale, max_len=4096)
    ok()
    check_attn(*short, q, ref, scale, 2.0 ** -11, flushed)


# ------------------------------------------------------------------ prompts
PROMPTS = [  # (lengths, rows before, rows behind, H, Hkv, d, dtype)
    ([1], 0, 0, 1, 1, 64, torch.bfloat16),
    ([1, 2, 0, 127, 128, 129], 0, 0, 2, 1, 64, torch.float16),
    ([128], 0, 0, 4, 2, 128, torch.bfloat16),
    ([300, 5, 257], 3, 9, 4, 2, 128, torch.bfloat16),
    ([513, 256, 255, 1], 1, 0, 3, 3, 128, torch.float16),
    ([700], 0, 5, 8, 1, 64, torch.bfloat16),
    ([0, 0, 40], 0, 0, 6, 2, 64, torch.bfloat16),
    ([1100, 385], 0, 0, 2, 2, 128, torch.bfloat16),
]


@pytest.mark.parametrize("lens,before,behind,H,Hkv,d,dtype", PROMPTS)
def test_prompt_attn(lens, before, behind, H, Hkv, d, dtype):
    g = rng(sum(lens) + H)
    starts = before + np.concatenate([[0], np.cumsum(lens)])
    T = int(starts[-1]) + behind
    qkv = randn(g, T, H + 2 * Hkv, d, dtype=dtype)
    q, k, v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    scale = 0.8 / np.sqrt(d)
    ref = orc.prompt_attn(f64(q), f64(k), f64(v), starts, scale)
    out = (torch.full((T, H, d), 5.0, dtype=dtype, device="cuda"), torch.full((H, T), 6.0, device="cuda"))
    # what lies outside the sequences must not matter
    qkv[:before] = float("nan")
    qkv[int(starts[-1]):] = float("inf")
    o, lse = aj.prompt_attn(q, k, v, ints(starts), scale=scale, out=out)
    ok()
    a, e = before, int(starts[-1])
    check_attn(o[a:e], lse[:, a:e], q, [x[a:e] if x.ndim == 3 else x[:, a:e] for x in ref], scale, HALF[dtype])
    for rows in (slice(0, a), slice(e, T)):
        assert (o[rows] == 5).all() and (lse[:, rows] == 6).all()
    again = aj.prompt_attn(q, k, v, ints(starts), scale=scale)
    assert torch.equal(o[a:e], again[0][a:e]) and torch.equal(lse[:, a:e], again[1][:, a:e])


@pytest.mark.parametrize("seqs,n,H,Hkv", [(27, 21, 2, 1), (10, 117, 2, 2), (2, 57, 4, 2)])
def test_cache_attn_repeats(seqs, n, H, Hkv):
    """One row tile of d = 128, the keys ready before their turn: each of many calls
    gives the first one's bits."""
    g = rng(seqs)
    lens = [900 + 131 * b for b in range(seqs)]
    pages = sum(-(-m // 32) for m in lens) + 2
    cache = filled(g, pages, Hkv, 32, 128)
    table = tables(g, pages, lens, 32)
    q = randn(g, seqs, n, H, 128, dtype=torch.float16)
    first = aj.cache_attn(q, cache, ints(lens), table)
    for _ in range(100):
        o, lse = aj.cache_attn(q, cache, ints(lens), table)
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])
    ok()
