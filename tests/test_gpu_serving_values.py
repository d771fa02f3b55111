"""The serving operators with values, scales and sizes far apart, calls repeated,
and what they leave behind: the status word and the tensors' versions.

The bounds are those of test_gpu_serving.py; what fp16 takes from small
probabilities is bounded key by key. A probability times its value scale is held
at 2^7 or more for the row's largest (at the running maximum, which is never above
the final one), so rounding takes at most 2^-25 / 2^7 of the largest, or the whole
of it: sum_j min(p_j b_j, 2^-32 max p b) |code_j|, over the keys that the row sees.
"""
import numpy as np
import pytest
import torch

import attention_jvp_attn_b200 as aj
from attention_jvp_attn_b200 import inputs as wl
from oracle import serving_oracle as orc
from test_gpu_serving import F8, check_attn, f64, filled, ints, ok, pool, randn, rng, same_codes, stale, tables

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


def taken(q, cache, v_scale, lens, table, causal, scale, k_scale=None):
    """What fp16 may take of each output: [B, n, H, d]."""
    B, n, H, d = q.shape
    group = H // cache.k.shape[1]
    one = np.ones_like(v_scale)
    out = np.zeros(q.shape)
    kc, vc = f64(cache.k), f64(cache.v)
    ks = f64(cache.k_scale) if k_scale is None else k_scale
    for b, m in enumerate(lens):
        k = orc.cache_values(kc, ks, table[b], m)
        code = np.abs(orc.cache_values(vc, one, table[b], m))
        size = orc.cache_values(np.ones_like(vc), v_scale, table[b], m)[..., 0]
        for h in range(H):
            for i in range(n):
                seen = min(max(m - n + 1 + i, 0), m) if causal else m
                if seen == 0:
                    continue
                x = scale * (k[h // group][:seen] @ f64(q[b, i, h]))
                p = np.exp(x - x.max())
                pb = p / p.sum() * size[h // group][:seen]
                out[b, i, h] = np.minimum(pb, 2.0 ** -32 * pb.max()) @ code[h // group][:seen]
    return out


# ------------------------------------------------------------------ scales and scores far apart
@pytest.mark.parametrize("up", [10, 20, 26])
@pytest.mark.parametrize("length,n,H,Hkv,d,dtype,width", [
    (500, 1, 4, 2, 64, torch.float16, 32), (500, 4, 4, 1, 128, torch.bfloat16, 32), (4900, 1, 2, 1, 128, torch.float16, 310),
    (500, 24, 2, 2, 64, torch.float16, 32), (700, 140, 1, 1, 128, torch.float16, 48)])
def test_one_page_of_a_large_scale(up, length, n, H, Hkv, d, dtype, width):
    """One token of large values raises its page's scale by 2^up and gets next to no
    probability; its page-mates hold zeros. The output is made of all other tokens."""
    g = rng(up + length + n)
    page = 16
    cache = filled(g, -(-length // page) + 2, Hkv, page, d)
    table = tables(g, cache.k.shape[0], [length], page, width)
    cache.k_scale.fill_(1.0)
    cache.v_scale.fill_(2.0 ** -7)
    cache.k.view(torch.uint8).zero_()
    first = cache.k.view(torch.uint8)[..., 0]  # scores are s q_0 k_0, with s = q_0 = 1
    at = table[0, 11].item()
    first[at] = torch.tensor([0.3125], device="cuda").to(F8).view(torch.uint8)
    first[at, :, 5] = torch.tensor([-40.0], device="cuda").to(F8).view(torch.uint8)
    cache.v_scale[at] = 2.0 ** (up - 7)
    cache.v.view(torch.uint8)[at] = 0
    cache.v.view(torch.uint8)[at, :, 5] = torch.tensor([448.0], device="cuda").to(F8).view(torch.uint8)
    q = randn(g, 1, n, H, d, dtype=dtype)
    q[..., 0] = 1.0
    tab = table.cpu().numpy()
    causal = n < 140
    ref = orc.cache_attn(f64(q), f64(cache.k), f64(cache.v), f64(cache.k_scale), f64(cache.v_scale), [length], tab, causal, 1.0)
    lost = taken(q, cache, f64(cache.v_scale), [length], tab, causal, 1.0)
    o, lse = aj.cache_attn(q, cache, ints([length]), table, causal=causal, scale=1.0)
    ok()
    check_attn(o, lse, q, ref, 1.0, 2.0 ** -11, lost)


@pytest.mark.parametrize("n,H,d,dtype", [(1, 4, 64, torch.bfloat16), (3, 4, 128, torch.float16), (60, 4, 64, torch.float16),
                                         (150, 2, 128, torch.bfloat16)])
def test_scales_of_any_size_key_by_key(n, H, d, dtype):
    """Value scales that differ by 2^20 from page to page, none a power of two."""
    g = rng(41 + n)
    cache = filled(g, 60, 2, 16, d)
    for s in (cache.k_scale, cache.v_scale):
        s.mul_(torch.exp(torch.rand(s.shape, generator=g, device="cuda")))
    cache.v_scale.mul_(torch.exp2(torch.randint(-10, 11, (60, 2), generator=g, device="cuda").float()))
    lens = [500, 290]
    table = tables(g, 60, lens, 16)
    tab = table.cpu().numpy()
    q = randn(g, 2, n, H, d, dtype=dtype)
    scale = 1 / np.sqrt(d)
    ref = orc.cache_attn(f64(q), f64(cache.k), f64(cache.v), f64(cache.k_scale), f64(cache.v_scale), lens, tab, True, scale)
    lost = taken(q, cache, f64(cache.v_scale), lens, tab, True, scale)
    o, lse = aj.cache_attn(q, cache, ints(lens), table, scale=scale)
    ok()
    check_attn(o, lse, q, ref, scale, 2.0 ** -11, lost)


@pytest.mark.parametrize("T,H,Hkv,d", [(300, 2, 1, 64), (700, 4, 2, 128), (1400, 64, 2, 64)])
def test_prompt_behind_a_sink(T, H, Hkv, d):
    """A first key 16 above all others in the exponent, with values of 0: fp16 must
    keep the others' probabilities."""
    g = rng(T)
    q, v = randn(g, T, H, d, dtype=torch.float16), randn(g, T, Hkv, d, dtype=torch.float16)
    k = torch.zeros(T, Hkv, d, dtype=torch.float16, device="cuda")
    q[..., 0] = 1.0
    k[0, :, 0] = 16.0
    v[0] = 0.0
    heads = slice(0, H, max(H // 4, 1))
    ref = orc.prompt_attn(f64(q[:, heads]), f64(k).repeat(H // Hkv, 1)[:, heads], f64(v).repeat(H // Hkv, 1)[:, heads], [0, T], 1.0)
    p = np.exp(-16.0) / (1.0 + np.arange(T) * np.exp(-16.0))  # of each other key, for row t
    top = 1.0 / (1.0 + np.arange(T) * np.exp(-16.0))
    sums = np.cumsum(np.abs(f64(v)), 0).repeat(H // Hkv, 1)[:, heads]
    lost = np.minimum(p, 2.0 ** -32 * top)[:, None, None] * sums
    o, lse = aj.prompt_attn(q, k, v, ints([0, T]), scale=1.0)
    ok()
    check_attn(o[:, heads], lse[heads], q, ref, 1.0, 2.0 ** -11, lost)


@pytest.mark.parametrize("size", [118, 127, -118, -126])
@pytest.mark.parametrize("n,H,d", [(1, 4, 64), (2, 8, 128), (40, 4, 128), (70, 4, 64)])
def test_queries_of_any_size(size, n, H, d):
    """bf16 queries at the ends of the type's range, their size taken back by the scale."""
    g = rng(n + H)
    cache = filled(g, 20, 2, 32, d)
    table = tables(g, 20, [300], 32)
    q = randn(g, 1, n, H, d).clamp(-1.5, 1.5)
    q = (q.double() * 2.0 ** size).to(torch.bfloat16)
    scale = 0.1 * 2.0 ** -size
    ref = orc.cache_attn(f64(q), f64(cache.k), f64(cache.v), f64(cache.k_scale), f64(cache.v_scale), [300],
                         table.cpu().numpy(), True, np.float64(np.float32(scale)))
    o, lse = aj.cache_attn(q, cache, ints([300]), table, scale=scale)
    ok()
    check_attn(o, lse, q, ref, scale, 2.0 ** -11, 300 * 448 * 2.0 ** -7 * 2.0 ** -25)


@pytest.mark.parametrize("n,H", [(1, 4), (6, 4), (40, 4)])
def test_scales_that_are_none(n, H):
    """Page scales of 0, below 0, NaN, infinite, too small and too large are read as
    the limits that they pass (a NaN as the smallest)."""
    g = rng(n)
    cache = filled(g, 30, 2, 16, 64)
    lens = [300, 130]
    table = tables(g, 30, lens, 16)
    for i, s in enumerate((0.0, -1.0, NAN, 2.0 ** -60, -INF)):
        cache.k_scale[table[0, 2 + i].item()] = s
        cache.v_scale[table[1, 1 + i].item()] = s
    cache.v_scale[table[0, 3].item(), 0] = INF
    cache.v_scale[table[0, 4].item(), 1] = 2.0 ** 50
    clamp = lambda t: np.where(np.isnan(f64(t)), 2.0 ** -40, np.clip(f64(t), 2.0 ** -40, 2.0 ** 40))
    ks, vs, tab = clamp(cache.k_scale), clamp(cache.v_scale), table.cpu().numpy()
    q = randn(g, 2, n, H, 64)
    ref = orc.cache_attn(f64(q), f64(cache.k), f64(cache.v), ks, vs, lens, tab, True, 0.125)
    lost = taken(q, cache, vs, lens, tab, True, 0.125, ks)
    o, lse = aj.cache_attn(q, cache, ints(lens), table)
    ok()
    check_attn(o, lse, q, ref, 0.125, 2.0 ** -11, lost)


def test_tiles_of_large_pages_in_many_pieces():
    """Pages of 128 tokens at d = 64 where the key tiles are shared out over all SMs."""
    g = rng(77)
    lens, n, H, Hkv = [9000, 150, 5000], 200, 4, 2
    pages = sum(-(-m // 128) for m in lens) + 2
    cache = filled(g, pages, Hkv, 128, 64)
    table = tables(g, pages, lens, 128)
    stale(cache, table, lens, 128)
    q = randn(g, 3, n, H, 64)
    at = [0, 1, 7, 100, 199]
    for causal in (True, False):
        o, lse = aj.cache_attn(q, cache, ints(lens), table, causal=causal, scale=0.1)
        ok()
        for b, m in enumerate(lens):
            k, v = (orc.cache_values(f64(c), f64(s), table[b].cpu().numpy(), m)
                    for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
            seen = np.array([max(m - n + 1 + i, 0) if causal else m for i in at])
            r = [orc.softmax_rows(f64(q[b, at, h]), k[h // 2], v[h // 2], 0.1, seen) for h in range(H)]
            ref = [np.stack([x[i] for x in r], 1 if r[0][i].ndim == 2 else 0) for i in range(5)]
            lost = m * 448 * 2.0 ** -7 * 2.0 ** -32 * ref[4].T[..., None]  # equal scales but for 2^2
            check_attn(o[b, at], lse[b][:, at], q[b], ref, 0.1, 2.0 ** -11, 4 * lost)


# ------------------------------------------------------------------ calls repeated
REPEATS = [  # (sequences, n, H, Hkv, d, dtype, shortest length)
    (2, 1, 4, 4, 64, torch.bfloat16, 300),     # 1 row, clusters
    (18, 1, 16, 2, 128, torch.float16, 200),   # 8 rows, clusters
    (9, 4, 8, 2, 64, torch.bfloat16, 200),     # 16 rows, clusters
    (3, 1, 2, 2, 128, torch.bfloat16, 4200),   # the same, the steps shared out
    (20, 1, 16, 2, 64, torch.float16, 2000),
    (5, 2, 16, 2, 128, torch.float16, 4200),
    (27, 21, 2, 1, 64, torch.float16, 900),    # one row tile
    (10, 60, 4, 2, 64, torch.bfloat16, 900),
    (10, 60, 4, 2, 128, torch.bfloat16, 900),
    (7, 130, 2, 2, 64, torch.float16, 900),    # two row tiles
    (7, 70, 4, 2, 128, torch.bfloat16, 900),
]


@pytest.mark.parametrize("seqs,n,H,Hkv,d,dtype,shortest", REPEATS)
def test_cache_attn_repeats_and_is_right(seqs, n, H, Hkv, d, dtype, shortest):
    """The first call against the oracle (some rows), then each of many calls against it."""
    g = rng(seqs + n)
    lens = [shortest + 131 * b for b in range(seqs)]
    pages = sum(-(-m // 32) for m in lens) + 2
    cache = filled(g, pages, Hkv, 32, d)
    table = tables(g, pages, lens, 32)
    q = randn(g, seqs, n, H, d, dtype=dtype)
    first = aj.cache_attn(q, cache, ints(lens), table, scale=0.05)
    ok()
    rows = sorted({0, n // 2, n - 1})
    for b in sorted({0, seqs // 2, seqs - 1}):
        m = lens[b]
        k, v = (orc.cache_values(f64(c), f64(s), table[b].cpu().numpy(), m)
                for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
        seen = np.array([m - n + 1 + i for i in rows])
        r = [orc.softmax_rows(f64(q[b, rows, h]), k[h * Hkv // H], v[h * Hkv // H], 0.05, seen) for h in range(H)]
        ref = [np.stack([x[i] for x in r], 1 if r[0][i].ndim == 2 else 0) for i in range(5)]
        lost = 4 * m * 448 * 2.0 ** -7 * 2.0 ** -32 * ref[4].T[..., None]
        check_attn(first[0][b, rows], first[1][b][:, rows], q[b], ref, 0.05, 2.0 ** -11, lost)
    for _ in range(50):
        o, lse = aj.cache_attn(q, cache, ints(lens), table, scale=0.05)
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])
    ok()


# ------------------------------------------------------------------ append
def test_append_of_a_skewed_batch():
    """One long sequence among a thousand single tokens: the mean is below five."""
    g = rng(55)
    new, page, heads, d = [1] * 500 + [3000] + [1] * 523, 128, 2, 128
    cached = [(i * 37) % 300 for i in range(1024)]
    lens = [a + b for a, b in zip(new, cached)]
    pages = sum(-(-n // page) for n in lens) + 2
    cache = pool(g, pages, heads, page, d)
    table = tables(g, pages, lens, page)
    starts = np.concatenate([[0], np.cumsum(new)])
    kv = randn(g, int(starts[-1]), 2 * heads, d, size=3.0)
    k, v = kv[:, :heads], kv[:, heads:]
    want_k = orc.append(f64(cache.k), f64(cache.k_scale), f64(k), starts, cached, table.cpu().numpy())
    want_v = orc.append(f64(cache.v), f64(cache.v_scale), f64(v), starts, cached, table.cpu().numpy())
    aj.cache_append(cache, k, v, ints(starts), ints(cached), table)
    ok()
    assert (f64(cache.k_scale) == want_k[1]).all() and (f64(cache.v_scale) == want_v[1]).all()
    same_codes(cache.k, want_k[0])
    same_codes(cache.v, want_v[0])


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("before,read", [(0.0, 2.0 ** -40), (-1.0, 2.0 ** -40), (NAN, 2.0 ** -40), (-INF, 2.0 ** -40),
                                         (2.0 ** -60, 2.0 ** -40), (2.0 ** 50, 2.0 ** 40), (INF, 2.0 ** 40)])
def test_append_behind_a_scale_that_is_none(new, before, read):
    """The scale of a page that keeps earlier tokens counts as the attention reads it."""
    g = rng(9)
    cache = filled(g, 4, 2, 64, 64)
    cache.k_scale[1], cache.v_scale[1] = before, before
    k, v = randn(g, new, 2, 64), randn(g, new, 2, 64, size=2.0 ** -30)
    scales = [f64(s).copy() for s in (cache.k_scale, cache.v_scale)]
    for s in scales:
        s[1] = read
    want_k = orc.append(f64(cache.k), scales[0], f64(k), [0, new], [11], [[1]])
    want_v = orc.append(f64(cache.v), scales[1], f64(v), [0, new], [11], [[1]])
    aj.cache_append(cache, k, v, ints([0, new]), ints([11]), ints([[1]]))
    ok()
    assert (f64(cache.k_scale) == want_k[1]).all() and (f64(cache.v_scale) == want_v[1]).all()
    same_codes(cache.k, want_k[0])
    same_codes(cache.v, want_v[0])


# ------------------------------------------------------------------ what a call leaves behind
def test_bad_index_does_not_fail_the_host_call():
    """A serving call's bad index is not an error of attn_jvp_host, and is reported after it."""
    w = wl.Workload("host_small", B=1, H=2, d=64, n_chunks=2, chunk_tokens=20, mode=wl.TEACHER_FORCING, seed=3)
    host = {n: t.cpu().pin_memory() for n, t in wl.make_inputs(w, device="cuda").items()}
    outs = [torch.empty_like(host["q"]).pin_memory() for _ in range(2)]
    lse = torch.empty(1, 2, host["q"].shape[1], dtype=torch.float32).pin_memory()
    cos, sin = aj.rope_tables(64, 8)
    aj.rope_at(randn(rng(1), 2, 1, 64), None, torch.tensor([3, 99], device="cuda"), cos, sin)
    staging = torch.empty(aj.host_staging_bytes(1, host["q"].shape[1], 2, 64, torch.bfloat16), dtype=torch.uint8, device="cuda")
    aj.attn_jvp_host(*(host[n] for n in ("q", "k", "v", "tq", "tk", "tv")), w.mode, w.chunk_tokens, w.n_chunks, staging,
                     (*outs, lse))
    assert aj.sync_status() == 7 and aj.sync_status() == 0


def test_written_tensors_get_a_new_version():
    """Autograd notices that a tensor which it saved was written over."""
    g = rng(2)
    q, k = randn(g, 4, 2, 64), randn(g, 4, 1, 64)
    cos, sin = aj.rope_tables(64, 8)
    pos, starts = ints([0, 1, 2, 3]), ints([0, 4])

    def raised(call, *written, kept=()):
        before = [t._version for t in (*written, *kept)]
        call()
        after = [t._version for t in (*written, *kept)]
        assert all(a > b for a, b in zip(after[:len(written)], before))
        assert after[len(written):] == before[len(written):]

    raised(lambda: aj.rope_at(q, k, pos, cos, sin, out=(q, k)), q, k, kept=(cos, sin, pos))
    raised(lambda: aj.rope_at(q, None, pos, cos, sin, out=(q, None)), q)
    cache = aj.paged_cache(2, 16, 1, 64)
    raised(lambda: aj.cache_append(cache, k, k, starts, ints([0]), ints([[1]])), *cache, kept=(k,))
    out = aj.prompt_attn(q, k, k, starts)
    raised(lambda: aj.prompt_attn(q, k, k, starts, out=out), *out, kept=(q, k))
    out = aj.cache_attn(q[None], cache, ints([4]), ints([[1]]))
    raised(lambda: aj.cache_attn(q[None], cache, ints([4]), ints([[1]]), out=out), *out, kept=(q, *cache))
    with torch.inference_mode():  # tensors without versions
        x = q.clone()
        aj.rope_at(x, None, pos, cos, sin, out=(x, None))
    ok()
    w = torch.ones(4, 2, 64, device="cuda", requires_grad=True)
    y = q.float()
    loss = (w * y).sum()
    aj.rope_at(y, None, pos, cos, sin, out=(y, None))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
