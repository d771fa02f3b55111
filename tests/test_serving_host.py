"""The serving operators on the host (no GPU): argument checks of the C ABI, which
every call here fails before any device call, the Python wrapper's own checks,
the rotation tables and the oracle's small parts."""
import ctypes
import math

import numpy as np
import pytest
import torch

import attention_jvp_attn_b200 as aj
from attention_jvp_attn_b200 import _abi
from oracle import serving_oracle as orc

BF16, F32, F16 = _abi.DTYPE_BF16, _abi.DTYPE_F32, _abi.DTYPE_F16
INVALID, UNSUPPORTED, MISALIGNED = _abi.ERR_INVALID_ARGUMENT, _abi.ERR_UNSUPPORTED, _abi.ERR_MISALIGNED
P = [0x10000 * (i + 1) for i in range(12)]  # fake, aligned device pointers: never used


@pytest.fixture(scope="module")
def lib():
    from attention_jvp_attn_b200 import build
    build.build()
    return _abi.load()


def S(token, head):
    return _abi.Strides(token, head)


def tables(cos=P[0], sin=P[1], n=100, rot=64, layout=0):
    return _abi.pack_rope_tables(cos or 0, sin or 0, n, rot, layout)


def cache(k=P[2], v=P[3], ks=P[4], vs=P[5], pages=9, page=64, strides=(8192, 4096, 64), scale=(1, 1)):
    return _abi.pack_cache(k or 0, v or 0, ks or 0, vs or 0, pages, page, *strides, *scale)


# ------------------------------------------------------------------ rotation
def rope(lib, T=8, H=2, Hkv=1, d=64, dtype=BF16, q=P[6], sq=(128, 64), k=P[7], sk=(64, 64), pos=P[8], pb=4,
         tab=None, qo=P[9], sqo=(128, 64), ko=P[10], sko=(64, 64), shape=True):
    sh = _abi.pack_tokens(T, H, Hkv, d, dtype, 0.0) if shape else None
    return lib.attn_jvp_rope_at(sh, q, S(*sq), k, S(*sk), pos, pb, tables() if tab is None else tab, 0, qo,
                                S(*sqo), ko, S(*sko), None)


@pytest.mark.parametrize("bad,code", [
    (dict(shape=False), INVALID), (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(Hkv=0), INVALID),
    (dict(d=96), UNSUPPORTED), (dict(dtype=9), UNSUPPORTED), (dict(q=None), INVALID), (dict(qo=None), INVALID),
    (dict(pos=None), INVALID), (dict(pb=2), INVALID), (dict(pos=P[8] + 2), MISALIGNED),
    (dict(q=P[6] + 8), MISALIGNED), (dict(k=None), INVALID), (dict(ko=None), INVALID), (dict(ko=P[10] + 2), MISALIGNED),
    (dict(sq=(130, 64)), MISALIGNED), (dict(sq=(-128, 64)), MISALIGNED), (dict(sqo=(64, 64)), INVALID),
    (dict(sqo=(128, 0)), INVALID), (dict(sko=(0, 64)), INVALID), (dict(T=2 ** 31), INVALID),
    (dict(tab=tables(cos=None)), INVALID), (dict(tab=tables(sin=P[1] + 4)), MISALIGNED), (dict(tab=tables(n=0)), INVALID),
    (dict(tab=tables(rot=24)), INVALID), (dict(tab=tables(rot=80)), INVALID), (dict(tab=tables(rot=0)), INVALID),
    (dict(tab=tables(layout=2)), INVALID)])
def test_rope_at_refuses(lib, bad, code):
    assert rope(lib, **bad) == code


def test_nothing_to_do_is_ok(lib):
    assert rope(lib, T=0, q=None, qo=None, pos=None) == _abi.OK
    assert append(lib, T=0) == _abi.OK and append(lib, B=0) == _abi.OK
    assert attn(lib, B=0) == _abi.OK and attn(lib, n=0) == _abi.OK
    assert prompt(lib, T=0) == _abi.OK and prompt(lib, B=0) == _abi.OK


# ------------------------------------------------------------------ append
def append(lib, T=8, Hkv=2, d=64, dtype=BF16, k=P[6], sk=(128, 64), v=P[7], sv=(128, 64), c=None, B=2, starts=P[8],
           cached=P[9], table=P[10], width=4, stride=4, rot=None):
    return lib.attn_jvp_cache_append(_abi.pack_tokens(T, 1, Hkv, d, dtype, 0.0), k, S(*sk), v, S(*sv),
                                     cache() if c is None else c, B, starts, cached, table, width, stride, rot, None)


@pytest.mark.parametrize("bad,code", [
    (dict(T=-1), INVALID), (dict(Hkv=0), INVALID), (dict(d=32), UNSUPPORTED), (dict(dtype=4), UNSUPPORTED),
    (dict(k=None), INVALID), (dict(v=P[7] + 4), MISALIGNED), (dict(sk=(132, 64)), MISALIGNED), (dict(B=-1), INVALID),
    (dict(starts=None), INVALID), (dict(cached=None), INVALID), (dict(table=None), INVALID), (dict(width=0), INVALID),
    (dict(stride=3), INVALID), (dict(rot=tables(rot=128)), INVALID), (dict(rot=tables(cos=P[0] + 1)), MISALIGNED),
    (dict(c=cache(k=None)), INVALID), (dict(c=cache(vs=None)), INVALID), (dict(c=cache(k=P[2] + 8)), MISALIGNED),
    (dict(c=cache(pages=0)), INVALID), (dict(c=cache(page=48)), UNSUPPORTED), (dict(c=cache(page=256)), UNSUPPORTED),
    (dict(c=cache(strides=(8192, 4096, 72))), MISALIGNED), (dict(c=cache(strides=(8192, 4096, 48))), INVALID),
    (dict(c=cache(strides=(8192, 32, 64))), INVALID), (dict(c=cache(strides=(2 ** 32, 4096, 64))), UNSUPPORTED),
    (dict(c=cache(scale=(0, 1))), INVALID), (dict(c=cache(scale=(2, 0))), INVALID), (dict(Hkv=32768), INVALID),
    (dict(width=2 ** 62, stride=2 ** 62), INVALID), (dict(T=2 ** 31), INVALID), (dict(B=2 ** 21), INVALID),
    (dict(starts=P[8] + 2), MISALIGNED), (dict(cached=P[9] + 1), MISALIGNED), (dict(table=P[10] + 2), MISALIGNED),
    (dict(c=cache(ks=P[4] + 2)), MISALIGNED)])
def test_cache_append_refuses(lib, bad, code):
    assert append(lib, **bad) == code


# ------------------------------------------------------------------ attention over the cache
def attn(lib, B=2, n=1, H=4, Hkv=2, d=64, dtype=BF16, scale=0.0, q=P[6], sq=(256, 256, 64), c=None, lens=P[7], table=P[8],
         width=4, stride=4, max_len=0, work=None, size=0, o=P[9], lse=P[10]):
    arr = (ctypes.c_int64 * 3)(*sq)
    return lib.attn_jvp_cache_attn(_abi.pack_shape(B, n, H, d, dtype, scale), Hkv, q, arr, cache() if c is None else c,
                                   lens, table, width, stride, max_len, 1, work, size, o, lse, None)


@pytest.mark.parametrize("bad,code", [
    (dict(B=-1), INVALID), (dict(n=-2), INVALID), (dict(H=0), INVALID), (dict(H=3), INVALID), (dict(Hkv=0), INVALID),
    (dict(d=32), UNSUPPORTED), (dict(dtype=F32), UNSUPPORTED), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(q=None), INVALID), (dict(q=P[6] + 2), MISALIGNED),
    (dict(sq=(260, 256, 64)), MISALIGNED), (dict(sq=(256, 256, -64)), INVALID), (dict(lens=None), INVALID),
    (dict(table=None), INVALID), (dict(o=None), INVALID), (dict(o=P[9] + 8), MISALIGNED), (dict(lse=None), INVALID),
    (dict(width=0), INVALID), (dict(width=2 ** 25), INVALID), (dict(max_len=-1), INVALID), (dict(c=cache(page=8)), UNSUPPORTED),
    (dict(B=65536), INVALID), (dict(width=2 ** 60, stride=2 ** 60), INVALID), (dict(n=2 ** 25), INVALID),
    (dict(H=65536), INVALID), (dict(c=cache(strides=(8192, 4096, 2 ** 32))), UNSUPPORTED),
    (dict(lens=P[7] + 2), MISALIGNED), (dict(table=P[8] + 1), MISALIGNED), (dict(lse=P[10] + 2), MISALIGNED)])
def test_cache_attn_refuses(lib, bad, code):
    assert attn(lib, **bad) == code


# ------------------------------------------------------------------ prompts
def prompt(lib, T=8, H=4, Hkv=2, d=64, dtype=BF16, scale=0.0, q=P[0], sq=(512, 64), k=P[1], sk=(512, 64), v=P[2],
           sv=(512, 64), B=1, starts=P[3], o=P[4], lse=P[5]):
    return lib.attn_jvp_prompt_attn(_abi.pack_tokens(T, H, Hkv, d, dtype, scale), q, S(*sq), k, S(*sk), v, S(*sv), B,
                                    starts, o, lse, None)


@pytest.mark.parametrize("bad,code", [
    (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(H=5), INVALID), (dict(Hkv=0), INVALID), (dict(d=80), UNSUPPORTED),
    (dict(dtype=F32), UNSUPPORTED), (dict(scale=float("nan")), INVALID), (dict(q=None), INVALID), (dict(k=P[1] + 2), MISALIGNED),
    (dict(v=None), INVALID), (dict(sv=(508, 64)), MISALIGNED), (dict(B=-1), INVALID), (dict(B=2 ** 21), INVALID),
    (dict(starts=None), INVALID), (dict(o=None), INVALID), (dict(o=P[4] + 8), MISALIGNED), (dict(lse=None), INVALID),
    (dict(sk=(512, 0)), INVALID), (dict(sq=(0, 64)), INVALID), (dict(sv=(32, 64)), INVALID), (dict(starts=P[3] + 2), MISALIGNED),
    (dict(lse=P[5] + 1), MISALIGNED)])
def test_prompt_attn_refuses(lib, bad, code):
    assert prompt(lib, **bad) == code


@pytest.mark.parametrize("bad", [dict(B=-1), dict(n=-1), dict(n=2 ** 62), dict(H=3), dict(H=0), dict(Hkv=0), dict(d=96),
                                 dict(dtype=F32), dict(max_len=-1), dict(max_len=2 ** 62)])
def test_workspace_bytes_refuses(lib, bad):
    a = dict(B=2, n=1, H=4, Hkv=2, d=64, dtype=BF16, max_len=5000) | bad
    shape = _abi.pack_shape(a["B"], a["n"], a["H"], a["d"], a["dtype"], 0.0)
    assert lib.attn_jvp_cache_attn_workspace_bytes(shape, a["Hkv"], a["max_len"]) == -1


def test_fp16_is_refused_elsewhere(lib):
    """The type that the serving operators add is not one of the other functions'."""
    s = _abi.Shape(1, 8, 2, 64, F16, 0.0)
    assert lib.attn_jvp_rope(ctypes.byref(s), *P[:10], None) == UNSUPPORTED
    assert lib.attn_jvp_fwd(ctypes.byref(s), *P[:6], _abi.Mask(0, 2, 2), *P[6:9], None) == UNSUPPORTED


def test_status_string(lib):
    assert "device" in _abi.status_string(_abi.ERR_BAD_INDEX)


# ------------------------------------------------------------------ the wrapper
def test_wrapper_refuses_host_tensors(lib):
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        aj.rope_at(x, x, i, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        aj.prompt_attn(x, x, x, i)
    with pytest.raises(ValueError, match="CUDA"):
        aj.cache_attn(x[None], None, i, i)
    with pytest.raises(ValueError):
        aj.cache_append(aj.paged_cache(2, 16, 2, 64, device="cpu"), x, x, i, i, i)
    with pytest.raises(ValueError, match=r"\[T, heads, d\]"):
        aj.rope_at(x[0], None, i, x, x)


def test_wrapper_refuses_what_is_no_tensor(lib):
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    c = aj.paged_cache(2, 16, 2, 64, device="cpu")
    for call in (lambda: aj.rope_at(None, x, i, x, x), lambda: aj.rope_at([1], x, i, x, x),
                 lambda: aj.cache_attn(3, c, i, i), lambda: aj.cache_append(c[:3], x, x, i, i, i),
                 lambda: aj.cache_append(None, x, x, i, i, i), lambda: aj.cache_append(c, x, 1.0, i, i, i),
                 lambda: aj.prompt_attn(x, x, None, i)):
        with pytest.raises(ValueError):
            call()


def test_binding_shares_the_process_cpp_runtime(lib):
    """Two C++ runtimes in one process crash when a message formats a number."""
    from attention_jvp_attn_b200 import build
    with open(build.BINDING, "rb") as f:
        assert b"\0libstdc++.so.6\0" in f.read()


def test_missing_binding_fails_loudly(lib, monkeypatch):
    """Without its binding an operator raises; nothing stands in for it."""
    import sys
    from attention_jvp_attn_b200 import serving
    monkeypatch.setattr(serving, "_bound", None)
    monkeypatch.delattr(aj, "_serving", raising=False)
    monkeypatch.setitem(sys.modules, "attention_jvp_attn_b200._serving", None)
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(RuntimeError, match="not built"):
        aj.prompt_attn(x, x, x, x)


@pytest.mark.parametrize("args", [(2, 24, 1, 64), (2, 16, 1, 96), (0, 16, 1, 64), (2, 16, 0, 64)])
def test_paged_cache_refuses(args):
    with pytest.raises(ValueError):
        aj.paged_cache(*args, device="cpu")


def test_paged_cache():
    c = aj.paged_cache(3, 32, 2, 128, device="cpu")
    assert c.k.shape == c.v.shape == (3, 2, 32, 128) and c.k.dtype == torch.float8_e4m3fn
    assert c.k_scale.shape == (3, 2) and c.v_scale.dtype == torch.float32


# ------------------------------------------------------------------ tables
def test_rope_tables_plain_and_far():
    cos, sin = aj.rope_tables(64, 131072, device="cpu")
    assert cos.shape == sin.shape == (131072, 32) and cos.dtype == torch.float32
    for p in (0, 1, 77, 131071):
        for i in (0, 5, 31):
            a = p * 10000.0 ** (-2 * i / 64)  # python's 64-bit floats
            assert abs(cos[p, i].item() - math.cos(a)) < 1e-6 and abs(sin[p, i].item() - math.sin(a)) < 1e-6


def test_rope_tables_scaled():
    freq = lambda c, s: torch.atan2(s[1].double(), c[1].double()).numpy()  # angle of position 1: the frequency
    base = freq(*aj.rope_tables(128, 2, device="cpu"))
    assert np.allclose(freq(*aj.rope_tables(128, 2, scaling="linear", factor=4.0, device="cpu")), base / 4, rtol=1e-5)
    ntk = freq(*aj.rope_tables(128, 2, scaling="base", factor=4.0, device="cpu"))
    assert abs(ntk[0] - base[0]) < 1e-6 and abs(ntk[-1] / base[-1] - 0.25) < 1e-4
    cos, sin = aj.rope_tables(128, 2, scaling="by_parts", factor=4.0, original_positions=4096, device="cpu")
    mag = torch.sqrt(cos.double() ** 2 + sin.double() ** 2)
    assert torch.allclose(mag, torch.full_like(mag, 0.1 * math.log(4.0) + 1.0), atol=1e-6)
    parts = freq(cos, sin) / base
    turns = 4096 * base / (2 * math.pi)
    assert np.allclose(parts[turns > 40], 1.0, atol=1e-5) and np.allclose(parts[turns < 0.8], 0.25, atol=1e-4)
    assert (np.diff(parts) <= 1e-6).all()


@pytest.mark.parametrize("kw", [dict(rot=8), dict(rot=40), dict(n_positions=0), dict(base=1.0), dict(factor=0.5),
                                dict(scaling="odd"), dict(scaling="by_parts"),
                                dict(scaling="by_parts", original_positions=10, fast_turns=1.0, slow_turns=2.0)])
def test_rope_tables_refuse(kw):
    with pytest.raises(ValueError):
        aj.rope_tables(**{"rot": 64, "n_positions": 8, "device": "cpu", **kw})


# ------------------------------------------------------------------ the oracle's own pins
def test_oracle_e4m3_is_torchs():
    x = np.concatenate([np.linspace(-500, 500, 4001), 2.0 ** np.linspace(-14, 9, 3001), [0.0, 448, 464, 1e30]])
    want = torch.from_numpy(np.clip(x, -448, 448)).to(torch.float64).to(torch.float8_e4m3fn).double().numpy()
    assert (orc.round_e4m3(x) == want).all()
    assert orc.round_e4m3(np.inf) == 448 and np.isnan(orc.round_e4m3(np.nan))


@pytest.mark.parametrize("x,e", [(448.0, 0), (448.0001, 1), (224.0, -1), (224.1, 0), (0.0, -32), (1e-30, -32), (1e30, 32),
                                 (1.75, -8), (1.7500001, -7)])
def test_oracle_needed_exp(x, e):
    assert orc.needed_exp(np.array([x, -x / 2, np.inf, np.nan])) == e


def test_oracle_attention_pins():
    """One key: its value; equal keys: the mean; no key: 0 and -inf."""
    v = np.arange(12.0).reshape(3, 4)
    o, lse, *_ = orc.softmax_rows(np.ones((3, 4)), np.zeros((3, 4)), v, 0.5, [1, 3, 0])
    assert np.allclose(o, [v[0], v.mean(0), np.zeros(4)]) and np.allclose(lse[:2], [0, math.log(3)]) and lse[2] == -np.inf


def test_oracle_rope_pins():
    cos, sin = np.array([[0.0] * 8]), np.array([[1.0] * 8])  # a quarter turn
    x = np.arange(16.0)[None, None]
    half = orc.rope(x, [0], cos, sin, "half")[0, 0]
    assert (half == np.concatenate([-x[0, 0, 8:], x[0, 0, :8]])).all()
    inter = orc.rope(x, [0], cos, sin, "interleaved")[0, 0]
    assert (inter[0::2] == -x[0, 0, 1::2]).all() and (inter[1::2] == x[0, 0, 0::2]).all()
    assert np.allclose(orc.rope(orc.rope(x, [0], cos, sin, "half"), [0], cos, sin, "half", True), x)
