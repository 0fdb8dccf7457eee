"""Host-side refusals of the calls on new tokens (append, window attention,
shared-prefix attention): every call below is invalid by construction or a
no-op, so none reaches a kernel launch, and they run without a GPU. Then the
rotary tables, and properties of the new sources."""
import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

from tests import step_common as sc

OK, INVALID, HEAD_DIM, BITS, ALIGN, DTYPE = range(6)
P = 1 << 20  # an aligned address that is never read
CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "turboquant_kv_cache_tq_gb300", "csrc")


@pytest.fixture(scope="module")
def tq():
    from turboquant_kv_cache_tq_gb300 import build

    build.build()
    import turboquant_kv_cache_tq_gb300 as tq

    tq.lib()
    return tq


def _cache(tq, cap=64, **bad):
    c = dict(k_codes=P, k_scales=P, k_zeros=P, v_codes=P, v_scales=P)
    c.update(bad)
    return tq.TQPackedCache(c["k_codes"], c["k_scales"], c["k_zeros"], c["v_codes"], c["v_scales"], cap)


def _apart(tq, cap=64):
    """A cache whose buffers do not share memory."""
    return tq.TQPackedCache(*[P + (i << 24) for i in range(5)], cap)


def _rows(tq, data=1 << 40, b=1 << 14, h=1 << 12, t=128):
    return tq.TQRows(data, b, h, t)


def _append(tq, q="rows", k="rows", v="rows", dtype=1, B=1, Hq=4, Hkv=2, N=8, D=128, cos=1 << 41, sin=1 << 42, length=64, R=128,
            inter=0, positions=None, lens=None, pad=None, count=None, cache=None, kb=8, ks=1, vb=3, q_out=1 << 43,
            new=1 << 44):
    c = _apart(tq) if cache is None else cache
    r = [_rows(tq) if x == "rows" else x for x in (q, k, v)]
    return tq.lib().tq_append_kv(*[None if x is None else ctypes.byref(x) for x in r], dtype, B, Hq, Hkv, N, D, cos, sin,
                                 length, R, inter, positions, lens, pad, count, ctypes.byref(c), kb, ks, vb, q_out, new, None)


def test_append_refusals(tq):
    assert _append(tq, B=0) == OK
    for kw in (dict(B=-1), dict(Hkv=0), dict(N=-1), dict(Hq=0), dict(k=None), dict(v=None), dict(R=3), dict(R=-2), dict(R=130),
               dict(length=0), dict(length=1 << 31), dict(cos=None), dict(sin=None), dict(new=None), dict(q_out=None),
               dict(cache=_cache(tq, -1)), dict(cache=_cache(tq, 1 << 31)), dict(cache=_cache(tq, 64, v_scales=0)),
               dict(B=1 << 31), dict(N=1 << 31), dict(B=1 << 16, N=1 << 16), dict(Hkv=1 << 30, N=4), dict(Hq=1 << 30, N=4),
               dict(k=_rows(tq, data=0)), dict(v=_rows(tq, data=0)), dict(q=_rows(tq, data=0)), dict(B=2, k=_rows(tq, b=-128)),
               dict(k=_rows(tq, h=-128)), dict(v=_rows(tq, t=-128)), dict(q=_rows(tq, t=1 << 60)),
               dict(cache=_cache(tq, 64))):  # (the cache's buffers share memory)
        assert _append(tq, **kw) == INVALID, kw
    for D in (0, 32, 96, 1024, -64):
        assert _append(tq, D=D, R=0) == HEAD_DIM
    for kw in (dict(kb=3, ks=0), dict(kb=4, ks=1), dict(vb=6), dict(vb=1)):
        assert _append(tq, **kw) == BITS, kw
    assert _append(tq, dtype=2) == DTYPE and _append(tq, dtype=-1) == DTYPE
    for kw in (dict(q=_rows(tq, data=P + 8)), dict(k=_rows(tq, data=P + 2)), dict(k=_rows(tq, t=4)), dict(v=_rows(tq, h=12)),
               dict(B=2, q=_rows(tq, b=1)), dict(dtype=0, k=_rows(tq, t=2)), dict(q_out=P + 8), dict(new=P + 2),
               dict(cos=P + 4), dict(sin=P + 8), dict(lens=P + 1), dict(pad=P + 2), dict(count=P + 3), dict(positions=P + 1),
               dict(cache=_cache(tq, 64, k_zeros=P + 2))):
        assert _append(tq, **kw) == ALIGN, kw


def test_append_refuses_shared_memory(tq):
    at = [P + (i << 24) for i in range(5)]
    for kw in (dict(q_out=1 << 40), dict(q_out=at[0]), dict(new=at[3]), dict(new=1 << 43), dict(lens=1 << 44, new=1 << 44),
               dict(count=at[1]), dict(k=_rows(tq, data=at[2])), dict(v=_rows(tq, data=at[4] - (1 << 13))), dict(cos=at[0]),
               dict(sin=1 << 43), dict(positions=at[4]), dict(pad=1 << 44)):
        assert _append(tq, **kw) == INVALID, kw


def _window(tq, q=P, B=1, Hq=4, N=8, cache=None, Hkv=2, T=64, D=128, kb=8, ks=1, vb=3, lens=None, pad=None, count=None,
            win=16, sinks=2, out=1 << 40, dtype=1, lse=None, ws=1 << 41, ws_bytes=1 << 39):
    c = _cache(tq) if cache is None else cache
    return tq.lib().tq_window_attention(q, B, Hq, N, ctypes.byref(c), Hkv, T, D, kb, ks, vb, lens, pad, count, win, sinks,
                                        ctypes.c_float(1.0), out, dtype, lse, ws, ws_bytes, None)


def test_window_refusals(tq):
    assert _window(tq, B=0) == OK
    for kw in (dict(B=-1), dict(Hq=0), dict(Hkv=0), dict(N=0), dict(T=-1), dict(T=65), dict(Hq=5), dict(q=0), dict(out=0),
               dict(ws=0), dict(ws_bytes=0), dict(ws_bytes=-1), dict(win=0), dict(win=-1), dict(sinks=-1),
               dict(cache=_cache(tq, v_codes=0)), dict(cache=_cache(tq, 1 << 40)), dict(B=1 << 32), dict(B=1 << 20, Hq=1 << 12),
               dict(N=(1 << 19) + 1), dict(N=1 << 40), dict(cache=_cache(tq, 1 << 31), T=(1 << 31) - 8)):
        assert _window(tq, **kw) == INVALID, kw
    for D in (0, 32, 96, 1024, -64):
        assert _window(tq, D=D) == HEAD_DIM
    for kw in (dict(kb=3, ks=0), dict(kb=4, ks=1), dict(vb=6)):
        assert _window(tq, **kw) == BITS, kw
    assert _window(tq, dtype=2) == DTYPE
    for kw in (dict(q=P + 8), dict(out=P + 2), dict(ws=P + 4), dict(cache=_cache(tq, k_scales=P + 2)), dict(lens=P + 2),
               dict(pad=P + 3), dict(count=P + 1), dict(lse=P + 1)):
        assert _window(tq, **kw) == ALIGN, kw
    for kw in (dict(out=P), dict(ws=P), dict(lse=P), dict(lse=1 << 40), dict(ws=1 << 40), dict(lens=1 << 41), dict(count=1 << 40)):
        assert _window(tq, **kw) == INVALID, kw
    assert tq.lib().tq_window_attention(P, 1, 4, 8, None, 2, 64, 128, 8, 1, 3, None, None, None, 4, 0, ctypes.c_float(1.0),
                                        P, 1, None, P, 1 << 39, None) == INVALID


def _prefix(tq, q=P, B=4, Hq=4, N=2, pre=None, Bp=2, Pn=32, plens=None, cache=None, Hkv=2, T=64, D=128, kb=8, ks=1, vb=3,
            lens=None, pad=None, count=None, out=1 << 40, dtype=1, lse=None, ws=1 << 41, ws_bytes=1 << 39):
    c, p = _cache(tq) if cache is None else cache, _cache(tq, 32) if pre is None else pre
    return tq.lib().tq_prefix_attention(q, B, Hq, N, ctypes.byref(p), Bp, Pn, plens, ctypes.byref(c), Hkv, T, D, kb, ks, vb,
                                        lens, pad, count, ctypes.c_float(1.0), out, dtype, lse, ws, ws_bytes, None)


def test_prefix_refusals(tq):
    assert _prefix(tq, B=0) == OK
    for kw in (dict(B=-1), dict(B=3), dict(Bp=0), dict(Bp=-2), dict(Hq=0), dict(N=0), dict(T=65), dict(Pn=33), dict(Pn=-1),
               dict(Hq=5), dict(q=0), dict(out=0), dict(ws=0), dict(ws_bytes=0), dict(pre=_cache(tq, 32, k_codes=0)),
               dict(cache=_cache(tq, v_codes=0)), dict(pre=_cache(tq, 1 << 40)), dict(B=1 << 20, Bp=1, N=1 << 10),
               dict(out=P), dict(ws=P), dict(plens=1 << 41)):
        assert _prefix(tq, **kw) == INVALID, kw
    assert _prefix(tq, D=100) == HEAD_DIM and _prefix(tq, vb=7) == BITS and _prefix(tq, dtype=5) == DTYPE
    for kw in (dict(q=P + 8), dict(out=P + 2), dict(pre=_cache(tq, 32, v_scales=P + 8)), dict(plens=P + 2), dict(lens=P + 1)):
        assert _prefix(tq, **kw) == ALIGN, kw


def test_workspace_sizes(tq):
    w, p = tq.lib().tq_window_attention_workspace_size, tq.lib().tq_prefix_attention_workspace_size
    for a in ((-1, 4, 2, 8, 128), (1, 0, 1, 8, 128), (1, 4, 0, 8, 128), (1, 4, 3, 8, 128), (1, 4, 2, 0, 128),
              (1 << 40, 4, 2, 8, 128), (1, 4, 2, 1 << 30, 128)):
        assert w(*a) == -INVALID, a
    for a in ((0, 4, 4, 2, 8, 128), (3, 4, 4, 2, 8, 128), (-1, 4, 4, 2, 8, 128), (1, 4, 4, 2, 0, 128)):
        assert p(*a) == -INVALID, a
    assert w(1, 4, 2, 8, 100) == -HEAD_DIM and p(1, 4, 4, 2, 8, 100) == -HEAD_DIM
    assert 0 < w(1, 4, 2, 1, 128) <= w(8, 4, 2, 1, 128) and 0 < p(1, 4, 4, 2, 1, 128) < 1 << 30
    assert p(1, 0, 4, 2, 1, 128) >= 0  # (an empty batch)
    with pytest.raises(tq.TQError):
        tq.tq_window_attention_workspace_size(1, 4, 3, 8, 128)
    with pytest.raises(tq.TQError):
        tq.tq_prefix_attention_workspace_size(3, 4, 4, 2, 8, 128)


def test_binding_refusals(tq):
    """What the binding sees before the library: shapes, types, devices."""
    cache = tq.alloc_cache(2, 2, 16, 64, 8, 3, device="cpu")
    k = torch.zeros((2, 2, 3, 64))
    lens = torch.zeros(2, dtype=torch.int32)
    for bad in (k[0], k.half(), k.double()):
        with pytest.raises(ValueError):
            tq.tq_append_kv(bad, bad, cache, lens, 8, True, 3)
    with pytest.raises(ValueError, match="CUDA device"):
        tq.tq_append_kv(k, k, cache, lens, 8, True, 3)
    dev = torch.device("cpu")
    for t in (k.transpose(2, 3), k[..., ::2]):
        with pytest.raises(ValueError, match="contiguous rows"):
            tq._rows(t, t.shape, torch.float32, "k", dev)
    q = torch.zeros((2, 4, 1, 64), dtype=torch.bfloat16)
    for call in (lambda q, **kw: tq.tq_window_attention(q, cache, 16, 8, True, 3, 4, **kw),
                 lambda q, **kw: tq.tq_prefix_attention(q, cache, 16, cache, 16, 8, True, 3, **kw)):
        with pytest.raises(ValueError, match="bfloat16"):
            call(q.float())
        with pytest.raises(ValueError, match="contiguous"):
            call(q[..., ::2])
        with pytest.raises(ValueError, match="out_dtype"):
            call(q, out_dtype=torch.float16)
        with pytest.raises(ValueError, match="CUDA device"):
            call(q)


def test_rope_tables(tq):
    def close(a, b):
        return np.abs(a.numpy().astype(np.float64) - b).max() <= 2.0 ** -24 + 1e-12

    R, n = 64, 300
    j = np.arange(R // 2)
    f = 10000.0 ** (-2 * j / R)
    at = np.arange(n)[:, None]
    for args, freq in ((dict(), f), (dict(scaling="linear", factor=4.0), f / 4),
                       (dict(scaling="base", factor=8.0), (10000.0 * 8 ** (R / (R - 2))) ** (-2 * j / R)),
                       (dict(base=5e5), 5e5 ** (-2 * j / R))):
        cos, sin = tq.rope_tables(R, n, device="cpu", **args)
        assert cos.dtype == sin.dtype == torch.float32 and cos.shape == sin.shape == (n, R // 2)
        assert close(cos, np.cos(at * freq)) and close(sin, np.sin(at * freq)), args
    # a larger base: the highest frequency stays, the lowest is divided by the factor
    cos, sin = tq.rope_tables(R, 2, scaling="base", factor=8.0, device="cpu")
    assert abs(math.atan2(sin[1, 0], cos[1, 0]) - 1) < 1e-6 and abs(math.atan2(sin[1, -1], cos[1, -1]) * 8 / f[-1] - 1) < 1e-5
    # bands: fast turns stay, slow ones are divided, and nothing jumps between
    cos, sin = tq.rope_tables(R, 2, scaling="bands", factor=8.0, original=8192, device="cpu")
    g = np.arctan2(sin[1].numpy(), cos[1].numpy()).astype(np.float64)
    turns = 8192 * f / (2 * math.pi)
    assert np.allclose(g[turns > 4], f[turns > 4], rtol=1e-5) and np.allclose(g[turns < 1], f[turns < 1] / 8, rtol=1e-5)
    assert (g <= f * (1 + 1e-5)).all() and (g >= f / 8 * (1 - 1e-5)).all() and (np.diff(g) < 0).all()
    for bad in (dict(rot_dim=3, length=4), dict(rot_dim=0, length=4), dict(rot_dim=4, length=0),
                dict(rot_dim=4, length=4, factor=0.5), dict(rot_dim=4, length=4, base=0.0),
                dict(rot_dim=4, length=4, scaling="other"), dict(rot_dim=2, length=4, scaling="base", factor=2.0),
                dict(rot_dim=4, length=4, scaling="bands", factor=2.0),
                dict(rot_dim=4, length=4, scaling="bands", factor=2.0, original=8, low=4.0, high=4.0)):
        with pytest.raises(ValueError):
            tq.rope_tables(device="cpu", **bad)


def test_the_rotation_turns():
    """The reference itself: lengths stay, positions add up, the rest of the row stays."""
    import turboquant_kv_cache_tq_gb300 as tq

    g = torch.Generator().manual_seed(1)
    x = torch.randn((1, 1, 2, 64), generator=g)
    for inter in (False, True):
        for R in (64, 20):
            cos, sin = tq.rope_tables(R, 50, device="cpu")
            y = sc.turned(x, cos, sin, np.array([[0, 7]]), inter)
            assert np.array_equal(y[..., 0, :], x[..., 0, :].numpy()) and np.array_equal(y[..., R:], x[..., R:].numpy())
            assert abs(np.linalg.norm(y[0, 0, 1]) - x[0, 0, 1].norm().item()) < 1e-5
            z = sc.turned(torch.from_numpy(sc.turned(x, cos, sin, np.array([[3, 4]]), inter)), cos, sin, np.array([[9, 8]]), inter)
            assert np.abs(z - sc.turned(x, cos, sin, np.array([[12, 12]]), inter)).max() < 1e-5


def test_what_a_token_sees_by_hand():
    m, there = sc.seen(2, 2, 6, lens=[6, 3], left_pad=[1, 0], count=[2, 1], window=2, sinks=1)
    assert m[0, 0].tolist() == [False, True, False, True, True, False]
    assert m[0, 1].tolist() == [False, True, False, False, True, True]
    assert m[1, 0].tolist() == [True, True, True, False, False, False] and not m[1, 1].any()
    assert there.tolist() == [[True, True], [True, False]]


def test_sources_of_the_new_calls():
    """Below a C entry point an exception ends the process; a device helper has a caller."""
    names = [n for n in sorted(os.listdir(CSRC)) if re.match(r"tq_(append|span_)", n)]
    assert len(names) >= 8
    text = {n: open(os.path.join(CSRC, n)).read() for n in sorted(os.listdir(CSRC)) if n.endswith((".cu", ".cuh", ".h"))}
    everything = "".join(text.values())
    for name in names:
        code = re.sub(r"//[^\n]*|/\*.*?\*/", "", text[name], flags=re.S)
        assert not re.search(r"std::(vector|string|map|function|mutex|lock_guard)|\bnew\b|\bthrow\b", code), name
        for helper in re.findall(r"__forceinline__ (?:static )?[\w:<> ]*?(\w+)\(", text[name]):
            if not helper[0].isupper():
                assert len(re.findall(r"\b%s\b" % helper, everything)) > 1, (name, helper)
