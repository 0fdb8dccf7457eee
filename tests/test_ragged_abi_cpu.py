"""Host-side refusals of the calls on ragged packed caches: every call below is
invalid by construction (or a no-op), so none reaches a kernel launch, and they
run without a GPU."""
import ctypes

import numpy as np
import pytest
import torch

from tests import ragged_common as rc

OK, INVALID, HEAD_DIM, BITS, ALIGN, DTYPE = range(6)
P = 1 << 20  # an aligned address that is never read


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


def _tree(tq, q=P, B=1, Hq=4, N=8, cache=None, Hkv=2, T=64, D=128, tree=None, parents=None, kb=8, ks=1, vb=3, lens=None,
          pad=None, out=P, dtype=1, lse=None, ws=P, ws_bytes=1 << 40):
    c = _cache(tq) if cache is None else cache
    t = _cache(tq, 8) if tree is None else tree
    return tq.lib().tq_tree_attention(q, B, Hq, N, ctypes.byref(c), Hkv, T, D, ctypes.byref(t), parents, kb, ks, vb, lens,
                                      pad, ctypes.c_float(1.0), out, dtype, lse, ws, ws_bytes, None)


def test_tree_refusals(tq):
    assert _tree(tq, B=0) == OK
    for kw in (dict(B=-1), dict(Hq=0), dict(Hkv=0), dict(N=0), dict(N=65, tree=_cache(tq, 65)), dict(T=-1), dict(T=65),
               dict(Hq=5), dict(q=0), dict(out=0), dict(ws=0), dict(ws_bytes=0), dict(tree=_cache(tq, 7)),
               dict(cache=_cache(tq, v_codes=0)), dict(tree=_cache(tq, 8, k_zeros=0)), dict(B=1 << 32),
               dict(B=1 << 20, Hq=1 << 12), dict(cache=_cache(tq, 1 << 40)), dict(ws_bytes=-1)):
        assert _tree(tq, **kw) == INVALID, kw
    for D in (0, 32, 96, 1024, -64):
        assert _tree(tq, D=D) == HEAD_DIM
    for kw in (dict(kb=3, ks=0), dict(kb=4, ks=1), dict(vb=6), dict(vb=1), dict(kb=0, ks=0)):
        assert _tree(tq, **kw) == BITS, kw
    assert _tree(tq, dtype=2) == DTYPE
    for kw in (dict(q=P + 8), dict(out=P + 2), dict(ws=P + 4), dict(cache=_cache(tq, k_scales=P + 2)),
               dict(tree=_cache(tq, 8, v_scales=P + 8)), dict(parents=P + 1), dict(lens=P + 2), dict(pad=P + 3),
               dict(lse=P + 1)):
        assert _tree(tq, **kw) == ALIGN, kw
    assert tq.lib().tq_tree_attention(P, 1, 4, 8, None, 2, 64, 128, None, None, 8, 1, 3, None, None,
                                      ctypes.c_float(1.0), P, 1, None, P, 1 << 40, None) == INVALID


def test_tree_workspace_refusals(tq):
    f = tq.lib().tq_tree_attention_workspace_size
    for a in ((-1, 4, 2, 8, 128), (1, 0, 1, 8, 128), (1, 4, 0, 8, 128), (1, 4, 3, 8, 128), (1, 4, 2, 0, 128),
              (1, 4, 2, 65, 128), (1 << 40, 4, 2, 8, 128)):
        assert f(*a) == -INVALID, a
    assert f(1, 4, 2, 8, 100) == -HEAD_DIM
    with pytest.raises(tq.TQError):
        tq.tq_tree_attention_workspace_size(1, 4, 3, 8, 128)


def _weights(tq, q=P, lse=P, B=1, Hq=4, N=8, kc=P, ks_=P, kz=P, Hkv=2, T=64, D=128, cap=64, kb=8, ks=1, lens=None,
             pad=None, path=None, n_path=None, Pn=8, w_in=None, w_out=P, w_cap=64):
    return tq.lib().tq_attention_weights(q, lse, B, Hq, N, kc, ks_, kz, Hkv, T, D, cap, kb, ks, lens, pad, path, n_path,
                                         Pn, ctypes.c_float(1.0), w_in, w_out, w_cap, None)


def test_weights_refusals(tq):
    assert _weights(tq, B=0) == OK
    assert _weights(tq, T=0, w_cap=0) == OK
    for kw in (dict(B=-1), dict(Hq=0), dict(Hkv=0), dict(N=0), dict(T=-1), dict(T=65), dict(w_cap=63), dict(Hq=5),
               dict(Pn=-1), dict(Pn=9), dict(path=P, Pn=32769), dict(q=0), dict(lse=0), dict(kc=0), dict(ks_=0),
               dict(kz=0), dict(w_out=0), dict(B=1 << 33), dict(cap=1 << 40)):
        assert _weights(tq, **kw) == INVALID, kw
    for D in (0, 100, 1024):
        assert _weights(tq, D=D) == HEAD_DIM
    assert _weights(tq, kb=3, ks=0) == BITS and _weights(tq, kb=2, ks=1) == BITS
    for kw in (dict(q=P + 8), dict(kc=P + 4), dict(ks_=P + 2), dict(kz=P + 8), dict(lse=P + 2), dict(lens=P + 1),
               dict(pad=P + 2), dict(path=P + 3), dict(n_path=P + 1), dict(w_in=P + 2), dict(w_out=P + 1)):
        assert _weights(tq, **kw) == ALIGN, kw


def _select(tq, w=P, B=1, H=2, T=64, w_cap=64, lens=None, pad=None, keep=8, recent=2, index=P, count=P):
    return tq.lib().tq_evict_select(w, B, H, T, w_cap, lens, pad, keep, recent, index, count, None)


def test_select_refusals(tq):
    assert _select(tq, B=0) == OK and _select(tq, H=0) == OK
    for kw in (dict(B=-1), dict(H=-1), dict(T=-1), dict(w_cap=63), dict(keep=-1, recent=-1), dict(recent=-1),
               dict(recent=9), dict(w=0), dict(index=0), dict(count=0), dict(keep=1 << 31), dict(B=1 << 31),
               dict(B=1 << 16, H=1 << 16)):
        assert _select(tq, **kw) == INVALID, kw
    for kw in (dict(w=P + 2), dict(index=P + 1), dict(count=P + 2), dict(lens=P + 1), dict(pad=P + 2)):
        assert _select(tq, **kw) == ALIGN, kw


def _gather(tq, src=None, dst=None, B=1, H=2, D=128, kb=8, vb=3, index=P, n=4, heads=0, count=None, off=None, length=P,
            sw=None, dw=None):
    s = _cache(tq) if src is None else src
    d = _cache(tq) if dst is None else dst
    return tq.lib().tq_cache_gather(ctypes.byref(s), ctypes.byref(d), B, H, D, kb, vb, index, n, heads, count, off,
                                    length, sw, dw, None)


def test_gather_refusals(tq):
    assert _gather(tq, B=0) == OK and _gather(tq, H=0) == OK and _gather(tq, n=0, length=None) == OK
    for kw in (dict(B=-1), dict(H=-1), dict(n=-1), dict(index=0), dict(src=_cache(tq, k_codes=0)),
               dict(dst=_cache(tq, v_scales=0)), dict(src=_cache(tq, -1)), dict(dst=_cache(tq, -1)), dict(sw=P),
               dict(B=1 << 30, H=4), dict(n=1 << 31), dict(src=_cache(tq, 1 << 40)), dict(B=1 << 20, n=1 << 20)):
        assert _gather(tq, **kw) == INVALID, kw
    assert _gather(tq, D=96) == HEAD_DIM
    assert _gather(tq, kb=3) == BITS and _gather(tq, vb=7) == BITS
    for kw in (dict(index=P + 2), dict(count=P + 1), dict(off=P + 2), dict(length=P + 1), dict(sw=P + 2, dw=P),
               dict(sw=P, dw=P + 1), dict(src=_cache(tq, k_codes=P + 8)), dict(dst=_cache(tq, v_codes=P + 4))):
        assert _gather(tq, **kw) == ALIGN, kw
    assert tq.lib().tq_cache_gather(None, None, 1, 2, 128, 8, 3, P, 4, 0, None, None, None, None, None, None) == INVALID


def test_token_counts_that_32_bits_do_not_hold_are_refused(tq):
    """Up to 2^31 - 2^13 tokens a sequence and kept tokens a row: past that the
    kernels' steps would leave 32 bits."""
    far = [P + (i << 40) for i in range(8)]
    for n in ((1 << 31) - (1 << 13) + 1, (1 << 31) - 128, (1 << 31) - 1):
        assert _select(tq, w=far[0], index=far[1], count=far[2], B=1, H=1, keep=n, recent=n) == INVALID, n
        assert _select(tq, w=far[0], index=far[1], count=far[2], B=1, H=1, T=n, w_cap=n) == INVALID, n
        assert _tree(tq, q=far[0], out=far[1], lse=far[2], ws=far[3], Hq=1, Hkv=1, T=n, cache=_cache(tq, n)) == INVALID, n
        assert _weights(tq, q=far[0], lse=far[1], w_out=far[2], Hq=1, Hkv=1, T=n, cap=n, w_cap=n) == INVALID, n


def test_overlaps_are_refused(tq):
    """Arrays that share memory, where the call does not allow it."""
    far = [P + (i << 30) for i in range(16)]
    distinct = dict(q=far[0], out=far[1], lse=far[2], ws=far[3], cache=_cache(tq), tree=_cache(tq, 8))
    for kw in (dict(out=far[0]), dict(out=far[0] + 4 * 8 * 128 * 2 - 16), dict(lse=far[0] + 4), dict(lse=far[1] + 8),
               dict(ws=far[0] - 16), dict(ws=far[1] - 16), dict(ws=far[2] - 16)):
        assert _tree(tq, **dict(distinct, **kw)) == INVALID, kw
    assert _weights(tq, w_in=far[1], w_out=far[1] + 4, q=far[0], lse=far[2]) == INVALID
    assert _weights(tq, w_in=far[1] + 2 * 64 * 4 - 4, w_out=far[1], q=far[0], lse=far[2]) == INVALID
    assert _weights(tq, w_out=far[2] + 4, q=far[0], lse=far[2]) == INVALID
    for kw in (dict(index=far[0]), dict(count=far[0]), dict(count=far[1] + 4), dict(lens=far[2]), dict(pad=far[2]),
               dict(lens=far[1] + 60)):
        assert _select(tq, **dict(dict(w=far[0], index=far[1], count=far[2]), **kw)) == INVALID, kw
    src = _cache(tq, 64, **{n: far[i] for i, n in enumerate(rc.CACHE_KEYS)})
    dst = {n: far[5 + i] for i, n in enumerate(rc.CACHE_KEYS)}
    apart = dict(src=src, dst=_cache(tq, 64, **dst), index=far[10], length=far[11], sw=far[12], dw=far[13])
    for kw in (dict(dst=src), dict(dst=_cache(tq, 64, **dict(dst, v_codes=far[1] + 16))), dict(dw=far[12] + 4),
               dict(off=far[11]), dict(count=far[11]), dict(length=far[10] + 12)):
        assert _gather(tq, **dict(apart, **kw)) == INVALID, kw


def test_every_written_array_is_held_apart(tq):
    """Each array that a call writes against each other one, by one element at
    either end."""
    far = [(i + 1) << 30 for i in range(24)]
    # (argument, bytes) of B = 1, Hq = 4, Hkv = 2, N = 8, T = capacity = 64, D = 128, k8 v3; the tree's capacity is 8
    names = rc.CACHE_KEYS
    X = (128, 8, 8, 48, 8)
    main = {n: far[i] for i, n in enumerate(names)}
    tree = {n: far[5 + i] for i, n in enumerate(names)}
    need = tq.lib().tq_tree_attention_workspace_size(1, 4, 2, 8, 128)
    base = dict(q=far[10], out=far[11], lse=far[12], ws=far[13], parents=far[14], lens=far[15], pad=far[16])
    size = dict(q=4 * 8 * 128 * 2, out=4 * 8 * 128 * 2, lse=4 * 8 * 4, ws=need, parents=8 * 4, lens=4, pad=4)
    reads = [(base[n], size[n]) for n in ("q", "parents", "lens", "pad")]
    reads += [(main[n], 2 * 64 * x) for n, x in zip(names, X)] + [(tree[n], 2 * 8 * x) for n, x in zip(names, X)]
    step = dict(out=16, lse=4, ws=16)

    def ends(at, length, own, step):
        """Places for an array of `own` bytes that share its last or first element with [at, at + length)."""
        return [(at + length - 1) // step * step, -(-(at - own + 1) // step) * step]

    def call(**kw):
        a = dict(base, **kw)
        return _tree(tq, cache=_cache(tq, 64, **main), tree=_cache(tq, 8, **tree), **a)

    for name in ("out", "lse", "ws"):
        for at, length in reads + [(base[n], size[n]) for n in ("out", "lse", "ws") if n != name]:
            for place in ends(at, length, size[name], step[name]):
                assert call(**{name: place}) == INVALID, (name, hex(at), hex(place))
    keys = dict(kc=far[0], ks_=far[1], kz=far[2])
    base_w = dict(keys, q=far[10], lse=far[12], lens=far[15], pad=far[16], path=far[17], n_path=far[18], w_in=far[19])
    sums = 2 * 64 * 4
    for at, length in ((far[0], 2 * 64 * 128), (far[1], 2 * 64 * 8), (far[2], 2 * 64 * 8), (far[10], 4 * 8 * 128 * 2),
                       (far[12], 4 * 8 * 4), (far[15], 4), (far[16], 4), (far[17], 8 * 4), (far[18], 4), (far[19], sums)):
        for place in ends(at, length, sums, 4):
            if place != far[19]:
                assert _weights(tq, w_out=place, **base_w) == INVALID, (hex(at), hex(place))
    dst = dict(tree)
    base_g = dict(index=far[14], length=far[15], sw=far[16], dw=far[17], count=far[18], off=far[19])
    for name, own in [(n, 2 * 64 * x) for n, x in zip(names, X)] + [("dw", 2 * 64 * 4), ("length", 4)]:
        others = [(main[n], 2 * 64 * x) for n, x in zip(names, X)]
        others += [(dst[n], 2 * 64 * x) for n, x in zip(names, X) if n != name]
        others += [(far[14], 4 * 4), (far[16], 2 * 64 * 4), (far[18], 4), (far[19], 4)]
        others += [(base_g[n], b) for n, b in (("dw", 2 * 64 * 4), ("length", 4)) if n != name]
        for at, length in others:
            for place in ends(at, length, own, 16 if name in dst else 4):
                d, g = (dict(dst, **{name: place}), base_g) if name in dst else (dst, dict(base_g, **{name: place}))
                assert _gather(tq, src=_cache(tq, 64, **main), dst=_cache(tq, 64, **d), **g) == INVALID, (name, hex(at))


def test_binding_refuses_wrong_tensors(tq):
    """Shapes, types and devices are checked before the library is called."""
    G = 4
    cache = {"k_codes": torch.zeros((1, 2, 16, 128), dtype=torch.uint8),
             "k_scales": torch.zeros((1, 2, 16, G), dtype=torch.float16),
             "k_zeros": torch.zeros((1, 2, 16, G), dtype=torch.float16),
             "v_codes": torch.zeros((1, 2, 16, 48), dtype=torch.uint8),
             "v_scales": torch.zeros((1, 2, 16, G), dtype=torch.float16)}
    q = torch.zeros((1, 4, 3, 128), dtype=torch.bfloat16)
    lse = torch.zeros((1, 4, 3))
    for bad in (dict(q=q.float()), dict(q=q[..., ::2]), dict(q=q[0]), dict(cache=dict(cache, k_scales=cache["k_scales"].float())),
                dict(cache=dict(cache, v_codes=cache["v_codes"][:, :, :8])), dict(vb=4), dict(out_dtype=torch.float16),
                dict(parents=torch.zeros((1, 3), dtype=torch.int64)), dict(parents=torch.zeros((1, 2), dtype=torch.int32)),
                dict(lens=torch.zeros((2,), dtype=torch.int32)), dict(q=q.expand(2, -1, -1, -1)), dict()):
        a = dict(q=q, cache=cache, vb=3, out_dtype=torch.bfloat16, parents=None, lens=None)
        a.update(bad)
        with pytest.raises(ValueError):  # the last: tensors on the host
            tq.tq_tree_attention(a["q"], a["cache"], 16, cache, 8, True, a["vb"], parents=a["parents"], lens=a["lens"],
                                 out_dtype=a["out_dtype"])
    with pytest.raises(ValueError):
        tq.tq_attention_weights(q, lse, cache, 16, 8, True)
    with pytest.raises(ValueError):
        tq.tq_attention_weights(q.float(), lse, cache, 16, 8, True)
    with pytest.raises(ValueError):
        tq.tq_evict_select(torch.zeros((1, 2, 16)), 16, 4, 1)
    with pytest.raises(ValueError):
        tq.tq_evict_select(torch.zeros((2, 16)), 16, 4, 1)
    with pytest.raises(ValueError):
        tq.tq_cache_gather(cache, cache, torch.zeros((1, 4), dtype=torch.int32))


def test_a_cache_without_room_has_no_weights(tq):
    assert _gather(tq, sw=P, dw=None, dst=_cache(tq, 0), n=0, length=None) == OK
    assert _gather(tq, sw=P, dw=None, dst=_cache(tq, 1), n=0, length=None) == INVALID


def test_cutting_into_less_room_than_the_budget_is_refused(tq):
    """A fresh cache too small for the kept tokens would lose the last of them,
    the recent ones."""
    cache = tq.alloc_cache(1, 2, 16, 64, 8, 3, device="cpu")
    w = torch.zeros((1, 2, 16))
    for keep, T, t_cap in ((8, 16, 7), (8, 16, 0), (12, 10, 9)):
        with pytest.raises(ValueError, match="t_cap"):
            tq.evict_rows(cache, w, T, keep, 2, t_cap=t_cap)
    for keep, T, t_cap in ((8, 16, 8), (12, 10, 10), (8, 16, None)):  # refused for the device alone
        with pytest.raises(ValueError, match="CUDA device"):
            tq.evict_rows(cache, w, T, keep, 2, t_cap=t_cap)


def test_a_stream_of_another_device_is_refused(tq):
    """(It was passed over, and the current stream of the tensors' device taken.)"""
    class Stream:
        device = torch.device("cuda", 1)

    with pytest.raises(ValueError, match="stream"):
        tq._elsewhere(torch.device("cuda", 0), Stream())
    assert tq._elsewhere(torch.device("cuda", 1), Stream()) is True


def test_reference_of_one_token_by_hand():
    """The reference itself: one key alone gives its own value row back, and
    lse is the score."""
    c = rc.random_cache(1, 1, 1, 64, 8, True, 8, 3)
    t = rc.random_cache(1, 1, 1, 64, 8, True, 8, 4)
    q = torch.zeros((1, 1, 1, 64), dtype=torch.bfloat16)
    out, lse, _, _ = rc.tree_reference(q, c, 1, t, 8, True, 8, lens=[0])
    _, v = rc.decoded(t, 1, 8, True, 8)
    assert np.allclose(out[0, 0, 0], v[0, 0, 0] @ rc.rotation(64)) and lse[0, 0, 0] == 0
    out, lse, _, _ = rc.tree_reference(q, c, 1, t, 8, True, 8)
    assert abs(lse[0, 0, 0] - np.log(2)) < 1e-12
    index, count = rc.select_reference(torch.tensor([[[1.0, 5.0, 5.0, 0.0, 2.0]]]), 5, 3, 1)
    assert index.tolist() == [[[1, 2, 4]]] and count.tolist() == [3]
