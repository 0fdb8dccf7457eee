"""GPU tests of tq_window_attention and tq_prefix_attention against references in
64 bits."""
import math

import numpy as np
import pytest
import torch

import turboquant_kv_cache_tq_gb300 as tq
from tests import step_common as sc
from tests.gpu_common import require_gpu

pytestmark = pytest.mark.gpu
MODES = [(2, False, 2), (4, False, 3), (5, False, 4), (8, False, 5), (8, True, 8)]
DTYPES = [torch.bfloat16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    yield
    assert tq.lib().tq_device_status(None) == 0


def _twice(call, need):
    """The outputs of a call; whatever the workspace and the outputs held, the same bits come."""
    got = []
    for fill in (0x00, 0xFF):
        got.append(call(torch.full((max(need, 16),), fill, dtype=torch.uint8, device="cuda")))
    for a, b in zip(*got):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    return got[0]


def window(B, Hkv, G, N, T, D, kb, ks, vb, win, sinks, dtype=torch.bfloat16, lens=None, left_pad=None, count=None,
           cap=None, seed=0, qscale=1.0, scale=None, edit=None, offset=0.0):
    c = sc.cache(B, Hkv, T, D, kb, ks, vb, seed, cap, offset)
    if edit is not None:
        edit(c)
    q = sc.normal((B, Hkv * G, N, D), seed + 5, qscale)
    args = dict(lens=sc.ints(lens), left_pad=sc.ints(left_pad), count=sc.ints(count), scale=scale, out_dtype=dtype)
    out, lse = _twice(lambda ws: tq.tq_window_attention(q, c, T, kb, ks, vb, win, sinks=sinks, workspace=ws, **args),
                      tq.tq_window_attention_workspace_size(B, Hkv * G, Hkv, N, D))
    ref = sc.reference(q, c, T, kb, ks, vb, lens, left_pad, count, win, sinks, scale, dtype=dtype)
    sc.check(out, lse, ref, "window")
    return out, lse, q, c


def prefix(Bp, S, Hkv, G, N, P, T, D, kb, ks, vb, dtype=torch.bfloat16, prefix_lens=None, lens=None, left_pad=None,
           count=None, cap=None, pcap=None, seed=0, qscale=1.0, scale=None, edit=None):
    B = Bp * S
    pre = sc.cache(Bp, Hkv, P, D, kb, ks, vb, seed, pcap)
    c = sc.cache(B, Hkv, T, D, kb, ks, vb, seed + 2, cap)
    if edit is not None:
        edit(pre, c)
    q = sc.normal((B, Hkv * G, N, D), seed + 5, qscale)
    args = dict(prefix_lens=sc.ints(prefix_lens), lens=sc.ints(lens), left_pad=sc.ints(left_pad), count=sc.ints(count),
                scale=scale, out_dtype=dtype)
    out, lse = _twice(lambda ws: tq.tq_prefix_attention(q, pre, P, c, T, kb, ks, vb, workspace=ws, **args),
                      tq.tq_prefix_attention_workspace_size(Bp, B, Hkv * G, Hkv, N, D))
    ref = sc.reference(q, c, T, kb, ks, vb, lens, left_pad, count, scale=scale, prefix=pre, P=P, prefix_lens=prefix_lens,
                       dtype=dtype)
    sc.check(out, lse, ref, "prefix")
    return out, lse


# ---- window ---------------------------------------------------------------------------
@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("kb,ks,vb", MODES)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N", [1, 5, 40])
def test_window_every_format(D, kb, ks, vb, dtype, N):
    window(2, 2, 4, N, 333, D, kb, ks, vb, 100, 3, dtype, lens=[333, 170], cap=336)


@pytest.mark.parametrize("win,sinks", [(1, 0), (1, 1), (1, 40), (7, 0), (16, 16), (17, 5), (64, 64), (65, 63), (128, 4),
                                       (299, 1), (300, 0), (10 ** 9, 0), (2 ** 40, 2 ** 40), (3, 299), (3, 1000)])
@pytest.mark.parametrize("N", [1, 3, 33, 140])
def test_window_shapes(win, sinks, N):
    window(3, 1, 3, N, 300, 128, 8, True, 3, win, sinks, torch.float32, lens=[300, 133, 64], left_pad=[0, 17, 60])


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257])
@pytest.mark.parametrize("D", [64, 128, 512])
def test_window_lengths(T, D):
    window(2, 2, 2, 1, T, D, 8, True, 8, 50, 2, lens=[T, (T + 1) // 2])
    window(1, 2, 2, min(T, 20), T, D, 8, True, 3, 50, 2)


@pytest.mark.parametrize("G,N", [(1, 1), (2, 1), (3, 2), (8, 1), (8, 2), (16, 1), (5, 3), (1, 16), (1, 17), (17, 1), (4, 16),
                                 (2, 32), (4, 17), (4, 32), (3, 43), (1, 129), (2, 200), (7, 37)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_window_rows(G, N, dtype):
    window(2, 2, G, N, 260, 128, 8, True, 3, 70, 5, dtype, lens=[260, 77])
    window(1, 1, G, N, 260, 256, 5, False, 5, 70, 5, dtype)


def test_window_empty_rows():
    """No tokens, fewer tokens than new ones, no new tokens, pads past the end."""
    for N in (1, 4, 50, 150):
        window(7, 2, 2, N, 90, 128, 8, True, 3, 20, 2, torch.float32, lens=[0, 1, 3, 90, 90, -5, 1000],
               left_pad=[0, 0, 2, 90, 89, 3, 200], count=[N, N, N, N, N, N, N])
        window(6, 2, 2, N, 90, 128, 8, True, 3, 20, 2, lens=[90, 90, 40, 40, 0, 1], count=[0, 1, -3, 1000, 0, N])
    assert window(2, 1, 1, 1, 0, 64, 8, True, 3, 5, 1, cap=0)[1].isneginf().all()
    out, lse = tq.tq_window_attention(sc.normal((0, 4, 1, 64), 1), tq.alloc_cache(0, 2, 8, 64, 8, 3), 8, 8, True, 3, 4)
    assert out.shape == (0, 4, 1, 64) and lse.shape == (0, 4, 1)


@pytest.mark.parametrize("cap", [301, 302, 304, 308, 320, 10000])
@pytest.mark.parametrize("D", [64, 128, 256, 512])
def test_window_capacities(cap, D):
    """Capacities that break the rows' alignment, and T far below the capacity."""
    for N in (1, 30, 70):
        window(2, 3, 2, N, 301, D, 2 if D == 64 else 5, False, 5 if D == 64 else 2, 100, 4, lens=[301, 150], cap=cap)


def test_window_scales():
    for N in (2, 20, 140):
        for scale in (-0.2, 0.0, 3.0):
            window(2, 2, 2, N, 200, 128, 8, True, 8, 60, 3, torch.float32, scale=scale, lens=[200, 9])


def test_window_large_scores():
    """Scores in the hundreds, whose maximum rises along the sequence."""
    for N in (1, 20, 40):
        window(1, 2, 4, N, 2000, 128, 8, True, 8, 1500, 4, torch.float32, qscale=30.0)
        window(1, 2, 4, N, 2000, 64, 8, False, 3, 5000, 0, qscale=30.0, offset=2.0)


def _poison(tokens, what):
    def edit(c):
        for b, h, t in tokens:
            if what == "value":
                c["v_scales"][b, h, t, 0] = math.inf
            elif what == "value nan":
                c["v_scales"][b, h, t, 1] = math.nan
            elif what == "key":
                c["k_scales"][b, h, t, 0] = math.nan
            else:
                c["k_zeros"][b, h, t, 1] = math.inf
    return edit


@pytest.mark.parametrize("what", ["value", "value nan", "key", "zero point"])
@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("dtype", DTYPES)
def test_window_bad_tokens(what, D, dtype):
    """Tokens that decode to NaN or infinities reach the rows that see them, and no other."""
    for N, G in ((1, 4), (4, 2), (30, 3), (70, 2)):
        T, win = 300, 60
        first = T - N
        tokens = [(0, 0, first - win + 1), (0, 1, 100), (1, 0, 5), (1, 1, 2), (2, 0, first - win + (N + 1) // 2), (2, 1, T - 1)]
        out, lse, _, _ = window(3, 2, G, N, T, D, 8, False, 8, win, 4, dtype, edit=_poison(tokens, what))
        assert not lse.isnan().all() and lse.isnan().any()


def test_window_queries_of_their_own_values():
    """A query of zeros weighs its tokens equally; one with an infinity spoils its own row only."""
    c = sc.cache(1, 1, 50, 128, 8, True, 8, 3)
    for N in (2, 20, 90):
        q = sc.normal((1, 2, N, 128), 1)
        q[0, 0, 0] = 0
        q[0, 1, 1, 7] = math.inf
        out, lse = tq.tq_window_attention(q, c, 50, 8, True, 8, 10, out_dtype=torch.float32)
        assert N > 50 or abs(lse[0, 0, 0].item() - math.log(10)) < 1e-6
        nan = out.isnan().any(-1)
        if N > 50:  # (its last 50 new tokens are all that the sequence has)
            assert not nan.any() and (lse[0, :, :N - 50] == -math.inf).all()
        else:
            assert nan[0, 1, 1] and nan.sum() == 1 and lse.isnan().sum() == 1


def test_window_many_sequences():
    r = np.random.RandomState(0)
    B = 100
    lens = r.randint(0, 400, B).tolist()
    pad = [int(n * r.rand() * 0.7) for n in lens]
    window(B, 2, 4, 1, 400, 128, 8, True, 3, 90, 4, lens=lens, left_pad=pad)
    window(B, 1, 4, 9, 400, 64, 4, False, 4, 90, 4, lens=lens, left_pad=pad, count=r.randint(0, 10, B).tolist())


def test_window_long_sequences():
    window(1, 1, 2, 1, 70000, 64, 8, True, 3, 10 ** 6, 0, torch.float32)
    window(1, 1, 2, 20, 30000, 128, 8, True, 8, 20000, 100, torch.float32)
    window(2, 1, 1, 1, 30000, 512, 5, False, 2, 9000, 30, lens=[30000, 9100])


# ---- prefix ---------------------------------------------------------------------------
@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("kb,ks,vb", MODES)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("S,N", [(2, 1), (9, 1), (5, 6)])
def test_prefix_every_format(D, kb, ks, vb, dtype, S, N):
    prefix(2, S, 2, 4, N, 200, 40, D, kb, ks, vb, dtype, prefix_lens=[200, 77], lens=[40 - i for i in range(2 * S)])


@pytest.mark.parametrize("P", [0, 1, 15, 16, 17, 63, 64, 65, 129, 1000])
@pytest.mark.parametrize("T", [1, 16, 65, 200])
def test_prefix_lengths(P, T):
    prefix(1, 3, 2, 2, 1, P, T, 128, 8, True, 3, torch.float32, lens=[T, max(T - 1, 1), (T + 1) // 2])
    prefix(1, 40, 1, 2, 1, P, T, 64, 8, True, 8)


@pytest.mark.parametrize("S,G,N", [(1, 1, 1), (1, 16, 1), (1, 17, 1), (16, 1, 1), (17, 1, 1), (2, 8, 1), (4, 4, 1), (4, 5, 1),
                                   (3, 4, 11), (64, 4, 1), (33, 4, 1), (2, 3, 50), (130, 1, 1), (12, 8, 3)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_prefix_rows(S, G, N, dtype):
    prefix(2, S, 1, G, N, 300, 60, 128, 8, True, 3, dtype, prefix_lens=[300, 250])
    prefix(1, S, 2, G, N, 150, 60, 512, 4, False, 5, dtype)


def test_prefix_empty_rows():
    for N in (1, 30, 80):
        # no own tokens but the new one, none at all, no prefix, neither
        prefix(2, 4, 2, 2, N, 100, 40, 128, 8, True, 3, torch.float32, prefix_lens=[100, 0],
               lens=[40, 1, 0, 20, 40, 1, 0, 20], left_pad=[0, 0, 0, 20, 0, 0, 0, 20])
        prefix(3, 2, 2, 2, N, 100, 40, 128, 8, True, 3, prefix_lens=[-4, 1000, 1], lens=[40, 30, 20, 10, -1, 50],
               count=[N, 0, 1, N, -2, 100], left_pad=[3, 0, 0, 2, 0, 39])
    prefix(1, 2, 1, 2, 1, 0, 30, 64, 8, True, 3, pcap=0)
    prefix(1, 2, 1, 2, 1, 30, 0, 64, 8, True, 3, cap=0)


@pytest.mark.parametrize("cap,pcap", [(61, 201), (62, 202), (64, 208), (500, 9000)])
@pytest.mark.parametrize("D", [64, 128, 256, 512])
def test_prefix_capacities(cap, pcap, D):
    prefix(2, 5, 2, 2, 1, 200, 61, D, 5, False, 3, prefix_lens=[200, 90], cap=cap, pcap=pcap)
    prefix(2, 2, 2, 2, 12, 200, 61, D, 2, False, 2, prefix_lens=[200, 90], cap=cap, pcap=pcap)
    prefix(2, 2, 2, 2, 50, 200, 61, D, 4, False, 4, prefix_lens=[200, 90], cap=cap, pcap=pcap)


def test_prefix_scales_and_large_scores():
    for S in (2, 12, 100):
        for scale in (-0.2, 0.0, 3.0):
            prefix(1, S, 2, 2, 1, 200, 60, 128, 8, True, 8, torch.float32, scale=scale)
        prefix(1, S, 2, 4, 1, 3000, 500, 128, 8, True, 8, torch.float32, qscale=30.0)


@pytest.mark.parametrize("what", ["value", "value nan", "key", "zero point"])
@pytest.mark.parametrize("D", [64, 128, 512])
def test_prefix_bad_tokens(what, D):
    for S, N in ((3, 1), (20, 1), (3, 9), (70, 1)):
        def edit(pre, c):
            _poison([(1, 0, 10), (0, 1, 70)], what)(pre)  # (70: behind prefix 0's end)
            _poison([(1, 1, 20), (2, 0, 0)], what)(c)
        prefix(2, S, 2, 2, N, 100, 30, D, 8, False, 8, prefix_lens=[70, 100], edit=edit,
               lens=[21 if b == 1 else 30 for b in range(2 * S)])


def test_prefix_equals_one_sequence():
    """A prefix and its continuation give what attention over both in one cache gives."""
    S, Hkv, G, P, T, D = 6, 2, 4, 500, 50, 128
    pre, own = sc.cache(1, Hkv, P, D, 8, True, 8, 1), sc.cache(S, Hkv, T, D, 8, True, 8, 3)
    whole = tq.alloc_cache(S, Hkv, P + T, D, 8, 8)
    for name in whole:
        whole[name][:, :, :P], whole[name][:, :, P:] = pre[name], own[name]
    q = sc.normal((S, Hkv * G, 1, D), 5)
    a, la = tq.tq_prefix_attention(q, pre, P, own, T, 8, True, 8, out_dtype=torch.float32)
    ref = sc.reference(q, whole, P + T, 8, True, 8)
    sc.check(a, la, ref)
    b, lb = tq.tq_window_attention(q, whole, P + T, 8, True, 8, P + T, out_dtype=torch.float32)
    sc.check(b, lb, ref)


# ---- together -------------------------------------------------------------------------
def test_steps_of_a_layer_in_a_graph():
    """Prompt, then single tokens: append and attend, eager and as one captured step, over a window and over a shared
    prefix; against references over the bytes that the cache then holds."""
    B, Hkv, G, D, cap, win, sinks = 4, 2, 4, 128, 200, 50, 4
    Hq = Hkv * G
    cos, sin = tq.rope_tables(D, 1000, scaling="bands", factor=8.0, original=256)
    pre = sc.cache(1, Hkv, 300, D, 8, True, 8, 90)
    cache = tq.alloc_cache(B, Hkv, cap, D, 8, 8)
    lens = sc.ints([0, 0, 0, 0])
    prompt = sc.normal((B, 60, Hq + 2 * Hkv, D), 1).transpose(1, 2)
    count = [60, 35, 1, 0]
    q, new = tq.tq_append_kv(prompt[:, Hq:Hq + Hkv], prompt[:, Hq + Hkv:], cache, lens, 8, True, 8, cos=cos, sin=sin,
                             q=prompt[:, :Hq], count=sc.ints(count))
    assert new.tolist() == count
    out, lse = tq.tq_window_attention(q, cache, cap, 8, True, 8, win, sinks=sinks, lens=new, count=sc.ints(count))
    sc.check(out, lse, sc.reference(q, cache, cap, 8, True, 8, count, None, count, win, sinks, dtype=torch.bfloat16))
    lens.copy_(new)
    token = sc.normal((B, 1, Hq + 2 * Hkv, D), 2)
    new = torch.empty_like(lens)
    q_out = torch.empty((B, Hq, 1, D), dtype=torch.bfloat16, device="cuda")

    def step():
        x = token.transpose(1, 2)
        tq.tq_append_kv(x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], cache, lens, 8, True, 8, cos=cos, sin=sin, q=x[:, :Hq],
                        q_out=q_out, new_lens=new)
        a = tq.tq_window_attention(q_out, cache, cap, 8, True, 8, win, sinks=sinks, lens=new)
        b = tq.tq_prefix_attention(q_out, pre, 300, cache, cap, 8, True, 8, lens=new)
        lens.copy_(new)
        return a, b

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a, b = step()
    for i in range(6):
        token.copy_(sc.normal(token.shape, 10 + i))
        graph.replay()
        at = lens.tolist()
        assert at == [n + 2 + i for n in count]
        sc.check(*a, sc.reference(q_out, cache, cap, 8, True, 8, at, window=win, sinks=sinks, dtype=torch.bfloat16))
        sc.check(*b, sc.reference(q_out, cache, cap, 8, True, 8, at, prefix=pre, P=300, dtype=torch.bfloat16))


def test_another_stream_and_two_calls_at_once():
    c, pre = sc.cache(3, 2, 400, 128, 8, True, 8, 1), sc.cache(1, 2, 400, 128, 8, True, 8, 5)
    qs = [sc.normal((3, 8, n, 128), n) for n in (1, 40)]
    want = [(tq.tq_window_attention(q, c, 400, 8, True, 8, 100), tq.tq_prefix_attention(q, pre, 400, c, 400, 8, True, 8))
            for q in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [(tq.tq_window_attention(q, c, 400, 8, True, 8, 100, stream=s),
                tq.tq_prefix_attention(q, pre, 400, c, 400, 8, True, 8, stream=s)) for q, s in zip(qs, streams)]
        torch.cuda.synchronize()
        for w, g in zip(want, got):
            for x, y in zip(w, g):
                assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


def test_outputs_and_workspaces_that_are_given():
    c, pre = sc.cache(2, 2, 100, 128, 8, True, 8, 1), sc.cache(1, 2, 90, 128, 8, True, 8, 5)
    q = sc.normal((2, 8, 3, 128), 1)
    for call, need in (
            (lambda **kw: tq.tq_window_attention(q, c, 100, 8, True, 8, 30, **kw),
             tq.tq_window_attention_workspace_size(2, 8, 2, 3, 128)),
            (lambda **kw: tq.tq_prefix_attention(q, pre, 90, c, 100, 8, True, 8, **kw),
             tq.tq_prefix_attention_workspace_size(1, 2, 8, 2, 3, 128))):
        want, log = call()
        out, lse = torch.full_like(q, 7.0), torch.full((2, 8, 3), 7.0, device="cuda")
        got = call(out=out, lse=lse, workspace=torch.empty(need, dtype=torch.uint8, device="cuda"))
        assert got[0] is out and got[1] is lse and torch.equal(out, want) and torch.equal(lse, log)
        with pytest.raises(tq.TQError):
            call(workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
        for bad in (dict(out=out.float()), dict(out=out[:1]), dict(lse=lse.double()), dict(lse=lse[..., :1]),
                    dict(workspace=torch.empty(need, dtype=torch.uint8)), dict(lens=sc.ints([1, 2, 3])),
                    dict(count=sc.ints([1, 2]).long()), dict(left_pad=sc.ints([1, 2], "cpu"))):
            with pytest.raises(ValueError):
                call(**bad)
    assert (out == want).all()  # (what was refused wrote nothing)
