"""GPU tests of tq_append_kv: the bytes of the turned, quantised tokens, where
they go, and everything else left as it was."""
import numpy as np
import pytest
import torch

import oracle
import turboquant_kv_cache_tq_gb300 as tq
from tests import step_common as sc
from tests.gpu_common import cache_to_numpy, compare_encoded, require_gpu

pytestmark = pytest.mark.gpu
MODES = [(2, False, 2), (4, False, 3), (5, False, 4), (8, False, 5), (8, True, 8)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _garbage(B, H, cap, D, kb, vb):
    c = tq.alloc_cache(B, H, cap, D, kb, vb)
    g = torch.Generator(device="cuda").manual_seed(7)
    for t in c.values():
        u = t.view(torch.uint8)
        u.copy_(torch.randint(0, 256, u.shape, generator=g, device="cuda", dtype=torch.uint8))
    return c


def check(B, Hkv, Hq, N, D, kb, ks, vb, R, dtype=torch.bfloat16, interleaved=False, cap=40, lens=None, left_pad=None,
          count=None, positions=None, length=64, with_q=True, fused=False, seed=0, scale=1.0):
    if fused:
        x = sc.normal((B, N, Hq + 2 * Hkv, D), seed, scale, dtype).transpose(1, 2)
        q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    else:
        q, k, v = (sc.normal((B, h, N, D), seed + i, scale, dtype) for i, h in enumerate((Hq, Hkv, Hkv)))
    q = q if with_q else None
    cos, sin = tq.rope_tables(R, length) if R else (None, None)
    cache = _garbage(B, Hkv, cap, D, kb, vb)
    after, qt, want = sc.append_reference(k, v, cache, lens, kb, ks, vb, cos, sin, interleaved, q, positions, left_pad, count)
    got_q, got = tq.tq_append_kv(k, v, cache, sc.ints(lens), kb, ks, vb, cos=cos, sin=sin, interleaved=interleaved, q=q,
                                 positions=sc.ints(positions), left_pad=sc.ints(left_pad), count=sc.ints(count))
    assert got.tolist() == want
    assert sc.same_bytes(cache, after)
    if with_q:
        assert got_q.dtype == dtype and torch.equal(got_q.cpu(), qt.to(dtype))
    else:
        assert got_q is None
    return cache


@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("kb,ks,vb", MODES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_every_format(D, kb, ks, vb, dtype):
    check(3, 2, 6, 5, D, kb, ks, vb, D, dtype, lens=[0, 7, 35], interleaved=kb == 5)


@pytest.mark.parametrize("D,R", [(64, 2), (64, 10), (64, 32), (64, 62), (128, 64), (128, 96), (128, 32), (256, 64), (256, 18),
                                 (512, 128), (512, 320), (512, 510), (128, 0)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_a_part_of_the_row(D, R, interleaved):
    check(2, 1, 3, 4, D, 8, True, 3, R, interleaved=interleaved, lens=[3, 9])
    check(2, 1, 3, 4, D, 4, False, 4, R, torch.float32, interleaved=interleaved, lens=[3, 9], fused=True)


@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("with_q", [False, True])
def test_strides_and_missing_queries(fused, with_q):
    check(5, 3, 6, 9, 128, 8, True, 3, 128, fused=fused, with_q=with_q, lens=[0, 1, 2, 30, 31])


def test_one_token_and_many():
    check(1, 1, 1, 1, 64, 8, True, 3, 64)
    check(70, 2, 4, 1, 128, 8, True, 3, 128, cap=8, lens=list(range(-3, 67)))
    check(2, 3, 3, 1337, 64, 5, False, 5, 64, cap=1400, lens=[11, 63], length=1400)


def test_ends_of_rows_and_counts():
    """Full rows, rows that fill up, no new tokens, clamped counts and lengths."""
    check(6, 2, 2, 6, 128, 8, True, 8, 128, cap=20, lens=[20, 17, 19, 5, -4, 500], count=[6, 6, 9, 0, -1, 2])
    check(2, 2, 2, 6, 128, 8, True, 8, 128, cap=20)  # (no lengths: the start)
    check(2, 2, 2, 0, 128, 8, True, 8, 128, cap=20, lens=[3, 25])
    check(1, 2, 2, 3, 64, 8, True, 8, 64, cap=0, lens=[0])
    q, n = tq.tq_append_kv(*(sc.normal((0, 2, 3, 64), 1) for _ in range(2)), tq.alloc_cache(0, 2, 8, 64, 8, 3), None, 8, True, 3)
    assert q is None and n.shape == (0,)


def test_positions():
    """Left pads shift them, own ones replace them, the ends of the table hold."""
    check(3, 2, 4, 5, 128, 8, True, 3, 128, lens=[10, 20, 30], left_pad=[4, 25, -3])
    check(3, 2, 4, 5, 128, 8, True, 3, 128, lens=[10, 20, 30], length=12)
    check(2, 2, 4, 3, 128, 8, True, 3, 64, lens=[10, 20], positions=[[5, -7, 63], [1 << 30, 64, 0]])


def test_lengths_near_the_largest_number():
    check(2, 1, 1, 3, 64, 8, True, 3, 64, lens=[2 ** 31 - 1, 2 ** 31 - 2], cap=8)


def test_the_oracle_gives_the_same_bytes():
    """Against the CPU oracle itself, not against this library's encode."""
    B, H, N, D, kb, ks, vb = 2, 3, 17, 128, 8, True, 5
    k, v = sc.normal((B, H, N, D), 1), sc.normal((B, H, N, D), 2)
    cos, sin = tq.rope_tables(D, 64)
    cache = tq.alloc_cache(B, H, N, D, kb, vb)
    tq.tq_append_kv(k, v, cache, None, kb, ks, vb, cos=cos, sin=sin)
    at = np.tile(np.arange(N), (B, 1))
    vf = v.float().cpu().numpy()
    ref = oracle.encode_kv(sc.turned(k, cos, sin, at, False), vf, kb, ks, vb)
    compare_encoded(cache_to_numpy(cache), ref, D, vb, v_input=vf.reshape(-1, D))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_infinities_zeros_and_constant_rows(dtype):
    B, H, N, D = 1, 2, 6, 128
    k, v = sc.normal((B, H, N, D), 1, dtype=dtype), sc.normal((B, H, N, D), 2, dtype=dtype)
    k[0, 0, 0] = 0
    k[0, 0, 1] = 1.5
    k[0, 0, 2, 5] = float("inf")
    k[0, 1, 3, 70] = float("nan")
    v[0, 0, 0] = 0
    v[0, 1, 2, 9] = float("-inf")
    v[0, 1, 4, 9] = float("nan")
    k[0, 1, 5] *= 1e30
    for R in (0, 32, 128):
        cos, sin = tq.rope_tables(R, 64) if R else (None, None)
        cache = _garbage(B, H, N, D, 8, 8)
        after, _, _ = sc.append_reference(k, v, cache, None, 8, True, 8, cos, sin)
        tq.tq_append_kv(k, v, cache, None, 8, True, 8, cos=cos, sin=sin)
        got, want = cache_to_numpy(cache), cache_to_numpy(after)
        compare_encoded(got, want, D, 8, v_input=np.zeros((B * H * N, D), np.float32))


def test_broadcast_rows():
    """Zero strides: every head and token gets the same row."""
    k = sc.normal((1, 1, 1, 64), 1).expand(2, 3, 4, 64)
    v = sc.normal((1, 1, 1, 64), 2).expand(2, 3, 4, 64)
    cache = tq.alloc_cache(2, 3, 8, 64, 8, 3)
    tq.tq_append_kv(k, v, cache, sc.ints([0, 2]), 8, True, 3)
    want = tq.alloc_cache(2, 3, 4, 64, 8, 3)
    tq.tq_encode_kv(k.contiguous(), v.contiguous(), 8, True, 3, want)
    for name in cache:
        assert torch.equal(cache[name][0, :, :4], want[name][0]) and torch.equal(cache[name][1, :, 2:6], want[name][1])


def test_on_another_stream_and_in_a_graph():
    B, H, N, D = 4, 2, 3, 128
    q, k, v = (sc.normal((B, h, N, D), i) for i, h in enumerate((4, H, H)))
    cos, sin = tq.rope_tables(D, 256)
    cache = tq.alloc_cache(B, H, 64, D, 8, 3)
    lens, new = sc.ints([0, 5, 9, 1]), torch.empty(B, dtype=torch.int32, device="cuda")
    q_out = torch.empty_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    tq.tq_append_kv(k, v, cache, lens, 8, True, 3, cos=cos, sin=sin, q=q, q_out=q_out, new_lens=new, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert new.tolist() == [3, 8, 12, 4]
    want = {n: t.clone() for n, t in cache.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tq.tq_append_kv(k, v, cache, lens, 8, True, 3, cos=cos, sin=sin, q=q, q_out=q_out, new_lens=new)
        lens.copy_(new)
    for step in range(5):  # five tokens groups more, each at the end of the last
        before = lens.tolist()
        after, qt, n = sc.append_reference(k, v, want, before, 8, True, 3, cos, sin, False, q)
        graph.replay()
        assert lens.tolist() == n and sc.same_bytes(cache, after) and torch.equal(q_out.cpu(), qt.bfloat16())
        want = after


def test_what_is_refused_writes_nothing():
    B, H, N, D = 2, 2, 3, 64
    k, v, q = (sc.normal((B, h, N, D), i) for i, h in enumerate((H, H, 4)))
    cos, sin = tq.rope_tables(D, 16)
    cache = _garbage(B, H, 10, D, 8, 3)
    before = {n: t.clone() for n, t in cache.items()}
    lens = sc.ints([0, 4])
    for bad in (dict(q=q[:, :, :2]), dict(q=q.float()), dict(q_out=torch.empty_like(q)), dict(cos=cos), dict(cos=cos[0], sin=sin[0]),
                dict(cos=cos, sin=sin[:8]), dict(cos=cos.double(), sin=sin.double()), dict(count=sc.ints([1])),
                dict(positions=sc.ints([0, 1])), dict(left_pad=sc.ints([1, 1], "cpu")), dict(new_lens=lens.float())):
        with pytest.raises(ValueError):
            tq.tq_append_kv(k, v, cache, lens, 8, True, 3, **bad)
    for bad in (dict(new_lens=lens), dict(q=q, q_out=q), dict(cos=torch.ones((4, 33), device="cuda"), sin=torch.ones((4, 33), device="cuda"))):
        with pytest.raises(tq.TQError):
            tq.tq_append_kv(k, v, cache, lens, 8, True, 3, **bad)
    odd = torch.empty((B, H, N, D + 4), dtype=torch.bfloat16, device="cuda")[..., :D]
    with pytest.raises(tq.TQError):  # (rows 136 bytes apart)
        tq.tq_append_kv(odd, v, cache, lens, 8, True, 3)
    torch.cuda.synchronize()
    assert sc.same_bytes(cache, before) and lens.tolist() == [0, 4]
