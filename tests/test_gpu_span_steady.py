"""GPU tests of the window and the shared-prefix attention in their steady state:
enough tiles a block that every ring of stages, barrier parity and running
maximum is gone through many times (test_gpu_span_attention.py has a few tiles a
block), many output rows, and two passes that run side by side."""
import pytest
import torch

import turboquant_kv_cache_tq_gb300 as tq
from tests import step_common as sc
from tests.gpu_common import require_gpu
from tests.test_gpu_span_attention import DTYPES, prefix, window

pytestmark = pytest.mark.gpu
FORMATS = {64: (8, False, 5), 128: (8, True, 8), 256: (4, False, 4), 512: (5, False, 3)}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    yield
    assert tq.lib().tq_device_status(None) == 0


@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("dtype", DTYPES)
def test_many_tiles_a_block_of_128_rows(D, dtype):
    """132 to 160 rows a kv head: two row blocks, each over all tiles."""
    T = 12000 if D <= 128 else 6000
    window(2, 8, 4, 40 if D == 64 else 33, T, D, *FORMATS[D], T, 0, dtype, lens=[T, T - 77], qscale=3.0, offset=0.3)
    window(2, 8, 4, 33, T, D, *FORMATS[D], T // 2, 1000, dtype, lens=[T, T - 77], left_pad=[0, 13])


@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("G,N", [(4, 1), (4, 3)])
def test_many_tiles_a_warp_of_few_rows(D, dtype, G, N):
    B, T = 16, 4000 if D <= 128 else 2000
    lens = [T - 91 * b for b in range(B)]
    window(B, 8, G, N, T, D, *FORMATS[D], T, 0, dtype, lens=lens, qscale=3.0, offset=0.3)
    window(B, 8, G, N, T, D, *FORMATS[D], T // 2, 100, dtype, lens=lens, left_pad=[b for b in range(B)], cap=T + 5)


@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("dtype", DTYPES)
def test_a_long_prefix(D, dtype):
    """Both passes over many tiles a block, side by side and (a capacity that is no multiple of 16) one after the other."""
    for cap in (1024, 1003):
        prefix(2, 20, 8, 4, 1, 5000, 1000, D, *FORMATS[D], dtype, prefix_lens=[5000, 4321],
               lens=[1000 - 20 * b for b in range(40)], cap=cap, qscale=3.0)


@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("dtype", DTYPES)
def test_many_rows(D, dtype):
    """More output rows than two waves of warps."""
    window(2, 4, 4, 300, 700, D, *FORMATS[D], 200, 5, dtype, lens=[700, 333], count=[300, 290])
    prefix(1, 2, 4, 4, 290, 100, 300, D, *FORMATS[D], dtype)


def test_a_short_prefix_beside_the_sequences():
    """A prefix that leaves SMs for the second pass, in a graph, called again and again: the second pass must not read what
    an append has not written yet, nor the combine what the first pass has not."""
    S, Hkv, G, P, cap, D = 8, 8, 4, 4096, 256, 128
    Hq = Hkv * G
    pre, cache = sc.cache(1, Hkv, P, D, 8, True, 3, 1), tq.alloc_cache(S, Hkv, cap, D, 8, 3)
    lens, new = sc.ints([0] * S), sc.ints([0] * S)
    x = torch.empty((S, 1, Hq + 2 * Hkv, D), dtype=torch.bfloat16, device="cuda")
    q = torch.empty((S, Hq, 1, D), dtype=torch.bfloat16, device="cuda")

    def step():
        y = x.transpose(1, 2)
        tq.tq_append_kv(y[:, Hq:Hq + Hkv], y[:, Hq + Hkv:], cache, lens, 8, True, 3, q=y[:, :Hq], q_out=q, new_lens=new)
        out = tq.tq_prefix_attention(q, pre, P, cache, cap, 8, True, 3, lens=new)
        lens.copy_(new)
        return out

    step()
    lens.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = step()
    lens.zero_()
    for i in range(40):
        x.copy_(sc.normal(x.shape, i))
        graph.replay()
        if i % 13 == 12 or i < 3:
            n = [i + 1] * S
            assert lens.tolist() == n
            sc.check(out, lse, sc.reference(q, cache, cap, 8, True, 3, n, prefix=pre, P=P, dtype=torch.bfloat16), "step %d" % i)


@pytest.mark.parametrize("N", [1, 20, 150])
def test_offsets_past_32_bits(N):
    """Keys and values of 4.5 GB each: the last tokens of the last head are appended and attended to beyond 2^32 bytes."""
    Hkv, G, D, cap, n = 8, 2, 512, 1_100_000, 256
    at = cap - n
    big, small = tq.alloc_cache(1, Hkv, cap, D, 8, 8), tq.alloc_cache(1, Hkv, n, D, 8, 8)
    k, v = sc.normal((1, Hkv, n, D), 1), sc.normal((1, Hkv, n, D), 2)
    assert big["k_codes"].numel() > 2 ** 32
    _, new = tq.tq_append_kv(k, v, big, sc.ints([at]), 8, True, 8)
    tq.tq_append_kv(k, v, small, None, 8, True, 8)
    assert new.tolist() == [cap]
    for name in big:
        assert torch.equal(big[name][:, :, at:], small[name]) and not big[name][:, :, :at].any()
    q = sc.normal((1, Hkv * G, N, D), 3)
    ref = sc.reference(q, small, n, 8, True, 8, window=100, dtype=torch.float32)
    out, lse = tq.tq_window_attention(q, big, cap, 8, True, 8, 100, out_dtype=torch.float32)
    sc.check(out, lse, ref, "window")
