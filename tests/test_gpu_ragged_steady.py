"""GPU tests of the tree attention and the weight sums one call after another."""
import pytest
import torch

import turboquant_kv_cache_tq_gb300 as tq
from tests.gpu_common import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _normal(shape, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).bfloat16()


def _cache(B, H, T, D, kb, ks, vb, seed, cap=None, ramp=None):
    """A packed cache of normal keys (plus ramp [T] in every element, when given) and values."""
    c = tq.alloc_cache(B, H, T if cap is None else cap, D, kb, vb)
    k = _normal((B, H, T, D), seed)
    if ramp is not None:
        k = (k.float() + ramp[:, None]).bfloat16()
    tq.tq_encode_kv(k, _normal((B, H, T, D), seed + 1), kb, ks, vb, c)
    return c


def test_calls_one_after_another():
    """Short calls of both kernels in a row on the same SMs, each the same bits
    as alone: a block's last asynchronous arrivals do not reach the next one's
    shared memory."""
    jobs = []
    for D, T in ((64, 70), (128, 130), (256, 40), (512, 33)):
        B, Hkv, G, N = 19, 8, 2, 4  # a block a segment, one to three tiles
        c, tree, q = _cache(B, Hkv, T, D, 8, True, 3, D), _cache(B, Hkv, N, D, 8, True, 3, D + 1), _normal((B, Hkv * G, N, D), D)
        for dtype in (torch.bfloat16, torch.float32):
            jobs.append(lambda q=q, c=c, T=T, tree=tree, dtype=dtype: tq.tq_tree_attention(q, c, T, tree, 8, True, 3, out_dtype=dtype))
        lse = jobs[-1]()[1]
        jobs.append(lambda q=q, c=c, T=T, lse=lse: (tq.tq_attention_weights(q, lse, c, T, 8, True),))
    alone = []
    for job in jobs:
        torch.cuda.synchronize()
        alone.append(job())
        torch.cuda.synchronize()
    for _ in range(30):
        got = [job() for job in jobs]
    torch.cuda.synchronize()
    assert tq.lib().tq_device_status(None) == 0
    for a, b in zip(alone, got):
        for x, y in zip(a, b):
            assert torch.equal(x, y)
