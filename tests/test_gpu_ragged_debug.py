"""The calls on ragged packed caches in the debug build of the library: every
output equals the release build's byte for byte, and no index check fails (see
test_gpu_debug_checks.py)."""
import numpy as np
import pytest
import torch

import turboquant_kv_cache_tq_gb300 as tq
from tests import ragged_common as rc
from tests.test_gpu_debug_checks import _bytes, _with, libs  # noqa: F401  (libs is a fixture)

pytestmark = pytest.mark.gpu


def _equal(a, b):
    for x, y in zip(a, b):
        assert np.array_equal(_bytes(x), _bytes(y))


@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("N,cap", [(4, 304), (7, 301)])  # bulk copies, narrow copies
def test_attention_and_weights_match_release(libs, D, N, cap):  # noqa: F811
    release, debug = libs
    B, Hkv, G, T = 3, 2, 4, 300
    kb, ks, vb = (8, True, 3) if D < 256 else (5, False, 5)
    main, tree = (rc.to_gpu(rc.random_cache(B, Hkv, n, D, kb, ks, vb, n)) for n in (cap, N))
    g = torch.Generator().manual_seed(D)
    q = torch.randn((B, Hkv * G, N, D), generator=g).to(torch.bfloat16).cuda()
    lens, pad = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([300, 0, 37], [5, 0, 20]))
    for dtype in (torch.bfloat16, torch.float32):
        outs = []
        for L in (release, debug):
            def run():
                out, lse = tq.tq_tree_attention(q, main, T, tree, kb, ks, vb, lens=lens, left_pad=pad, out_dtype=dtype)
                w = tq.tq_attention_weights(q, lse, main, T, kb, ks, lens=lens, left_pad=pad)
                return out, lse, w
            outs.append(_with(L, run))
        _equal(*outs)
    assert debug.tq_device_status(None) == 0 and release.tq_device_status(None) == 0


def test_choice_and_gather_match_release(libs):  # noqa: F811
    release, debug = libs
    B, Hkv, T, D = 3, 2, 5000, 128
    cache = rc.to_gpu(rc.random_cache(B, Hkv, T, D, 8, True, 3, 1))
    score = torch.rand((B, Hkv, T), generator=torch.Generator().manual_seed(2)).cuda()
    lens = torch.tensor([5000, 0, 777], dtype=torch.int32, device="cuda")
    outs = []
    for L in (release, debug):
        def run():
            index, n = tq.tq_evict_select(score, T, 900, 64, lens=lens)
            dst = {k: torch.zeros_like(v) for k, v in tq.alloc_cache(B, Hkv, 1000, D, 8, 3).items()}
            _, length = tq.tq_cache_gather(cache, dst, index, n)
            return [index, n, length] + [dst[k] for k in rc.CACHE_KEYS]
        outs.append(_with(L, run))
    _equal(*outs)
    assert debug.tq_device_status(None) == 0 and release.tq_device_status(None) == 0
