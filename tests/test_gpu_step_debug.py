"""The calls on new tokens in the debug build of the library: every output equals
the release build's byte for byte, and no index check fails (see
test_gpu_debug_checks.py)."""
import numpy as np
import pytest
import torch

import turboquant_kv_cache_tq_gb300 as tq
from tests import step_common as sc
from tests.test_gpu_debug_checks import _bytes, _with, libs  # noqa: F401  (libs is a fixture)

pytestmark = pytest.mark.gpu


def _same(release, debug, run):
    a, b = _with(release, run), _with(debug, run)
    for x, y in zip(a, b):
        assert np.array_equal(_bytes(x), _bytes(y))


@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("N,cap", [(1, 304), (3, 301), (40, 304), (40, 301)])
def test_attention_matches_release(libs, D, N, cap):  # noqa: F811
    release, debug = libs
    B, Hkv, G, T, P = 4, 2, 4, 300, 200
    kb, ks, vb = (8, True, 3) if D < 256 else (5, False, 5)
    cache, pre = sc.cache(B, Hkv, T, D, kb, ks, vb, 1, cap), sc.cache(2, Hkv, P, D, kb, ks, vb, 5, cap - 100)
    q = sc.normal((B, Hkv * G, N, D), 9)
    lens, pad, count, plens = (sc.ints(x) for x in ([300, 0, 37, 299], [5, 0, 20, 0], [N, N, 1, N], [200, 33]))
    for dtype in (torch.bfloat16, torch.float32):
        _same(release, debug, lambda: tq.tq_window_attention(q, cache, T, kb, ks, vb, 50, sinks=3, lens=lens, left_pad=pad,
                                                             count=count, out_dtype=dtype))
        _same(release, debug, lambda: tq.tq_prefix_attention(q, pre, P, cache, T, kb, ks, vb, prefix_lens=plens, lens=lens,
                                                             left_pad=pad, count=count, out_dtype=dtype))
    assert debug.tq_device_status(None) == 0 and release.tq_device_status(None) == 0


@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_append_matches_release(libs, D, dtype):  # noqa: F811
    release, debug = libs
    B, Hkv, Hq, N, cap = 5, 2, 6, 7, 30
    q, k, v = (sc.normal((B, h, N, D), i, dtype=dtype) for i, h in enumerate((Hq, Hkv, Hkv)))
    cos, sin = tq.rope_tables(D // 2, 64)
    lens, count = sc.ints([0, 30, 27, -2, 2 ** 31 - 3]), sc.ints([7, 7, 7, 3, 7])

    def run():
        c = tq.alloc_cache(B, Hkv, cap, D, 5, 3)
        q_out, new = tq.tq_append_kv(k, v, c, lens, 5, False, 3, cos=cos, sin=sin, q=q, count=count)
        return [q_out, new, *c.values()]

    _same(release, debug, run)
    assert debug.tq_device_status(None) == 0 and release.tq_device_status(None) == 0
