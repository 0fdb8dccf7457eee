"""Sizes near the ends of their types in the calls on new tokens. Every call below is
refused by its sizes, so none reaches a kernel launch, and they run without a GPU."""
import ctypes
import os
import re

import pytest
import torch

INVALID = 1
MOST = 2 ** 31 - 2 ** 13  # the most tokens of a sequence
EVERY = 2 ** 63 - 1


@pytest.fixture(scope="module")
def tq():
    from turboquant_kv_cache_tq_gb300 import build

    build.build()
    import turboquant_kv_cache_tq_gb300 as tq

    tq.lib()
    return tq


def _window(tq, B, Hq, Hkv, N, D, T, window, sinks):
    """A call over addresses that are never read, far enough apart for any cache."""
    at = [(i + 1) << 50 for i in range(8)]
    cache = tq.TQPackedCache(*at[:5], T)
    return tq.lib().tq_window_attention(at[5], B, Hq, N, ctypes.byref(cache), Hkv, T, D, 8, 1, 8, None, None, None, window,
                                        sinks, ctypes.c_float(1.0), at[6], 1, None, at[7], 1 << 49, None)


@pytest.mark.parametrize("B,Hq,Hkv,N,D", [(64, 4, 2, 1, 128), (64, 2, 2, 1, 512), (32, 4, 2, 512, 128), (64, 2, 2, 300, 512)])
@pytest.mark.parametrize("window,sinks", [(1, EVERY), (4096, EVERY), (MOST - 1, EVERY), (1, EVERY - 4), (1, MOST), (1, MOST + 5),
                                          (MOST - 1, 0), (MOST, 0), (EVERY, 0), (EVERY, EVERY)])
def test_tiles_of_a_call_are_counted_for_any_window_and_sinks(tq, B, Hq, Hkv, N, D, window, sinks):
    """Few rows and many over sequences whose tiles pass 32 bits in all: refused, however
    the window and the first tokens say that a row sees all of its sequence (a sum
    that wraps would be a negative number of tiles, which no limit stops)."""
    assert _window(tq, B, Hq, Hkv, N, D, MOST, window, sinks) == INVALID


def test_a_kernel_that_starts_without_a_wait_acquires():
    """Of two kernels of a call that run side by side, the second may read what the kernel
    before the call wrote only after it has acquired what the first released, and waits
    where it has not: the start of a dependent kernel orders no memory."""
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "turboquant_kv_cache_tq_gb300", "csrc")
    text = open(os.path.join(csrc, "tq_span_attention.cuh")).read()
    begin = re.search(r"void begin\(\) const \{(.*?)\n  \}\n", text, re.S).group(1)
    begin = re.sub(r"\s*//[^\n]*", "", begin)
    second, first = begin.split("return;")
    assert re.search(r"if \(order == 2\) \{.*ld\.acquire\.gpu.*if \(seen != call\) pdl_wait\(\);", second, re.S)
    assert re.search(r"pdl_wait\(\);.*st\.release\.gpu.*__syncthreads\(\);.*pdl_launch_dependents\(\);", first, re.S)


class _Like:
    """What the binding asks of a tensor before it takes the tensor's address."""

    def __init__(self, t, device):
        self.t, self.dtype, self.shape, self.device = t, t.dtype, t.shape, device

    def get_device(self):
        return self.device.index

    def stride(self):
        return self.t.stride()

    def numel(self):
        return self.t.numel()

    def data_ptr(self):
        return 1 << 40


def test_the_binding_takes_contiguous_rows_only(tq):
    dev = torch.device("cuda", 0)
    k = torch.zeros((2, 2, 64, 64))
    for t in (k, k[:, :1], k[:, :, 3:5], k[:1].expand(4, 2, 64, 64), k.transpose(1, 2)):
        r = tq._rows(_Like(t, dev), t.shape, torch.float32, "k", dev)
        assert (r.data, r.stride_b, r.stride_h, r.stride_t) == (1 << 40, *t.stride()[:3])
    for t in (k.transpose(2, 3), k[..., ::2], k.permute(3, 1, 2, 0)):
        with pytest.raises(ValueError, match="contiguous rows"):
            tq._rows(_Like(t, dev), t.shape, torch.float32, "k", dev)
    for x, shape, dtype in ((_Like(k, torch.device("cuda", 1)), k.shape, torch.float32), (_Like(k, dev), (2, 2, 64, 32), torch.float32),
                            (_Like(k, dev), k.shape, torch.bfloat16)):
        with pytest.raises(ValueError, match="contiguous rows"):
            tq._rows(x, shape, dtype, "k", dev)


def test_numbers_of_tokens_past_64_bits(tq, monkeypatch):
    """ctypes drops the bits above 64: what the binding passes on has to fit."""
    passed, cache = {}, tq.alloc_cache(1, 2, 16, 64, 8, 3, device="cpu")

    class Library:
        def tq_window_attention_workspace_size(self, *a):
            return 16

        tq_prefix_attention_workspace_size = tq_window_attention_workspace_size

        def tq_window_attention(self, *a):
            passed.update(T=a[6], window=a[14], sinks=a[15])

        def tq_prefix_attention(self, *a):
            passed.update(P=a[6], T=a[10])

    monkeypatch.setattr(tq, "lib", Library)
    monkeypatch.setattr(tq, "_elsewhere", lambda device, stream: False)
    monkeypatch.setattr(tq, "_current_stream", lambda device: 0)
    monkeypatch.setattr(tq, "_packed", lambda *a: tq.TQPackedCache())
    q = torch.zeros((1, 4, 1, 64), dtype=torch.bfloat16)
    for x, want in ((5, 5), (0, 0), (-1, -1), (EVERY, EVERY), (EVERY + 1, EVERY), (2 ** 64, EVERY), (2 ** 64 + 5, EVERY),
                    (2 ** 100, EVERY), (-5, -1), (-2 ** 64, -1), (-2 ** 64 + 5, -1)):
        tq.tq_window_attention(q, cache, x, 8, True, 3, x, x)
        assert passed == dict(T=want, window=want, sinks=want), x
        passed.clear()
        tq.tq_prefix_attention(q, cache, x, cache, x, 8, True, 3)
        assert passed == dict(P=want, T=want), x
        passed.clear()
