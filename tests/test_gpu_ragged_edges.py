"""GPU tests of the calls on ragged packed caches at the ends of what they
accept: budgets and caches of nothing, full rows, capacities far beyond the
sequences."""
import ctypes

import numpy as np
import pytest
import torch

import turboquant_kv_cache_tq_gb300 as tq
from tests import ragged_common as rc
from tests.gpu_common import cache_to_numpy, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _int(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def test_cutting_to_nothing():
    cache = rc.to_gpu(rc.random_cache(2, 3, 20, 128, 8, True, 3, 1))
    w = torch.rand((2, 3, 20), device="cuda")
    for t_cap in (None, 4):
        cut, cw, length = tq.evict_rows(cache, w, 20, 0, 0, lens=_int([20, 7]), t_cap=t_cap)
        assert length.tolist() == [0, 0]
        assert cut["k_codes"].shape[2] == cw.shape[2] == (t_cap or 0)


def test_cutting_a_cache_without_room():
    cache = tq.alloc_cache(2, 3, 0, 128, 8, 3)
    w = torch.zeros((2, 3, 0), device="cuda")
    index, count = tq.tq_evict_select(w, 0, 5, 2)
    assert (index == -1).all() and count.tolist() == [0, 0]
    cut, cw, length = tq.evict_rows(cache, w, 0, 5, 2)
    assert length.tolist() == [0, 0] and cut["k_codes"].shape[2] == 5 and (cw == 0).all()


def test_a_path_that_does_not_fit_into_its_row():
    """What fits is appended, new - lens tokens; with that as n_path the weight
    sums see the same observers at the same tokens as a reference of the kept
    part of the path."""
    B, Hkv, G, N, D, cap = 3, 2, 2, 6, 128, 40
    main = rc.random_cache(B, Hkv, cap, D, 8, True, 3, 1)
    draft = rc.random_cache(B, Hkv, N, D, 8, True, 3, 2)
    dm, dt = rc.to_gpu(main), rc.to_gpu(draft)
    lens, path, n_path = [38, 40, 20], [[0, 1, 3, 5], [0, 2, 3, 4], [1, 2, 4, 5]], [4, 3, 4]
    sums = torch.ones((B, Hkv, cap), device="cuda")
    new = tq.commit_path(dm, _int(lens), dt, _int(path), _int(n_path), weights=sums)
    assert new.tolist() == [40, 40, 24]
    after, ow, _ = rc.gather_reference(draft, main, np.array(path), n_path, lens, None, np.ones((B, Hkv, cap), np.float32))
    for k, v in cache_to_numpy(dm).items():
        assert np.array_equal(v, after[k]), k
    assert np.array_equal(sums.cpu().numpy(), ow)
    q = torch.randn((B, Hkv * G, N, D), generator=torch.Generator().manual_seed(3)).bfloat16()
    lse = torch.full((B, Hkv * G, N), 4.0)
    appended = new - _int(lens)
    assert appended.tolist() == [2, 0, 4]
    got = tq.tq_attention_weights(q.cuda(), lse.cuda(), dm, cap, 8, True, path=_int(path), n_path=appended, lens=new,
                                  weights=sums)
    rc.check_weights(got, rc.weights_reference(q, lse, after, cap, 8, True, path, [2, 0, 4], [40, 40, 24], None, None,
                                               torch.tensor(ow), cap))


@pytest.mark.parametrize("given", [False, True])
def test_weights_in_arrays_far_longer_than_the_sequences(given):
    """Every element outside the sequences is copied or zeroed, at both ends."""
    B, Hkv, G, N, T, D, w_cap = 2, 3, 2, 3, 130, 128, 131073
    cache = rc.random_cache(B, Hkv, T, D, 8, True, 3, 1)
    g = torch.Generator().manual_seed(2)
    q, lse = torch.randn((B, Hkv * G, N, D), generator=g).bfloat16(), torch.full((B, Hkv * G, N), 5.0)
    w = torch.rand((B, Hkv, w_cap), generator=g) if given else None
    lens, pad = [130, 41], [5, 40]
    out = torch.full((B, Hkv, w_cap), 7.0, device="cuda")
    got = tq.tq_attention_weights(q.cuda(), lse.cuda(), rc.to_gpu(cache), T, 8, True, lens=_int(lens), left_pad=_int(pad),
                                  weights=None if w is None else w.cuda(), out=out)
    rc.check_weights(got, rc.weights_reference(q, lse, cache, T, 8, True, None, None, lens, pad, None, w, w_cap))
    before = torch.zeros((B, Hkv, w_cap)) if w is None else w
    for b in range(B):
        assert torch.equal(got[b, :, lens[b]:].cpu(), before[b, :, lens[b]:])
        assert torch.equal(got[b, :, :pad[b]].cpu(), before[b, :, :pad[b]])


def test_weights_and_choice_clamp_lengths_outside_the_range():
    B, T, D = 4, 70, 128
    lens, pad = [71, -5, 2**31 - 1, 10], [-7, 3, 2**31 - 1, 10]
    cache = rc.random_cache(B, 1, T, D, 8, True, 3, 1)
    g = torch.Generator().manual_seed(2)
    q, lse, w = torch.randn((B, 2, 3, D), generator=g).bfloat16(), torch.full((B, 2, 3), 4.0), torch.rand((B, 1, T), generator=g)
    for in_place in (False, True):
        dw = w.cuda()
        got = tq.tq_attention_weights(q.cuda(), lse.cuda(), rc.to_gpu(cache), T, 8, True, lens=_int(lens), left_pad=_int(pad),
                                      weights=dw, out=dw if in_place else None)
        rc.check_weights(got, rc.weights_reference(q, lse, cache, T, 8, True, None, None, lens, pad, None, w))
    index, count = tq.tq_evict_select(w.cuda(), T, 9, 4, lens=_int(lens), left_pad=_int(pad))
    want, wc = rc.select_reference(w, T, 9, 4, lens, pad)
    assert np.array_equal(index.cpu().numpy(), want) and np.array_equal(count.cpu().numpy(), wc)


def test_weights_of_as_many_observers_as_a_call_takes():
    """65536 rows of a kv head: 256 rounds of columns."""
    G, P, T, D = 16, 4096, 4500, 64
    c = tq.alloc_cache(1, 1, T, D, 8, 3)
    g = torch.Generator(device="cuda").manual_seed(1)
    k = torch.randn((1, 1, T, D), generator=g, device="cuda").bfloat16()
    tq.tq_encode_kv(k, k, 8, True, 3, c)
    q = torch.randn((1, G, P, D), generator=g, device="cuda").bfloat16()
    lse = 8 + torch.rand((1, G, P), generator=g, device="cuda")
    got = tq.tq_attention_weights(q, lse, c, T, 8, True)[0, 0].double()
    K = tq.tq_decode_kv(c, T, 8, True, 3)[0][0, 0].double()
    want, tol = torch.zeros(T, dtype=torch.float64, device="cuda"), torch.zeros(T, dtype=torch.float64, device="cuda")
    sees = torch.arange(T, device="cuda") <= T - P + torch.arange(P, device="cuda")[:, None]
    for h in range(G):
        s = D ** -0.5 * (q[0, h].double() @ K.T)
        w = torch.where(sees, (s - lse[0, h].double()[:, None]).exp(), 0.0)
        mag = D ** -0.5 * (q[0, h].double().abs() @ K.abs().T)
        # (the derivation is weights_reference's)
        e = (D / 16 + 4) * 2 * rc.HALF * mag + (s.abs() + lse[0, h].double()[:, None].abs()) * 2.0 ** -22 + 2.0 ** -21
        want += w.sum(0)
        tol += (w * (e + (G * P + 2) * 2 * rc.HALF)).sum(0)
    off = (got - want).abs() - tol
    assert (off <= 0).all(), off.max()
    with pytest.raises(tq.TQError):  # one more
        tq.tq_attention_weights(q, lse, c, T, 8, True, path=torch.zeros((1, P + 1), dtype=torch.int32, device="cuda"))


def test_batches_of_nothing():
    cache, tree = tq.alloc_cache(0, 2, 16, 64, 8, 3), tq.alloc_cache(0, 2, 3, 64, 8, 3)
    q = torch.empty((0, 4, 3, 64), dtype=torch.bfloat16, device="cuda")
    out, lse = tq.tq_tree_attention(q, cache, 16, tree, 8, True, 3)
    assert out.shape == (0, 4, 3, 64) and lse.shape == (0, 4, 3)
    w = tq.tq_attention_weights(q, lse, cache, 16, 8, True)
    none = torch.empty((0,), dtype=torch.int32, device="cuda")
    new = tq.commit_path(cache, none, tree, torch.empty((0, 2), dtype=torch.int32, device="cuda"), none, weights=w)
    cut, cw, length = tq.evict_rows(cache, w, 16, 4, 1, lens=new)
    assert cut["k_codes"].shape[:3] == (0, 2, 4) and cw.shape == (0, 2, 4) and length.shape == (0,)


def _pieces(seed):
    B, Hkv, G, N, T, D = 2, 2, 2, 5, 700, 128
    main, tree = (rc.to_gpu(rc.random_cache(B, Hkv, n, D, 8, True, 3, n + seed)) for n in (T, N))
    q = torch.randn((B, Hkv * G, N, D), generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()

    def call():
        out, lse = tq.tq_tree_attention(q, main, T, tree, 8, True, 3)
        w = tq.tq_attention_weights(q, lse, main, T, 8, True)
        return (out, lse, w, *tq.tq_evict_select(w, T, 99, 9))

    return call


def test_two_graphs_replayed_at_once():
    """Two captured calls, replayed on two streams at the same time."""
    calls = [_pieces(1), _pieces(2)]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    graphs, got, streams = [], [], [torch.cuda.Stream() for _ in calls]
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(c())
        graphs.append(g)
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


def test_calls_of_two_host_threads():
    import threading

    calls = [_pieces(3), _pieces(4)]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    got = [None, None]

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(30):
                got[i] = calls[i]()
            s.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for a, b in zip(want, got):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


def test_views_into_larger_storage():
    """Contiguous views at 16-byte offsets are taken, at others refused."""
    main, tree = (rc.to_gpu(rc.random_cache(1, 2, n, 64, 8, True, 3, n)) for n in (100, 4))
    q = torch.randn((1, 4, 4, 64), generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    room = torch.empty(q.numel() + 8, dtype=torch.bfloat16, device="cuda")
    want = tq.tq_tree_attention(q, main, 100, tree, 8, True, 3)
    view = room[8:].view(q.shape)
    view.copy_(q)
    got = tq.tq_tree_attention(view, main, 100, tree, 8, True, 3)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    for call in (lambda x: tq.tq_tree_attention(x, main, 100, tree, 8, True, 3),
                 lambda x: tq.tq_attention_weights(x, want[1], main, 100, 8, True)):
        with pytest.raises(tq.TQError):
            call(room[1:1 + q.numel()].view(q.shape))


def test_a_refused_launch_does_not_fail_the_next_call():
    """A launch that the host refuses (on the legacy stream, while a stream that
    waits for it is captured) is that call's error alone."""
    B, Hkv, G, N, T, D = 1, 2, 2, 4, 100, 64
    main, tree = (rc.to_gpu(rc.random_cache(B, Hkv, n, D, 8, True, 3, n)) for n in (T, N))
    q = torch.randn((B, Hkv * G, N, D), generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    out, lse = torch.empty_like(q), torch.empty((B, Hkv * G, N), device="cuda")
    ws = torch.empty(tq.tq_tree_attention_workspace_size(B, Hkv * G, Hkv, N, D), dtype=torch.uint8, device="cuda")
    w = torch.zeros((B, Hkv, T), device="cuda")
    index, count = torch.empty((B, Hkv, 9), dtype=torch.int32, device="cuda"), torch.empty((B,), dtype=torch.int32, device="cuda")
    dst, length = tq.alloc_cache(B, Hkv, 9, D, 8, 3), torch.empty((B,), dtype=torch.int32, device="cuda")
    path = torch.zeros((B, 2), dtype=torch.int32, device="cuda")
    calls = [lambda: tq.tq_tree_attention(q, main, T, tree, 8, True, 3, out=out, lse=lse, workspace=ws),
             lambda: tq.tq_attention_weights(q, lse, main, T, 8, True, weights=w, out=w),
             lambda: tq.tq_evict_select(w, T, 9, 3, index=index, count=count),
             lambda: tq.tq_cache_gather(main, dst, path, dst_len=length)]
    assert torch.cuda.current_stream().cuda_stream == 0
    for call in calls:  # what a first call sets up
        call()
    torch.cuda.synchronize()
    driver = ctypes.CDLL("libcuda.so.1")
    for call in calls:
        stream, graph = ctypes.c_void_p(), ctypes.c_void_p()
        assert driver.cuStreamCreate(ctypes.byref(stream), 0) == 0
        assert driver.cuStreamBeginCapture_v2(stream, 0) == 0
        try:
            with pytest.raises(tq.TQError) as refused:
                call()
        finally:
            driver.cuStreamEndCapture(stream, ctypes.byref(graph))
            driver.cuStreamDestroy_v2(stream)
        assert refused.value.status == 6  # TQ_ERR_CUDA
        call()
    torch.cuda.synchronize()
    assert torch.isfinite(lse).all() and count.tolist() == [9] and length.tolist() == [2]
