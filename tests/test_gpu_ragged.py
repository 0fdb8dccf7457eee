"""GPU tests of the calls on ragged packed caches against plain 64-bit
references (tests/ragged_common.py, with the derivation of every tolerance):
tree attention, attention weight sums, the choice of the tokens that stay, the
copy of tokens between caches, and a decoding step made of all of them.
"""
import ctypes

import numpy as np
import pytest
import torch

import turboquant_kv_cache_tq_gb300 as tq
from tests import ragged_common as rc
from tests.gpu_common import cache_to_numpy, require_gpu

pytestmark = pytest.mark.gpu

KEY_MODES = [(2, False), (4, False), (5, False), (8, False), (8, True)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _q(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).bfloat16()


def _int(a):
    return None if a is None else torch.tensor(a, dtype=torch.int32, device="cuda")


def _parents(B, N, seed, absent=True):
    r = np.random.RandomState(seed)
    p = np.array([[r.randint(-1, i) if i else -1 for i in range(N)] for _ in range(B)], dtype=np.int32)
    if absent and N > 3:
        p[-1, N // 2] = -2  # and with it what hangs on it
        p[0, N - 1] = N - 1  # no earlier node
    return p


def run_tree(B, Hkv, G, N, T, D, kb, ks, vb, seed=0, lens=None, left_pad=None, parents="random", t_cap=None,
             out_dtype=torch.float32, qscale=1.0, edit=None, tree_cap=None, **kw):
    main = rc.random_cache(B, Hkv, T, D, kb, ks, vb, seed, t_cap=t_cap)
    tree = rc.random_cache(B, Hkv, N, D, kb, ks, vb, seed + 1, t_cap=tree_cap)
    if edit is not None:
        edit(main, tree)
    q = _q((B, Hkv * G, N, D), seed + 2, qscale)
    par = _parents(B, N, seed) if isinstance(parents, str) else parents
    got, lse = tq.tq_tree_attention(q.cuda(), rc.to_gpu(main), T, rc.to_gpu(tree), kb, ks, vb, parents=_int(par),
                                    lens=_int(lens), left_pad=_int(left_pad), out_dtype=out_dtype, **kw)
    torch.cuda.synchronize()
    ref = rc.tree_reference(q, main, T, tree, kb, ks, vb, par, lens, left_pad, dtype=out_dtype)
    return got, lse, ref


# ---- tree attention ---------------------------------------------------------------
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kb,ks", KEY_MODES)
@pytest.mark.parametrize("D", [64, 128, 256, 512])
def test_tree_all_formats(D, kb, ks, dtype):
    T = {64: 201, 128: 141, 256: 77, 512: 53}[D]
    for vb in (2, 3, 4, 5, 8):
        got, lse, ref = run_tree(2, 2, 3, 5, T, D, kb, ks, vb, seed=D + 10 * kb + vb, lens=[T, T // 2 + 1],
                                 left_pad=[0, 5], out_dtype=dtype)
        rc.check_tree(got, lse, ref, "D%d k%d%s v%d" % (D, kb, "s" if ks else "", vb))


@pytest.mark.parametrize("B,Hkv,G,N,T,D", [
    (1, 1, 1, 1, 1, 64), (1, 1, 1, 1, 0, 128), (1, 2, 4, 1, 300, 128), (3, 1, 1, 64, 65, 128), (1, 1, 16, 2, 64, 64),
    (2, 2, 5, 7, 128, 128), (1, 1, 8, 64, 130, 128), (1, 1, 3, 43, 129, 256), (1, 1, 8, 17, 31, 512),
    (1, 1, 33, 4, 63, 64), (2, 1, 2, 16, 127, 64), (1, 3, 4, 33, 257, 128), (1, 1, 4, 64, 40, 512),
    (1, 1, 4, 8, 65, 256), (5, 1, 1, 3, 1, 512),
])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_tree_shapes(B, Hkv, G, N, T, D, dtype):
    lens = None if B == 1 else [max(0, T - 9 * b) for b in range(B)]
    got, lse, ref = run_tree(B, Hkv, G, N, T, D, 8, True, 3, seed=B + G + N + T, lens=lens, out_dtype=dtype)
    rc.check_tree(got, lse, ref)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_tree_long_ragged(D, dtype):
    got, lse, ref = run_tree(3, 2, 2, 6, 2500, D, 8, True, 4, seed=5, lens=[2500, 0, 1411], left_pad=[17, 3, 1409],
                             qscale=2.0, out_dtype=dtype)
    rc.check_tree(got, lse, ref)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D", [64, 128, 256, 512])
def test_tree_sharp_rows_and_rising_maximum(D, dtype):
    """Rows whose weight sits on few keys, and keys that grow along the cache,
    so that a running maximum rises at nearly every tile."""
    def edit(main, tree):
        ramp = np.linspace(0.05, 4.0, main["k_scales"].shape[2]).astype(np.float32)[None, None, :, None]
        s = main["k_scales"].view(np.float16)
        s[...] = (s.astype(np.float32) * ramp).astype(np.float16)

    got, lse, ref = run_tree(1, 2, 4, 4, 300, D, 8, True, 8, seed=3, qscale=4.0, edit=edit, out_dtype=dtype)
    rc.check_tree(got, lse, ref)


@pytest.mark.parametrize("scale", [-0.11, 0.0, 1e-30, 3.0])
def test_tree_scales(scale):
    """Negative, zero, tiny and large softmax scales (hidden tokens stay hidden)."""
    main, tree = (rc.random_cache(1, 2, n, 128, 8, True, 3, n) for n in (150, 6))
    q, par = _q((1, 4, 6, 128), 2), _parents(1, 6, 3)
    got, lse = tq.tq_tree_attention(q.cuda(), rc.to_gpu(main), 150, rc.to_gpu(tree), 8, True, 3, parents=_int(par),
                                    left_pad=_int([5]), scale=scale, out_dtype=torch.float32)
    rc.check_tree(got, lse, rc.tree_reference(q, main, 150, tree, 8, True, 3, par, None, [5], scale))
    got, lse = tq.tq_tree_attention(q.cuda(), rc.to_gpu(main), 150, rc.to_gpu(tree), 8, True, 3, parents=_int(par),
                                    left_pad=_int([5]), scale=scale)
    rc.check_tree(got, lse, rc.tree_reference(q, main, 150, tree, 8, True, 3, par, None, [5], scale, torch.bfloat16))


def test_tree_lengths_outside_the_range_are_clamped():
    got, lse, ref = run_tree(4, 1, 2, 3, 70, 128, 8, True, 3, lens=[71, -5, 2**31 - 1, 10],
                             left_pad=[-7, 3, 2**31 - 1, 10])
    rc.check_tree(got, lse, ref)


def test_tree_rows_without_a_key():
    """No node present: zeros and -inf everywhere; an absent node's descendants
    are absent."""
    N = 6
    par = np.array([[-2] * N, [-1, 0, -3, 2, 5, 1]], dtype=np.int32)
    got, lse, ref = run_tree(2, 2, 2, N, 50, 128, 8, True, 3, parents=par)
    rc.check_tree(got, lse, ref)
    assert torch.isneginf(lse[0]).all() and (got[0] == 0).all()
    assert torch.isneginf(lse[1, :, 2:5]).all() and torch.isfinite(lse[1, :, [0, 1, 5]]).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D", [64, 128, 256, 512])
def test_tree_masked_places_hold_nan_and_infinity(D, dtype):
    """Scales and zero points of NaN and infinity outside [left_pad, lens) and
    in branches that a node is not on: nothing of them reaches a row; a row
    that attends to one is NaN as a whole."""
    T, N = 90, 6
    par = np.array([[-1, 0, 0, 1, 2, -1]] * 2, dtype=np.int32)

    def edit(main, tree):
        for name, bad in (("k_scales", 0x7E00), ("k_zeros", 0x7C00), ("v_scales", 0x7C00)):
            main[name][:, :, :7] = bad
            main[name][:, :, 70:] = bad
        tree["v_scales"][0, :, 1, 0] = 0x7C00   # an infinite value group: nodes 1 and 3
        tree["k_scales"][0, :, 2, -1] = 0x7E00  # a NaN key: nodes 2 and 4
        tree["v_scales"][1, :, 5, -1] = 0xFE00  # a NaN value group: node 5

    got, lse, ref = run_tree(2, 2, 2, N, T, D, 8, True, 3, parents=par, lens=[70, 66], left_pad=[7, 9], edit=edit,
                             out_dtype=dtype)
    rc.check_tree(got, lse, ref)
    assert torch.isnan(lse[0, :, 1:5]).all() and torch.isfinite(lse[0, :, [0, 5]]).all()
    assert torch.isnan(lse[1, :, 5]).all() and torch.isfinite(lse[1, :, :5]).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_tree_bad_values_in_the_sequence(dtype):
    """A value group with an infinite scale and a constant key group inside the
    range: every row of that batch row and head is NaN, no other."""
    def edit(main, tree):
        main["v_scales"][0, 0, 33, 1] = 0x7C00
        main["k_zeros"][1, 1, 99, 2] = 0xFC00

    got, lse, ref = run_tree(2, 2, 2, 3, 128, 128, 8, True, 3, parents=None, edit=edit, out_dtype=dtype)
    rc.check_tree(got, lse, ref)
    assert torch.isnan(lse[0, :2]).all() and torch.isfinite(lse[0, 2:]).all()
    assert torch.isnan(lse[1, 2:]).all() and torch.isfinite(lse[1, :2]).all()


def test_tree_capacities_that_no_tile_divides():
    for D in (64, 128, 256, 512):
        for kb, ks, vb in ((8, True, 3), (5, False, 5), (2, False, 2)):
            for dtype in (torch.float32, torch.bfloat16):
                got, lse, ref = run_tree(2, 3, 2, 5, 61, D, kb, ks, vb, t_cap=67, tree_cap=11, lens=[61, 47],
                                         out_dtype=dtype)
                rc.check_tree(got, lse, ref, "D%d k%d v%d" % (D, kb, vb))


def test_tree_equals_decode_attention_on_the_appended_cache():
    """A chain of drafted tokens is a causal tail: the same rows as
    tq_decode_attention gives once the chain is in the cache (both are within
    the tolerance of the exact result, so within twice of each other)."""
    B, Hkv, G, N, T, D = 2, 2, 2, 4, 156, 128
    main = rc.random_cache(B, Hkv, T + N, D, 8, True, 3, 1, t_cap=160)
    q = _q((B, Hkv * G, N, D), 2)
    dev = rc.to_gpu(main)
    tree = {k: v[:, :, T:T + N].contiguous() for k, v in dev.items()}
    got, lse = tq.tq_tree_attention(q.cuda(), dev, T, tree, 8, True, 3, out_dtype=torch.float32)
    other = tq.tq_decode_attention(q.cuda(), dev, T + N, 8, True, 3, out_dtype=torch.float32)
    ref = rc.tree_reference(q, main, T, cache_to_numpy(tree), 8, True, 3)
    rc.check_tree(got, lse, ref)
    err = (got.double() - other.double()).norm(dim=-1).cpu().numpy()
    assert np.all(err <= 2 * ref[2])


def test_tree_writes_nothing_beside_its_rows():
    B, Hkv, G, N, D = 1, 2, 3, 5, 128
    main, tree = (rc.to_gpu(rc.random_cache(B, Hkv, 40, D, 8, True, 3, s)) for s in (1, 2))
    q = _q((B, Hkv * G, N, D), 3).cuda()
    n, m = q.numel(), B * Hkv * G * N
    out = torch.full((n + 256,), 7.0, device="cuda")
    lse = torch.full((m + 64,), 7.0, device="cuda")
    need = tq.tq_tree_attention_workspace_size(B, Hkv * G, Hkv, N, D)
    ws = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    a, b = out[:n].view(B, Hkv * G, N, D), lse[:m].view(B, Hkv * G, N)
    tq.tq_tree_attention(q, main, 40, tree, 8, True, 3, out_dtype=torch.float32, out=a, lse=b, workspace=ws[:need])
    want, wl = tq.tq_tree_attention(q, main, 40, tree, 8, True, 3, out_dtype=torch.float32)
    assert torch.equal(a, want) and torch.equal(b, wl)
    assert (out[n:] == 7).all() and (lse[m:] == 7).all() and (ws[need:] == 0x5A).all()


def test_tree_equal_calls_give_equal_bits():
    main, tree = (rc.to_gpu(rc.random_cache(2, 2, n, 128, 8, True, 3, n)) for n in (700, 12))
    q = _q((2, 8, 12, 128), 3).cuda()
    first = tq.tq_tree_attention(q, main, 700, tree, 8, True, 3)
    for _ in range(5):
        again = tq.tq_tree_attention(q, main, 700, tree, 8, True, 3)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_tree_captured_and_replayed_with_new_lengths():
    B, Hkv, G, N, T, D = 2, 2, 2, 5, 200, 128
    main, tree = rc.random_cache(B, Hkv, T, D, 8, True, 3, 1), rc.random_cache(B, Hkv, N, D, 8, True, 3, 2)
    q = _q((B, Hkv * G, N, D), 3)
    dm, dt, dq = rc.to_gpu(main), rc.to_gpu(tree), q.cuda()
    lens, par = _int([10, 20]), _int(_parents(B, N, 1))
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        tq.tq_tree_attention(dq, dm, T, dt, 8, True, 3, parents=par, lens=lens)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = tq.tq_tree_attention(dq, dm, T, dt, 8, True, 3, parents=par, lens=lens, out_dtype=torch.float32)
    for new in ([200, 1], [0, 137], [64, 65]):
        lens.copy_(_int(new))
        g.replay()
        torch.cuda.synchronize()
        ref = rc.tree_reference(q, main, T, tree, 8, True, 3, par.cpu().numpy(), new)
        rc.check_tree(out, lse, ref)


def test_tree_on_two_streams_at_once():
    main, tree = (rc.to_gpu(rc.random_cache(2, 2, n, 128, 8, True, 3, n)) for n in (900, 8))
    q = [_q((2, 8, 8, 128), s).cuda() for s in (1, 2)]
    want = [tq.tq_tree_attention(x, main, 900, tree, 8, True, 3)[0] for x in q]
    streams = [torch.cuda.Stream() for _ in q]
    torch.cuda.synchronize()
    for _ in range(10):
        got = [tq.tq_tree_attention(x, main, 900, tree, 8, True, 3, stream=s)[0] for x, s in zip(q, streams)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_tree_many_batch_rows():
    """More rows than a warp counts at a time, many of them short or empty."""
    lens = [(7 * b) % 41 for b in range(70)]
    for dtype in (torch.float32, torch.bfloat16):
        got, lse, ref = run_tree(70, 1, 2, 2, 40, 128, 8, True, 3, lens=lens, out_dtype=dtype)
        rc.check_tree(got, lse, ref)


def _roomy(main, cap):
    """The same tokens at the start of a cache of `cap` tokens whose other bytes are all ones."""
    big = {}
    for k, v in rc.to_gpu(main).items():
        big[k] = torch.full((*v.shape[:2], cap, v.shape[3]), 255, dtype=torch.uint8, device="cuda") if v.dtype == torch.uint8 \
            else torch.full((*v.shape[:2], cap, v.shape[3]), -1, dtype=torch.int16, device="cuda").view(torch.float16)
        big[k][:, :, :v.shape[2]] = v
    return big


@pytest.mark.parametrize("kb,ks", KEY_MODES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,N", [(4, 16), (1, 1), (3, 5), (2, 31), (1, 64)])
def test_tree_two_lanes_a_row(D, kb, ks, G, N):
    """The bound T of the lengths, not the lengths, decides how rows are laid out: few
    rows and a large T give each two lanes."""
    B, Hkv, T, cap = 3, 2, 201, 26112
    lens, pad = [201, 64, 0], [0, 5, 0]
    vb = {(2, False): 2, (4, False): 3, (5, False): 4, (8, False): 5, (8, True): 8}[(kb, ks)]
    main, tree = (rc.random_cache(B, Hkv, n, D, kb, ks, vb, n + D) for n in (T, N))
    if kb == 4:
        main["v_scales"][0, 1, 40, 1] = 0x7C00  # attended to by one row's second head
        tree["v_scales"][1, :, N - 1, 0] = 0xFE00
    q, par = _q((B, Hkv * G, N, D), 4), _parents(B, N, N)
    got, lse = tq.tq_tree_attention(q.cuda(), _roomy(main, cap), cap, rc.to_gpu(tree), kb, ks, vb, parents=_int(par),
                                    lens=_int(lens), left_pad=_int(pad))
    torch.cuda.synchronize()
    rc.check_tree(got, lse, rc.tree_reference(q, main, T, tree, kb, ks, vb, par, lens, pad, dtype=torch.bfloat16))


def test_tree_caches_in_pinned_host_memory():
    """Buffers in pinned host memory give the same bits as in device memory."""
    B, Hkv, G, N, T, D = 2, 2, 2, 4, 150, 128
    main, tree = (rc.to_gpu(rc.random_cache(B, Hkv, n, D, 8, True, 3, n)) for n in (T, N))
    q = _q((B, Hkv * G, N, D), 4).cuda()
    want, wl = tq.tq_tree_attention(q, main, T, tree, 8, True, 3)
    ww = tq.tq_attention_weights(q, wl, main, T, 8, True)
    hm, ht = ({k: v.cpu().pin_memory() for k, v in c.items()} for c in (main, tree))
    out, lse, w = torch.empty_like(want), torch.empty_like(wl), torch.empty_like(ww)
    ws = torch.empty(tq.tq_tree_attention_workspace_size(B, Hkv * G, Hkv, N, D), dtype=torch.uint8, device="cuda")
    views = [tq.TQPackedCache(*(c[n].data_ptr() for n in rc.CACHE_KEYS), c["k_codes"].shape[2]) for c in (hm, ht)]
    s = torch.cuda.current_stream().cuda_stream
    assert tq.lib().tq_tree_attention(q.data_ptr(), B, Hkv * G, N, ctypes.byref(views[0]), Hkv, T, D,
                                      ctypes.byref(views[1]), None, 8, 1, 3, None, None, ctypes.c_float(D ** -0.5),
                                      out.data_ptr(), 1, lse.data_ptr(), ws.data_ptr(), ws.numel(), s) == 0
    assert tq.lib().tq_attention_weights(q.data_ptr(), lse.data_ptr(), B, Hkv * G, N, hm["k_codes"].data_ptr(),
                                         hm["k_scales"].data_ptr(), hm["k_zeros"].data_ptr(), Hkv, T, D, T, 8, 1, None,
                                         None, None, None, N, ctypes.c_float(D ** -0.5), None, w.data_ptr(), T, s) == 0
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, wl) and torch.equal(w, ww)


def test_offsets_past_32_bits():
    """The last head of a cache whose buffers pass 2^32 bytes: the bits that the
    same tokens give in a small cache (equal lengths are cut the same way)."""
    B, Hkv, N, T, D, cap = 1, 4, 3, 200, 128, 9 << 20
    small, tree = (rc.to_gpu(rc.random_cache(B, Hkv, n, D, 8, True, 8, n)) for n in (208, N))
    big = tq.alloc_cache(B, Hkv, cap, D, 8, 8)
    assert big["k_codes"].numel() > 1 << 32
    for k in rc.CACHE_KEYS:
        big[k][:, :, :208] = small[k]
    q, lens = _q((B, 2 * Hkv, N, D), 4).cuda(), _int([T])
    for dtype in (torch.float32, torch.bfloat16):
        a = tq.tq_tree_attention(q, small, T, tree, 8, True, 8, lens=lens, out_dtype=dtype)
        b = tq.tq_tree_attention(q, big, T, tree, 8, True, 8, lens=lens, out_dtype=dtype)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    wa, wb = (tq.tq_attention_weights(q, a[1], c, T, 8, True, lens=lens) for c in (small, big))
    assert torch.equal(wa, wb)
    # tokens at the far end of every head, there and back
    index = torch.arange(N, dtype=torch.int32, device="cuda")[None]
    far = _int([cap - N])
    _, length = tq.tq_cache_gather(tree, big, index, dst_off=far)
    assert length.tolist() == [cap]
    back = tq.alloc_cache(B, Hkv, N, D, 8, 8)
    tq.tq_cache_gather(big, back, index + (cap - N))
    for k in rc.CACHE_KEYS:
        assert torch.equal(back[k].view(torch.uint8), tree[k].view(torch.uint8))


# ---- weight sums ------------------------------------------------------------------
def run_weights(B, Hkv, G, N, T, D, kb, ks, seed=0, lens=None, left_pad=None, path=None, n_path=None, t_cap=None,
                w_cap=None, start=False, in_place=False, lse=None, edit=None, qscale=1.0):
    cache = rc.random_cache(B, Hkv, T, D, kb, ks, 8, seed, t_cap=t_cap)
    if edit is not None:
        edit(cache)
    q = _q((B, Hkv * G, N, D), seed + 1, qscale)
    g = torch.Generator().manual_seed(seed)
    if lse is None:
        lse = np.log(max(T, 1)) + 0.5 + torch.rand((B, Hkv * G, N), generator=g)
    w_cap = T if w_cap is None else w_cap
    w = torch.rand((B, Hkv, w_cap), generator=g) if start or in_place else None
    dw = None if w is None else w.cuda()
    out = dw if in_place else torch.full((B, Hkv, w_cap), 7.0, device="cuda")
    got = tq.tq_attention_weights(q.cuda(), lse.cuda(), rc.to_gpu(cache), T, kb, ks, path=_int(path),
                                  n_path=_int(n_path), lens=_int(lens), left_pad=_int(left_pad), weights=dw, out=out)
    torch.cuda.synchronize()
    assert got is out
    ref = rc.weights_reference(q, lse, cache, T, kb, ks, path, n_path, lens, left_pad, None, w, w_cap)
    rc.check_weights(got, ref)
    return got, w


@pytest.mark.parametrize("kb,ks", KEY_MODES)
@pytest.mark.parametrize("D", [64, 128, 256, 512])
def test_weights_all_formats(D, kb, ks):
    T = {64: 201, 128: 141, 256: 77, 512: 53}[D]
    run_weights(2, 2, 3, 5, T, D, kb, ks, seed=D + kb, lens=[T, T // 2], left_pad=[0, 6], start=True)


@pytest.mark.parametrize("B,Hkv,G,N,T,D", [
    (1, 1, 1, 1, 1, 64), (1, 2, 4, 1, 300, 128), (2, 1, 4, 64, 130, 128), (1, 1, 8, 64, 70, 128), (1, 1, 16, 33, 129, 64),
    (1, 1, 5, 13, 128, 256), (1, 1, 8, 40, 60, 512), (1, 1, 4, 200, 257, 128), (3, 2, 1, 2, 127, 128),
    (1, 1, 3, 100, 90, 512),
])
def test_weights_shapes(B, Hkv, G, N, T, D):
    run_weights(B, Hkv, G, N, T, D, 8, True, seed=T + N, lens=None if B == 1 else [max(0, T - 11 * b) for b in range(B)])


def test_weights_many_batch_rows():
    run_weights(70, 1, 2, 3, 40, 128, 8, True, lens=[(7 * b) % 41 for b in range(70)],
                n_path=[b % 4 for b in range(70)], path=[[0, 1, 2]] * 70, start=True)


@pytest.mark.parametrize("D", [64, 128, 256, 512])
def test_weights_capacities_that_no_tile_divides(D):
    for kb, ks in ((8, True), (5, False)):
        run_weights(2, 3, 2, 5, 61, D, kb, ks, t_cap=67, lens=[61, 40])


def test_weights_paths():
    """Paths of every length, entries outside the nodes, counts outside the
    range, capacities beyond T, sums in place."""
    path = [[0, 2, 5, 7], [1, 1, 3, 3], [-1, 4, 8, 2], [7, 6, 5, 0], [0, 1, 2, 3]]
    for in_place in (False, True):
        got, w = run_weights(5, 2, 3, 8, 90, 128, 8, True, lens=[90, 71, 3, 50, 0], left_pad=[0, 70, 0, 8, 0], path=path,
                             n_path=[4, 3, 9, -2, 4], t_cap=97, w_cap=93, start=True, in_place=in_place)
        assert torch.equal(got[:, :, 90:].cpu(), w[:, :, 90:])
        assert torch.equal(got[3].cpu(), w[3]) and torch.equal(got[4].cpu(), w[4])


def test_weights_rows_without_a_key_add_nothing():
    lse = torch.full((1, 4, 3), -float("inf"))
    lse[:, :, 1] = 3.0
    got, w = run_weights(1, 2, 2, 3, 66, 128, 8, True, lse=lse, start=True)


@pytest.mark.parametrize("D", [64, 512])
def test_weights_masked_places_hold_nan(D):
    def edit(cache):
        for name in ("k_scales", "k_zeros"):
            cache[name][:, :, :5] = 0x7E00
            cache[name][:, :, 60:] = 0x7C00

    got, w = run_weights(1, 2, 2, 3, 80, D, 8, True, lens=[60], left_pad=[5], start=True, edit=edit)
    assert torch.isfinite(got).all()

    def spoil(cache):
        cache["k_scales"][0, 0, 40] = 0x7E00  # a NaN key: NaN at that token alone

    got, w = run_weights(1, 2, 2, 3, 80, D, 8, True, edit=spoil)
    assert torch.isnan(got[0, 0, 40]) and torch.isfinite(got).sum() == got.numel() - 1


def test_weights_equal_calls_give_equal_bits():
    cache = rc.to_gpu(rc.random_cache(2, 2, 500, 128, 8, True, 8, 1))
    q, lse = _q((2, 8, 20, 128), 3).cuda(), torch.full((2, 8, 20), 6.0, device="cuda")
    first = tq.tq_attention_weights(q, lse, cache, 500, 8, True)
    for _ in range(5):
        assert torch.equal(first, tq.tq_attention_weights(q, lse, cache, 500, 8, True))


# ---- choice -----------------------------------------------------------------------
def check_select(w, T, keep, recent, lens=None, left_pad=None):
    index = torch.full((w.shape[0], w.shape[1], keep), 77, dtype=torch.int32, device="cuda")
    got, count = tq.tq_evict_select(w.cuda(), T, keep, recent, lens=_int(lens), left_pad=_int(left_pad), index=index)
    torch.cuda.synchronize()
    want, wc = rc.select_reference(w, T, keep, recent, lens, left_pad)
    assert np.array_equal(count.cpu().numpy(), wc)
    assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("T", [0, 1, 2, 31, 33, 255, 1023, 1024, 1025, 5000, 20011])
def test_select_sizes(T):
    g = torch.Generator().manual_seed(T)
    w = torch.randn((2, 3, T + 3), generator=g)
    for keep in sorted({0, 1, T // 3, max(T - 1, 0), T, T + 5}):
        for recent in sorted({0, keep // 4, keep}):
            check_select(w, T, keep, recent, lens=[T, T - T // 3], left_pad=[0, T // 5])


def test_select_ties_and_special_values():
    g = torch.Generator().manual_seed(1)
    inf, nan = float("inf"), float("nan")
    w = torch.randint(0, 4, (1, 4, 700), generator=g).float()
    w[0, 1] = 0.0
    w[0, 2] = torch.tensor([0.0, -0.0, nan, -inf, inf, 1e-45, -1e-45])[torch.randint(0, 7, (700,), generator=g)]
    w[0, 3] = nan
    for keep in (1, 99, 350, 699):
        check_select(w, 700, keep, 0)
        check_select(w, 700, keep, keep // 2)


def test_select_one_long_row():
    g = torch.Generator().manual_seed(2)
    w = (torch.rand((1, 2, 200003), generator=g) ** 8).half().float()
    check_select(w, 200003, 70001, 1000, lens=[200001], left_pad=[3])


@pytest.mark.parametrize("T", [8193, 16384, 16385, 40000])
def test_select_more_rows_than_the_gpu_has_sms(T):
    g = torch.Generator().manual_seed(T)
    w = (torch.rand((40, 5, T), generator=g) ** 6).half().float()
    check_select(w, T, T // 4, 100, lens=[T - 37 * b for b in range(40)], left_pad=[b for b in range(40)])


@pytest.mark.parametrize("T", [65536, 140000])
def test_select_eight_blocks_a_row(T):
    w = torch.rand((1, 2, T), generator=torch.Generator().manual_seed(T)).half().float()
    check_select(w, T, T // 3, 77, lens=[T - 5], left_pad=[9])


def test_select_many_rows():
    g = torch.Generator().manual_seed(3)
    check_select(torch.rand((40, 8, 300), generator=g), 300, 100, 10, lens=[(7 * b) % 301 for b in range(40)])


# ---- copy -------------------------------------------------------------------------
def check_gather(src, dst, index, count=None, dst_off=None, sw=None, dw=None):
    ds, dd = rc.to_gpu(src), rc.to_gpu(dst)
    gw = None if dw is None else torch.tensor(dw, device="cuda")
    got, length = tq.tq_cache_gather(ds, dd, _int(index), count=_int(count), dst_off=_int(dst_off),
                                     src_weights=None if sw is None else torch.tensor(sw, device="cuda"), dst_weights=gw)
    torch.cuda.synchronize()
    want, ow, wl = rc.gather_reference(src, dst, index, count, dst_off, sw, dw)
    back = cache_to_numpy(got)
    for k in rc.CACHE_KEYS:
        assert np.array_equal(back[k], want[k]), k
        assert np.array_equal(cache_to_numpy(ds)[k], src[k]), k
    assert np.array_equal(length.cpu().numpy(), wl)
    if dw is not None:
        assert np.array_equal(gw.cpu().numpy(), ow)


@pytest.mark.parametrize("D", [64, 128, 256, 512])
def test_gather_all_formats(D):
    r = np.random.RandomState(D)
    for kb, ks in KEY_MODES:
        for vb in (2, 3, 4, 5, 8):
            src = rc.random_cache(2, 3, 37, D, kb, ks, vb, D + kb + vb, t_cap=39)
            dst = rc.random_cache(2, 3, 31, D, kb, ks, vb, D + kb + vb + 1)
            check_gather(src, dst, r.randint(0, 39, (2, 3, 23)), count=[23, 11], dst_off=[0, 9],
                         sw=r.rand(2, 3, 39).astype(np.float32), dw=r.rand(2, 3, 31).astype(np.float32))


@pytest.mark.parametrize("n", [1, 63, 64, 65, 1000])
def test_gather_sizes_and_bad_entries(n):
    """Equal indices, indices outside the source, destinations past the
    capacity, counts and offsets outside their ranges."""
    r = np.random.RandomState(n)
    src = rc.random_cache(4, 2, 50, 128, 8, True, 3, 1)
    dst = rc.random_cache(4, 2, n + 5, 128, 8, True, 3, 2)
    index = r.randint(-3, 55, (4, n)).astype(np.int32)
    index[0, 0] = 2**31 - 1
    index[1, -1] = -(2**31)
    check_gather(src, dst, index, count=[n, n // 2, n + 9, -1], dst_off=[5, 9, -4, 2**31 - 1], dw=r.rand(4, 2, n + 5).astype(np.float32))
    check_gather(src, dst, index)


def test_gather_nothing():
    src, dst = rc.random_cache(2, 1, 5, 64, 8, True, 3, 1), rc.random_cache(2, 1, 9, 64, 8, True, 3, 2)
    check_gather(src, dst, np.zeros((2, 0), np.int32), dst_off=[4, 100])


# ---- together ---------------------------------------------------------------------
def test_a_decoding_step_of_all_of_them():
    """Draft, attend, commit, sum the weights, cut, and attend again, all in one
    captured graph replayed for a second step; each part against its reference
    on the bytes that it was given."""
    B, Hkv, G, N, T, D, kb, ks, vb = 2, 2, 4, 7, 160, 128, 8, True, 3
    cap, keep = 176, 96
    main = rc.to_gpu(rc.random_cache(B, Hkv, T - 20, D, kb, ks, vb, 1, t_cap=cap))
    lens = _int([T - 20, 100])
    weights = torch.zeros((B, Hkv, cap), device="cuda")
    kd, vd = (_q((B, Hkv, N, D), s).cuda() for s in (2, 3))
    q = _q((B, Hkv * G, N, D), 4).cuda()
    par, path, n_path = _int([[-1, 0, 0, 1, 2, 2, 4], [-1, -1, 1, 1, 3, 4, 5]]), _int([[0, 2, 4, 6], [1, 3, 0, 0]]), _int([4, 2])
    tree = tq.alloc_cache(B, Hkv, N, D, kb, vb)

    def step():
        tq.tq_encode_kv(kd, vd, kb, ks, vb, tree)
        out, lse = tq.tq_tree_attention(q, main, T, tree, kb, ks, vb, parents=par, lens=lens, out_dtype=torch.float32)
        new = tq.commit_path(main, lens, tree, path, n_path, weights=weights)
        tq.tq_attention_weights(q, lse, main, T, kb, ks, path=path, n_path=n_path, lens=new, weights=weights, out=weights)
        cut, cw, cl = tq.evict_rows(main, weights, T, keep, 16, lens=new)
        lens.copy_(new)
        return out, lse, new, cut, cw, cl

    def check(before, lens0, w0, r):
        out, lse, new, cut, cw, cl = r
        tn, l0 = cache_to_numpy(tree), lens0.tolist()
        rc.check_tree(out, lse, rc.tree_reference(q, before, T, tn, kb, ks, vb, par.cpu().numpy(), l0))
        index = path.cpu().numpy()
        after, _, nl = rc.gather_reference(tn, before, index, n_path.tolist(), l0)
        assert nl.tolist() == new.tolist()
        now = cache_to_numpy(main)
        for k in rc.CACHE_KEYS:
            assert np.array_equal(now[k], after[k]), k
        for b in range(B):
            w0[b, :, l0[b]:nl[b]] = 0.0
        rc.check_weights(weights, rc.weights_reference(q, lse, after, T, kb, ks, index, n_path.tolist(), nl.tolist(),
                                                       weights=w0, w_cap=cap))
        # every observer's weights add up to one
        added = (weights - w0.cuda()).double().sum(-1).cpu().numpy()
        assert np.allclose(added, G * n_path.cpu().numpy()[:, None], rtol=1e-4)
        idx, cnt = rc.select_reference(weights, T, keep, 16, nl.tolist())
        kept, kw, kl = rc.gather_reference(after, {k: np.zeros_like(v.cpu().numpy().view(after[k].dtype)) for k, v in cut.items()},
                                           idx, cnt.tolist(), None, weights.cpu().numpy(), np.zeros((B, Hkv, keep), np.float32))
        assert kl.tolist() == cl.tolist() == [keep, keep] and np.array_equal(cw.cpu().numpy(), kw)
        got = cache_to_numpy(cut)
        for k in rc.CACHE_KEYS:
            assert np.array_equal(got[k], kept[k]), k
        out2, lse2 = tq.tq_tree_attention(q, cut, keep, tree, kb, ks, vb, parents=par, lens=cl)
        rc.check_tree(out2, lse2, rc.tree_reference(q, kept, keep, tn, kb, ks, vb, par.cpu().numpy(), cl.tolist(),
                                                    dtype=torch.bfloat16))

    state = lambda: (cache_to_numpy(main), lens.clone(), weights.cpu().clone())  # noqa: E731
    s = state()
    r = step()
    torch.cuda.synchronize()
    check(*s, r)
    s = state()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = step()
    for _ in range(2):
        s = state()
        g.replay()
        torch.cuda.synchronize()
        check(*s, r)


def test_calls_on_another_stream_than_the_current_one():
    B, Hkv, G, N, T, D = 1, 2, 2, 4, 300, 128
    main, tree = (rc.to_gpu(rc.random_cache(B, Hkv, n, D, 8, True, 3, n)) for n in (T, N))
    q = _q((B, Hkv * G, N, D), 4).cuda()
    w = torch.rand((B, Hkv, T), device="cuda")
    want = tq.tq_tree_attention(q, main, T, tree, 8, True, 3)
    ww = tq.tq_attention_weights(q, want[1], main, T, 8, True, weights=w)
    cut = tq.evict_rows(main, ww, T, 99, 9)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = tq.tq_tree_attention(q, main, T, tree, 8, True, 3, stream=s)
    gw = tq.tq_attention_weights(q, got[1], main, T, 8, True, weights=w, stream=s)
    gc = tq.evict_rows(main, gw, T, 99, 9, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(gw, ww)
    assert torch.equal(gc[1], cut[1]) and torch.equal(gc[2], cut[2])
    for k in rc.CACHE_KEYS:
        assert torch.equal(gc[0][k].view(torch.uint8), cut[0][k].view(torch.uint8))


def test_refusals_launch_nothing():
    """Bad sizes are turned into errors on the host; the outputs keep their bytes."""
    main, tree = (rc.to_gpu(rc.random_cache(1, 1, n, 64, 8, True, 3, n)) for n in (16, 4))
    q = _q((1, 2, 4, 64), 1).cuda()
    out = torch.full((1, 2, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(tq.TQError):
        tq.tq_tree_attention(q, main, 17, tree, 8, True, 3, out=out)  # T past the capacity
    with pytest.raises(tq.TQError):
        tq.tq_tree_attention(q, main, 16, tree, 8, True, 3, out=out, workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        tq.tq_tree_attention(q, main, 16, tree, 8, True, 3, out=out, lens=torch.tensor([1], device="cuda"))  # int64
    with pytest.raises(ValueError):
        tq.tq_tree_attention(q, main, 16, tree, 8, True, 3, out=out, lens=torch.tensor([1], dtype=torch.int32))  # on the host
    with pytest.raises(ValueError):
        tq.tq_tree_attention(q, main, 16, tree, 8, True, 4, out=out)  # the buffers' widths
    torch.cuda.synchronize()
    assert (out == 7).all()
