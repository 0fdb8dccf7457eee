"""GPU tests of the tree attention and the weight sums in their steady state:
enough tiles a block that every ring of stages, barrier parity and running
maximum is gone through many times (test_gpu_ragged.py has one or two tiles a
block), against 64-bit references computed on the GPU with the tolerances of
ragged_common.py."""
import math

import numpy as np
import pytest
import torch

import turboquant_kv_cache_tq_gb300 as tq
from tests import ragged_common as rc
from tests.gpu_common import require_gpu

pytestmark = pytest.mark.gpu

# Tokens of a tile at most, and what a block's tiles have to exceed: twice the
# eight tiles for which marks of bad values are kept, the longest of the rings.
TILE = {64: 64, 128: 64, 256: 32, 512: 32}
DEPTH = 16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _int(a):
    return None if a is None else torch.tensor(a, dtype=torch.int32, device="cuda")


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


def _decoded(c, T, kb, ks, vb):
    """K and rotated V of tokens [0, T) as float64 (test_gpu_parity.py pins both decodes to the oracle)."""
    k = tq.tq_decode_kv(c, T, kb, ks, vb)[0]
    v = tq.tq_decode_kv_rotated(c, T, kb, ks, vb)[1]
    return k.double(), v.double()


def _reach(parents):
    """[N, N]: whether node i attends to node j."""
    N = len(parents)
    m = np.zeros((N, N), bool)
    for i in range(N):
        m[i, rc.chain(parents, i)] = True
    return torch.tensor(m, device="cuda")


def _rises(s, D, groups):
    """Tiles at which a row's maximum rises past what the kernels let a weight
    grow to, seen by every groups-th tile from the first on (rows of s [R, T],
    scores in units of log 2): the least over the rows."""
    n = s.shape[-1] // TILE[D]
    tiles = s[:, : n * TILE[D]].unflatten(-1, (n, TILE[D])).amax(-1)[:, ::groups]
    m, count = tiles[:, 0], torch.zeros(len(s), device=s.device)
    for j in range(1, tiles.shape[1]):
        up = tiles[:, j] > m + 8
        m, count = torch.where(up, tiles[:, j], m), count + up
    return int(count.min())


def check_tree_call(B, Hkv, G, N, T, D, kb, ks, vb, seed, dtype, lens=None, pad=None, cap=None, tree_cap=None, ramp=None,
                    qscale=1.0, parents="random", edit=None, rises=0):
    """One call with many tiles a block against the formula, and the same bits from a second one."""
    value_halves = 2 if D == 512 else 1
    blocks = -(-G * N // 128)
    real = [(0 if pad is None else pad[b], T if lens is None else lens[b]) for b in range(B)]
    tiles = sum(-(-(hi - lo) // TILE[D]) for lo, hi in real) * Hkv * value_halves * blocks
    assert tiles > DEPTH * torch.cuda.get_device_properties(0).multi_processor_count, "too few tiles a block"
    main = _cache(B, Hkv, T, D, kb, ks, vb, seed, cap, ramp)
    tree = _cache(B, Hkv, N, D, kb, ks, vb, seed + 10, tree_cap, None if ramp is None else ramp[-1:].expand(N))
    if edit is not None:
        edit(main, tree)
    r = np.random.RandomState(seed)
    if isinstance(parents, str):
        parents = np.array([[r.randint(-1, i) if i else -1 for i in range(N)] for _ in range(B)])
        if N > 3:
            parents[-1, N // 2] = -2
    q = _normal((B, Hkv * G, N, D), seed + 20, qscale)
    if ramp is not None:  # queries with a sum of about D
        q = (q.float() + 1).bfloat16()
    need = tq.tq_tree_attention_workspace_size(B, Hkv * G, Hkv, N, D)
    got = []
    for fill in (0x00, 0xFF):  # what the workspace held does not matter
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        got.append(tq.tq_tree_attention(q, main, T, tree, kb, ks, vb, parents=_int(parents), lens=_int(lens),
                                        left_pad=_int(pad), out_dtype=dtype, workspace=ws))
    (out, lse), again = got
    torch.cuda.synchronize()
    assert tq.lib().tq_device_status(None) == 0
    for a, b in zip((out, lse), again):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), "equal calls give other bits"
    K, V = _decoded(main, T, kb, ks, vb)
    Kt, Vt = _decoded(tree, N, kb, ks, vb)
    turn = torch.tensor(rc.rotation(D), device="cuda")
    scale, half = D ** -0.5, rc.HALF
    weight = 2.0 ** -27 if dtype == torch.float32 else 2.0 ** -18
    rounding = 0.0 if dtype == torch.float32 else torch.finfo(dtype).eps / 2
    seen_rises = []
    for b in range(B):
        lo, hi = real[b]
        reach = _reach(parents[b]).repeat(G, 1)  # rows (g, node)
        for h in range(Hkv):
            x = q[b].view(Hkv, G * N, D)[h].double()
            k, v = torch.cat([K[b, h, lo:hi], Kt[b, h]]), torch.cat([V[b, h, lo:hi], Vt[b, h]])
            mask = torch.cat([reach.any(-1, keepdim=True).expand(-1, hi - lo), reach], -1)
            bad = ~torch.isfinite(torch.cat([c["v_scales"][b, h, at].float() for c, at in
                                             ((main, slice(lo, hi)), (tree, slice(0, N)))])).all(-1)
            raw = scale * (x @ k.T)
            spoiled = (mask & (bad | raw.isnan())).any(-1)
            s = torch.where(mask & ~raw.isnan(), raw, -math.inf)
            empty = ~mask.any(-1)
            m = torch.where(empty, 0.0, s.amax(-1))
            p = (s - m[:, None]).exp()
            den = p.sum(-1)
            vf = torch.where(bad[:, None], 0.0, v)
            want = (p @ vf) / torch.where(empty, 1.0, den)[:, None] @ turn
            wl = torch.where(empty, -math.inf, m + den.log())
            want[spoiled], wl[spoiled] = math.nan, math.nan
            kf = torch.nan_to_num(k, 0.0, 0.0, 0.0).abs()
            mag = torch.where(mask, scale * (x.abs() @ kf.T), 0.0).amax(-1)
            top = torch.where(torch.isfinite(s), s.abs(), 0.0).amax(-1)
            # (the derivation is tree_reference's)
            e = (D / 16 + 4) * 2 * half * mag + top * 2.0 ** -22 + 2.0 ** -21
            steps = (mask.sum(-1) / 16 + 32 + math.log2(D)) * 2 * half
            tol = (2 * (e + weight) + 2 * steps) * (mask * vf.norm(dim=-1)).amax(-1)
            ltol = e + steps + wl.abs() * 4 * half + 2.0 ** -21
            g, gl = out[b].view(Hkv, G * N, D)[h].double(), lse[b].view(Hkv, G * N)[h].double()
            what = "row %d head %d" % (b, h)
            assert torch.equal(g.isnan(), want.isnan()) and torch.equal(gl.isnan(), wl.isnan()), what
            assert (g[empty] == 0).all() and torch.isneginf(gl[empty]).all(), what
            fine = ~empty & ~spoiled
            err = (g - want)[fine].norm(dim=-1) / (tol[fine] + rounding * (want[fine].norm(dim=-1) + tol[fine]))
            lerr = (gl - wl)[fine].abs() / ltol[fine]
            if fine.any():
                assert err.max() <= 1, "%s: an output is %.3g times its tolerance off" % (what, err.max())
                assert lerr.max() <= 1, "%s: an lse is %.3g times its tolerance off" % (what, lerr.max())
                if rises:
                    seen_rises.append(_rises(s[fine][:, : hi - lo] / math.log(2), D, 2 if D <= 128 else 1))
    if rises:
        assert min(seen_rises) >= rises, "the maximum rises %d times only" % min(seen_rises)
    return out, lse


# sequences, kv heads, tokens: 20 to 30 tiles a block of 152, most of them of one segment
SIZES = {64: (8, 8, 4096), 128: (8, 8, 4096), 256: (8, 4, 4096), 512: (3, 4, 4096)}


def _ramp(T, D):
    """What grows along the keys, so that (q about one in every element, scaled
    by D^-1/2) scores rise by 12 a pair of tiles where two groups take the tiles
    in turn, else by 10 a tile: 17 and 14 units of log 2, where the running
    maximum follows from 8 on. Scores beside that vary by about one."""
    rise = 6 if D <= 128 else 10
    return torch.arange(T, device="cuda") * (rise / TILE[D] / math.sqrt(D))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("G,N", [(4, 8), (5, 16)])  # few rows, more than 64 of them
def test_tree_maximum_rises_many_times_in_a_block(D, dtype, G, N):
    B, Hkv, T = SIZES[D]
    check_tree_call(B, Hkv, G, N, T, D, 8, True, 8, D + G, dtype, ramp=_ramp(T, D), qscale=0.5, rises=20)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("cap,tree_cap", [(4352, 16), (4307, 11)])  # bulk copies, narrow copies
def test_tree_ragged_rows_of_many_tiles(D, dtype, cap, tree_cap):
    """Unequal lengths and pads; heads change inside a block at other tiles of the rings."""
    B, Hkv, _ = SIZES[D]
    T = 4301
    lens = [T - 97 * b for b in range(B)]
    pad = [(13 * b) % 50 for b in range(B)]
    for kb, ks, vb in ((8, True, 3), (5, False, 5), (2, False, 2), (4, False, 4)):
        check_tree_call(B, Hkv, 2, 7, T, D, kb, ks, vb, D + kb + vb, dtype, lens=lens, pad=pad, cap=cap,
                        tree_cap=tree_cap, qscale=2.0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D", [64, 128, 256, 512])
def test_tree_marks_of_bad_values_in_far_tiles(D, dtype):
    """Value groups with infinite and NaN scales at places far apart, in a few
    heads, in one node of a tree, and outside the sequences: the rows that
    attend to one are NaN, all others are right."""
    B, Hkv, T = SIZES[D]
    N, G = 6, 4
    lens, pad = [T - 5 * b for b in range(B)], [20] * B
    par = np.array([[-1, 0, 0, 1, 2, -1]] * B)

    def edit(main, tree):
        inf, nan = math.inf, math.nan
        main["v_scales"][0, 0, 25, 0] = inf
        main["v_scales"][0, 1, T - 1, 1] = nan
        main["v_scales"][1, 2, T // 2 + 3, 0] = -inf
        main["v_scales"][1, 2, T // 2 + 700, 1] = nan
        main["v_scales"][:, :, :20] = inf
        for b in range(B):
            main["v_scales"][b, :, lens[b]:] = nan
        tree["v_scales"][2, :, 1, 0] = inf
        tree["v_scales"][0, 3, 5, 1] = nan

    out, lse = check_tree_call(B, Hkv, G, N, T, D, 8, True, 3, D, dtype, lens=lens, pad=pad, edit=edit, parents=par)
    rows = lse.view(B, Hkv, G, N).isnan()
    assert rows[0, :2].all() and rows[1, 2].all() and rows[2, :, :, [1, 3]].all() and rows[0, 3, :, 5].all()
    assert int(rows.sum()) == 3 * G * N + Hkv * G * 2 + G


@pytest.mark.parametrize("D", [64, 128, 256, 512])
def test_tree_more_rows_than_a_block_and_a_rising_maximum(D):
    B, Hkv, T = SIZES[D]
    B = (B + 1) // 2
    check_tree_call(B, Hkv, 3, 50, T, D, 8, False, 5, D, torch.bfloat16, ramp=_ramp(T, D), qscale=0.5, rises=20)


# ---- weight sums ------------------------------------------------------------------
def check_weights_call(B, Hkv, G, N, T, D, kb, ks, seed, lens=None, pad=None, cap=None, in_place=False, n_path=None,
                       path=None):
    P = N if path is None else len(path[0])
    token_rows = 128 if D <= 128 else 64
    real = [(0 if pad is None else pad[b], T if lens is None else lens[b]) for b in range(B)]
    tiles = sum(-(-(hi - lo) // token_rows) for lo, hi in real) * Hkv
    assert tiles > DEPTH * torch.cuda.get_device_properties(0).multi_processor_count, "too few tiles a block"
    c = _cache(B, Hkv, T, D, kb, ks, 2, seed, cap)
    q = _normal((B, Hkv * G, N, D), seed + 2)
    g = torch.Generator(device="cuda").manual_seed(seed)
    lse = math.log(T) + 0.5 + torch.rand((B, Hkv * G, N), generator=g, device="cuda")
    lse[0, 0, 0] = -math.inf
    start = torch.rand((B, Hkv, T), generator=g, device="cuda")
    got = []
    for _ in range(2):
        w = start.clone()
        out = w if in_place else torch.full_like(w, 7.0)
        tq.tq_attention_weights(q, lse, c, T, kb, ks, path=_int(path), n_path=_int(n_path), lens=_int(lens),
                                left_pad=_int(pad), weights=w, out=out)
        got.append(out)
    torch.cuda.synchronize()
    assert tq.lib().tq_device_status(None) == 0
    assert torch.equal(*got), "equal calls give other bits"
    K = _decoded(c, T, kb, ks, 2)[0]
    scale, half = D ** -0.5, rc.HALF
    t = torch.arange(T, device="cuda")
    for b in range(B):
        lo, hi = real[b]
        n = P if n_path is None else min(max(n_path[b], 0), P)
        nodes = list(range(n)) if path is None else path[b][:n]
        last = hi - n + torch.arange(n, device="cuda")
        sees = (t >= lo) & (t <= last[:, None])  # [n, T]
        for h in range(Hkv):
            x = q[b].view(Hkv, G, N, D)[h][:, nodes].double()
            ls = lse[b].view(Hkv, G, N)[h][:, nodes].double()[..., None]
            s = scale * (x @ K[b, h].T)
            w = torch.where(sees & (ls != -math.inf), (s - ls).exp(), 0.0)
            mag = scale * (x.abs() @ K[b, h].abs().T)
            # (the derivation is weights_reference's)
            e = (D / 16 + 4) * 2 * half * mag + (s.abs() + torch.where(ls == -math.inf, 0.0, ls.abs())) * 2.0 ** -22 + 2.0 ** -21
            want = start[b, h].double() + w.sum((0, 1))
            tol = start[b, h].double() * 2 * half + (w * (e + (G * n + 2) * 2 * half)).sum((0, 1))
            off = (got[0][b, h].double() - want).abs() - tol
            assert (off <= 0).all(), "row %d head %d: off by %.3g beyond its tolerance" % (b, h, off.max())
            outside = (t < lo) | (t >= hi)
            assert torch.equal(got[0][b, h][outside], start[b, h][outside])


WEIGHT_SIZES = {64: (8, 8, 6100), 128: (8, 8, 6100), 256: (8, 4, 6100), 512: (8, 4, 6100)}


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256, 512])
def test_weights_rounds_of_columns_over_many_tiles(D, in_place):
    """More observers than a round's columns, many tiles a block, heads that change inside a block."""
    B, Hkv, T = WEIGHT_SIZES[D]
    lens, pad = [T - 61 * b for b in range(B)], [(17 * b) % 40 for b in range(B)]
    P = {64: 90, 128: 90, 256: 45, 512: 45}[D]  # with four heads 360 columns (of 256), 180 (of 128 or 64)
    check_weights_call(B, Hkv, 4, P, T, D, 8, True, D, lens=lens, pad=pad, in_place=in_place,
                       n_path=[P - 11 * b for b in range(B)] if D <= 128 else [P - 5 * b for b in range(B)])


@pytest.mark.parametrize("D", [64, 128, 256, 512])
def test_weights_short_paths_and_narrow_copies_over_many_tiles(D):
    B, Hkv, T = WEIGHT_SIZES[D]
    path = [[(3 * i + b) % 16 for i in range(6)] for b in range(B)]
    for kb, ks in ((8, False), (5, False), (2, False)):
        check_weights_call(B, Hkv, 3, 16, T, D, kb, ks, D + kb, cap=6103, lens=[T - 3 * b for b in range(B)], path=path,
                           n_path=[1 + b % 6 for b in range(B)])


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
