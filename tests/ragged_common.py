"""Plain references, in 64 bits, of the calls on ragged packed caches, and the
tolerances of their tests.

Decoded keys and rotated values come from the CPU oracle's bf16 decode of the
same packed bytes; everything after that is numpy in double precision.
"""
from __future__ import annotations

import math

import numpy as np
import torch

import oracle
from tests.gpu_common import cache_from_numpy

CACHE_KEYS = ("k_codes", "k_scales", "k_zeros", "v_codes", "v_scales")
HALF = 2.0 ** -24  # half a step of fp32, relative


def bits_of(t):
    return t.cpu().contiguous().view(torch.int16).numpy().view(np.uint16)


def bf16(t):
    return t.detach().cpu().float().numpy().astype(np.float64)


def encode(k, v, kb, ks, vb, t_cap=None):
    from tests.gpu_common import oracle_encode

    return oracle_encode(k, v, kb, ks, vb, t_cap=t_cap)


def random_cache(B, H, T, D, kb, ks, vb, seed, t_cap=None, kscale=1.0, vscale=1.0):
    """A packed cache of normal keys and values (numpy dict)."""
    g = torch.Generator().manual_seed(seed)
    k = (torch.randn((B, H, T, D), generator=g) * kscale).bfloat16()
    v = (torch.randn((B, H, T, D), generator=g) * vscale).bfloat16()
    return encode(k, v, kb, ks, vb, t_cap=t_cap)


def to_gpu(cache):
    return cache_from_numpy(cache)


def decoded(cache, T, kb, ks, vb):
    """K and rotated V of tokens [0, T) as float64 [B, H, T, D]."""
    if T == 0:
        B, H = cache["k_codes"].shape[:2]
        D = cache["k_scales"].shape[-1] * 32
        return np.zeros((B, H, 0, D)), np.zeros((B, H, 0, D))
    k, v = oracle.decode_kv(cache, T, kb, ks, vb, out_dtype=oracle.BF16, rotated_v=True)
    return oracle.bf16_bits_to_f32(k).astype(np.float64), oracle.bf16_bits_to_f32(v).astype(np.float64)


def hadamard(D):
    h = np.ones((1, 1))
    while h.shape[0] < D:
        h = np.block([[h, h], [h, -h]])
    return h


def rotation(D):
    """The inverse value rotation as a matrix: y = x @ rotation(D)."""
    sign = np.array(oracle.sign_vector(D), dtype=np.float64)
    return hadamard(D) / math.sqrt(D) * sign


def chain(parents, i):
    """The nodes node i attends to ([] when it is absent)."""
    seen = []
    while True:
        seen.append(i)
        up = int(parents[i])
        if up == -1:
            return seen
        if up < 0 or up >= i:
            return []
        i = up


def ranges(B, T, lens, left_pad):
    out = []
    for b in range(B):
        hi = T if lens is None else min(max(int(lens[b]), 0), T)
        lo = 0 if left_pad is None else min(max(int(left_pad[b]), 0), hi)
        out.append((lo, hi))
    return out


def tree_reference(q, cache, T, tree, kb, ks, vb, parents=None, lens=None, left_pad=None, scale=None,
                   dtype=torch.float32):
    """-> (out, lse, tolerance of a row's 2-norm, tolerance of lse), float64.

    Tolerances. With exact products of bf16 operands, what the kernels round is
    (1) a score: at most D / 16 + 4 accumulations in fp32, each at most one
    step (2^-23) of the sum of the products' magnitudes, so the weight's
    exponent is off by ds = (D / 16 + 4) 2^-23 scale sum |q K|, and the
    multiplication by scale log2(e), the subtraction of the running maximum
    and exp2 add 2^-22 of the largest |score| and 2^-21; (2) the weights, as
    two bf16 parts for a bf16 output (2^-18), as three for an fp32 one (2^-27);
    (3) the sums over tokens, at most one step for each
    of T / 16 + 32 partial sums and merges; the weights' own sum the same; the
    inverse rotation one step a stage. A relative error e of the weights moves
    the output by at most 2 e max_t |V_t| (2-norm, which the rotation keeps),
    since numerator and denominator may be off by e each."""
    B, Hq, N, D = q.shape
    Hkv = cache["k_codes"].shape[1]
    G = Hq // Hkv
    scale = D ** -0.5 if scale is None else scale
    with np.errstate(all="ignore"):
        K, V = decoded(cache, T, kb, ks, vb)
        Kt, Vt = decoded(tree, N, kb, ks, vb)
    q = bf16(q)
    out = np.zeros((B, Hq, N, D))
    lse = np.full((B, Hq, N), -np.inf)
    tol, ltol = np.zeros((B, Hq, N)), np.zeros((B, Hq, N))
    R = rotation(D)
    rg = ranges(B, T, lens, left_pad)
    sv, st = cache["v_scales"].view(np.float16), tree["v_scales"].view(np.float16)
    for b in range(B):
        lo, hi = rg[b]
        for i in range(N):
            seen = chain(parents[b], i) if parents is not None else list(range(i + 1))
            if not seen:
                continue
            seen = sorted(seen)
            for hq in range(Hq):
                h = hq // G
                k = np.concatenate([K[b, h, lo:hi], Kt[b, h, seen]])
                v = np.concatenate([V[b, h, lo:hi], Vt[b, h, seen]])
                ok = np.isfinite(sv[b, h, lo:hi]).all() and np.isfinite(st[b, h, seen]).all()
                with np.errstate(all="ignore"):
                    s = scale * (k @ q[b, hq, i])
                    if np.isnan(s).any() or not ok or np.isposinf(s).any():
                        out[b, hq, i], lse[b, hq, i] = np.nan, np.nan
                        continue
                    m = s.max()
                    p = np.exp(s - m)
                    out[b, hq, i] = (p @ v) / p.sum() @ R
                    lse[b, hq, i] = m + np.log(p.sum())
                    mag = abs(scale) * (np.abs(k) @ np.abs(q[b, hq, i])).max()
                e = (D / 16 + 4) * 2 * HALF * mag + np.abs(s).max() * 2.0 ** -22 + 2.0 ** -21
                steps = (len(s) / 16 + 32 + math.log2(D)) * 2 * HALF
                tol[b, hq, i] = (2 * (e + (2.0 ** -27 if dtype == torch.float32 else 2.0 ** -18)) + 2 * steps) * np.sqrt((v * v).sum(-1)).max()
                ltol[b, hq, i] = e + steps + abs(lse[b, hq, i]) * 4 * HALF + 2.0 ** -21
    return out, lse, tol, ltol


def check_tree(got, got_lse, ref, what=""):
    out, lse, tol, ltol = ref
    dtype = got.dtype
    g = got.detach().cpu().float().numpy().astype(np.float64)
    gl = got_lse.detach().cpu().numpy().astype(np.float64)
    nan = np.isnan(lse)
    assert np.array_equal(np.isnan(g), np.isnan(out)), "%s: NaN rows differ" % what
    assert np.array_equal(np.isnan(gl), nan), "%s: NaN lse differ" % what
    empty = np.isneginf(lse)
    assert np.all(g[empty] == 0) and np.all(np.isneginf(gl[empty])), "%s: rows without a key" % what
    fine = ~nan & ~empty
    if not fine.any():
        return
    rounding = 0.0 if dtype == torch.float32 else torch.finfo(dtype).eps / 2
    err = np.sqrt(((g - out)[fine] ** 2).sum(-1))
    lim = tol[fine] + rounding * (np.sqrt((out[fine] ** 2).sum(-1)) + tol[fine])
    worst = (err / lim).max()
    assert worst <= 1, "%s: a row is %.3g times its tolerance off" % (what, worst)
    lerr = (np.abs(gl[fine] - lse[fine]) / ltol[fine]).max()
    assert lerr <= 1, "%s: an lse is %.3g times its tolerance off" % (what, lerr)


def weights_reference(q, lse, cache, T, kb, ks, path=None, n_path=None, lens=None, left_pad=None, scale=None,
                      weights=None, w_cap=None):
    """-> (weights, tolerance), float64 [B, Hkv, w_cap]. A term's exponent is
    off as in tree_reference, its exp by 2^-21 of itself more, and the sum by
    one step for each of its terms."""
    B, Hq, N, D = q.shape
    Hkv = cache["k_codes"].shape[1]
    G = Hq // Hkv
    scale = D ** -0.5 if scale is None else scale
    w_cap = T if w_cap is None else w_cap
    K = decoded(dict(cache), T, kb, ks, 8)[0] if "v_codes" in cache else decoded_keys(cache, T, kb, ks)
    q, lse = bf16(q), lse.detach().cpu().numpy().astype(np.float64)
    out = np.zeros((B, Hkv, w_cap)) if weights is None else weights.detach().cpu().numpy().astype(np.float64)
    tol = np.abs(out) * 2 * HALF
    path = None if path is None else np.asarray(path)
    P = N if path is None else path.shape[1]
    rg = ranges(B, T, lens, left_pad)
    for b in range(B):
        lo, hi = rg[b]
        n = P if n_path is None else min(max(int(n_path[b]), 0), P)
        for i in range(n):
            node = i if path is None else int(path[b, i])
            last = hi - n + i
            if node < 0 or node >= N or last < lo:
                continue
            for hq in range(Hq):
                if np.isneginf(lse[b, hq, node]):
                    continue
                k = K[b, hq // G, lo:last + 1]
                with np.errstate(all="ignore"):
                    x = scale * (k @ q[b, hq, node])
                    w = np.exp(x - lse[b, hq, node])
                    mag = abs(scale) * (np.abs(k) @ np.abs(q[b, hq, node]))
                    e = (D / 16 + 4) * 2 * HALF * mag + (np.abs(x) + abs(lse[b, hq, node])) * 2.0 ** -22 + 2.0 ** -21
                    out[b, hq // G, lo:last + 1] += w
                    tol[b, hq // G, lo:last + 1] += w * (e + (G * n + 2) * 2 * HALF)
    return out, tol


def decoded_keys(cache, T, kb, ks):
    B, H, cap = cache["k_codes"].shape[:3]
    G = cache["k_scales"].shape[-1]
    full = dict(cache, v_codes=np.zeros((B, H, cap, G * 8), np.uint8), v_scales=np.zeros((B, H, cap, G), np.uint16))
    return decoded(full, T, kb, ks, 2)[0]


def check_weights(got, ref, what=""):
    want, tol = ref
    g = got.detach().cpu().numpy().astype(np.float64)
    assert np.array_equal(np.isnan(g), np.isnan(want)), "%s: NaN differ" % what
    fine = np.isfinite(want)
    assert np.array_equal(g[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)]), "%s: infinities differ" % what
    err = np.abs(g[fine] - want[fine]) - tol[fine]
    assert np.all(err <= 0), "%s: off by %.3g beyond its tolerance" % (what, err.max())


def select_reference(weights, T, keep, recent, lens=None, left_pad=None):
    w = weights.detach().cpu().numpy()
    B, H = w.shape[:2]
    index = np.full((B, H, keep), -1, np.int32)
    count = np.zeros((B,), np.int32)
    for b, (lo, hi) in enumerate(ranges(B, T, lens, left_pad)):
        count[b] = min(hi - lo, keep)
        for h in range(H):
            if hi - lo <= keep:
                chosen = list(range(lo, hi))
            else:
                late = list(range(hi - recent, hi))
                rest = range(lo, hi - recent)
                key = {t: (-np.inf if np.isnan(w[b, h, t]) else w[b, h, t]) for t in rest}
                chosen = sorted(sorted(rest, key=lambda t: (-key[t], t))[: keep - recent]) + late
            index[b, h, : len(chosen)] = chosen
    return index, count


def gather_reference(src, dst, index, count=None, dst_off=None, src_weights=None, dst_weights=None):
    """dst (numpy dicts), its weights and lengths after the copy."""
    index = np.asarray(index)
    B, H, s_cap = src["k_codes"].shape[:3]
    d_cap = dst["k_codes"].shape[2]
    n = index.shape[-1]
    out = {k: dst[k].copy() for k in CACHE_KEYS}
    ow = None if dst_weights is None else np.array(dst_weights, copy=True)
    length = np.zeros((B,), np.int32)
    for b in range(B):
        c = n if count is None else min(max(int(count[b]), 0), n)
        off = 0 if dst_off is None else max(int(dst_off[b]), 0)
        length[b] = min(off + c, d_cap)
        for h in range(H):
            for j in range(c):
                t = int(index[b, h, j] if index.ndim == 3 else index[b, j])
                if not 0 <= t < s_cap or off + j >= d_cap:
                    continue
                for k in CACHE_KEYS:
                    out[k][b, h, off + j] = src[k][b, h, t]
                if ow is not None:
                    ow[b, h, off + j] = 0.0 if src_weights is None else src_weights[b, h, t]
    return out, ow, length
