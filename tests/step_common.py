"""Plain references, in 64 bits, of the calls on new tokens (append, window
attention, shared-prefix attention), and the tolerances of their tests."""
from __future__ import annotations

import math

import numpy as np
import torch

import turboquant_kv_cache_tq_gb300 as tq
from tests import ragged_common as rc

HALF = 2.0 ** -24  # half a step of fp32, relative


def ints(a, device="cuda"):
    return None if a is None else torch.tensor(a, dtype=torch.int32, device=device)


def normal(shape, seed, scale=1.0, dtype=torch.bfloat16, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)
    return (torch.randn(shape, generator=g, device=device) * scale).to(dtype)


def cache(B, H, T, D, kb, ks, vb, seed, cap=None, offset=0.0):
    """A packed cache of normal keys and values; what lies behind T is garbage."""
    c = tq.alloc_cache(B, H, T if cap is None else cap, D, kb, vb)
    for t in c.values():
        t.view(torch.uint8).fill_(0xFF)  # (scales and zero points of NaN)
    if B and T:
        tq.tq_encode_kv(normal((B, H, T, D), seed) + offset, normal((B, H, T, D), seed + 1), kb, ks, vb, c)
    return c


def decoded(c, T, kb, ks, vb):
    """K and rotated V of tokens [0, T) in float64 (test_gpu_parity.py pins both decodes to the oracle)."""
    B, H = c["k_codes"].shape[:2]
    D = c["k_scales"].shape[-1] * 32
    if not T or not B:
        return (torch.zeros((B, H, T, D), dtype=torch.float64, device="cuda"),) * 2
    k = tq.tq_decode_kv(c, T, kb, ks, vb)[0]
    v = tq.tq_decode_kv_rotated(c, T, kb, ks, vb)[1]
    return k.double(), v.double()


def clamp(x, B, lo, hi, default):
    return [min(max(int(default if x is None else x[b]), lo), hi) for b in range(B)]


def seen(B, N, T, lens=None, left_pad=None, count=None, window=1 << 30, sinks=0):
    """[B, N, T]: which of its sequence's tokens a new token sees; and [B, N], which new tokens there are."""
    hi = clamp(lens, B, 0, T, T)
    n_new = clamp(count, B, 0, N, N)
    out, there = np.zeros((B, N, T), bool), np.zeros((B, N), bool)
    for b in range(B):
        lo = 0 if left_pad is None else min(max(int(left_pad[b]), 0), hi[b])
        for n in range(n_new[b]):
            p = hi[b] - n_new[b] + n
            if p < lo:
                continue
            there[b, n] = True
            for a, z in ((lo, min(lo + sinks, p + 1)), (max(lo, p - window + 1), p + 1)):
                out[b, n, a:z] = True
    return out, there


def reference(q, c, T, kb, ks, vb, lens=None, left_pad=None, count=None, window=1 << 30, sinks=0, scale=None,
              prefix=None, P=0, prefix_lens=None, dtype=torch.float32):
    """-> (out, lse, tolerance of a row's 2-norm, tolerance of lse), float64 on the GPU.

    Tolerances. With exact products of bf16 operands, what the kernels round is
    (1) a score: at most D / 16 + 4 accumulations in fp32, each at most one
    step (2^-23) of the sum of the products' magnitudes, so the weight's
    exponent is off by ds = (D / 16 + 4) 2^-23 scale sum |q K|, and the
    multiplication by scale log2(e), the subtraction of the running maximum
    and exp2 add 2^-22 of the largest |score| and 2^-21; (2) the weights, as
    two bf16 parts for a bf16 output (2^-18), as three for an fp32 one (2^-27);
    (3) the sums over tokens, at most one step for each of t / 16 + 64 partial
    sums and merges of t tokens; the weights' own sum the same; the inverse rotation one step a
    stage. A relative error e of the weights moves the output by at most 2 e
    max_t |V_t| (2-norm, which the rotation keeps), since numerator and
    denominator may be off by e each."""
    B, Hq, N, D = q.shape
    Hkv = c["k_codes"].shape[1]
    G = Hq // Hkv
    scale = D ** -0.5 if scale is None else scale
    K, V = decoded(c, T, kb, ks, vb)
    bad = ~torch.isfinite(c["v_scales"][:, :, :T].float()).all(-1)
    mask, there = (torch.tensor(x, device="cuda") for x in seen(B, N, T, lens, left_pad, count, window, sinks))
    if prefix is not None:
        Bp = prefix["k_codes"].shape[0]
        Kp, Vp = decoded(prefix, P, kb, ks, vb)
        bp = ~torch.isfinite(prefix["v_scales"][:, :, :P].float()).all(-1)
        n = torch.tensor(clamp(prefix_lens, Bp, 0, P, P), device="cuda")
        mp = (torch.arange(P, device="cuda") < n[:, None])
        Kp, Vp, bp, mp = (x.repeat_interleave(B // Bp, 0) for x in (Kp, Vp, bp, mp))
        K, V, bad = torch.cat([Kp, K], 2), torch.cat([Vp, V], 2), torch.cat([bp, bad], 2)
        mask = torch.cat([mp[:, None] & there[..., None], mask], 2)
    qq = q.double().view(B, Hkv, G, N, D)
    out = torch.zeros((B, Hkv, G, N, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hkv, G, N), -math.inf, dtype=torch.float64, device="cuda")
    tol, ltol = torch.zeros_like(lse), torch.zeros_like(lse)
    turn = torch.tensor(rc.rotation(D), device="cuda")
    for b in range(B):
        for n in range(N):
            t = mask[b, n].nonzero()[:, 0]
            if not len(t):
                continue
            k, v = K[b][:, t], V[b][:, t]
            s = scale * torch.einsum("htd,hgd->hgt", k, qq[b, :, :, n])
            nan = s.isnan().any(-1) | (s == math.inf).any(-1) | bad[b][:, t].any(-1)[:, None]
            m = s.amax(-1, keepdim=True)
            p = (s - m).exp()
            o = torch.einsum("hgt,htd->hgd", p, v) / p.sum(-1, keepdim=True)
            out[b, :, :, n] = torch.where(nan[..., None], math.nan, o @ turn)
            lse[b, :, :, n] = torch.where(nan, math.nan, (m + p.sum(-1, keepdim=True).log())[..., 0])
            mag = abs(scale) * torch.einsum("htd,hgd->hgt", k.abs(), qq[b, :, :, n].abs()).amax(-1)
            e = (D / 16 + 4) * 2 * HALF * mag + s.abs().amax(-1) * 2.0 ** -22 + 2.0 ** -21
            steps = (len(t) / 16 + 64 + math.log2(D)) * 2 * HALF
            vmax = v.square().sum(-1).sqrt().amax(-1)[:, None]
            tol[b, :, :, n] = (2 * (e + (2.0 ** -27 if dtype == torch.float32 else 2.0 ** -18)) + 2 * steps) * vmax
            ltol[b, :, :, n] = e + steps + lse[b, :, :, n].abs() * 4 * HALF + 2.0 ** -21
    return [x.view(B, Hq, *x.shape[3:]) for x in (out, lse, tol, ltol)]


def check(got, got_lse, ref, what=""):
    out, lse, tol, ltol = ref
    g, gl = got.double(), got_lse.double()
    nan = lse.isnan()
    assert torch.equal(g.isnan(), out.isnan()), "%s: NaN rows differ" % what
    assert torch.equal(gl.isnan(), nan), "%s: NaN lse differ" % what
    empty = lse == -math.inf
    assert (g[empty] == 0).all() and (gl[empty] == -math.inf).all(), "%s: rows without a key" % what
    fine = ~nan & ~empty
    if not fine.any():
        return
    f32 = got.dtype == torch.float32
    rounding = 0.0 if f32 else torch.finfo(got.dtype).eps / 2
    err = (g - out)[fine].norm(dim=-1)
    lim = tol[fine] + rounding * (out[fine].norm(dim=-1) + tol[fine])
    worst = (err / lim).max().item()
    assert worst <= 1, "%s: a row is %.3g times its tolerance off" % (what, worst)
    lerr = ((gl[fine] - lse[fine]).abs() / ltol[fine]).max().item()
    assert lerr <= 1, "%s: an lse is %.3g times its tolerance off" % (what, lerr)


# ---- append ---------------------------------------------------------------------------
def turned(x, cos, sin, positions, interleaved):
    """Rows [B, H, N, D] in fp32, every product and sum rounded once (numpy)."""
    x = x.detach().float().cpu().numpy().astype(np.float32)
    cos, sin = (t.cpu().numpy() for t in (cos, sin))
    R = 2 * cos.shape[1]
    at = np.clip(np.asarray(positions, dtype=np.int64), 0, cos.shape[0] - 1)
    c, s = cos[at][:, None], sin[at][:, None]
    out = x.copy()
    i = np.arange(R // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
    with np.errstate(all="ignore"):
        out[..., a] = x[..., a] * c - x[..., b] * s
        out[..., b] = x[..., b] * c + x[..., a] * s
    return out


def append_reference(k, v, before, lens, kb, ks, vb, cos=None, sin=None, interleaved=False, q=None, positions=None,
                     left_pad=None, count=None):
    """-> (the cache's bytes after the call as torch tensors on the GPU, turned q in fp32 or None, new lengths). The
    bytes of a token are those that tq_encode_kv gives for the turned fp32 key and the value."""
    B, H, N, D = k.shape
    cap = before["k_codes"].shape[2]
    off = [max(int(x), 0) for x in lens] if lens is not None else [0] * B
    n_new = clamp(count, B, 0, N, N)
    if positions is None:
        pad = [0] * B if left_pad is None else [min(max(int(left_pad[b]), 0), off[b]) for b in range(B)]
        positions = np.array([[off[b] - pad[b] + n for n in range(N)] for b in range(B)]).reshape(B, N)
    kt = k.float().cpu().numpy() if cos is None else turned(k, cos, sin, positions, interleaved)
    after = {name: t.clone() for name, t in before.items()}
    if B and N:
        new = tq.alloc_cache(B, H, N, D, kb, vb)
        tq.tq_encode_kv(torch.from_numpy(kt).cuda().contiguous(), v.float().contiguous(), kb, ks, vb, new)
        for b in range(B):
            m = max(min(n_new[b], cap - off[b]), 0)
            for name in after:
                after[name][b, :, off[b]:off[b] + m] = new[name][b, :, :m]
    qt = None
    if q is not None:
        qt = torch.from_numpy(turned(q, cos, sin, positions, interleaved) if cos is not None else q.float().cpu().numpy())
    return after, qt, [min(off[b] + n_new[b], cap) for b in range(B)]


def same_bytes(a, b):
    return all(torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8)) for k in a)
