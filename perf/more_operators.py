"""Cases of one layer's step on ragged packed caches, the plain forms of its operators and their exact results.

The operators: new tokens rotated to their positions, quantised and written at every sequence's own end (`append`),
attention of new tokens over a sliding window and a few first tokens of each sequence (`window`), and attention over a
prefix that several sequences share and over each sequence's own tokens (`prefix`).

A packed cache row (batch row, kv head, token) holds keys as codes with an fp16 scale and zero point per group of 32
elements, K = bf16((code + zero) * scale), and rotated values as table indices with an fp16 scale per group,
V = bf16(centroid * scale); attention runs on the rotated values, and its output is turned back by the Hadamard
transform / sqrt(D) and the sign vector. The codec fixes every rounding of an encode (fp32, one rounding an operation),
so the packed bytes are whole numbers that have one right value.
"""
import math
import random

import torch

own = False

GROUP = 32
#: Centroids of the value tables by bit width (the cache format's constants).
CENTROIDS = {
    2: (
        -1.51447499, -0.45822522, 0.4486323, 1.51215208,
    ),
    3: (
        -2.15194988, -1.34390998, -0.756009996, -0.245089993, 0.245089993, 0.756009996, 1.34390998, 2.15194988,
    ),
    4: (
        -2.76566267, -2.09952307, -1.6401931, -1.27662992, -0.960249186, -0.673130453, -0.403818518, -0.142727122,
        0.117162906, 0.379088163, 0.647577643, 0.93377775, 1.25230753, 1.62176251, 2.07574821, 2.72072792,
    ),
    5: (
        -3.34820437, -2.7744689, -2.39178157, -2.08856535, -1.83827627, -1.62735081, -1.4368273, -1.25994205,
        -1.09586811, -0.941173851, -0.793228626, -0.650904477, -0.511321127, -0.37372008, -0.2373216, -0.102789663,
        0.0317942873, 0.164198548, 0.300100625, 0.439542502, 0.580825627, 0.727580249, 0.873896539, 1.02939796,
        1.19426072, 1.37287045, 1.56764567, 1.77888131, 2.02251363, 2.30951571, 2.66635156, 3.2329483,
    ),
    8: (
        -4.50567865, -4.45461845, -4.43628597, -4.40158939, -4.36323977, -4.33219719, -4.29750061, -4.26280403,
        -4.22810793, -4.19341183, -4.15871525, -4.12401867, -4.0944376, -4.04575825, -4.00262117, -4.00217152,
        -3.94239211, -3.91680169, -3.8863256, -3.84775352, -3.79886436, -3.76279426, -3.74451518, -3.70696044,
        -3.67462158, -3.63148546, -3.59501195, -3.58025694, -3.53995252, -3.50384212, -3.46715689, -3.4281671,
        -3.39812803, -3.36313319, -3.32746673, -3.29197431, -3.2577858, -3.22009683, -3.19298172, -3.15723801,
        -3.11180258, -3.08213401, -3.05064034, -3.01481104, -2.98015881, -2.94645143, -2.91119051, -2.87472129,
        -2.84122705, -2.80610228, -2.77168679, -2.73760104, -2.70292187, -2.66344619, -2.63037777, -2.59961796,
        -2.56089878, -2.52527523, -2.49475455, -2.46137404, -2.42400932, -2.38777113, -2.35051441, -2.31639862,
        -2.28237486, -2.24365282, -2.20979595, -2.17706394, -2.14471698, -2.11136937, -2.07867384, -2.04449439,
        -2.00639272, -1.96986961, -1.93009889, -1.89317, -1.8589747, -1.82121062, -1.78488111, -1.74654865,
        -1.71034062, -1.67431962, -1.63937545, -1.60405171, -1.57082164, -1.53654802, -1.50356638, -1.4691751,
        -1.43506563, -1.40220082, -1.36889982, -1.33558917, -1.30184495, -1.26983678, -1.23553228, -1.20119047,
        -1.16646945, -1.13050497, -1.09593332, -1.06143272, -1.02749336, -0.994027138, -0.960926235, -0.92738539,
        -0.892908275, -0.859346271, -0.826147497, -0.793744266, -0.758828282, -0.723001719, -0.687129736,
        -0.651774585, -0.616251647, -0.581151485, -0.546266854, -0.511128128, -0.475061059, -0.439445883,
        -0.404982328, -0.369819641, -0.334137887, -0.299191833, -0.264652461, -0.231688678, -0.200136259,
        -0.167214751, -0.134137928, -0.100328237, -0.0657153204, -0.031323947, 0.00434282701, 0.0403724611,
        0.074515067, 0.107615396, 0.140435055, 0.174268574, 0.208128259, 0.243044406, 0.277972639, 0.31494686,
        0.350885689, 0.387439877, 0.422298372, 0.456864834, 0.491283506, 0.525663376, 0.558622718, 0.591042757,
        0.624955237, 0.659494579, 0.694283545, 0.727847457, 0.762456179, 0.79638499, 0.830988765, 0.864448369,
        0.898106396, 0.932024539, 0.966624379, 1.00069964, 1.03437936, 1.06806338, 1.10186052, 1.13556361, 1.17071009,
        1.20386875, 1.23885643, 1.27442825, 1.31021035, 1.34411871, 1.37696886, 1.40916574, 1.44245946, 1.47704709,
        1.51275897, 1.54820752, 1.58390474, 1.61932015, 1.65540004, 1.69247389, 1.72731769, 1.76187444, 1.79856312,
        1.83496022, 1.87118769, 1.90620697, 1.94272494, 1.98070216, 2.01647091, 2.0498004, 2.08364153, 2.11928773,
        2.15560579, 2.18980479, 2.22491336, 2.25726533, 2.2943573, 2.33088923, 2.36460924, 2.39812469, 2.43361306,
        2.46727657, 2.50339603, 2.53576612, 2.57121992, 2.60696888, 2.64032793, 2.67307615, 2.70947099, 2.74528575,
        2.77945948, 2.81456661, 2.85181594, 2.88525105, 2.91967273, 2.95498037, 2.98756051, 3.02149129, 3.0616591,
        3.10226703, 3.14550018, 3.17241645, 3.20520377, 3.23778415, 3.26746464, 3.30144954, 3.33452749, 3.36958742,
        3.40689158, 3.44204021, 3.46366453, 3.50248289, 3.55081081, 3.57493377, 3.60472679, 3.64016843, 3.69267416,
        3.7173543, 3.74880195, 3.79786205, 3.81671, 3.85657883, 3.890836, 3.92172647, 3.97400618, 4.00900364,
        4.0296216, 4.07956123, 4.09901381, 4.13371038, 4.17270517, 4.19839382, 4.23779917, 4.27249575, 4.30719233,
        4.34188843,
    ),
}
#: Boundaries between the values' table entries, where they are not the centroids' fp32 midpoints.
BOUNDARIES = {3: (-1.74793005, -1.04996002, -0.500549972, 0.0, 0.500549972, 1.04996002, 1.74793005)}
#: Rotation signs by head_dim: bit j of the number is set where element j has sign -1.
SIGNS = {
    64: 0x62de4802b769548e,
    128: 0x146059de4a8337d56a9c02506a39df0d,
    256: 0xfe8bc3575730d96bb2275d733a2ff29bd39c5ec9a96d146f10cd4a1162e63012,
    512: 0x296b9d6d520e4bef8ea79bc28a8214525d81721f3204a3c59a4c151811873e8477bacaba542ade30e9dd12439b477c8f5ccad261d439e46362fbe30d70364bbd,
}

BUFFERS = ("k_codes", "k_scales", "k_zeros", "v_codes", "v_scales")
KEY_MODES = ((2, False), (4, False), (5, False), (8, False), (8, True))


# ---- cases -------------------------------------------------------------------------------------------------------
def listed():
    return [
        # one token of one short sequence, the smallest head_dim: nothing but latency
        dict(name="append_tiny", op="append", B=1, Hkv=2, G=2, D=64, N=1, cap=48, R=64, inter=False, bands=False,
             fused=False, f32=False, given=False, kb=8, ks=True, vb=3, pad=False, short=False),
        # a decode step of 64 sequences of an 8B-shaped layer, straight from the fused projection
        dict(name="append_8b_decode", op="append", B=64, Hkv=8, G=4, D=128, N=1, cap=1056, R=128, inter=False,
             bands=True, fused=True, f32=False, given=False, kb=8, ks=True, vb=3, pad=False, short=False),
        # prompts of unequal lengths up to 2048 tokens, four at once
        dict(name="append_prompt", op="append", B=4, Hkv=8, G=4, D=128, N=2048, cap=4096, R=128, inter=False,
             bands=True, fused=True, f32=False, given=False, kb=8, ks=True, vb=8, pad=False, short=True),
        # wide heads of which a quarter turns, interleaved pairs, fp32 inputs, positions of their own
        dict(name="append_hd256_part", op="append", B=8, Hkv=4, G=4, D=256, N=33, cap=777, R=64, inter=True,
             bands=False, fused=False, f32=True, given=True, kb=5, ks=False, vb=5, pad=True, short=False),
        # one token of one short sequence, fp32 outputs
        dict(name="window_tiny", op="window", B=1, Hkv=2, G=2, D=64, N=1, T=40, window=16, sinks=4, kb=8, ks=True,
             vb=3, f32=True, pad=False, short=False),
        # a decode step of 32 sequences of up to 16384 tokens that look 4096 back
        dict(name="window_decode", op="window", B=32, Hkv=8, G=4, D=128, N=1, T=16384, window=4096, sinks=64, kb=8,
             ks=True, vb=8, f32=False, pad=False, short=False),
        # chunks of 512 prompt tokens, two prompts at once, that look 2048 back
        dict(name="window_chunk", op="window", B=2, Hkv=8, G=4, D=128, N=512, T=8192, window=2048, sinks=4, kb=8,
             ks=True, vb=3, f32=False, pad=False, short=True),
        # the widest heads, three tokens at once, left-padded rows
        dict(name="window_hd512", op="window", B=4, Hkv=2, G=4, D=512, N=3, T=8192, window=1024, sinks=7, kb=5,
             ks=False, vb=5, f32=False, pad=True, short=False),
        # two answers to one short prompt, fp32 outputs
        dict(name="prefix_tiny", op="prefix", Bp=1, S=2, Hkv=2, G=2, D=64, N=1, P=48, T=8, kb=8, ks=True, vb=3,
             f32=True, pad=False, short=False),
        # eight beams after a prompt of 4096 tokens, an 8B-shaped layer
        dict(name="prefix_8b_beams", op="prefix", Bp=1, S=8, Hkv=8, G=4, D=128, N=1, P=4096, T=256, kb=8, ks=True,
             vb=3, f32=False, pad=False, short=False),
        # 64 conversations that begin with the same 8192 tokens
        dict(name="prefix_batch", op="prefix", Bp=1, S=64, Hkv=8, G=4, D=128, N=1, P=8192, T=1024, kb=8, ks=True,
             vb=8, f32=False, pad=False, short=False),
        # four prompts of unequal lengths, six answers each, wide heads, up to three new tokens at once
        dict(name="prefix_groups_hd256", op="prefix", Bp=4, S=6, Hkv=4, G=4, D=256, N=3, P=6001, T=301, kb=4,
             ks=False, vb=4, f32=False, pad=True, short=True),
    ]


MOST_CACHE = 32 * 8 * 16384 * 128  # cached elements of the largest listed case
MOST_SCORES = 2 * 32 * 512 * 8192  # scores of the largest one, before its window
MOST_FLOPS = 4 * 2 * 32 * 512 * 1800 * 128
MOST_BYTES = 298_000_000
MOST_NEW = 4 * 2048 * 48 * 128     # new elements of the largest append


def _log(rng, lo, hi):
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    """One more case, no dearer than the largest listed one."""
    while True:
        c = _draw(rng)
        w = work(c)
        if w["bytes"] <= MOST_BYTES and w["flops"] <= MOST_FLOPS:
            return c


def _draw(rng):
    op = rng.choice(("append", "window", "window", "prefix", "prefix"))
    Hkv, G, D = rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 3, 4, 5, 8)), rng.choice((64, 128, 128, 256, 512))
    kb, ks = rng.choice(KEY_MODES)
    c = dict(op=op, Hkv=Hkv, G=G, D=D, kb=kb, ks=ks, vb=rng.choice((2, 3, 4, 5, 8)), f32=rng.random() < 0.3,
             pad=rng.random() < 0.3, short=rng.random() < 0.4)
    if op == "append":
        B, N = _log(rng, 1, 64), 1 if rng.random() < 0.4 else _log(rng, 1, 2048)
        N = max(1, min(N, MOST_NEW // (B * Hkv * (G + 2) * D)))
        R = rng.choice((0, D, D, D, D // 2, D // 4, 2 * rng.randint(1, D // 2)))
        cap = N + _log(rng, 1, max(1, min(2048, MOST_CACHE // (B * Hkv * D) - N)))
        return dict(c, B=B, N=N, cap=cap, R=R, inter=rng.random() < 0.5, bands=rng.random() < 0.5,
                    fused=rng.random() < 0.5, given=rng.random() < 0.3)
    N = rng.choice((1, 1, 1, rng.randint(2, 16), _log(rng, 2, 512)))
    if op == "window":
        B, T = _log(rng, 1, 32), _log(rng, 1, 32768)
        N = max(1, min(N, MOST_SCORES // (B * Hkv * G * 64)))
        T = max(1, min(T, MOST_CACHE // (B * Hkv * D), MOST_SCORES // (B * Hkv * G * N)))
        window, sinks = _log(rng, 1, T), rng.choice((0, 1, 4, rng.randint(1, 100)))
        if rng.random() < 0.2:
            window = T
        window = max(1, min(window, MOST_FLOPS // (4 * D * B * Hkv * G * N) - sinks))
        return dict(c, B=B, N=N, T=T, window=window, sinks=sinks)
    Bp, S = rng.choice((1, 1, 2, 3, 4)), _log(rng, 1, 64)
    N = max(1, min(N, MOST_FLOPS // (4 * D * Bp * S * Hkv * G * 256)))
    most = min(MOST_FLOPS // (4 * D * Bp * S * Hkv * G * N), MOST_SCORES // (Bp * S * Hkv * G * N))
    T = max(1, min(_log(rng, 1, 4096), MOST_CACHE // (2 * Bp * S * Hkv * D), most // 2))
    P = max(1, min(_log(rng, 1, 32768), MOST_CACHE // (2 * Bp * Hkv * D), most // 2))
    return dict(c, Bp=Bp, S=S, N=N, P=P, T=T)


# Lengths, pads and counts go by the case alone (the seed only deals them out to the rows), so that the work of a case
# does not depend on its seed.
def _batch(c):
    return c["Bp"] * c["S"] if c["op"] == "prefix" else c["B"]


def _lens(c):
    """Tokens of each sequence: before an append, or with the new tokens."""
    B, T = _batch(c), c["cap"] - c["N"] if c["op"] == "append" else c["T"]
    return [T - (i * (T // 2)) // max(B - 1, 1) for i in range(B)]


def _pads(c):
    return [(n * (i % 4)) // 8 if c["pad"] else 0 for i, n in enumerate(_lens(c))]


def _counts(c):
    """New tokens of each sequence."""
    return [c["N"] - (i % 5) * c["N"] // 8 if c["short"] else c["N"] for i in range(_batch(c))]


def _prefixes(c):
    return [c["P"] - (i * (c["P"] // 3)) // max(c["Bp"] - 1, 1) for i in range(c["Bp"])]


def work(c):
    Hkv, G, D, N, B = c["Hkv"], c["G"], c["D"], c["N"], _batch(c)
    row = D * (c["kb"] + c["vb"]) // 8 + 3 * (D // GROUP) * 2  # bytes of a packed token
    if c["op"] == "append":
        size, new = 4 if c["f32"] else 2, sum(_counts(c))
        tables = 4 * c["R"] * B * N
        return {"bytes": Hkv * new * (2 * D * size + row) + 2 * Hkv * G * B * N * D * size + tables + 12 * B, "flops": 0}
    sees, read = 0, 0  # pairs of a new token and a cached one; cached tokens that any new one sees
    window = c["window"] if c["op"] == "window" else c["T"] + 1
    sinks = c["sinks"] if c["op"] == "window" else 0
    for n, lo, count in zip(_lens(c), _pads(c), _counts(c)):
        first = n
        for p in range(max(n - count, lo), n):
            start = max(lo, p - window + 1)
            sees += p + 1 - start + max(0, min(lo + sinks, start) - lo)
            first = min(first, start)
        if n > max(n - count, lo):
            read += n - first + max(0, min(lo + sinks, first) - lo)
    if c["op"] == "prefix":
        lens = _prefixes(c)
        read += sum(lens)
        sees += sum(lens[b // c["S"]] * count for b, count in enumerate(_counts(c)))
    rows = B * Hkv * G * N
    return {"bytes": Hkv * read * row + rows * (D * (6 if c["f32"] else 4) + 4) + 12 * B, "flops": 4 * D * Hkv * G * sees}


# ---- inputs ------------------------------------------------------------------------------------------------------
def _signs(D, device):
    n = SIGNS[D]
    return torch.tensor([-1.0 if n >> j & 1 else 1.0 for j in range(D)], device=device)


def _hadamard(D, device, dtype=torch.float32):
    """The Sylvester Hadamard matrix: entry (i, j) is -1 to the number of ones in i & j."""
    i = torch.arange(D, device=device)
    both = i[:, None] & i[None, :]
    ones = sum((both >> k) & 1 for k in range(9))
    return (1 - 2 * (ones % 2)).to(dtype)


def _pack(codes, bits):
    """Codes [..., D] (uint8) as a little-endian bitstream along the last axis."""
    if bits == 8:
        return codes
    b = (codes[..., None] >> torch.arange(bits, device=codes.device, dtype=torch.uint8)) & 1
    b = b.reshape(*codes.shape[:-1], codes.shape[-1] * bits // 8, 8)
    return (b << torch.arange(8, device=codes.device, dtype=torch.uint8)).sum(-1, dtype=torch.uint8)


def _encode_keys(x, bits, signed):
    """fp32 rows -> packed codes, scales, zero points; each operation rounds once, and divisions are by tensors (a
    division by a number may be a product with its reciprocal)."""
    g = x.unflatten(-1, (-1, GROUP))
    lo, hi = g.amin(-1), g.amax(-1)
    most = 2 ** (bits - 1) - 1 if signed else 2 ** bits - 1
    scale = (hi - lo) / torch.full_like(lo, 2 * most if signed else most)
    se = scale + 1e-8
    zero = ((hi + lo) / (se * 2) if signed else lo / se).round()
    code = (g / se[..., None] - zero[..., None]).round().clamp(-most if signed else 0, most)
    return _pack((code.to(torch.int16) & 255).to(torch.uint8).flatten(-2).contiguous(), bits), scale.half(), zero.half()


def _encode_values(x, bits):
    """fp32 rows -> packed table indices, scales: signs, Hadamard butterflies in ascending strides, / sqrt(D); the
    squares of a group are added up pairwise."""
    D = x.shape[-1]
    y = x * _signs(D, x.device)
    h = 1
    while h < D:
        y = y.unflatten(-1, (-1, 2, h))
        y = torch.stack((y[..., 0, :] + y[..., 1, :], y[..., 0, :] - y[..., 1, :]), -2).flatten(-3)
        h *= 2
    y = y * torch.full((), D ** -0.5, device=x.device)
    g = y.unflatten(-1, (-1, GROUP))
    sq = g * g
    while sq.shape[-1] > 1:
        sq = sq[..., ::2] + sq[..., 1::2]
    rms = (sq[..., 0] * (1 / GROUP)).sqrt()
    inv = torch.ones_like(rms) / (rms + 1e-8)
    table = torch.tensor(CENTROIDS[bits], device=x.device)
    edges = torch.tensor(BOUNDARIES[bits], device=x.device) if bits in BOUNDARIES else (table[1:] + table[:-1]) / 2
    # (64 bits: the product is compared with the boundaries before any rounding)
    idx = torch.bucketize(g.double() * inv[..., None].double(), edges.double())
    return _pack(idx.to(torch.uint8).flatten(-2).contiguous(), bits), rms.half()


def _cache(gen, B, H, cap, D, kb, ks, vb):
    """A packed cache of keys with an offset a channel (as keys of trained models have) and of normal values, encoded
    as the codec encodes them."""
    offset = torch.randn((H, 1, D), generator=gen, device="cuda")
    parts = []
    for _ in range(B):  # (a row at a time: what an encode needs beside its result is much larger)
        k = torch.randn((H, cap, D), generator=gen, device="cuda") + offset
        v = torch.randn((H, cap, D), generator=gen, device="cuda")
        parts.append((*_encode_keys(k, kb, ks), *_encode_values(v, vb)))
    return {name: torch.stack([p[i] for p in parts]) for i, name in enumerate(BUFFERS)}


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _tables(R, length, bands):
    """cos and sin of position * frequency, [length, R / 2]; bands: low frequencies 8 times lower and a smooth passage
    to the high ones, for contexts longer than the trained one."""
    f = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device="cuda") / R)
    if bands:
        turns = 8192 * f / (2 * math.pi)
        keep = ((turns - 1) / 3).clamp(0, 1)
        f = f * keep + f / 8 * (1 - keep)
    angle = torch.arange(length, dtype=torch.float64, device="cuda")[:, None] * f
    return angle.cos().float(), angle.sin().float()


def prepare(c, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)
    s, B, Hkv, G, N, D = dict(c), _batch(c), c["Hkv"], c["G"], c["N"], c["D"]
    rows = list(range(B))
    rng.shuffle(rows)
    lens, pads, counts = _lens(c), _pads(c), _counts(c)
    s["B"] = B
    s["lens"] = _ints([lens[i] for i in rows])
    s["left_pad"] = _ints([pads[i] for i in rows]) if c["pad"] else None
    s["count"] = _ints([counts[i] for i in rows]) if c["short"] else None
    if c["op"] == "append":
        dtype = torch.float32 if c["f32"] else torch.bfloat16
        heads = Hkv * (G + 2)
        new = torch.randn((B, N, heads, D), generator=gen, device="cuda")
        new[:, :, Hkv * G:Hkv * (G + 1)] += torch.randn((Hkv, D), generator=gen, device="cuda")
        new = new.to(dtype).transpose(1, 2)  # heads of one projection, a token's side by side
        if not c["fused"]:
            new = new.contiguous()
        s["q"], s["k"], s["v"] = new[:, :Hkv * G], new[:, Hkv * G:Hkv * (G + 1)], new[:, Hkv * (G + 1):]
        if not c["fused"]:
            s["q"], s["k"], s["v"] = (x.contiguous() for x in (s["q"], s["k"], s["v"]))
        length = 4 * c["cap"]
        s["cos"], s["sin"] = _tables(c["R"], length, c["bands"]) if c["R"] else (None, None)
        # positions of their own: of sequences that lost tokens on the way
        s["positions"] = (s["lens"][:, None] + _ints([rng.randrange(2 * c["cap"]) for _ in range(B)])[:, None]
                          + torch.arange(N, dtype=torch.int32, device="cuda")).contiguous() if c["given"] else None
        s["cache"] = _cache(gen, B, Hkv, c["cap"], D, c["kb"], c["ks"], c["vb"])
        s["q_out"] = torch.empty((B, Hkv * G, N, D), dtype=dtype, device="cuda")
        return s
    s["scale"] = 1 / math.sqrt(D)
    # queries that look at some keys much more than at others
    s["q"] = (2 * torch.randn((B, Hkv * G, N, D), generator=gen, device="cuda")).bfloat16()
    s["cache"] = _cache(gen, B, Hkv, c["T"], D, c["kb"], c["ks"], c["vb"])
    if c["op"] == "prefix":
        s["prefix"] = _cache(gen, c["Bp"], Hkv, c["P"], D, c["kb"], c["ks"], c["vb"])
        s["prefix_lens"] = _ints(_prefixes(c))
    # what the plain form reads and the codec has built in: the value table and the rotation
    s["table"] = torch.tensor(CENTROIDS[c["vb"]], device="cuda")
    s["hadamard"], s["signs"] = _hadamard(D, "cuda"), _signs(D, "cuda")
    return s


# ---- plain forms -------------------------------------------------------------------------------------------------
def _codes(packed, bits, D):
    if bits == 8:
        return packed.int()
    bit = torch.arange(D, device=packed.device) * bits
    wide = torch.nn.functional.pad(packed, (0, 1)).int()
    return ((wide[..., bit >> 3] | wide[..., (bit >> 3) + 1] << 8) >> (bit & 7)) & (2 ** bits - 1)


def _keys(cache, D, bits, signed):
    codes = cache["k_codes"].view(torch.int8).int() if signed else _codes(cache["k_codes"], bits, D)
    x = codes.unflatten(-1, (-1, GROUP)).float()
    x = (x + cache["k_zeros"].float()[..., None]) * cache["k_scales"].float()[..., None]
    return x.flatten(-2).bfloat16().float()


def _values(cache, D, bits, table):
    x = table[_codes(cache["v_codes"], bits, D)].unflatten(-1, (-1, GROUP))
    return (x * cache["v_scales"].float()[..., None]).flatten(-2).bfloat16().float()


def _turn(x, cos, sin, R, inter):
    """Rows [B, H, N, D] turned by their positions' angles [B, N, R / 2]."""
    cos, sin = cos[:, None], sin[:, None]
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if inter else (x[..., :R // 2], x[..., R // 2:R])
    c, d = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((c, d), -1).flatten(-2) if inter else torch.cat((c, d), -1)
    return torch.cat((turned, x[..., R:]), -1)


def _plain_append(s):
    B, N, cap, R = s["B"], s["N"], s["cap"], s["R"]
    n = torch.arange(N, device="cuda")
    q, k, v = (s[name].float() for name in "qkv")
    if R:
        if s["positions"] is not None:
            at = s["positions"]
        else:
            at = s["lens"][:, None] - (s["left_pad"][:, None] if s["left_pad"] is not None else 0) + n
        at = at.long().clamp(0, s["cos"].shape[0] - 1)
        cos, sin = s["cos"][at], s["sin"][at]
        q, k = (_turn(x, cos, sin, R, s["inter"]) for x in (q, k))
    packed = dict(zip(BUFFERS, (*_encode_keys(k, s["kb"], s["ks"]), *_encode_values(v, s["vb"]))))
    count = s["count"] if s["count"] is not None else torch.full((B,), N, device="cuda")
    to = s["lens"][:, None] + n
    b, m = torch.nonzero((n < count[:, None]) & (to < cap), as_tuple=True)
    for name in BUFFERS:
        s["cache"][name][b, :, to[b, m].long()] = packed[name][b, :, m]
    s["q_out"].copy_(q)
    return {"q": s["q_out"], "cache": s["cache"], "lens": (s["lens"] + count).clamp(max=cap).to(torch.int32)}


def _seen(s):
    """[B, N, T]: which of its sequence's tokens a new token sees."""
    N, T = s["N"], s["T"]
    t = torch.arange(T, device="cuda")
    n = torch.arange(N, device="cuda")
    count = s["count"] if s["count"] is not None else torch.full_like(s["lens"], N)
    lo = (s["left_pad"] if s["left_pad"] is not None else torch.zeros_like(s["lens"]))[:, None, None]
    p = (s["lens"] - count)[:, None, None] + n[:, None]
    seen = (t >= lo) & (t <= p)
    if s["op"] == "window":
        seen = seen & ((t > p - s["window"]) | (t < lo + s["sinks"]))
    return seen & (n < count[:, None])[..., None]


def _plain_attention(s):
    B, Hkv, G, N, D, T = (s[k] for k in ("B", "Hkv", "G", "N", "D", "T"))
    q = s["q"].float().view(B, Hkv, G * N, D)
    seen = _seen(s)[:, None].expand(B, G, N, T).reshape(B, 1, G * N, T)
    k, v = _keys(s["cache"], D, s["kb"], s["ks"]), _values(s["cache"], D, s["vb"], s["table"])
    x = torch.where(seen, s["scale"] * (q @ k.transpose(-1, -2)), -math.inf)
    shared = None
    if s["op"] == "prefix":
        Bp, S, P = s["Bp"], s["S"], s["P"]
        together = q.view(Bp, S, Hkv, G * N, D).transpose(1, 2).reshape(Bp, Hkv, S * G * N, D)
        y = s["scale"] * (together @ _keys(s["prefix"], D, s["kb"], s["ks"]).transpose(-1, -2))
        there = torch.arange(P, device="cuda") < s["prefix_lens"][:, None]
        y = torch.where(there[:, None, None], y, -math.inf)
        y = y.view(Bp, Hkv, S, G * N, P).transpose(1, 2).reshape(B, Hkv, G * N, P)
        # (a new token that its sequence does not have sees nothing)
        new = _seen(s).any(-1)[:, None].expand(B, G, N).reshape(B, 1, G * N, 1)
        shared = torch.where(new, y, -math.inf)
    most = x.amax(-1, keepdim=True)
    if shared is not None:
        most = torch.maximum(most, shared.amax(-1, keepdim=True))
    most = torch.where(most == -math.inf, 0.0, most)
    p = (x - most).exp()
    den, o = p.sum(-1, keepdim=True), p @ v
    if shared is not None:
        p = (shared - most).exp()
        den = den + p.sum(-1, keepdim=True)
        p = p.view(Bp, S, Hkv, G * N, P).transpose(1, 2).reshape(Bp, Hkv, S * G * N, P)
        more = (p @ _values(s["prefix"], D, s["vb"], s["table"])).view(Bp, Hkv, S, G * N, D)
        o = o + more.transpose(1, 2).reshape(B, Hkv, G * N, D)
    o = o / torch.where(den == 0, 1.0, den)
    o = (o @ s["hadamard"]) * (1 / math.sqrt(D)) * s["signs"]
    lse = (most + den.log())[..., 0]
    return {"out": o.view(B, Hkv * G, N, D).to(torch.float32 if s["f32"] else torch.bfloat16),
            "lse": lse.view(B, Hkv * G, N)}


def run(s):
    op = s["op"]
    if own:
        import turboquant_kv_cache_tq_gb300 as tq

        if op == "append":
            q, lens = tq.tq_append_kv(
                s["k"], s["v"], s["cache"], s["lens"], s["kb"], s["ks"], s["vb"], cos=s["cos"], sin=s["sin"],
                interleaved=s["inter"], q=s["q"], positions=s["positions"], left_pad=s["left_pad"], count=s["count"],
                q_out=s["q_out"])
            return {"q": q, "cache": s["cache"], "lens": lens}
        kind = torch.float32 if s["f32"] else torch.bfloat16
        if op == "window":
            out, lse = tq.tq_window_attention(
                s["q"], s["cache"], s["T"], s["kb"], s["ks"], s["vb"], s["window"], sinks=s["sinks"], lens=s["lens"],
                left_pad=s["left_pad"], count=s["count"], scale=s["scale"], out_dtype=kind)
        else:
            out, lse = tq.tq_prefix_attention(
                s["q"], s["prefix"], s["P"], s["cache"], s["T"], s["kb"], s["ks"], s["vb"],
                prefix_lens=s["prefix_lens"], lens=s["lens"], left_pad=s["left_pad"], count=s["count"],
                scale=s["scale"], out_dtype=kind)
        return {"out": out, "lse": lse}
    return _plain_append(s) if op == "append" else _plain_attention(s)


# ---- exact results -----------------------------------------------------------------------------------------------
def _bitwise(packed, bits):
    """Codes of a bitstream, from its single bits."""
    b = (packed[..., None] >> torch.arange(8, device=packed.device, dtype=torch.uint8)) & 1
    b = b.flatten(-2).unflatten(-1, (-1, bits)).to(torch.int64)
    return (b << torch.arange(bits, device=packed.device)).sum(-1)


def _exact_keys(cache, at, bits, signed):
    b, tokens = at
    code = _bitwise(cache["k_codes"][b, :, tokens], bits).double()
    code = torch.where(code > 127, code - 256, code) if signed else code
    zero, scale = (cache[k][b, :, tokens].double().repeat_interleave(GROUP, -1) for k in ("k_zeros", "k_scales"))
    moved = (code + zero).float().double()  # the format's roundings: fp32 after each operation, then bf16
    return (moved * scale).float().bfloat16().double()


def _exact_values(cache, at, bits):
    b, tokens = at
    c = torch.tensor(CENTROIDS[bits], device="cuda", dtype=torch.float32).double()
    scale = cache["v_scales"][b, :, tokens].double().repeat_interleave(GROUP, -1)
    return (c[_bitwise(cache["v_codes"][b, :, tokens], bits)] * scale).float().bfloat16().double()


def _exact_append(c, s):
    """The turned queries; the packed bytes are whole numbers (every rounding of an encode is the codec's)."""
    B, Hq, N, D = s["q"].shape
    out = s["q"].double()
    lens = s["lens"].tolist()
    pads = s["left_pad"].tolist() if s["left_pad"] is not None else [0] * B
    for b in range(B if c["R"] else 0):
        at = s["positions"][b] if c["given"] else torch.arange(lens[b] - pads[b], lens[b] - pads[b] + N, device="cuda")
        angle = torch.complex(s["cos"][at.long()].double(), s["sin"][at.long()].double())
        i = torch.arange(c["R"] // 2, device="cuda")
        x, y = (2 * i, 2 * i + 1) if c["inter"] else (i, i + c["R"] // 2)
        z = torch.complex(out[b][..., x], out[b][..., y]) * angle
        out[b][..., x], out[b][..., y] = z.real, z.imag
    return {"q": out, "cache": {name: None for name in BUFFERS}, "lens": None}


def exact(c, seed):
    B, Hkv, G, N, D = _batch(c), c["Hkv"], c["G"], c["N"], c["D"]
    if c["op"] != "append" and B * Hkv * G * N * (c["T"] + c.get("P", 0)) * D > 2e13:
        return None
    s = prepare(c, seed)
    if c["op"] == "append":
        return _exact_append(c, s)
    lens, counts = s["lens"].tolist(), s["count"].tolist() if s["count"] is not None else [N] * B
    pads = s["left_pad"].tolist() if s["left_pad"] is not None else [0] * B
    out = torch.zeros((B, Hkv * G, N, D), dtype=torch.float64, device="cuda")
    logs = torch.full((B, Hkv * G, N), -math.inf, dtype=torch.float64, device="cuda")
    turn = _hadamard(D, "cuda", torch.float64) / math.sqrt(D) * _signs(D, "cuda").double()
    shared = {}
    for b in range(B):
        lo, hi, count = pads[b], lens[b], counts[b]
        own_at = (b, slice(lo, hi))
        k, v = _exact_keys(s["cache"], own_at, c["kb"], c["ks"]), _exact_values(s["cache"], own_at, c["vb"])
        first = 0
        if c["op"] == "prefix":
            g = b // c["S"]
            if g not in shared:
                at = (g, slice(0, _prefixes(c)[g]))
                shared = {g: (_exact_keys(s["prefix"], at, c["kb"], c["ks"]), _exact_values(s["prefix"], at, c["vb"]))}
            k, v = torch.cat([shared[g][0], k], 1), torch.cat([shared[g][1], v], 1)
            first = _prefixes(c)[g]
        t = torch.arange(k.shape[1], device="cuda") - first + lo  # (below lo: the prefix)
        for n0 in range(0, count, 64):
            n = torch.arange(n0, min(n0 + 64, count), device="cuda")
            p = (hi - count + n)[:, None]
            hide = (t > p) | (p < lo)
            if c["op"] == "window":
                hide = hide | ((t <= p - c["window"]) & (t >= lo + c["sinks"]))
            q = s["q"][b][:, n].double().view(Hkv, G, len(n), D)
            x = (torch.einsum("hgnd,htd->hgnt", q, k) / math.sqrt(D)).masked_fill(hide, -math.inf)
            empty = (x == -math.inf).all(-1, keepdim=True)
            w = torch.softmax(x.masked_fill(empty, 0.0), -1).masked_fill(empty, 0.0)
            o = torch.einsum("hgnt,htd->hgnd", w, v) if k.shape[1] else torch.zeros_like(q)
            out[b, :, n] = (o @ turn).view(Hkv * G, len(n), D)
            logs[b, :, n] = torch.logsumexp(x, -1).view(Hkv * G, len(n)) if k.shape[1] else -math.inf
    return {"out": out, "lse": logs}
