"""Cases of the operators on ragged packed caches, their plain forms and their exact results.

The operators: attention of a tree of drafted tokens over a packed cache (`tree`), the sums of attention weights per
cached token (`weights`), the choice of the tokens that stay when a cache is cut (`select`) and the copy of chosen
tokens from one packed cache into another (`gather`), which commits an accepted path and compacts a cut cache.

A packed cache row (batch row, kv head, token) holds keys as codes with an fp16 scale and zero point per group of 32
elements, K = bf16((code + zero) * scale), and rotated values as table indices with an fp16 scale per group,
V = bf16(centroid * scale); attention runs on the rotated values, and its output is turned back by the Hadamard
transform / sqrt(D) and the sign vector.
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
        # the first draft on a short prompt, the smallest head_dim and fp32 outputs: nothing but latency
        dict(name="tree_tiny", op="tree", B=1, Hkv=2, G=2, D=64, T=16, N=5, kb=8, ks=True, vb=3, f32=True, pad=False),
        # a 32-node draft tree over one 4096-token layer of an 8B-shaped model (8 kv heads, 32 query heads)
        dict(name="tree_8b_layer", op="tree", B=1, Hkv=8, G=4, D=128, T=4096, N=32, kb=8, ks=True, vb=3, f32=False,
             pad=False),
        # a batch of 32 sequences of unequal lengths up to 8192 tokens, 16-node trees of unequal sizes
        dict(name="tree_long_context", op="tree", B=32, Hkv=8, G=4, D=128, T=8192, N=16, kb=8, ks=True, vb=8,
             f32=False, pad=False),
        # wide heads, 26-node trees: 104 query rows a kv head
        dict(name="tree_hd256", op="tree", B=4, Hkv=4, G=4, D=256, T=8192, N=26, kb=8, ks=True, vb=4, f32=False,
             pad=False),
        # the widest heads, an odd key width, left-padded rows
        dict(name="tree_hd512", op="tree", B=2, Hkv=2, G=4, D=512, T=16384, N=12, kb=5, ks=False, vb=5, f32=False,
             pad=True),
        # the weights that the last 64 tokens of a prompt give to the prompt, by which it is cut
        dict(name="weights_8b_window", op="weights", B=1, Hkv=8, G=4, D=128, T=4096, N=64, P=64, path=False, kb=8,
             ks=True, pad=False),
        # the weights of an accepted path (1 to 6 of 16 nodes) in every sequence of a batch
        dict(name="weights_long_context", op="weights", B=32, Hkv=8, G=4, D=128, T=8192, N=16, P=6, path=True, kb=8,
             ks=True, pad=False),
        # which 1000 of a 4096-token layer stay, the last 128 among them
        dict(name="select_8b_layer", op="select", B=1, Hkv=8, T=4096, keep=1000, recent=128, pad=False),
        # the same for a batch of unequal lengths
        dict(name="select_long_context", op="select", B=32, Hkv=8, T=8192, keep=2048, recent=256, pad=False),
        # an accepted path of 1 to 6 nodes goes from the draft's cache to the end of each sequence
        dict(name="commit_long_context", op="gather", B=32, Hkv=8, D=128, T=8192, cap=8256, src=16, n=6, heads=False,
             append=True, kb=8, vb=8),
        # a cut cache of a batch, 2048 of up to 8192 tokens a head
        dict(name="compact_long_context", op="gather", B=32, Hkv=8, D=128, T=8192, cap=2112, src=8256, n=2048,
             heads=True, append=False, kb=8, vb=3),
        # a cut cache with the widest rows
        dict(name="compact_hd512", op="gather", B=2, Hkv=2, D=512, T=16384, cap=5000, src=16384, n=4999, heads=True,
             append=False, kb=8, vb=5),
    ]


MOST_TOKENS = 32 * 8 * 8192  # cached rows of the largest listed case, each of 128 elements
MOST_FLOPS = 4 * MOST_TOKENS * 128 * 64


def _log(rng, lo, hi):
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    op = rng.choice(("tree", "tree", "tree", "weights", "weights", "select", "gather"))
    B, Hkv, T = _log(rng, 1, 32), rng.choice((1, 2, 4, 8)), _log(rng, 1, 32768)
    if op == "select":
        T = min(T, MOST_TOKENS // (B * Hkv))
        keep = _log(rng, 1, T)
        return dict(op=op, B=B, Hkv=Hkv, T=T, keep=keep, recent=rng.randint(0, keep), pad=rng.random() < 0.5)
    D = rng.choice((64, 128, 128, 256, 512))
    kb, ks = rng.choice(KEY_MODES)
    T = max(1, min(T, MOST_TOKENS * 128 // (B * Hkv * D)))
    if op == "gather":
        append = rng.random() < 0.4
        n = rng.randint(1, 16) if append else _log(rng, 1, T)
        return dict(op=op, B=B, Hkv=Hkv, D=D, T=T, cap=T + n if append else n + rng.randint(0, 9),
                    src=16 if append else T, n=n, heads=not append, append=append, kb=kb, vb=rng.choice((2, 3, 4, 5, 8)))
    G, N = rng.choice((1, 2, 3, 4, 5, 8)), _log(rng, 1, 64)
    T = max(1, min(T, MOST_FLOPS // (4 * B * Hkv * D * G * N)))
    if op == "weights":
        path = rng.random() < 0.6
        return dict(op=op, B=B, Hkv=Hkv, G=G, D=D, T=T, N=N, P=min(N, rng.randint(1, 8)) if path else N, path=path,
                    kb=kb, ks=ks, pad=rng.random() < 0.3)
    return dict(op=op, B=B, Hkv=Hkv, G=G, D=D, T=T, N=N, kb=kb, ks=ks, vb=rng.choice((2, 3, 4, 5, 8)),
                f32=rng.random() < 0.3, pad=rng.random() < 0.3)


# Lengths, pads and path lengths go by the case alone (the seed only deals them out to the rows), so that the work of
# a case does not depend on its seed.
def _lens(c):
    B, T = c["B"], c["T"]
    return [T - (i * (T // 2)) // max(B - 1, 1) for i in range(B)]


def _pads(c):
    return [(n * (i % 4)) // 8 if c.get("pad") else 0 for i, n in enumerate(_lens(c))]


def _counts(c, most):
    return [most - i % most for i in range(c["B"])]


def work(c):
    op, B, Hkv = c["op"], c["B"], c["Hkv"]
    tokens = sum(n - p for n, p in zip(_lens(c), _pads(c)))
    if op == "select":
        kept = sum(min(c["keep"], n - p) for n, p in zip(_lens(c), _pads(c)))
        return {"bytes": 4 * Hkv * (tokens + kept) + 12 * B, "flops": 0}
    D = c["D"]
    key = D * c["kb"] // 8 + D // 8
    if op == "weights":
        rows = c["G"] * sum(_counts(c, c["P"]) if c["path"] else [c["N"]] * B)
        per_row = [c["G"] * n for n in (_counts(c, c["P"]) if c["path"] else [c["N"]] * B)]
        flops = sum(2 * D * Hkv * r * (n - p) for r, n, p in zip(per_row, _lens(c), _pads(c)))
        return {"bytes": Hkv * (tokens * key + 8 * B * c["T"] + rows * (2 * D + 4)), "flops": flops}
    row = key + D * c["vb"] // 8 + D // 16
    if op == "gather":
        kept = Hkv * sum(_counts(c, c["n"]) if c["append"] else [c["n"]] * B)
        return {"bytes": kept * (2 * row + (4 if c["append"] else 8 + 4)) + 12 * B, "flops": 0}
    rows = c["G"] * c["N"]
    return {"bytes": Hkv * ((tokens + B * c["N"]) * row + B * rows * (D * (6 if c["f32"] else 4) + 4)),
            "flops": 4 * D * Hkv * rows * tokens}


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
    g = x.unflatten(-1, (-1, GROUP))
    lo, hi = g.amin(-1), g.amax(-1)
    scale = ((hi - lo) / (2 ** bits - 1)).half()
    s = scale.float().clamp_min(1e-8)
    first = -128 if signed else 0
    zero = ((lo / s).round() - first).half()
    code = ((g / s[..., None]).round() - zero.float()[..., None]).clamp(first, first + 2 ** bits - 1)
    return _pack((code.to(torch.int16) & 255).to(torch.uint8).flatten(-2).contiguous(), bits), scale, zero


def _encode_values(x, bits):
    D = x.shape[-1]
    y = (x * _signs(D, x.device)) @ _hadamard(D, x.device) * (1 / math.sqrt(D))
    g = y.unflatten(-1, (-1, GROUP))
    scale = g.square().mean(-1).sqrt().half()
    table = torch.tensor(CENTROIDS[bits], device=x.device)
    idx = torch.bucketize(g / scale.float()[..., None].clamp_min(1e-8), (table[1:] + table[:-1]) / 2)
    return _pack(idx.to(torch.uint8).flatten(-2).contiguous(), bits), scale


def _cache(gen, B, H, cap, D, kb, ks, vb, keys=True):
    """A packed cache of keys with an offset a channel (as keys of trained models have) and of normal values, encoded
    as the codec encodes them."""
    out = {}
    offset = torch.randn((1, H, 1, D), generator=gen, device="cuda")
    k = torch.randn((B, H, cap, D), generator=gen, device="cuda") + offset
    out["k_codes"], out["k_scales"], out["k_zeros"] = _encode_keys(k, kb, ks)
    del k
    if vb:
        out["v_codes"], out["v_scales"] = _encode_values(torch.randn((B, H, cap, D), generator=gen, device="cuda"), vb)
    return out


def _deal(values, rng):
    values = list(values)
    rng.shuffle(values)
    return values


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(c, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)
    B, Hkv, T, op = c["B"], c["Hkv"], c["T"], c["op"]
    s = dict(c)
    rows = _deal(range(B), rng)
    lens, pads = _lens(c), _pads(c)
    s["lens"] = _ints([lens[i] for i in rows])
    s["left_pad"] = _ints([pads[i] for i in rows]) if c.get("pad") else None
    if op == "select":
        # sums of attention weights: a few large, most small, and many equal ones (tokens that nothing looked at)
        w = torch.rand((B, Hkv, T), generator=gen, device="cuda")
        s["weights"] = torch.where(w < 0.2, torch.zeros_like(w), (w ** 8 * 64).half().float())
        return s
    D, kb = c["D"], c["kb"]
    if op == "gather":
        n, src = c["n"], c["src"]
        s["source"] = _cache(gen, B, Hkv, src, D, kb, False, c["vb"])
        if c["append"]:
            # an increasing path of drafted nodes, and how many of them were accepted
            order = torch.rand((B, src), generator=gen, device="cuda").argsort(-1)[:, :n]
            s["index"] = order.sort(-1).values.to(torch.int32)
            s["count"] = _ints([_counts(c, n)[i] for i in rows])
            s["offset"] = s["lens"]
            s["dst"] = _cache(gen, B, Hkv, c["cap"], D, kb, False, c["vb"])
            s["src_weights"] = None
        else:
            order = torch.rand((B, Hkv, T), generator=gen, device="cuda").argsort(-1)[..., :n]
            s["index"] = order.sort(-1).values.to(torch.int32)
            s["count"] = s["offset"] = None
            s["dst"] = {k: torch.zeros((B, Hkv, c["cap"], v.shape[-1]), dtype=v.dtype, device="cuda")
                        for k, v in s["source"].items()}
            s["src_weights"] = torch.rand((B, Hkv, src), generator=gen, device="cuda")
        s["dst_weights"] = torch.rand((B, Hkv, c["cap"]), generator=gen, device="cuda")
        return s
    G, N, ks = c["G"], c["N"], c["ks"]
    s["scale"] = 1 / math.sqrt(D)
    # queries that look at some keys much more than at others
    s["q"] = (2 * torch.randn((B, Hkv * G, N, D), generator=gen, device="cuda")).bfloat16()
    s["cache"] = _cache(gen, B, Hkv, T, D, kb, ks, c.get("vb"))
    if op == "tree":
        s["tree"] = _cache(gen, B, Hkv, N, D, kb, ks, c["vb"])
        # each node hangs on a random earlier one or on the sequence's end; trees of a batch have unequal sizes
        parents = [[rng.randint(max(-1, i - 6), i - 1) if i < N - (b % 4) * (N // 8) else -2 for i in range(N)]
                   for b in range(B)]
        s["parents"] = _ints(parents)
        # what the plain form reads and the codec has built in: the value table and the rotation
        s["table"] = torch.tensor(CENTROIDS[c["vb"]], device="cuda")
        s["hadamard"], s["signs"] = _hadamard(D, "cuda"), _signs(D, "cuda")
        return s
    P = c["P"]
    if c["path"]:
        s["path"] = _ints([sorted(rng.sample(range(N), P)) for _ in range(B)])
        s["n_path"] = _ints([_counts(c, P)[i] for i in rows])
    else:
        s["path"] = s["n_path"] = None
    q, mask, taken = _observers(s)
    x = torch.where(mask, s["scale"] * (q @ _keys(s["cache"], D, kb, ks).transpose(-1, -2)), -math.inf)
    lse = torch.logsumexp(x, -1).unflatten(-1, (G, P))
    at = torch.full((B, Hkv, G, N), -math.inf, device="cuda")
    s["lse"] = at.scatter_(-1, taken.long()[:, None, None].expand(B, Hkv, G, P), lse).view(B, Hkv * G, N)
    s["weights"] = torch.rand((B, Hkv, T), generator=gen, device="cuda")
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


def _ancestors(parents):
    """[B, N, N]: whether node i attends to node j: j is i or one of i's ancestors, and i's chain ends at -1."""
    N = parents.shape[-1]
    j = torch.arange(N, device=parents.device)
    up = ((parents[..., None] == j) & (j < j[:, None])).float()
    reach = torch.linalg.matrix_power(up + torch.eye(N, device=parents.device), N) > 0
    present = (reach & (parents == -1)[:, None, :]).any(-1)
    return reach & present[..., None], present


def _plain_tree(s):
    B, Hkv, G, N, D, T = (s[k] for k in ("B", "Hkv", "G", "N", "D", "T"))
    q = s["q"].float().view(B, Hkv, G * N, D)
    k = torch.cat([_keys(s["cache"], D, s["kb"], s["ks"]), _keys(s["tree"], D, s["kb"], s["ks"])], 2)
    v = torch.cat([_values(x, D, s["vb"], s["table"]) for x in (s["cache"], s["tree"])], 2)
    reach, present = _ancestors(s["parents"])
    t = torch.arange(T, device="cuda")
    seen = t < s["lens"][:, None]
    if s["left_pad"] is not None:
        seen = seen & (t >= s["left_pad"][:, None])
    mask = torch.cat([seen[:, None] & present[..., None], reach], -1)  # [B, N, T + N]
    mask = mask[:, None].expand(B, G, N, T + N).reshape(B, 1, G * N, T + N)
    x = torch.where(mask, s["scale"] * (q @ k.transpose(-1, -2)), -math.inf)
    most = x.amax(-1, keepdim=True)
    most = torch.where(most == -math.inf, 0.0, most)
    p = (x - most).exp()
    den = p.sum(-1, keepdim=True)
    o = (p @ v) / torch.where(den == 0, 1.0, den)
    o = (o @ s["hadamard"]) * (1 / math.sqrt(D)) * s["signs"]
    lse = (most + den.log())[..., 0]
    return {"out": o.view(B, Hkv * G, N, D).to(torch.float32 if s["f32"] else torch.bfloat16),
            "lse": lse.view(B, Hkv * G, N)}


def _observers(s):
    """The query rows that count, [B, Hkv, G * P, D] in fp32, and which keys each of them sees."""
    B, Hkv, G, N, P, D, T = (s[k] for k in ("B", "Hkv", "G", "N", "P", "D", "T"))
    i = torch.arange(P, device="cuda")
    taken = s["path"] if s["path"] is not None else i.expand(B, P)
    count = s["n_path"] if s["n_path"] is not None else torch.full((B,), P, device="cuda")
    at = taken.long()[:, None, :, None].expand(B, Hkv * G, P, D)
    q = s["q"].float().gather(2, at).view(B, Hkv, G * P, D)
    t = torch.arange(T, device="cuda")
    last = s["lens"][:, None] - count[:, None] + i
    mask = (t <= last[..., None]) & (i < count[:, None])[..., None]  # [B, P, T]
    if s["left_pad"] is not None:
        mask = mask & (t >= s["left_pad"][:, None, None])
    return q, mask[:, None].expand(B, G, P, T).reshape(B, 1, G * P, T), taken


def _plain_weights(s):
    B, Hkv, G, P, D = (s[k] for k in ("B", "Hkv", "G", "P", "D"))
    q, mask, taken = _observers(s)
    at = taken.long()[:, None, :].expand(B, Hkv * G, P)
    lse = s["lse"].gather(2, at).view(B, Hkv, G * P, 1)
    x = s["scale"] * (q @ _keys(s["cache"], D, s["kb"], s["ks"]).transpose(-1, -2))
    w = torch.where(mask & (lse != -math.inf), (x - lse).exp(), 0.0)
    return s["weights"] + w.sum(2)


def _plain_select(s):
    w, keep, recent, T = s["weights"], s["keep"], s["recent"], s["T"]
    t = torch.arange(T, device="cuda")
    n = s["lens"][:, None]
    first = s["left_pad"][:, None] if s["left_pad"] is not None else torch.zeros_like(n)
    valid = (t >= first) & (t < n)
    whole = n - first <= keep
    late = valid & (t >= n - recent)
    rest = (valid & ~late)[:, None].expand_as(w)
    key = torch.where(w.isnan(), -math.inf, w)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices  # the lowest index first among equals
    order = order.gather(-1, torch.sort(rest.gather(-1, order).int(), dim=-1, descending=True, stable=True).indices)
    rank = torch.empty_like(order).scatter_(-1, order, t.expand_as(order))
    chosen = (rest & (rank < keep - recent)) | late[:, None]
    chosen = torch.where(whole[:, None], valid[:, None], chosen)
    index = torch.where(chosen, t, T).sort(-1).values[..., :keep]
    return {"index": torch.where(index == T, -1, index).to(torch.int32),
            "count": (n - first).clamp(0, keep)[:, 0].to(torch.int32)}


def _plain_gather(s):
    B, Hkv, cap, src, n = (s[k] for k in ("B", "Hkv", "cap", "src", "n"))
    j = torch.arange(n, device="cuda")
    index = (s["index"] if s["heads"] else s["index"][:, None]).expand(B, Hkv, n).long()
    count = s["count"] if s["count"] is not None else torch.full((B,), n, device="cuda")
    offset = s["offset"] if s["offset"] is not None else torch.zeros_like(count)
    to = (offset[:, None] + j)[:, None].expand(B, Hkv, n).long()
    go = (j < count[:, None])[:, None].expand(B, Hkv, n) & (to < cap)
    row = torch.arange(B * Hkv, device="cuda").view(B, Hkv, 1)
    at, to = (row * src + index)[go], (row * cap + to)[go]
    for k in BUFFERS:
        s["dst"][k].view(B * Hkv * cap, -1)[to] = s["source"][k].view(B * Hkv * src, -1)[at]
    s["dst_weights"].view(-1)[to] = s["src_weights"].view(-1)[at] if s["src_weights"] is not None else 0.0
    return {"dst": s["dst"], "weights": s["dst_weights"], "len": (offset + count).clamp(max=cap).to(torch.int32)}


def run(s):
    op = s["op"]
    if own:
        import turboquant_kv_cache_tq_gb300 as tq

        if op == "tree":
            out, lse = tq.tq_tree_attention(
                s["q"], s["cache"], s["T"], s["tree"], s["kb"], s["ks"], s["vb"], parents=s["parents"],
                lens=s["lens"], left_pad=s["left_pad"], scale=s["scale"],
                out_dtype=torch.float32 if s["f32"] else torch.bfloat16)
            return {"out": out, "lse": lse}
        if op == "weights":
            return tq.tq_attention_weights(
                s["q"], s["lse"], s["cache"], s["T"], s["kb"], s["ks"], path=s["path"], n_path=s["n_path"],
                lens=s["lens"], left_pad=s["left_pad"], scale=s["scale"], weights=s["weights"])
        if op == "select":
            index, count = tq.tq_evict_select(s["weights"], s["T"], s["keep"], s["recent"], lens=s["lens"],
                                              left_pad=s["left_pad"])
            return {"index": index, "count": count}
        dst, length = tq.tq_cache_gather(
            s["source"], s["dst"], s["index"], count=s["count"], dst_off=s["offset"],
            src_weights=s["src_weights"], dst_weights=s["dst_weights"])
        return {"dst": dst, "weights": s["dst_weights"], "len": length}
    return {"tree": _plain_tree, "weights": _plain_weights, "select": _plain_select, "gather": _plain_gather}[op](s)


# ---- exact results -----------------------------------------------------------------------------------------------
def _bitwise(packed, bits):
    """Codes of a bitstream, from its single bits."""
    b = (packed[..., None] >> torch.arange(8, device=packed.device, dtype=torch.uint8)) & 1
    b = b.flatten(-2).unflatten(-1, (-1, bits)).to(torch.int64)
    return (b << torch.arange(bits, device=packed.device)).sum(-1)


def _exact_keys(cache, b, bits, signed):
    code = _bitwise(cache["k_codes"][b], bits).double()
    code = torch.where(code > 127, code - 256, code) if signed else code
    zero, scale = (cache[k][b].double().repeat_interleave(GROUP, -1) for k in ("k_zeros", "k_scales"))
    moved = (code + zero).float().double()  # the format's roundings: fp32 after each operation, then bf16
    return (moved * scale).float().bfloat16().double()


def _exact_values(cache, b, bits):
    c = torch.tensor(CENTROIDS[bits], device="cuda", dtype=torch.float32).double()
    scale = cache["v_scales"][b].double().repeat_interleave(GROUP, -1)
    return (c[_bitwise(cache["v_codes"][b], bits)] * scale).float().bfloat16().double()


def _chains(parents):
    """For each node the set of nodes that it attends to, by walking up from it."""
    sets = []
    for i in range(len(parents)):
        seen, at = [], i
        while 0 <= at and at not in seen:
            seen.append(at)
            up = parents[at]
            at = up if up < at else -2
        sets.append(seen if at == -1 else [])
    return sets


def exact(c, seed):
    if c["op"] in ("select", "gather"):
        return None
    s = prepare(c, seed)
    B, Hkv, G, N, D, T = (c[k] for k in ("B", "Hkv", "G", "N", "D", "T"))
    lens, pads = s["lens"].tolist(), s["left_pad"].tolist() if s["left_pad"] is not None else [0] * B
    t = torch.arange(T, device="cuda")
    if c["op"] == "weights":
        total = s["weights"].double()
        for b in range(B):
            nodes = s["path"][b].tolist() if c["path"] else list(range(N))
            nodes = nodes[: s["n_path"][b].item()] if c["path"] else nodes
            k = _exact_keys(s["cache"], b, c["kb"], c["ks"])
            for i, node in enumerate(nodes):
                q = s["q"][b, :, node].double().view(Hkv, G, D)
                lse = s["lse"][b, :, node].double().view(Hkv, G, 1)
                w = torch.exp(torch.einsum("hgd,htd->hgt", q, k) / math.sqrt(D) - lse).masked_fill(lse == -math.inf, 0.0)
                total[b] += w.sum(1) * ((t >= pads[b]) & (t <= lens[b] - len(nodes) + i))
        return total
    out = torch.zeros((B, Hkv * G, N, D), dtype=torch.float64, device="cuda")
    logs = torch.full((B, Hkv * G, N), -math.inf, dtype=torch.float64, device="cuda")
    turn = _hadamard(D, "cuda", torch.float64) / math.sqrt(D) * _signs(D, "cuda").double()
    for b in range(B):
        lo, hi = pads[b], lens[b]
        k = torch.cat([_exact_keys(s["cache"], b, c["kb"], c["ks"])[:, lo:hi], _exact_keys(s["tree"], b, c["kb"], c["ks"])], 1)
        v = torch.cat([_exact_values(s["cache"], b, c["vb"])[:, lo:hi], _exact_values(s["tree"], b, c["vb"])], 1)
        for i, chain in enumerate(_chains(s["parents"][b].tolist())):
            if not chain:
                continue
            hide = torch.ones(k.shape[1], dtype=torch.bool, device="cuda")
            hide[: max(hi - lo, 0)] = False
            hide[[max(hi - lo, 0) + j for j in chain]] = False
            q = s["q"][b, :, i].double().view(Hkv, G, D)
            x = (torch.einsum("hgd,htd->hgt", q, k) / math.sqrt(D)).masked_fill(hide, -math.inf)
            o = torch.einsum("hgt,htd->hgd", torch.softmax(x, -1), v)
            out[b, :, i] = (o @ turn).view(Hkv * G, D)
            logs[b, :, i] = torch.logsumexp(x, -1).view(Hkv * G)
    return {"out": out, "lse": logs}
