"""The gated feed-forward block of an adapted model and its 8-bit activation checkpoints, as measured cases.

Three kinds of case:

``act8``   bf16 rows compressed to 8 bits (E4M3 codes, one power-of-two scale per 32 columns) and
           expanded again: what a trainer does to an activation between its forward and its backward.
``gated``  h = act(g) * u with g = x.Wg^T + s_a (x.A0_a).B0_a and u = x.Wu^T + s_a (x.A1_a).B1_a, each
           token with its own adapter a (-1: none); with ``save`` also g and u as 8-bit checkpoints.
``grad``   the block's backward on a frozen base from those checkpoints: dX and the adapters' dA and dB,
           and on request h again (the down projection's input). x comes in 16 or in 8 bits.
"""
import math

import torch

own = False

_BLOCK = 32  # columns that share a scale


def listed():
    return [
        # one decode batch's hidden states kept for a step (a launch-bound call)
        dict(name="act8_small", kind="act8", M=64, N=4096),
        # an up projection's activations of one training batch
        dict(name="act8_large", kind="act8", M=2704, N=11008),
        # rows whose last block is half full, an odd number of them
        dict(name="act8_ragged", kind="act8", M=1531, N=5136),
        # decoding one sequence: weights streamed for one token
        dict(name="gated_one_token", kind="gated", M=1, K=4096, F=11008, n=8, r=16, ids="uniform", act="silu", save=False),
        # a decode batch, each request with its own adapter, a few with none
        dict(name="gated_decode", kind="gated", M=36, K=4096, F=11008, n=32, r=16, ids="distinct", act="silu", save=False),
        # the same on the large projection, popular adapters shared
        dict(name="gated_decode_large", kind="gated", M=16, K=8192, F=28672, n=16, r=16, ids="zipf", act="silu", save=False),
        # prefill of eight requests, tokens sorted by adapter, ragged length
        dict(name="gated_prefill", kind="gated", M=2704, K=4096, F=11008, n=8, r=64, ids="sorted", act="silu", save=False),
        # a training forward that keeps its pre-activations in 8 bits
        dict(name="gated_train", kind="gated", M=2048, K=4096, F=11008, n=2, r=16, ids="sorted", act="silu", save=True),
        # a small model's training backward: odd token count and widths, gelu
        dict(name="grad_small", kind="grad", M=333, K=1040, F=2768, n=5, r=8, ids="zipf", act="gelu", x8=False, h=True),
        # the training backward, every kept activation in 8 bits, h for the down projection
        dict(name="grad_train", kind="grad", M=2048, K=4096, F=11008, n=2, r=16, ids="sorted", act="silu", x8=True, h=True),
        # many tenants trained in one batch
        dict(name="grad_tenants", kind="grad", M=512, K=4096, F=11008, n=48, r=32, ids="zipf", act="silu", x8=False, h=False),
        # a frozen block without adapters between two trained ones: dX alone
        dict(name="grad_frozen", kind="grad", M=1024, K=4096, F=11008, n=0, r=16, ids="uniform", act="silu", x8=False, h=False),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    kind = rng.choice(("act8", "gated", "grad"))
    if kind == "act8":
        return dict(kind=kind, M=_log(rng, 1, 2704), N=_log(rng, 256, 11008, 16))
    save = kind == "grad" or rng.random() < 0.4
    while True:
        M, K, F = _log(rng, 1, 2704), _log(rng, 256, 8192, 8), _log(rng, 256, 28672, 8)
        r, n = rng.choice((8, 16, 32, 64)), rng.choice((0, 1, 2, 5, 16, 48))
        K, F = (K // 16 * 16, F // 16 * 16) if save else (K, F)
        if M * K * F <= 2048 * 4096 * 11008 and M * n * r <= 2048 * 512 and n * r * (K + F) <= 1 << 26:
            break
    ids = rng.choice(("uniform", "zipf", "sorted"))
    c = dict(kind=kind, M=M, K=K, F=F, n=n, r=r, ids=ids, act=rng.choice(("silu", "gelu")))
    if kind == "gated":
        c["save"] = save
    else:
        c["x8"], c["h"] = rng.random() < 0.5, rng.random() < 0.5
    return c


def _ids(c, gen, dev):
    M, n = c["M"], c["n"]
    if n == 0:
        return torch.full((M,), -1, dtype=torch.int32, device=dev)
    if c["ids"] == "distinct":
        ids = torch.cat([torch.arange(n, device=dev), torch.full((M - n,), -1, device=dev)])
        return ids[torch.randperm(M, generator=gen, device=dev)].to(torch.int32)
    if c["ids"] == "uniform":
        return torch.randint(0, n, (M,), generator=gen, device=dev, dtype=torch.int32)
    if c["ids"] == "sorted":
        return torch.randint(0, n, (M,), generator=gen, device=dev, dtype=torch.int32).sort().values
    w = torch.arange(1, n + 1, device=dev, dtype=torch.float64) ** -1.1  # popularity by a Zipf law
    ids = torch.multinomial(w, M, replacement=True, generator=gen).to(torch.int32)
    return torch.where(torch.rand(M, generator=gen, device=dev) < 0.05, -1, ids).to(torch.int32)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    c = case

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen, device=dev) * std).to(torch.bfloat16)

    def activations(rows, cols):  # columns of unlike magnitude, as hidden states have
        size = torch.exp(torch.randn(cols, generator=gen, device=dev) * 0.5)
        return (torch.randn(rows, cols, generator=gen, device=dev) * size).to(torch.bfloat16)

    if c["kind"] == "act8":
        s = dict(c=c, x=activations(c["M"], c["N"]), back=torch.empty(c["M"], c["N"], dtype=torch.bfloat16, device=dev))
        if own:
            from adapter_gemm_builder_b200 import lora as L
            s["kept"] = L.Act8(c["M"], c["N"])
        return s
    M, K, F, n, r = c["M"], c["K"], c["F"], c["n"], c["r"]
    s = dict(c=c, ids=_ids(c, gen, dev))
    s["Wg"], s["Wu"] = normal(F, K, std=K ** -0.5), normal(F, K, std=K ** -0.5)
    if n:
        s["ranks"] = torch.randint(1, r + 1, (n,), generator=gen, device=dev, dtype=torch.int32)
        s["ranks"][0] = r
        s["scales"] = torch.rand(n, generator=gen, device=dev) + 0.5
        s["A"], s["B"] = normal(2, n, K, r, std=K ** -0.5), normal(2, n, r, F, std=r ** -0.5)
    x = normal(M, K)
    if c["kind"] == "gated":
        s["x"] = x
        s["h"] = torch.empty(M, F, dtype=torch.bfloat16, device=dev)
    else:
        s["x8"] = _compress(x) if c["x8"] else None
        s["x"] = None if c["x8"] else x
        s["g8"], s["u8"] = _compress(normal(M, F)), _compress(normal(M, F))
        s["dh"] = normal(M, F, std=0.02)
        s["dX"] = torch.empty(M, K, dtype=torch.bfloat16, device=dev)
        s["dA"] = torch.empty_like(s["A"]) if n else None
        s["dB"] = torch.empty_like(s["B"]) if n else None
        s["h"] = torch.empty(M, F, dtype=torch.bfloat16, device=dev) if c["h"] else None
    if own:  # what a program keeps: the pool's handle, the batch's segments, a workspace
        from adapter_gemm_builder_b200 import lora as L
        s["pool"] = L.Pool(s["A"], s["B"], s["ranks"], s["scales"]) if n else None
        s["seg"] = None
        if n:
            s["seg"] = L.Segments(M, n)
            L.lora_build_segments(s["ids"], n, s["seg"])
        s["act"] = {"silu": L.LORA_ACT_SILU, "gelu": L.LORA_ACT_GELU}[c["act"]]
        if c["kind"] == "gated":
            s["ws"] = L.workspace(L.LORA_OP_BF16_GATED, M, K, s["pool"])
            s["save"] = (L.Act8(M, F), L.Act8(M, F)) if c["save"] else None
            s["saved"] = [torch.empty(M, F, dtype=torch.bfloat16, device=dev) for _ in (0, 1)] if c["save"] else None
        else:
            s["ws"] = L.workspace(L.LORA_OP_BF16_GATED_BACKWARD, M, F, s["pool"])
            s["kept"] = [L.Act8.of(*s[k]) if s[k] is not None else None for k in ("g8", "u8", "x8")]
    return s


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    from adapter_gemm_builder_b200 import lora as L
    c = s["c"]
    if c["kind"] == "act8":
        L.act8_compress_rows(s["x"], s["kept"])
        L.act8_expand_rows(s["kept"], s["back"])
        return s["back"]
    if c["kind"] == "gated":
        L.bf16_gated_gemm_lora_epilogue(s["x"], s["Wg"], s["Wu"], s["pool"], s["seg"], s["h"], s["ws"], act=s["act"], save=s["save"])
        if not c["save"]:
            return s["h"]
        L.act8_expand_rows(s["save"][0], s["saved"][0])
        L.act8_expand_rows(s["save"][1], s["saved"][1])
        return s["h"], s["saved"]
    g8, u8, x8 = s["kept"]
    L.bf16_gated_lora_backward(s["dh"], s["Wg"], s["Wu"], s["pool"], s["seg"], g8, u8, x8 if c["x8"] else s["x"],
                               s["dX"], s["dA"], s["dB"], s["ws"], act=s["act"], h=s["h"])
    return {k: s[k] for k in ("dX", "dA", "dB", "h") if s[k] is not None}


# ---------------------------------------------------------------- the plain form, 32 bits

def _blocks(x):
    """x [M][N] as [M][blocks][32], the last block filled with zeros."""
    return torch.nn.functional.pad(x, (0, -x.shape[1] % _BLOCK)).reshape(x.shape[0], -1, _BLOCK)


def _power(e):
    """2^e in 32 bits for whole e in -126 .. 127, from its bits."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _compress(x):
    """E4M3 codes [M][N] and E8M0 scales [M][ceil(N / 32)]: the scale of a block is the smallest power of two
    2^p with amax <= 448 2^p (biased by 127, at least 0)."""
    b = _blocks(x.float())
    amax = b.abs().amax(-1)
    m, e = torch.frexp(amax)  # amax = m 2^e, 1/2 <= m < 1; 448 = 7/8 2^9
    biased = torch.where(amax > 0, (e - 9 + (m > 0.875) + 127).clamp(0, 254), 0)
    codes = (b * _power(127 - biased[..., None])).to(torch.float8_e4m3fn)
    return codes.reshape(x.shape[0], -1)[:, :x.shape[1]].contiguous().view(torch.uint8), biased.to(torch.uint8)


def _expand(codes, scales):
    b = _blocks(codes.view(torch.float8_e4m3fn).float())
    return (b * 0.5 * _power(scales.int()[..., None] - 126)).reshape(codes.shape[0], -1)[:, :codes.shape[1]]


def _act(kind, z):
    """The activation and its derivative."""
    if kind == "silu":
        p = 1 / (1 + torch.exp(-z))
        return z * p, p * (1 + z * (1 - p))
    cdf = 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
    return z * cdf, cdf + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)


def _stacked(s):
    """Both slices of the pool side by side, [2][K][n r] and [2][n r][F], columns past a rank zero, and the
    token mask [M][n r] that holds a token's scale at its own adapter's columns."""
    n, r = s["c"]["n"], s["c"]["r"]
    live = torch.arange(r, device=s["ranks"].device) < s["ranks"][:, None]
    A = torch.where(live[None, :, None, :], s["A"].float(), 0).permute(0, 2, 1, 3).reshape(2, -1, n * r)
    B = torch.where(live[None, :, :, None], s["B"].float(), 0).reshape(2, n * r, -1)
    mine = (s["ids"][:, None] == torch.arange(n, device=s["ids"].device)) * s["scales"]
    return A, B, mine.repeat_interleave(r, 1)


def _run_plain(s):
    c = s["c"]
    if c["kind"] == "act8":
        return _expand(*_compress(s["x"])).to(torch.bfloat16)
    Wg, Wu = s["Wg"].float(), s["Wu"].float()
    if c["n"]:
        A, B, mine = _stacked(s)
    if c["kind"] == "gated":
        x = s["x"].float()
        g, u = x @ Wg.T, x @ Wu.T
        if c["n"]:
            g, u = g + (x @ A[0] * mine) @ B[0], u + (x @ A[1] * mine) @ B[1]
        h = (_act(c["act"], g)[0] * u).to(torch.bfloat16)
        return (h, [_expand(*_compress(z)).to(torch.bfloat16) for z in (g, u)]) if c["save"] else h
    g, u, dh = _expand(*s["g8"]), _expand(*s["u8"]), s["dh"].float()
    a, da = _act(c["act"], g)
    dg, du = dh * u * da, dh * a
    dX = dg @ Wg + du @ Wu
    out = {}
    if c["n"]:
        x = _expand(*s["x8"]) if c["x8"] else s["x"].float()
        tg, tu = dg @ B[0].T * mine, du @ B[1].T * mine
        dX = dX + tg @ A[0].T + tu @ A[1].T
        dA = torch.stack([x.T @ tg, x.T @ tu]).reshape(2, c["K"], c["n"], c["r"]).permute(0, 2, 1, 3)
        dB = torch.stack([(x @ A[0] * mine).T @ dg, (x @ A[1] * mine).T @ du]).reshape(2, c["n"], c["r"], c["F"])
        out["dA"], out["dB"] = dA.to(torch.bfloat16).contiguous(), dB.to(torch.bfloat16)
    out["dX"] = dX.to(torch.bfloat16)
    if c["h"]:
        out["h"] = (a * u).to(torch.bfloat16)
    return out


# ---------------------------------------------------------------- the definition, 64 bits

def _power64(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _round8(x):
    """The values a block-scaled 8-bit copy of x (64 bits) stands for, by arithmetic alone: four significant
    bits, steps of 2^-9 of the block's unit at the least."""
    M, N = x.shape
    wide = torch.zeros(M, -(-N // _BLOCK) * _BLOCK, dtype=torch.float64, device=x.device)
    wide[:, :N] = x
    b = wide.view(M, -1, _BLOCK)
    top = b.abs().amax(-1, keepdim=True)
    p = torch.ceil(torch.log2(torch.where(top > 0, top / 448, 1.0)))
    p = torch.where(top > 448 * _power64(p), p + 1, torch.where(top <= 448 * _power64(p - 1), p - 1, p)).clamp(-127, 127)
    unit = _power64(p)
    v = (b / unit).abs()
    step = _power64(torch.floor(torch.log2(v.clamp_min(2.0 ** -6))) - 3)
    step = torch.where(v >= 16 * step, 2 * step, torch.where((v < 8 * step) & (step > 2.0 ** -9), step / 2, step))
    return (torch.sign(b) * torch.round(v / step) * step * unit).view(M, -1)[:, :N]


def _from8(codes, scales):
    c, e = codes.int(), scales.double() - 127
    low, mid = (c & 7).double(), (c >> 3) & 15
    v = torch.where(mid == 0, low * 2.0 ** -9, (8 + low) * _power64(mid - 10))
    v = torch.where(c >= 128, -v, v)
    return v * _power64(e).repeat_interleave(_BLOCK, 1)[:, :c.shape[1]]


def exact(case, seed):
    s = prepare(case, seed)
    c = s["c"]
    d = torch.float64
    if c["kind"] == "act8":
        return _round8(s["x"].to(d))
    n = c["n"]
    members = [(a, int(s["ranks"][a]), float(s["scales"][a]), (s["ids"] == a).nonzero()[:, 0]) for a in range(n)]

    def value(z):
        if c["act"] == "silu":
            return z * torch.sigmoid(z), torch.sigmoid(z) + z * torch.sigmoid(z) * torch.sigmoid(-z)
        P = torch.special.ndtr(z)
        return z * P, P + z * torch.exp(-z * z / 2) / (2 * math.pi) ** 0.5

    if c["kind"] == "gated":
        x, pre = s["x"].to(d), []
        for i, W in enumerate((s["Wg"], s["Wu"])):
            z = x @ W.to(d).T
            for a, r, scale, t in members:
                z[t] += scale * (x[t] @ s["A"][i, a, :, :r].to(d)) @ s["B"][i, a, :r].to(d)
            pre.append(z)
        h = value(pre[0])[0] * pre[1]
        return (h, [_round8(z) for z in pre]) if c["save"] else h
    g, u, dh = _from8(*s["g8"]), _from8(*s["u8"]), s["dh"].to(d)
    x = _from8(*s["x8"]) if c["x8"] else s["x"].to(d)
    a0, a1 = value(g)
    ds = (dh * u * a1, dh * a0)
    dX, out = torch.zeros(c["M"], c["K"], dtype=d, device=g.device), {}
    if n:
        out["dA"] = torch.zeros(s["A"].shape, dtype=d, device=g.device)
        out["dB"] = torch.zeros(s["B"].shape, dtype=d, device=g.device)
    for i, W in enumerate((s["Wg"], s["Wu"])):
        dX += ds[i] @ W.to(d)
        for a, r, scale, t in members:
            Aa, Ba = s["A"][i, a, :, :r].to(d), s["B"][i, a, :r].to(d)
            back = scale * ds[i][t] @ Ba.T
            dX[t] += back @ Aa.T
            out["dA"][i, a, :, :r] = x[t].T @ back
            out["dB"][i, a, :r] = scale * (x[t] @ Aa).T @ ds[i][t]
    out["dX"] = dX
    if c["h"]:
        out["h"] = a0 * u
    return out


def work(case):
    """Inputs and outputs once; products and sums of the projections and the adapters' terms."""
    c = case
    if c["kind"] == "act8":  # in and out, and the codes and scales written and read between
        return {"bytes": c["M"] * (4 * c["N"] + 2 * (c["N"] + -(-c["N"] // _BLOCK))), "flops": 4 * c["M"] * c["N"]}
    M, K, F, n, r = (c[k] for k in "MKFnr")
    kept = F + -(-F // _BLOCK)
    pool = 4 * min(n, M) * r * (K + F)  # A and B of both slices, 16 bits
    lora = 4 * M * r * (K + F) if n else 0
    if c["kind"] == "gated":
        saved = 2 * M * (2 * kept + 2 * F) if c["save"] else 0  # written, read and expanded
        return {"bytes": 2 * M * K + 4 * F * K + pool + 2 * M * F + saved, "flops": 4 * M * K * F + lora}
    x = 0 if not n else M * (K + -(-K // _BLOCK)) if c["x8"] else 2 * M * K
    nbytes = 2 * M * F + 2 * M * kept + 4 * F * K + 2 * M * K + x + 2 * pool + (2 * M * F if c["h"] else 0)
    return {"bytes": nbytes, "flops": 4 * M * K * F + 3 * lora}
