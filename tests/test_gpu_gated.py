"""GPU tests of the gated feed-forward block (bf16_gated_gemm_lora_epilogue) and its backward
(bf16_gated_lora_backward) against the formulas in 64 bits.

Every bound is elementwise and counted before the first run. U = 2^-8 is a bf16 rounding
(half a step), a sum of n fp32 terms on the tensor cores is off by at most n 2^-23 of the sum
of its terms' magnitudes (each partial sum rounded or cut to 24 bits), the operands hi + lo of the
adapters' term carry 2^-16 of v, the activation's exp and division 2^-18."""
import numpy as np
import pytest
import torch

from adapter_gemm_builder_b200 import lora as L
from adapter_gemm_builder_b200 import workloads as wl

pytestmark = pytest.mark.gpu

U, ACC, HILO, FN = 2.0 ** -8, 2.0 ** -23, 2.0 ** -16, 2.0 ** -18
ACTS = {"silu": L.LORA_ACT_SILU, "gelu": L.LORA_ACT_GELU}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    L.load()


def act64(kind, z):
    if kind == "silu":
        p = torch.sigmoid(z)
        return z * p, p * (1 + z * (1 - p))
    P = 0.5 * torch.erfc(-z * 0.5 ** 0.5)  # (special.ndtr loses its digits below -5: 6.1e-16 for 6.2e-16 at -8)
    return z * P, P + z * torch.exp(-z * z / 2) / (2 * np.pi) ** 0.5


class Problem:
    """Inputs of one block; the pool's padding past each rank is NaN."""

    def __init__(self, M, K, F, n, r, ids="uniform", seed=0, none_frac=0.1, ranks=None):
        self.M, self.K, self.F, self.n, self.r = M, K, F, n, r
        gen = torch.Generator().manual_seed(seed * 1000003 + M * 31 + K * 7 + F)
        def normal(*s, std=1.0):
            return (torch.randn(*s, generator=gen) * std).bfloat16()
        self.x, self.Wg, self.Wu = normal(M, K), normal(F, K, std=K ** -0.5), normal(F, K, std=K ** -0.5)
        self.dh = normal(M, F)
        self.ids = np.full(M, -1, np.int32)
        if n:
            rng = np.random.default_rng(seed + M)
            self.ids = wl.make_ids(ids, rng, M, n, none_frac) if isinstance(ids, str) else np.asarray(ids, np.int32)
            self.ranks = torch.as_tensor(ranks if ranks is not None else rng.integers(1, r + 1, n), dtype=torch.int32)
            self.scales = torch.rand(n, generator=gen) + 0.5
            self.A, self.B = normal(2, n, K, r, std=K ** -0.5), normal(2, n, r, F, std=r ** -0.5)
            for a in range(n):
                self.A[:, a, :, int(self.ranks[a]):] = float("nan")
                self.B[:, a, int(self.ranks[a]):] = float("nan")

    def device(self):
        """pool, segments (None without adapters)."""
        if not self.n:
            return None, None
        pool = L.Pool(self.A.cuda(), self.B.cuda(), self.ranks.cuda(), self.scales.cuda())
        seg = L.Segments(self.M, self.n)
        L.lora_build_segments(torch.from_numpy(self.ids).cuda(), self.n, seg)
        return pool, seg

    def adapters(self):
        for a in range(self.n):
            t = torch.from_numpy(np.flatnonzero(self.ids == a))
            if len(t):
                r = int(self.ranks[a])
                yield a, t, r, float(self.scales[a])

    def pre(self):
        """g, u and how far an fp32 computation of them may be off."""
        x, out = self.x.double(), []
        for s, W in enumerate((self.Wg, self.Wu)):
            z = x @ W.double().T
            e = (self.K + 64) * ACC * (x.abs() @ W.double().abs().T)
            for a, t, r, sc in self.adapters():
                A, B = self.A[s, a, :, :r].double(), self.B[s, a, :r].double()
                v = sc * x[t] @ A
                ev = HILO * v.abs() + (self.K + 8) * ACC * sc * (x[t].abs() @ A.abs())
                z[t] += v @ B
                e[t] += ev @ B.abs() + (self.K + 64) * ACC * (v.abs() @ B.abs())
            out += [z, e + 2.0 ** -23 * z.abs()]
        return out


def guarded(op, M, K, pool):
    """A workspace of exactly the asked size with 64 KB of 0xff behind it."""
    n = L.lora_workspace_size(op, M, K, pool)
    room = torch.full((n + 65536,), 0xff, dtype=torch.uint8, device="cuda")
    room[:n] = L.workspace(op, M, K, pool)[:n]
    return room, room[:n]


def forward(p, act="silu", save=False, stream=None):
    pool, seg = p.device()
    x, Wg, Wu = p.x.cuda(), p.Wg.cuda(), p.Wu.cuda()
    h = torch.full((p.M + 1, p.F), 7.0, dtype=torch.bfloat16, device="cuda")
    kept = (L.Act8(p.M, p.F), L.Act8(p.M, p.F)) if save else None
    room, ws = guarded(L.LORA_OP_BF16_GATED, p.M, p.K, pool)
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    L.bf16_gated_gemm_lora_epilogue(x, Wg, Wu, pool, seg, h[:p.M], ws, act=ACTS[act], save=kept, stream=stream)
    torch.cuda.synchronize()
    assert (room[ws.numel():] == 0xff).all()
    st, detail = L.lora_workspace_status(ws)
    assert st == L.LORA_OK, hex(detail)
    assert (h[p.M] == 7).all()  # the row behind the last is left alone
    return h[:p.M].cpu().double(), kept


def within(got, want, bound, what):
    assert torch.isfinite(got).all(), f"{what}: {int((~torch.isfinite(got)).sum())} non-finite of {got.numel()}"
    over = ((got - want).abs() - bound)
    i = int(over.argmax())
    assert over.max() <= 0, (f"{what}: {int((over > 0).sum())} of {over.numel()} off; worst at "
                             f"{np.unravel_index(i, tuple(got.shape))}: {got.flatten()[i]} for {want.flatten()[i]}, bound {bound.flatten()[i]}")


def check_forward(p, act, h):
    g, eg, u, eu = p.pre()
    a, d = act64(act, g)
    # |act'| <= 1.13 for both activations
    e = 1.13 * eg * (u.abs() + eu) + a.abs() * eu + FN * (a * u).abs()
    within(h, a * u, e + U * ((a * u).abs() + e) + 1e-30, "h")


FORWARD = [
    # M, K, F, n, r, ids
    (1, 64, 16, 0, 8, "uniform"), (1, 8, 8, 1, 8, "uniform"), (1, 4096, 264, 3, 16, "identical"),
    (2, 72, 40, 2, 8, "uniform"), (16, 512, 1000, 16, 16, "zipf"), (36, 256, 640, 32, 16, "uniform"),
    (127, 200, 136, 5, 32, "zipf"), (128, 64, 128, 1, 64, "uniform"), (129, 1024, 392, 4, 64, "zipf"),
    (300, 128, 4096, 3, 16, "sorted_zipf"), (257, 328, 2064, 130, 8, "uniform"), (640, 192, 24, 2, 32, "sorted_zipf"),
    (1025, 96, 520, 7, 64, "zipf"),
    # wide enough for pairs of CTAs: whole and ragged pairs, the odd CTA without tokens, many adapters
    (512, 128, 9600, 0, 8, "uniform"), (700, 136, 9496, 3, 16, "sorted_zipf"), (1100, 64, 5000, 300, 8, "uniform"),
    (2049, 72, 3000, 9, 64, "zipf"),
    # tiles shared between CTAs: parts of a tile summed by whichever is done last
    (300, 4096, 1000, 3, 16, "zipf"), (513, 2048, 5000, 2, 32, "sorted_zipf"), (130, 8192, 272, 40, 64, "uniform"),
    # a token tile full of different adapters, one tile and two
    (128, 512, 1040, 128, 64, "uniform"), (256, 264, 9600, 256, 32, "uniform"),
]


@pytest.mark.parametrize("M,K,F,n,r,ids", FORWARD)
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_forward(M, K, F, n, r, ids, act):
    p = Problem(M, K, F, n, r, ids)
    check_forward(p, act, forward(p, act)[0])


@pytest.mark.parametrize("M,K,F,n,r,ids", [(1, 64, 16, 0, 8, "uniform"), (5, 128, 48, 2, 8, "uniform"),
                                           (130, 256, 1040, 5, 16, "zipf"), (513, 200, 272, 3, 64, "sorted_zipf"),
                                           (256, 64, 4112, 2, 32, "identical"), (600, 96, 9616, 4, 64, "sorted_zipf"),
                                           (400, 4096, 1200, 3, 32, "zipf"),
                                           # mixed over many adapters: rows copied by adapter
                                           (700, 136, 9504, 40, 16, "uniform"), (1030, 72, 4112, 130, 32, "zipf")])
def test_forward_with_checkpoints(M, K, F, n, r, ids):
    """h as without them; a block's scale is the rule's for a largest element within the error of the
    sum, and an element is within half an E4M3 step (2^-4, or half the smallest step) of g or u."""
    p = Problem(M, K, F, n, r, ids)
    h, kept = forward(p, save=True)
    check_forward(p, "silu", h)
    g, eg, u, eu = p.pre()
    for z, e, k in ((g, eg, kept[0]), (u, eu, kept[1])):
        X = 2.0 ** (k.scales.cpu().double() - 127)
        pad = -F % 32
        blocks = lambda t: torch.nn.functional.pad(t, (0, pad)).view(M, -1, 32).abs().amax(-1)
        top, err = blocks(z), blocks(e)
        assert (top - err <= 448 * X).all() and (top + err > 224 * X).all()
        Xc = X.repeat_interleave(32, 1)[:, :F]
        back = torch.empty(M, F, dtype=torch.bfloat16, device="cuda")
        L.act8_expand_rows(k, back)
        within(back.cpu().double(), z, e + 2.0 ** -4 * (z.abs() + e) + 2.0 ** -10 * Xc, "checkpoint")


def compress(z):
    """A checkpoint of fp32 values through the library, and the values it stands for."""
    a = L.Act8(*z.shape)
    L.act8_compress_rows(z.bfloat16().cuda(), a)
    back = torch.empty(*z.shape, dtype=torch.bfloat16, device="cuda")
    L.act8_expand_rows(a, back)
    return a, back.cpu().double()


def backward(p, act="silu", x8=False, h=False, seed=5):
    gen = torch.Generator().manual_seed(seed)
    g8, g = compress(1.5 * torch.randn(p.M, p.F, generator=gen))
    u8, u = compress(torch.randn(p.M, p.F, generator=gen))
    pool, seg = p.device()
    x = p.x.cuda()
    xv = p.x.double()
    if x8:
        x, xv = compress(p.x.float())
    dX = torch.full((p.M + 1, p.K), 7.0, dtype=torch.bfloat16, device="cuda")
    dA = dB = None
    if p.n:
        dA = torch.full((2, p.n, p.K, p.r), float("nan"), dtype=torch.bfloat16, device="cuda")
        dB = torch.full((2, p.n, p.r, p.F), float("nan"), dtype=torch.bfloat16, device="cuda")
    hb = torch.full((p.M + 1, p.F), 7.0, dtype=torch.bfloat16, device="cuda") if h else None
    room, ws = guarded(L.LORA_OP_BF16_GATED_BACKWARD, p.M, p.F, pool)
    L.bf16_gated_lora_backward(p.dh.cuda(), p.Wg.cuda(), p.Wu.cuda(), pool, seg, g8, u8, x if p.n else None, dX[:p.M],
                               dA, dB, ws, act=ACTS[act], h=hb[:p.M] if h else None)
    torch.cuda.synchronize()
    assert (room[ws.numel():] == 0xff).all()
    st, detail = L.lora_workspace_status(ws)
    assert st == L.LORA_OK, hex(detail)
    assert (dX[p.M] == 7).all() and (not h or (hb[p.M] == 7).all())
    return dict(g=g, u=u, x=xv, dX=dX[:p.M], dA=dA, dB=dB, h=hb[:p.M] if h else None)


def check_backward(p, act, o):
    dh = p.dh.double()
    a, d = act64(act, o["g"])
    ds = (dh * o["u"] * d, dh * a)
    # a rounding to bf16 and the activation's own error (the derivative's terms sum to 1.2 at most)
    eds = (U * ds[0].abs() + 4 * FN * (dh * o["u"]).abs(), U * ds[1].abs() + FN * ds[1].abs())
    dX, eX = torch.zeros(p.M, p.K, dtype=torch.float64), torch.zeros(p.M, p.K, dtype=torch.float64)
    for s, W in enumerate((p.Wg, p.Wu)):
        W = W.double()
        dX += ds[s] @ W
        eX += eds[s] @ W.abs() + (2 * p.F + 128) * ACC * ((ds[s].abs() + eds[s]) @ W.abs())
    dA, eA = torch.zeros(2, p.n, p.K, p.r, dtype=torch.float64), torch.zeros(2, p.n, p.K, p.r, dtype=torch.float64)
    dB, eB = torch.zeros(2, p.n, p.r, p.F, dtype=torch.float64), torch.zeros(2, p.n, p.r, p.F, dtype=torch.float64)
    for ad, t, r, sc in p.adapters():
        n_t = len(t) + 64
        for s in range(2):
            A, B, x, D, eD = p.A[s, ad, :, :r].double(), p.B[s, ad, :r].double(), o["x"][t], ds[s][t], eds[s][t]
            w = sc * D @ B.T
            ew = sc * (eD @ B.abs().T + (p.F + 8) * ACC * ((D.abs() + eD) @ B.abs().T))
            dX[t] += w @ A.T
            eX[t] += (ew + U * (w.abs() + ew)) @ A.abs().T + (2 * p.F + 128) * ACC * ((w.abs() + ew) @ A.abs().T)
            v = sc * x @ A
            ev = (p.K + 8) * ACC * sc * (x.abs() @ A.abs()) + HILO * v.abs()
            ew = ew + HILO * w.abs()
            dA[s, ad, :, :r] = x.T @ w
            eA[s, ad, :, :r] = x.abs().T @ ew + n_t * ACC * (x.abs().T @ (w.abs() + ew))
            dB[s, ad, :r] = v.T @ D
            eB[s, ad, :r] = v.abs().T @ eD + ev.T @ (D.abs() + eD) + n_t * ACC * ((v.abs() + ev).T @ (D.abs() + eD))
    within(o["dX"].cpu().double(), dX, eX + U * (dX.abs() + eX), "dX")
    if p.n:
        within(o["dA"].cpu().double(), dA, eA + U * (dA.abs() + eA), "dA")
        within(o["dB"].cpu().double(), dB, eB + U * (dB.abs() + eB), "dB")
        for ad in range(p.n):  # past the rank, and adapters without tokens: zeros
            r = int(p.ranks[ad]) if (p.ids == ad).any() else 0
            assert not o["dA"][:, ad, :, r:].any() and not o["dB"][:, ad, r:].any()
    if o["h"] is not None:
        want = a * o["u"]
        within(o["h"].cpu().double(), want, (U + 2 * FN) * want.abs(), "h")


@pytest.mark.parametrize("M,K,F,n,r,ids,act,x8,h", [
    (1, 8, 16, 0, 8, "uniform", "silu", False, False), (1, 64, 16, 1, 8, "uniform", "silu", False, True),
    (3, 80, 48, 2, 8, "uniform", "gelu", True, False), (37, 264, 272, 40, 16, "uniform", "silu", False, True),
    (64, 512, 256, 6, 32, "zipf", "gelu", True, True), (150, 200, 1040, 3, 64, "sorted_zipf", "silu", False, False),
    (333, 1040, 400, 5, 8, "zipf", "gelu", False, True), (128, 256, 128, 0, 8, "uniform", "gelu", False, True),
    (1030, 336, 144, 4, 16, "sorted_zipf", "silu", True, False), (256, 640, 208, 2, 64, "identical", "silu", True, True),
    # pairs of CTAs
    (512, 9600, 80, 0, 8, "uniform", "silu", False, False), (900, 9576, 48, 5, 64, "sorted_zipf", "silu", False, True),
    (1281, 5008, 112, 200, 8, "uniform", "gelu", True, False),
    # long sums: every tile shared, few tokens and many
    (1, 128, 8192, 1, 16, "identical", "silu", False, False), (20, 1040, 4112, 7, 32, "uniform", "silu", True, True),
    (300, 520, 6000, 0, 8, "uniform", "silu", False, False), (700, 1000, 3008, 6, 64, "zipf", "gelu", False, True),
    # many adapters mixed over several tiles: rows by adapter, with shared tiles and without
    (300, 528, 6000, 60, 16, "uniform", "silu", True, True), (520, 264, 1040, 130, 32, "zipf", "gelu", False, False),
])
def test_backward(M, K, F, n, r, ids, act, x8, h):
    p = Problem(M, K, F, n, r, ids)
    check_backward(p, act, backward(p, act, x8, h))


def test_backward_against_differences():
    """A difference of the library's own forward along a direction: L(x) = sum dh h. The step e = 2^-5
    moves x exactly (bf16 grid of 2^-6), the difference quotient is off by the curvature (second
    differences cancel to e^2 / 6 times the third derivative, measured in 64 bits below) and the
    checkpoints' half steps, both counted through the formula in 64 bits."""
    p = Problem(48, 64, 96, 3, 8, "uniform", seed=2)
    p.x = (torch.randint(-64, 65, (48, 64), generator=torch.Generator().manual_seed(9)).float() / 64).bfloat16()
    dirn = torch.randint(-1, 2, (48, 64), generator=torch.Generator().manual_seed(10)).float()
    e = 2.0 ** -5
    base = p.x.float()
    ends = []
    for sign in (1, -1):
        p.x = (base + sign * e * dirn).bfloat16()
        assert torch.equal(p.x.float(), base + sign * e * dirn)
        ends.append(((forward(p)[0] * p.dh.double()).sum(), p))
        g, _, u, _ = p.pre()
        ends[-1] += ((act64("silu", g)[0] * u * p.dh.double()).sum(), (act64("silu", g)[0] * u * p.dh.double()).abs().sum())
    quotient, exact_q = (ends[0][0] - ends[1][0]) / (2 * e), (ends[0][2] - ends[1][2]) / (2 * e)
    # both ends' h are rounded to bf16: 2^-8 of each term at the most
    assert abs(quotient - exact_q) <= 1.1 * U * (ends[0][3] + ends[1][3]) / (2 * e)
    p.x = base.bfloat16()
    _, kept = forward(p, save=True)
    pool, seg = p.device()
    dX = torch.empty(48, 64, dtype=torch.bfloat16, device="cuda")
    dA, dB = torch.empty_like(pool.A), torch.empty_like(pool.B)
    ws = L.workspace(L.LORA_OP_BF16_GATED_BACKWARD, 48, 96, pool)
    L.bf16_gated_lora_backward(p.dh.cuda(), p.Wg.cuda(), p.Wu.cuda(), pool, seg, *kept, p.x.cuda(), dX, dA, dB, ws)
    slope = (dX.cpu().double() * dirn.double()).sum()
    # the slope in 64 bits, and what half an E4M3 step of g and u (2^-4 of each) moves it
    g, _, u, _ = p.pre()
    dh = p.dh.double()
    def linear(s):
        z = dirn.double() @ (p.Wg, p.Wu)[s].double().T
        for a, t, r, sc in p.adapters():
            z[t] += sc * dirn.double()[t] @ p.A[s, a, :, :r].double() @ p.B[s, a, :r].double()
        return z
    tg, tu = linear(0), linear(1)
    a0, d0 = act64("silu", g)
    exact = (dh * (u * d0 * tg + a0 * tu)).sum()
    assert abs(exact - exact_q) <= 0.05 * abs(exact) + 0.5  # the curvature, in 64 bits on both sides
    # |act''| <= 1/2 for silu; roundings of dg, du and dX at the end
    moved = (dh.abs() * (2.0 ** -4 * u.abs() * (d0.abs() + 0.5 * g.abs()) * tg.abs() + 2.0 ** -4 * 1.13 * g.abs() * tu.abs())).sum()
    rounded = 3 * U * (dh.abs() * (u.abs() * 1.13 * tg.abs() + a0.abs() * tu.abs())).sum() + U * (dX.cpu().double().abs()).sum()
    assert abs(slope - exact) <= moved + rounded


def test_together_as_a_training_step_and_graph():
    """The block as a trainer uses it: forward with checkpoints, the down projection by
    bf16_gemm_lora_epilogue, backward from the checkpoints with h again, captured as one graph and
    replayed on other inputs: bit for bit what the calls give on their own."""
    M, K, F, n, r = 200, 256, 400, 3, 16
    p = Problem(M, K, F, n, r, "sorted_zipf", seed=4)
    pool, seg = p.device()
    gen = torch.Generator().manual_seed(8)
    Wd = (torch.randn(K, F, generator=gen) * F ** -0.5).bfloat16().cuda()
    x, dh, Wg, Wu = p.x.cuda(), p.dh.cuda(), p.Wg.cuda(), p.Wu.cuda()
    x8, g8, u8 = L.Act8(M, K), L.Act8(M, F), L.Act8(M, F)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    out = dict(h=torch.empty(M, F, **bf), y=torch.empty(M, K, **bf), dX=torch.empty(M, K, **bf), h2=torch.empty(M, F, **bf),
               dA=torch.empty_like(pool.A), dB=torch.empty_like(pool.B))
    wf, wd = L.workspace(L.LORA_OP_BF16_GATED, M, K, pool), L.workspace(L.LORA_OP_BF16_GEMM, M, F, None)
    wb = L.workspace(L.LORA_OP_BF16_GATED_BACKWARD, M, F, pool)

    def step(o):
        L.act8_compress_rows(x, x8)
        L.bf16_gated_gemm_lora_epilogue(x, Wg, Wu, pool, seg, o["h"], wf, save=(g8, u8))
        L.bf16_gemm_lora_epilogue(o["h"], Wd, None, None, o["y"], wd)
        L.bf16_gated_lora_backward(dh, Wg, Wu, pool, seg, g8, u8, x8, o["dX"], o["dA"], o["dB"], wb, h=o["h2"])

    step(out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(out)
    for seed in (1, 2):
        x.copy_(torch.randn(M, K, generator=torch.Generator().manual_seed(seed)).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        got = {k: v.clone() for k, v in out.items()}
        step(out)
        torch.cuda.synchronize()
        for k in out:
            assert torch.equal(got[k], out[k]), k
    for w in (wf, wd, wb):
        assert L.lora_workspace_status(w)[0] == L.LORA_OK


def test_other_stream_bad_ids_and_repeat():
    """On a side stream; ids outside the pool are served as -1; the same call twice gives the same bits."""
    p = Problem(70, 128, 256, 4, 16, "uniform", seed=6)
    p.ids[::7] = 9  # counted as bad, no adapter
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    h, _ = forward(p, stream=s)
    p.ids[p.ids == 9] = -1
    check_forward(p, "silu", h)
    h2, _ = forward(p)
    assert torch.equal(h, h2)


@pytest.mark.parametrize("M,K,F,n,r", [(1000, 136, 9496, 40, 16), (641, 264, 7000, 100, 8)])
def test_runs_of_tokens_in_any_order(M, K, F, n, r):
    """Requests one after the other, adapters in no order: some tiles' tokens are a run, others are gathered
    from everywhere, and tokens without an adapter lie between them."""
    rng = np.random.default_rng(M)
    ids = np.repeat(rng.integers(-1, n, 40), rng.integers(1, 60, 40)).astype(np.int32)
    ids = np.concatenate([np.full(300, n - 1, np.int32), ids, rng.integers(-1, n, M).astype(np.int32)])[:M]
    p = Problem(M, K, F, n, r, ids, seed=8)
    h, _ = forward(p)
    check_forward(p, "silu", h)
    assert torch.equal(h, forward(p)[0])


def test_non_finite_rows_stay_in_their_rows():
    p = Problem(140, 64, 96, 3, 8, "uniform", seed=7)
    clean, _ = forward(p)
    p.x[3, 5], p.x[131, 0] = float("nan"), float("inf")
    dirty, _ = forward(p)
    keep = torch.ones(140, dtype=torch.bool)
    keep[[3, 131]] = False
    assert torch.equal(clean[keep], dirty[keep])
    assert not torch.isfinite(dirty[3]).any()


@pytest.mark.parametrize("M,K,F,r", [(40, 256, 512, 16), (200, 128, 304, 8), (700, 136, 9504, 64)])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_a_broken_adapter_stays_with_its_tokens(M, K, F, r, value):
    """One adapter's B (forward) or A (backward) holds an infinity or NaN: the rows of its tokens are NaN,
    the other rows, and the other adapters' gradients, are bit for bit what they are without it."""
    p = Problem(M, K, F, 4, r, "uniform", seed=11, ranks=[r, max(1, r - 3), r, 1])
    mine = torch.from_numpy(p.ids == 1)
    clean, kept = forward(p, save=True)
    o = backward(p)
    A, B = p.A.clone(), p.B.clone()
    p.B[1, 1, 0, F // 2] = value
    dirty, bad = forward(p, save=True)
    assert torch.equal(clean[~mine], dirty[~mine]) and torch.isnan(dirty[mine]).all()
    other = (~mine).cuda()
    for a, b in zip(kept, bad):
        assert torch.equal(a.codes[other], b.codes[other]) and torch.equal(a.scales[other], b.scales[other])
    p.B, p.A = B, A
    p.A[0, 1, K // 2, 0] = value
    d = backward(p)
    assert torch.equal(o["dX"][other], d["dX"][other]) and torch.isnan(d["dX"][mine.cuda()]).all()
    for g in ("dA", "dB"):
        for a in (0, 2, 3):
            assert torch.equal(o[g][:, a], d[g][:, a])


def test_more_than_four_billion_elements():
    """Offsets past 32 bits: the last rows of 2^18 tokens by F 16400, forward with checkpoints and backward."""
    M, K, F, n, r = 1 << 18, 64, 16400, 2, 8
    p = Problem(150, K, F, n, r, "uniform", seed=14, none_frac=0.0)
    pool, _ = p.device()
    tail = p.M
    ids = torch.full((M,), -1, dtype=torch.int32, device="cuda")
    ids[-tail:] = torch.from_numpy(p.ids).cuda()
    seg = L.Segments(M, n)
    L.lora_build_segments(ids, n, seg)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    x, h = torch.zeros(M, K, **bf), torch.empty(M, F, **bf)
    x[-tail:] = p.x.cuda()
    Wg, Wu = p.Wg.cuda(), p.Wu.cuda()
    g8, u8 = L.Act8(M, F), L.Act8(M, F)
    ws = L.workspace(L.LORA_OP_BF16_GATED, M, K, pool)
    L.bf16_gated_gemm_lora_epilogue(x, Wg, Wu, pool, seg, h, ws, save=(g8, u8))
    torch.cuda.synchronize()
    assert L.lora_workspace_status(ws)[0] == L.LORA_OK
    check_forward(p, "silu", h[-tail:].cpu().double())
    assert not h[:-tail:997].any()
    values = []
    for k in (g8, u8):
        v = torch.empty(tail, F, **bf)
        L.act8_expand_rows(L.Act8.of(k.codes[-tail:], k.scales[-tail:]), v)
        values.append(v.cpu().double())
    dh = h.zero_()  # its buffer again
    dh[-tail:] = p.dh.cuda()
    dX, dA, dB = torch.empty(M, K, **bf), torch.empty_like(pool.A), torch.empty_like(pool.B)
    ws = L.workspace(L.LORA_OP_BF16_GATED_BACKWARD, M, F, pool)
    L.bf16_gated_lora_backward(dh, Wg, Wu, pool, seg, g8, u8, x, dX, dA, dB, ws)
    torch.cuda.synchronize()
    assert L.lora_workspace_status(ws)[0] == L.LORA_OK
    assert not dX[:-tail:997].any()
    check_backward(p, "silu", dict(g=values[0], u=values[1], x=p.x.double(), dX=dX[-tail:], dA=dA, dB=dB, h=None))


def test_captured_as_the_very_first_call():
    """In a process of its own: nothing ran before the capture."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = """
import torch
from adapter_gemm_builder_b200 import lora as L
M, K, F = 600, 96, 9616
bf = dict(dtype=torch.bfloat16, device="cuda")
x, Wg, Wu, h = torch.randn(M, K, **bf), torch.randn(F, K, **bf), torch.randn(F, K, **bf), torch.empty(M, F, **bf)
dh, dX = torch.randn(M, F, **bf), torch.empty(M, K, **bf)
g8, u8 = L.Act8(M, F), L.Act8(M, F)
wf, wb = L.workspace(L.LORA_OP_BF16_GATED, M, K, None), L.workspace(L.LORA_OP_BF16_GATED_BACKWARD, M, F, None)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    L.bf16_gated_gemm_lora_epilogue(x, Wg, Wu, None, None, h, wf, save=(g8, u8))
    L.bf16_gated_lora_backward(dh, Wg, Wu, None, None, g8, u8, None, dX, None, None, wb)
g.replay()
torch.cuda.synchronize()
a, b = h.clone(), dX.clone()
L.bf16_gated_gemm_lora_epilogue(x, Wg, Wu, None, None, h, wf, save=(g8, u8))
L.bf16_gated_lora_backward(dh, Wg, Wu, None, None, g8, u8, None, dX, None, None, wb)
torch.cuda.synchronize()
assert torch.equal(a, h) and torch.equal(b, dX)
print("same")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=180)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


def test_two_graphs_with_a_workspace_each_on_two_streams():
    """Two captured calls replayed at the same time, each with its own workspace."""
    p = Problem(150, 256, 1040, 5, 16, "uniform", seed=12)
    pool, seg = p.device()
    x, Wg, Wu = p.x.cuda(), p.Wg.cuda(), p.Wu.cuda()
    want, _ = forward(p)
    runs = []
    for _ in range(2):
        h = torch.zeros(150, 1040, dtype=torch.bfloat16, device="cuda")
        ws = L.workspace(L.LORA_OP_BF16_GATED, 150, 256, pool)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            L.bf16_gated_gemm_lora_epilogue(x, Wg, Wu, pool, seg, h, ws)
        runs.append((g, h, ws, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for g, _, _, s in runs:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for _, h, ws, _ in runs:
        assert L.lora_workspace_status(ws)[0] == L.LORA_OK
        assert torch.equal(h.cpu().double(), want)


def test_backward_twice_gives_the_same_bits():
    """Shared tiles are finished by whichever piece is done last, the sum is the same."""
    p = Problem(180, 512, 6000, 3, 16, "uniform", seed=13)
    a = backward(p)
    for _ in range(5):
        b = backward(p)
        for k in ("dX", "dA", "dB"):
            assert torch.equal(a[k], b[k]), k


@pytest.mark.parametrize("M,K,F", [(300, 256, 512), (700, 136, 9496)])  # single CTAs, pairs
def test_wait_runs_out_then_next_call_is_correct(M, K, F):
    """The bounded wait: a stalled launch returns and reports it, the next call is right."""
    for n in (0, 3):
        p = Problem(M, K, F, n, 16, "uniform", seed=8)
        pool, seg = p.device()
        h = torch.empty(p.M, p.F, dtype=torch.bfloat16, device="cuda")
        ws = L.workspace(L.LORA_OP_BF16_GATED, p.M, p.K, pool)
        args = (p.x.cuda(), p.Wg.cuda(), p.Wu.cuda(), pool, seg, h, ws)
        torch.cuda.synchronize()
        L.lora_debug_set_wait_limit(1_000_000, inject_stall=True)
        try:
            L.bf16_gated_gemm_lora_epilogue(*args)
            torch.cuda.synchronize()
        finally:
            L.lora_debug_set_wait_limit(0, False)
        assert L.lora_workspace_status(ws)[0] == L.LORA_ERR_TIMEOUT
        if n:
            L.lora_segments_status(seg)  # the shrink before it stalled too
        L.bf16_gated_gemm_lora_epilogue(*args)
        torch.cuda.synchronize()
        assert L.lora_workspace_status(ws)[0] == L.LORA_OK
        check_forward(p, "silu", h.cpu().double())
