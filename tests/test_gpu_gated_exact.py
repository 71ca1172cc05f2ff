"""The gated block's backward on whole numbers, bit for bit, on each way its dX product can go: tiles whole or
shared in pieces, of one CTA or a pair, in the caller's order or by adapter.

g = 8 everywhere with the erf activation: act(8) = 8 and act'(8) = 1 to 1e-14, so dg = dh u and du = 8 dh are
whole numbers that bf16 holds, and so are h = 8 u and every partial sum (all below 2^24, or multiples of 8
below 2^27): the only rounding is the outputs', to the nearest bf16. An adapter's first two ranks nearly cancel:
A[:, 1] = -A[:, 0] and B[1] is B[0] but for a few ones, while u of either is about 6 F, past 8 bits and within
16: dX shows a lost low half of u."""
import numpy as np
import pytest
import torch

from adapter_gemm_builder_b200 import lora as L
from test_gpu_gated import guarded


class Whole:
    def __init__(self, M, K, F, n, r, seed=0, device="cuda"):
        self.M, self.K, self.F, self.n, self.r, self.device = M, K, F, n, r, device
        gen = torch.Generator().manual_seed(seed * 7919 + M * 31 + K * 7 + F)

        def whole(lo, hi, *s):
            return torch.randint(lo, hi + 1, s, generator=gen).bfloat16().to(device)

        def sparse(*s):  # -1, 0 or 1, one in eight not zero
            return (torch.randint(-1, 2, s, generator=gen) * (torch.rand(s, generator=gen) < 3 / 16)).bfloat16().to(device)

        self.x, self.dh, self.u = whole(-1, 1, M, K), whole(1, 3, M, F), whole(1, 2, M, F)
        self.Wg, self.Wu = sparse(F, K), sparse(F, K)
        self.ids = np.full(M, -1, np.int32)
        if n:
            rng = np.random.default_rng(seed + M)
            self.ids = rng.integers(0, n, M).astype(np.int32)
            self.ids[rng.random(M) < 0.1] = -1
            self.ids[0] = 0
            self.ranks = torch.as_tensor(rng.integers(2, r + 1, n), dtype=torch.int32)
            self.scales = torch.as_tensor(rng.integers(1, 3, n), dtype=torch.float32)
            self.A, self.B = sparse(2, n, K, r), whole(-1, 1, 2, n, r, F)
            self.A[..., 0] = whole(-1, 1, 2, n, K)
            self.A[..., 1] = -self.A[..., 0]
            self.B[:, :, 0] = whole(1, 3, 2, n, F)
            self.B[:, :, 1] = self.B[:, :, 0] + sparse(2, n, F)
            for a in range(n):
                self.A[:, a, :, int(self.ranks[a]):] = float("nan")
                self.B[:, a, int(self.ranks[a]):] = float("nan")

    def formula(self, low_halves=True, stage=None):
        """dX, dA, dB, h in 64 bits. low_halves False: u only to 8 bits; stage: these 64 columns of F left
        out of dX's sum."""
        d = torch.float64
        dh = self.dh.to(d)
        ds = (dh * self.u.to(d), 8 * dh)
        dX = torch.zeros(self.M, self.K, dtype=d, device=self.device)
        for D, W in zip(ds, (self.Wg, self.Wu)):
            if stage is not None:
                D = D.clone()
                D[:, 64 * stage:64 * stage + 64] = 0
            dX += D @ W.to(d)
        out = dict(dX=dX, h=8 * self.u.to(d))
        if not self.n:
            return out
        out["dA"] = torch.zeros(2, self.n, self.K, self.r, dtype=d, device=self.device)
        out["dB"] = torch.zeros(2, self.n, self.r, self.F, dtype=d, device=self.device)
        x = self.x.to(d)
        for a in range(self.n):
            t = torch.from_numpy(np.flatnonzero(self.ids == a)).to(self.device)
            R, s_a = int(self.ranks[a]), float(self.scales[a])
            for s in range(2) if len(t) else ():
                A, B = self.A[s, a, :, :R].to(d), self.B[s, a, :R].to(d)
                w, v = s_a * ds[s][t] @ B.T, s_a * x[t] @ A
                # 16 significant bits: u's sums are multiples of s_a, or of 8 s_a
                assert w.abs().max() < s_a * (1, 8)[s] * 2 ** 16 and v.abs().max() < 2 ** 16
                dX[t] += (w if low_halves else w.bfloat16().to(d)) @ A.T
                out["dA"][s, a, :, :R] = x[t].T @ w
                out["dB"][s, a, :R] = v.T @ ds[s][t]
        return out

    def arguments(self, x8=False):
        pool = seg = None
        if self.n:
            pool = L.Pool(self.A, self.B, self.ranks.cuda(), self.scales.cuda())
            seg = L.Segments(self.M, self.n)
            L.lora_build_segments(torch.from_numpy(self.ids).cuda(), self.n, seg)

        def kept(t):
            k, back = L.Act8(*t.shape), torch.empty_like(t)
            L.act8_compress_rows(t, k)
            L.act8_expand_rows(k, back)
            assert torch.equal(back, t)
            return k

        bf = dict(dtype=torch.bfloat16, device="cuda")
        out = dict(dX=torch.full((self.M, self.K), 7.0, **bf), h=torch.full((self.M, self.F), 7.0, **bf))
        if self.n:
            out["dA"], out["dB"] = torch.full(self.A.shape, 7.0, **bf), torch.full(self.B.shape, 7.0, **bf)
        room, ws = guarded(L.LORA_OP_BF16_GATED_BACKWARD, self.M, self.F, pool)
        x = None if not self.n else kept(self.x) if x8 else self.x
        args = (self.dh, self.Wg, self.Wu, pool, seg, kept(torch.full_like(self.u, 8.0)), kept(self.u), x, out["dX"],
                out.get("dA"), out.get("dB"), ws)
        return args, out, room

    def plan(self, pool):
        return L.lora_debug_gated_plan(True, self.M, self.K, self.F, False, pool)


def check(p, out, room, ws):
    torch.cuda.synchronize()
    st, detail = L.lora_workspace_status(ws)
    assert st == L.LORA_OK, hex(detail)
    assert (room[ws.numel():] == 0xff).all()
    for k, want in p.formula().items():
        assert torch.equal(out[k], want.float().bfloat16()), k


# M, K, F, adapters, r; the plan: pairs of CTAs, whole tiles, tiles shared in pieces, rows by adapter
WAYS = [
    (70, 200, 272, 5, 64, (0, 1, 0, 0)),
    (1, 128, 8192, 1, 16, (0, 0, 1, 0)), (100, 528, 8192, 16, 16, (0, 0, 1, 0)), (100, 528, 8192, 0, 8, (0, 0, 1, 0)),
    (333, 1040, 400, 5, 8, (1, 1, 0, 0)), (520, 264, 1040, 130, 32, (1, 1, 0, 1)),
    (300, 528, 6000, 0, 8, (1, 0, 1, 0)), (300, 528, 6000, 60, 16, (1, 0, 1, 0)),
    (300, 528, 6000, 200, 32, (1, 0, 1, 1)),
    (1200, 4096, 6000, 0, 8, (1, 1, 1, 0)), (1200, 4096, 6000, 3, 16, (1, 1, 1, 0)),
    (1200, 4096, 6000, 100, 32, (1, 1, 1, 1)),
]


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,F,n,r,way", WAYS)
def test_backward_of_whole_numbers(M, K, F, n, r, way):
    p = Whole(M, K, F, n, r)
    args, out, room = p.arguments(x8=K % 16 == 0 and M % 2 == 0)
    plan = p.plan(args[3])
    assert (plan["pair"], plan["whole_tiles"] > 0, plan["whole_tiles"] < plan["tiles"], plan["by_adapter"]) == way, plan
    L.bf16_gated_lora_backward(*args, act=L.LORA_ACT_GELU, h=out["h"])
    check(p, out, room, args[-1])


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,F,n,r", [(70, 200, 272, 0, 8), (70, 200, 272, 5, 64), (100, 528, 8192, 0, 8), (100, 528, 8192, 16, 16),
                                       (520, 264, 1040, 130, 32), (300, 528, 6000, 0, 8), (300, 528, 6000, 200, 32)])
def test_a_wait_of_the_backward_runs_out(M, K, F, n, r):
    """The bounded waits of the dX product (a CTA, a pair, shared tiles, with adapters and without): a launch
    whose loads never begin on one CTA returns and reports it, and the next call on the same workspace is right."""
    p = Whole(M, K, F, n, r)
    args, out, room = p.arguments()
    torch.cuda.synchronize()
    L.lora_debug_set_wait_limit(1_000_000, inject_stall=True)
    try:
        L.bf16_gated_lora_backward(*args, act=L.LORA_ACT_GELU, h=out["h"])
        torch.cuda.synchronize()
    finally:
        L.lora_debug_set_wait_limit(0, False)
    assert L.lora_workspace_status(args[-1])[0] == L.LORA_ERR_TIMEOUT
    L.bf16_gated_lora_backward(*args, act=L.LORA_ACT_GELU, h=out["h"])
    check(p, out, room, args[-1])


@pytest.mark.parametrize("M,K,F,n,r", [(70, 200, 272, 5, 64), (1, 128, 8192, 1, 16), (100, 528, 2048, 16, 16)])
def test_the_whole_numbers_tell(M, K, F, n, r):
    """On the CPU: u to 8 bits, or 64 columns of the sum left out, is another dX after the rounding."""
    p = Whole(M, K, F, n, r, device="cpu")
    right = p.formula()["dX"].float().bfloat16()
    own = torch.from_numpy(p.ids >= 0)
    other = p.formula(low_halves=False)["dX"].float().bfloat16()
    # a row of a short sum may have both ranks' u off by the same amount
    assert (other != right)[own].any(1).double().mean() > 0.75
    for stage in (0, F // 128, (F - 1) // 64):
        other = p.formula(stage=stage)["dX"].float().bfloat16()
        assert (other != right).any(1).all()


def test_the_plan_hook_refuses():
    bad = [(0, 64, 96, None), (8, 60, 96, None), (8, 64, 4, None)]
    bad += [(8, 64, 96, L.Pool(torch.zeros(2, 4, k, 16), torch.zeros(2, 4, 16, f))) for k, f in ((128, 96), (64, 104))]
    bad += [(8, 64, 96, L.Pool(torch.zeros(1, 4, 64, 16), torch.zeros(1, 4, 16, 96)))]
    for M, K, F, pool in bad:
        with pytest.raises(L.LoraError):
            L.lora_debug_gated_plan(True, M, K, F, False, pool)
    plan = L.lora_debug_gated_plan(False, 8, 64, 96)
    assert plan["tiles"] == plan["whole_tiles"] >= 1 and plan["pieces"] == 1
