"""GPU tests of the gated block at the ends of the number range: what the formulas in 64 bits give for
infinite and very large intermediate values, the library gives too."""
import numpy as np
import pytest
import torch

from adapter_gemm_builder_b200 import lora as L
from test_gpu_gated import FN, U, Problem, act64, backward, compress, forward, within

pytestmark = pytest.mark.gpu

INF = float("inf")


def same_with_infinities(got, want, keep):
    """Infinities and NaN where the formula has them (within `keep`, the elements of a sign that no rounding
    decides)."""
    assert torch.equal(torch.isnan(got)[keep], torch.isnan(want)[keep])
    over = torch.isinf(want) & keep
    assert over.any() and torch.equal(got[over], want[over])
    assert torch.isfinite(got[torch.isfinite(want) & keep]).all()


SHAPES = [(1, 64, 48, 1, 16), (40, 256, 512, 4, 16), (200, 128, 304, 5, 8), (700, 136, 9504, 40, 64)]


@pytest.mark.parametrize("M,K,F,n,r", SHAPES)
def test_an_infinite_v_gives_infinities(M, K, F, n, r):
    """One element of A[1] is infinite, so v = x.A is infinite in one column and u = +-inf by the sign of B:
    h = act(g) u is an infinity of that sign, not NaN. The other tokens do not see it."""
    a = n - 1
    ids = np.arange(M) % n
    p = Problem(M, K, F, n, r, ids, seed=21, ranks=[r] * (n - 1) + [max(1, r - 3)])
    p.x[:, 3] = torch.where(p.x[:, 3] == 0, 1.0, p.x[:, 3])
    p.B[1] = torch.where(p.B[1] == 0, torch.ones_like(p.B[1]), p.B[1])
    mine = torch.from_numpy(ids == a)
    clean, _ = forward(p)
    p.A[1, a, 3, 0] = INF
    h, kept = forward(p, save=True)
    g, eg, u, _ = p.pre()
    z = act64("silu", g)[0] * u
    # where g is zero within its error the sign of act(g) is open
    same_with_infinities(h, z, mine[:, None] & (g.abs() > eg) & (g > -80))
    assert torch.equal(h[~mine], clean[~mine])
    back = torch.empty(M, F, dtype=torch.bfloat16, device="cuda")
    L.act8_expand_rows(kept[1], back)
    assert torch.isnan(back.cpu()[mine]).all() and torch.isfinite(back.cpu()[~mine]).all()  # kept as NaN


@pytest.mark.parametrize("M,K,F,n,r", SHAPES)
def test_an_infinite_u_or_v_in_the_backward(M, K, F, n, r):
    """B[0] of one adapter with one token holds an infinity: u = d.B^T is infinite in one rank, dX = +-inf by the
    sign of A and dA's column of that rank +-inf by the sign of x. Then A[1] holds one: v = x.A and dB's row."""
    a = n - 1
    ids = np.arange(M) % max(n - 1, 1) if n > 1 else np.full(M, -1)
    t = M // 2
    ids[t] = a
    p = Problem(M, K, F, n, r, ids, seed=22, ranks=[r] * (n - 1) + [max(1, r - 3)])
    R = max(1, r - 3)
    for z in (p.x, p.A, p.B, p.dh):
        z[z == 0] = 1.0
    clean = backward(p)
    B = p.B.clone()
    p.B[0, a, 0, F // 2] = INF
    o = backward(p)
    act, slope = act64("silu", clean["g"])
    dg = p.dh.double() * clean["u"] * slope
    sign = torch.sign(dg[t, F // 2])
    assert sign != 0 and abs(slope[t, F // 2]) > 1e-4  # the sign is the formula's, not a rounding's
    assert torch.equal(o["dX"][t].cpu().double(), sign * torch.sign(p.A[0, a, :, 0].double()) * INF)
    assert torch.equal(o["dA"][0, a, :, 0].cpu().double(), sign * torch.sign(p.x[t].double()) * INF)
    assert torch.isfinite(o["dA"][0, a, :, 1:]).all() and torch.equal(o["dA"][1], clean["dA"][1])
    assert torch.equal(o["dB"], clean["dB"])
    rest = torch.arange(M, device="cuda") != t
    assert torch.equal(o["dX"][rest], clean["dX"][rest])
    p.B = B
    p.A[1, a, 3, 0] = INF
    o = backward(p)
    du = p.dh.double() * act
    live = du[t] != 0
    want = torch.sign(p.x[t, 3].double()) * torch.sign(du[t]) * INF
    assert live.any() and torch.equal(o["dB"][1, a, 0].cpu().double()[live], want[live])
    assert torch.equal(o["dB"][1, a, 1:], clean["dB"][1, a, 1:]) and torch.equal(o["dB"][0], clean["dB"][0])
    assert torch.equal(o["dX"][rest], clean["dX"][rest])


@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_a_finite_v_past_the_largest_bf16(sign):
    """v = 2^127 (1 + 127/128) + 1.5 2^119 is finite in 32 bits and would round to an infinity in bf16: u = v B
    with B = 2^-126 is 3.996, and h = act(g) u with g = 4."""
    M, K, F = 3, 64, 16
    p = Problem(M, K, F, 1, 8, np.zeros(M), seed=23, ranks=[1])
    for z in (p.x, p.Wg, p.Wu, p.A, p.B):
        z.zero_()
    p.scales[:] = 1.0
    p.x[:, 0], p.x[:, 1], p.x[:, 2] = sign * 2.0 ** 64, sign * 2.0 ** 60, 4.0
    p.Wg[:, 2] = 1.0
    p.A[1, 0, 0, 0], p.A[1, 0, 1, 0] = 2.0 ** 63 * (1 + 127 / 128), 1.5 * 2.0 ** 59
    p.B[1, 0, 0] = 2.0 ** -126
    h, _ = forward(p)
    v = sign * (2.0 ** 127 * (1 + 127 / 128) + 1.5 * 2.0 ** 119)
    want = torch.full((M, F), v * 2.0 ** -126, dtype=torch.float64) * act64("silu", torch.tensor(4.0, dtype=torch.float64))[0]
    # v's halves 2^-16, the activation, a rounding to bf16
    within(h, want, (2.0 ** -16 + FN + U) * 1.01 * want.abs(), "h")


@pytest.mark.parametrize("save", [False, True])
def test_silu_far_below_zero(save):
    """silu(g) = g exp(g) / (1 + exp(g)) down to g = -88, where 1 + exp(-g) is past 2^126: the product with a
    large u is an ordinary number. g = -k / 4 is a sum of one exact product, u = 2^100."""
    K, F = 64, 32
    M = 4 * 88 - 4 * 60
    p = Problem(M, K, F, 0, 8, seed=24)
    for z in (p.x, p.Wg, p.Wu):
        z.zero_()
    k = torch.arange(4 * 60, 4 * 88) + 1
    p.x[:, 0], p.x[:, 1], p.x[:, 2] = -(k // 4).float(), -(k % 4).float() / 4, 2.0 ** 100
    p.Wg[:, 0] = p.Wg[:, 1] = 1.0
    p.Wu[:, 2] = 1.0
    h, _ = forward(p, save=save)
    g = (-k.double() / 4)[:, None].expand(M, F)
    want = g * torch.exp(g) / (1 + torch.exp(g)) * 2.0 ** 100
    # exp of the fast kind: 2 + 1.173 |g| units of 2^-23; then a product, a sum and a division
    within(h, want, (U + 2.0 ** -23 * (2 + 1.173 * g.abs()) + 2.0 ** -20) * 1.01 * want.abs(), "h")


def test_silu_gradient_far_below_zero():
    """The same range in the backward: dg = dh u act'(g), du = dh act(g) through dX with a weight of one. g comes
    from its checkpoint: -88 to -64 in steps of 8 are among its values exactly, and 2^60 times 2^40 keeps the
    products in range."""
    K, F = 16, 32
    g = -torch.arange(64.0, 89.0, 8.0)
    M = len(g)
    p = Problem(M, K, F, 0, 8, seed=25)
    p.Wg.zero_(), p.Wu.zero_()
    p.Wg[0, 0], p.Wu[0, 8] = 1.0, 1.0
    p.dh = torch.full((M, F), 2.0 ** 60).bfloat16()
    g8, gv = compress(g[:, None].expand(M, F))
    u8, uv = compress(torch.full((M, F), 2.0 ** 40))
    assert (gv == g[:, None]).all() and (uv == 2.0 ** 40).all()
    dX, h = torch.empty(M, K, dtype=torch.bfloat16, device="cuda"), torch.empty(M, F, dtype=torch.bfloat16, device="cuda")
    ws = L.workspace(L.LORA_OP_BF16_GATED_BACKWARD, M, F, None)
    L.bf16_gated_lora_backward(p.dh.cuda(), p.Wg.cuda(), p.Wu.cuda(), None, None, g8, u8, None, dX, None, None, ws, h=h)
    z = g.double()
    e = torch.exp(z) / (1 + torch.exp(z))
    act, slope = z * e, e * (1 + z * (1 - e))
    rel = (2 * U + 2.0 ** -23 * (2 + 1.173 * 88) + 2.0 ** -19) * 1.01  # two roundings to bf16
    dX, h = dX.cpu().double(), h.cpu().double()
    for got, want, what in ((dX[:, 0], slope * 2.0 ** 100, "dg"), (dX[:, 8], act * 2.0 ** 60, "du"), (h[:, 0], act * 2.0 ** 40, "h")):
        within(got, want, rel * want.abs(), what)
    assert not dX[:, [1, 9]].any()
