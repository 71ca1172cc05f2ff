"""GPU tests of the 8-bit activation checkpoints (act8_compress_rows, act8_expand_rows).

The reference computes the definition in 64 bits on the CPU: X is the smallest power of two
with amax <= 448 X, the code the E4M3 value nearest to x / X (ties to even), NaN for a
non-finite x. Both directions are exact arithmetic with one rounding, so codes, scales and
expanded bits have to be equal."""
import math

import numpy as np
import pytest
import torch

from adapter_gemm_builder_b200 import lora as L

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    L.load()


# the 127 finite magnitudes of E4M3, by the format's definition
E4M3 = np.array([m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)][:127])


def nearest_codes(v):
    """E4M3 codes of finite |v| <= 448: nearest, ties to the even code; sign in bit 7."""
    a = np.abs(v)
    hi = np.clip(np.searchsorted(E4M3, a), 0, 126)
    lo = np.clip(hi - 1, 0, 126)
    dl, dh = a - E4M3[lo], E4M3[hi] - a
    c = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return (c + 128 * np.signbit(v)).astype(np.uint8)


def compress_ref(x):
    """x: float64 [M, N] of bf16 values -> codes, scales."""
    M, N = x.shape
    nb = -(-N // 32)
    codes, scales = np.zeros((M, N), np.uint8), np.zeros((M, nb), np.uint8)
    for m in range(M):
        for b in range(nb):
            v = x[m, b * 32:(b + 1) * 32]
            ok = np.isfinite(v)
            amax = np.abs(v[ok]).max(initial=0.0)
            p = -127
            if amax > 0:
                p = max(-127, math.frexp(amax / 448)[1])          # amax / 448 < 2^p
                if p > -127 and amax <= 448 * 2.0 ** (p - 1):
                    p -= 1
            scales[m, b] = p + 127
            codes[m, b * 32:(b + 1) * 32] = np.where(ok, nearest_codes(np.where(ok, v, 0) / 2.0 ** p), 0x7f)
    return codes, scales


def run_compress(x):
    M, N = x.shape
    guard = 64
    codes = torch.full((M * N + guard,), 0xAB, dtype=torch.uint8, device="cuda")
    nb = -(-N // 32)
    scales = torch.full((M * nb + guard,), 0xAB, dtype=torch.uint8, device="cuda")
    a = L.Act8.of(codes[:M * N].view(M, N), scales[:M * nb].view(M, nb))
    L.act8_compress_rows(x.cuda(), a)
    torch.cuda.synchronize()
    assert (codes[M * N:] == 0xAB).all() and (scales[M * nb:] == 0xAB).all()
    return a


@pytest.mark.parametrize("M,N", [(1, 16), (1, 32), (3, 48), (7, 272), (5, 256), (33, 1040), (64, 4096), (300, 528)])
def test_compress_and_expand(M, N):
    gen = torch.Generator().manual_seed(M * 10000 + N)
    x = (torch.randn(M, N, generator=gen) * torch.exp(4 * torch.randn(M, N, generator=gen))).bfloat16()
    if M > 1:
        x[1] = 0
        x[0, :16] = torch.randn(16, generator=gen).bfloat16() * 2.0 ** -125
    codes, scales = compress_ref(x.double().numpy())
    a = run_compress(x)
    assert np.array_equal(a.scales.cpu().numpy(), scales)
    got = a.codes.cpu().numpy()
    zero = (got & 127) == 0  # the sign of a zero carries nothing
    assert np.array_equal(np.where(zero, got & 127, got), np.where((codes & 127) == 0, codes & 127, codes))
    back = torch.full((M + 1, N), 7.0, dtype=torch.bfloat16, device="cuda")
    L.act8_expand_rows(a, back[:M])
    val = np.where(codes >= 128, -1, 1) * E4M3[codes & 127] * 2.0 ** (scales.repeat(32, 1)[:, :N].astype(np.float64) - 127)
    assert torch.equal(back[:M].cpu(), torch.from_numpy(val).float().bfloat16())
    assert (back[M] == 7).all()


def test_compress_borders_and_non_finite():
    """Blocks whose largest element is on, just below or just above 448 2^k, over the exponents of
    bf16; infinities and NaN become NaN and leave their block's scale alone."""
    rows = []
    for k in (-141, -133, -120, -119, -60, 0, 8, 60, 118, 119):
        for top in (447.0, 448.0, 450.0, 446.0, 256.0, 255.0, 480.0):
            v = torch.randn(32, generator=torch.Generator().manual_seed(int(top) + k + 500)).double().clamp(-3, 3) * 64
            v[5] = top
            rows.append((v * 2.0 ** k).float().bfloat16())
    x = torch.stack(rows)
    x = x[torch.isfinite(x.float()).all(1)]
    codes, scales = compress_ref(x.double().numpy())
    a = run_compress(x)
    assert np.array_equal(a.scales.cpu().numpy(), scales)
    got = a.codes.cpu().numpy()
    assert np.array_equal(np.where((got & 127) == 0, 0, got), np.where((codes & 127) == 0, 0, codes))

    y = torch.randn(6, 80, generator=torch.Generator().manual_seed(3)).bfloat16()
    y[0, 3], y[1, 40], y[2, 70], y[3, :32], y[4] = float("inf"), float("-inf"), float("nan"), float("nan"), float("inf")
    codes, scales = compress_ref(y.double().numpy())
    a = run_compress(y)
    got = a.codes.cpu().numpy()
    assert np.array_equal(a.scales.cpu().numpy(), scales)
    assert np.array_equal(got & 127, codes & 127)
    back = torch.empty_like(y, device="cuda")
    L.act8_expand_rows(a, back)
    assert torch.equal(torch.isnan(back).cpu(), ~torch.isfinite(y.float()))


def test_expand_every_code_and_scale():
    """All 256 codes under all 256 scales (255: NaN), rounded once to bf16."""
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1).cuda()
    scales = torch.arange(256, dtype=torch.uint8)[:, None].repeat(1, 8).cuda()
    x = torch.empty(256, 256, dtype=torch.bfloat16, device="cuda")
    L.act8_expand_rows(L.Act8.of(codes, scales), x)
    c = np.arange(256)
    v = np.where(c >= 128, -1.0, 1.0) * np.concatenate([E4M3, [np.nan]])[c & 127]
    want = v[None, :] * 2.0 ** (np.arange(256)[:, None] - 127.0)
    want[255] = np.nan
    # float64 -> float32 is exact here: four significant bits, no smaller than 2^-136
    want = torch.from_numpy(want).float().bfloat16()
    assert torch.equal(torch.isnan(x).cpu(), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(x.cpu().float(), nan=0.0, posinf=1.0, neginf=-1.0),
                       torch.nan_to_num(want.float(), nan=0.0, posinf=1.0, neginf=-1.0))


def test_more_than_four_billion_elements():
    """Offsets past 32 bits: the last rows of 2^18 x 16400 elements are what they are alone."""
    M, N = 1 << 18, 16400
    x = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(3, N, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    x[-3:] = tail
    a = L.Act8(M, N)
    L.act8_compress_rows(x, a)
    b = L.Act8(3, N)
    L.act8_compress_rows(tail, b)
    assert torch.equal(a.codes[-3:], b.codes) and torch.equal(a.scales[-3:], b.scales)
    x.fill_(1)
    L.act8_expand_rows(a, x)
    y = torch.empty_like(tail)
    L.act8_expand_rows(b, y)
    assert torch.equal(x[-3:], y) and not x[:-3:4097].any()


def test_empty_stream_and_graph():
    """No rows: nothing is launched. Captured with its expansion, replayed on new inputs."""
    L.act8_compress_rows(torch.empty(0, 32, dtype=torch.bfloat16, device="cuda"), L.Act8(0, 32))
    x = torch.randn(40, 2064, device="cuda").bfloat16()
    a, back = L.Act8(40, 2064), torch.empty(40, 2064, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        L.act8_compress_rows(x, a)
        L.act8_expand_rows(a, back)
    for seed in (1, 2):
        x.copy_(torch.randn(40, 2064, generator=torch.Generator().manual_seed(seed)).bfloat16())
        graph.replay()
        b, want = L.Act8(40, 2064), torch.empty_like(back)
        L.act8_compress_rows(x, b)
        L.act8_expand_rows(b, want)
        torch.cuda.synchronize()
        assert torch.equal(back, want)
