"""Host-side checks of the 8-bit checkpoints and the gated block: refusals come before any launch
(no GPU needed), and the workspace sizes hold what the calls put there."""
import ctypes

import pytest
import torch

from adapter_gemm_builder_b200 import build as lbuild
from adapter_gemm_builder_b200 import lora as L


@pytest.fixture(scope="module")
def lib():
    lbuild.build()
    return L.load()


def _pool(**kw):
    d = dict(A=16, B=32, ranks=None, scales=None, n_slices=2, n_adapters=4, h_in=64, h_out=96, r_max=16)
    d.update(kw)
    return L.lora_pool_t(*(d[k] for k in ("A", "B", "ranks", "scales", "n_slices", "n_adapters", "h_in", "h_out", "r_max")))


def _seg(T=8, n=4):
    return L.lora_segments_t(16, 32, 48, 64, 80, 96, T, n)


P = ctypes.c_void_p
REF = ctypes.byref


def test_act8_refusals(lib):
    a = L.lora_act8_t(1024, 2048)
    for f, args in ((lib.act8_compress_rows, lambda x, M, N, c: (x, M, N, c, None)),
                    (lib.act8_expand_rows, lambda x, M, N, c: (c, M, N, x, None))):
        assert f(*args(P(4096), 4, 24, REF(a))) == L.LORA_ERR_INVALID_ARG      # N % 16
        assert f(*args(P(4096), 4, 0, REF(a))) == L.LORA_ERR_INVALID_ARG
        assert f(*args(P(4096), -1, 32, REF(a))) == L.LORA_ERR_INVALID_ARG
        assert f(*args(None, 4, 32, REF(a))) == L.LORA_ERR_INVALID_ARG
        assert f(*args(P(4104), 4, 32, REF(a))) == L.LORA_ERR_INVALID_ARG      # x not 16-byte aligned
        assert f(*args(P(4096), 4, 32, None)) == L.LORA_ERR_INVALID_ARG
        assert f(*args(P(4096), 4, 32, REF(L.lora_act8_t(1032, 2048)))) == L.LORA_ERR_INVALID_ARG
        assert f(*args(P(4096), 4, 32, REF(L.lora_act8_t(1024, None)))) == L.LORA_ERR_INVALID_ARG
        assert f(*args(P(4096), 1 << 30, 512, REF(a))) == L.LORA_ERR_UNSUPPORTED
        assert f(*args(None, 0, 32, None)) == L.LORA_OK                        # no rows: nothing to do


def _forward(lib, **kw):
    d = dict(x=P(1024), M=8, K=64, F=96, Wg=P(2048), Wu=P(4096), act=0, pool=None, seg=None, h=P(8192), g8=None, u8=None,
             ws=P(16384), n=1 << 30, stream=None)
    d.update(kw)
    return lib.bf16_gated_gemm_lora_epilogue(*d.values())


def _backward(lib, **kw):
    a = L.lora_act8_t(1024, 2048)
    d = dict(x=None, x8=None, dh=P(1024), M=8, K=64, F=96, Wg=P(2048), Wu=P(4096), act=0, pool=None, seg=None, g8=REF(a),
             u8=REF(a), h=None, dX=P(8192), dA=None, dB=None, ws=P(16384), n=1 << 30, stream=None)
    d.update(kw)
    return lib.bf16_gated_lora_backward(*d.values())


BAD = L.LORA_ERR_INVALID_ARG


@pytest.mark.parametrize("kw,code", [
    (dict(M=0), BAD), (dict(K=60), BAD), (dict(F=4), BAD), (dict(Wg=None), BAD), (dict(Wu=P(4104)), BAD), (dict(act=2), BAD),
    (dict(M=(1 << 24) + 1), L.LORA_ERR_UNSUPPORTED), (dict(ws=None), L.LORA_ERR_WORKSPACE), (dict(n=128), L.LORA_ERR_WORKSPACE),
    (dict(ws=P(16392)), L.LORA_ERR_WORKSPACE),
    (dict(pool=REF(_pool(n_slices=1)), seg=REF(_seg())), BAD),   # two slices: gate and up
    (dict(pool=REF(_pool(h_in=128)), seg=REF(_seg())), BAD),
    (dict(pool=REF(_pool(h_out=64)), seg=REF(_seg())), BAD),
    (dict(pool=REF(_pool(r_max=24)), seg=REF(_seg())), L.LORA_ERR_UNSUPPORTED),
    (dict(pool=REF(_pool())), BAD),                              # no segments
    (dict(pool=REF(_pool()), seg=REF(_seg(T=7))), BAD),
    (dict(pool=REF(_pool()), seg=REF(_seg(n=5))), BAD),
])
def test_gated_shared_refusals(lib, kw, code):
    assert _forward(lib, **kw) == code
    more = dict(x=P(1024), dA=P(32768), dB=P(65536)) if "pool" in kw else {}
    assert _backward(lib, **kw, **more) == code


def test_forward_refusals(lib):
    a = L.lora_act8_t(1024, 2048)
    assert _forward(lib, x=None) == BAD and _forward(lib, h=None) == BAD and _forward(lib, h=P(8200)) == BAD
    assert _forward(lib, g8=REF(a)) == BAD                                    # one checkpoint only
    assert _forward(lib, g8=REF(a), u8=REF(a), F=104) == BAD                  # F % 16 with checkpoints
    assert _forward(lib, g8=REF(a), u8=REF(L.lora_act8_t(None, 2048))) == BAD


def test_backward_refusals(lib):
    a = L.lora_act8_t(1024, 2048)
    both = dict(pool=REF(_pool()), seg=REF(_seg()), dA=P(32768), dB=P(65536))
    assert _backward(lib, F=104) == BAD and _backward(lib, dh=None) == BAD and _backward(lib, dX=None) == BAD
    assert _backward(lib, g8=None) == BAD and _backward(lib, u8=None) == BAD and _backward(lib, h=P(8200)) == BAD
    assert _backward(lib, **both) == BAD                                      # neither x nor x8
    assert _backward(lib, **both, x=P(1024), x8=REF(a)) == BAD                # both
    assert _backward(lib, **{**both, "dA": None}, x=P(1024)) == BAD
    assert _backward(lib, **{**both, "pool": REF(_pool(h_in=72))}, K=72, x8=REF(a)) == BAD  # x8 needs K % 16


def test_workspace_sizes(lib):
    none = ctypes.c_size_t(-1).value
    size = lib.lora_workspace_size
    F, B = L.LORA_OP_BF16_GATED, L.LORA_OP_BF16_GATED_BACKWARD
    assert size(F, 8, 64, None) == 256
    assert size(B, 8, 96, None) >= 256 + 2 * 8 * 96 * 2 + 148 * 3 * 128 * 256 * 4   # dg, du, pieces of shared tiles
    p = _pool()
    # v in fp32 and its three bf16 parts, both slices; the backward: dg, du, x, u and v's parts
    assert size(F, 8, 64, REF(p)) >= 256 + 2 * 8 * 16 * (4 + 6)
    assert size(B, 8, 96, REF(p)) >= 256 + 2 * 8 * 96 * 2 + 8 * 64 * 2 + 2 * 8 * 16 * (4 + 6 + 6)
    assert size(F, 8, 72, REF(p)) == none and size(B, 8, 64, REF(p)) == none   # not the pool's h_in, h_out
    assert size(F, 0, 64, None) == none and size(F, 8, 0, None) == none
    assert size(F, 8, 64, REF(_pool(n_slices=1))) == none


def test_binding_refuses_other_tensors():
    x = torch.zeros(4, 32, dtype=torch.bfloat16)
    with pytest.raises(L.LoraError):
        L.act8_compress_rows(x, L.Act8(4, 32, device="cpu"))                   # not on a GPU
    with pytest.raises(L.LoraError):
        L.Act8.of(torch.zeros(4, 48, dtype=torch.uint8), torch.zeros(4, 1, dtype=torch.uint8))
    with pytest.raises(L.LoraError):
        L.Act8.of(torch.zeros(4, 48, dtype=torch.int8), torch.zeros(4, 2, dtype=torch.uint8))
    W = torch.zeros(48, 32, dtype=torch.bfloat16)
    with pytest.raises(L.LoraError):
        L.bf16_gated_gemm_lora_epilogue(x, W, W, None, None, torch.zeros(4, 48, dtype=torch.bfloat16), x)
