"""The e2m1 entry points without a GPU: refused before anything is launched; the
tests' own arithmetic against worked values."""
import ctypes

import pytest
import torch

import fp4_testutil as f4
import unpermute_combine_gb300 as moe
from unpermute_combine_gb300 import build as libbuild

P = ctypes.c_void_p
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
fake, other = P(0x1000), P(0x8000)     # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return moe.load_library()


def quantize(lib, x=fake, dt=1, T=4, H=64, block=16, g=None, q=fake, s=fake):
    return lib.moe_quantize_fp4(x, dt, T, H, block, g, q, s, None)


def permute(lib, x=fake, dt=1, T=4, H=64, block=16, g=None, k=2, n=8, pos=fake, q=fake, s=fake):
    return lib.moe_permute_quantize_fp4(x, dt, T, H, block, g, k, n, pos, q, s, None)


def dequantize(lib, q=fake, s=fake, T=4, H=64, block=16, g=None, x=fake):
    return lib.moe_dequantize_fp4(q, s, T, H, block, g, x, None)


@pytest.mark.parametrize("call", [quantize, permute, dequantize])
def test_quantizers_refuse(lib, call):
    for kw in (dict(T=-1), dict(H=-32), dict(H=48), dict(x=None), dict(q=None), dict(s=None),
               dict(x=P(0x1008)), dict(q=P(0x1004)), dict(g=P(0x1002)), dict(block=32, g=fake)):
        assert call(lib, **kw) == INVALID, kw
    for kw in (dict(block=8), dict(block=64), dict(block=0), dict(H=1 << 29), dict(T=1 << 31)):
        assert call(lib, **kw) == UNSUPPORTED, kw
    for kw in (dict(T=0, x=None, q=None, s=None), dict(H=0, x=None, q=None, s=None)):
        assert call(lib, **kw) == OK, kw


def test_quantizers_refuse_types_and_slots(lib):
    for call in (quantize, permute):
        assert call(lib, dt=2) == INVALID and call(lib, dt=7) == INVALID
    for kw in (dict(k=0), dict(n=-1), dict(pos=None), dict(pos=P(0x1001))):
        assert permute(lib, **kw) == INVALID, kw
    assert permute(lib, k=33) == UNSUPPORTED


def pack(lib, w=fake, E=2, N=128, K=64, gu=0, block=16, g=None, q=fake, s=fake):
    return lib.moe_pack_fp4(w, E, N, K, gu, block, g, q, s, None)


def test_pack_refuses(lib):
    for kw in (dict(E=0), dict(N=-1), dict(K=48), dict(w=None), dict(q=None), dict(s=None),
               dict(w=P(0x1008)), dict(q=P(0x1008)), dict(s=P(0x1008)), dict(block=32, g=fake)):
        assert pack(lib, **kw) == INVALID, kw
    for kw in (dict(gu=1, N=192), dict(block=48)):
        assert pack(lib, **kw) == UNSUPPORTED, kw
    assert pack(lib, N=0, w=None) == OK
    assert moe.moe_pack_fp4_scales_size(3, 200, 288, 16) == 3 * 2 * 2 * 2048
    assert moe.moe_pack_fp4_scales_size(3, 200, 288, 32) == 3 * 2 * 2 * 1024
    assert lib.moe_pack_fp4_scales_size(3, 200, 288, 16, None) == INVALID


def matmul(lib, x=fake, xs=fake, w=fake, ws=fake, a=None, off=fake, M=4, E=2, N=64, K=64, block=16,
           y=other, wk=fake, n=1 << 30):
    return lib.moe_grouped_matmul_fp4(x, xs, w, ws, a, off, M, E, N, K, block, y, wk, n, None)


def swiglu(lib, x=fake, xs=fake, w=fake, ws=fake, d=fake, ds=fake, a=None, ad=None, hs=None, off=fake,
           M=4, E=2, N=64, K=64, block=16, y=other, wk=fake, n=1 << 30):
    return lib.moe_grouped_swiglu_fp4(x, xs, w, ws, d, ds, a, ad, hs, off, M, E, K, N, block, y, wk, n,
                                      None)


@pytest.mark.parametrize("call", [matmul, swiglu])
def test_products_refuse(lib, call):
    for kw in (dict(M=-1), dict(E=0), dict(N=0), dict(K=0), dict(x=None), dict(xs=None), dict(w=None),
               dict(ws=None), dict(off=None), dict(y=None), dict(x=P(0x1008)), dict(w=P(0x1008)),
               dict(ws=P(0x1008)), dict(y=P(0x1008)), dict(a=P(0x1002)), dict(off=P(0x1002))):
        assert call(lib, **kw) == INVALID, kw
    for kw in (dict(E=1025), dict(K=48), dict(N=12), dict(block=64), dict(M=1 << 31), dict(K=1 << 24),
               dict(E=1024, N=1 << 22)):
        assert call(lib, **kw) == UNSUPPORTED, kw
    assert call(lib, wk=None) == WORKSPACE and call(lib, wk=P(0x1080)) == WORKSPACE
    assert call(lib, n=255) == WORKSPACE


def test_swiglu_refuses(lib):
    for kw in (dict(d=None), dict(ds=None), dict(d=P(0x1008)), dict(ds=P(0x1008)), dict(ad=P(0x1002)),
               dict(hs=P(0x1002)), dict(block=32, hs=fake)):
        assert swiglu(lib, **kw) == INVALID, kw
    assert swiglu(lib, K=96) == UNSUPPORTED and swiglu(lib, N=96) == UNSUPPORTED
    n = moe.moe_grouped_swiglu_fp4_workspace_size(100, 2, 64, 64, 16)
    assert n % 256 == 0 and n >= 256 + 100 * 32 + 100 * 16
    assert swiglu(lib, M=100, n=n - 1) == WORKSPACE
    assert moe.moe_grouped_swiglu_fp4_workspace_size(0, 2, 64, 64, 16) == 256


def test_binding_refuses_host_tensors():
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    for call in (lambda: moe.moe_quantize_fp4(x), lambda: moe.moe_pack_fp4(x[None]),
                 lambda: moe.moe_dequantize_fp4(x, x)):
        with pytest.raises(ValueError):
            call()


def test_worked_values():
    """One block by hand: largest 7.5, g = 1: 7.5 / 6 = 1.25, which e4m3 has."""
    x = torch.zeros(16)
    x[:9] = torch.tensor([7.5, -7.5, 0.3125, 0.31, -1.5625, 2.1875, 3.125, 4.375, 6.25])
    codes, byte, step = f4.quantize(x, 16)
    assert byte.item() == 0x3A and step.item() == 1.25          # 1.25 = 2^0 * (1 + 2/8)
    # quotients 6, -6, 0.25 (tie), 0.248, -1.25 (tie), 1.75 (tie), 2.5 (tie), 3.5 (tie), 5 (tie)
    assert codes[:9].tolist() == [7, 15, 0, 0, 8 + 2, 4, 4, 6, 6]
    codes, byte, step = f4.quantize(torch.cat([x, x]), 32)
    assert byte.item() == 127 and step.item() == 1.0            # floor(log2 7.5) - 2 = 0
    assert codes[:9].tolist() == [7, 15, 1, 1, 8 + 3, 4, 5, 6, 7]
    assert f4.pairs(torch.tensor([1, 2, 3, 4], dtype=torch.uint8)).tolist() == [0x21, 0x43]
    at = f4.packed_at(300, 512, 16)
    assert sorted(at.view(-1).tolist()) == sorted(set(at.view(-1).tolist()))
    assert at[0, :5].tolist() == [0, 1, 2, 3, 512] and at[33, 0] == 20 and at[128, 0] == 4096
    assert f4.in_turn(128)[[0, 63, 64, 128]].tolist() == [0, 63, 128, 64]


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("E,H,I", [(1, 4096, 4096), (8, 512, 1408), (64, 7168, 2048), (256, 7168, 2048),
                                   (300, 2048, 1024)])
def test_workspace_sizes_do_not_fall(E, H, I, block):
    """One workspace, of the largest call, serves every call of fewer rows."""
    step = lambda f: [f(M) for M in [*range(0, 1300), *range(1300, 20000, 97), 65536, 1 << 20]]
    for sizes in (step(lambda M: moe.moe_grouped_matmul_fp4_workspace_size(M, E, I, H, block)),
                  step(lambda M: moe.moe_grouped_swiglu_fp4_workspace_size(M, E, H, I, block))):
        assert all(a <= b for a, b in zip(sizes, sizes[1:]))
