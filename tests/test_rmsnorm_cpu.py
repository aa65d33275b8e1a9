"""Host-side validation of the norm calls: refused before anything is launched."""
import ctypes

import pytest

import unpermute_combine_gb300 as moe
from unpermute_combine_gb300 import build as libbuild

P = ctypes.c_void_p
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
fake = P(0x1000)                 # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return moe.load_library()


def norm(lib, x=fake, res=None, dt=1, w=fake, wdt=1, T=4, H=64, eps=1e-6, ho=None, out=fake):
    return lib.moe_rmsnorm(x, res, dt, w, wdt, T, H, eps, ho, out, None)


def quant(lib, x=fake, res=None, dt=1, w=fake, wdt=1, T=4, H=64, eps=1e-6, block=32, ho=None,
          q=fake, sc=fake):
    return lib.moe_rmsnorm_quantize_fp8(x, res, dt, w, wdt, T, H, eps, block, ho, q, sc, None)


def back(lib, g=fake, gh=None, h=fake, dt=1, w=fake, wdt=1, T=4, H=64, eps=1e-6, gx=fake, gw=fake,
         ws=fake, n=1 << 30):
    return lib.moe_rmsnorm_backward(g, gh, h, dt, w, wdt, T, H, eps, gx, gw, ws, n, None)


@pytest.mark.parametrize("call", [norm, quant, back])
def test_shared_refusals(lib, call):
    assert call(lib, dt=2) == INVALID and call(lib, wdt=2) == INVALID
    assert call(lib, T=-1) == INVALID and call(lib, H=-64) == INVALID
    assert call(lib, eps=-1e-6) == INVALID and call(lib, eps=float("nan")) == INVALID
    assert call(lib, T=1 << 31) == UNSUPPORTED and call(lib, H=1 << 31) == UNSUPPORTED
    assert call(lib, w=None) == INVALID


def test_norm(lib):
    assert norm(lib, x=None) == INVALID and norm(lib, out=None) == INVALID
    assert norm(lib, res=fake) == INVALID                      # nowhere to store the sum
    assert norm(lib, res=fake, ho=fake, out=fake) == INVALID   # two outputs in one place
    assert norm(lib, x=None, w=None, out=None, T=0) == OK
    assert norm(lib, x=None, w=None, out=None, H=0) == OK


def test_elements_off_their_boundaries(lib):
    odd, half = P(0x1001), P(0x1002)
    for kw in (dict(x=odd), dict(w=odd), dict(out=odd), dict(res=odd, ho=fake), dict(res=half, ho=odd),
               dict(x=half, dt=0), dict(out=half, dt=0), dict(w=half, wdt=0)):
        assert norm(lib, **{**dict(out=P(0x8000)), **kw}) == INVALID, kw
    for kw in (dict(g=odd), dict(h=odd), dict(gx=odd), dict(gh=odd), dict(w=odd), dict(gw=half),
               dict(g=half, dt=0), dict(w=half, wdt=0)):
        assert back(lib, **kw) == INVALID, kw


def test_quantize(lib):
    assert quant(lib, q=None) == INVALID and quant(lib, sc=None) == INVALID
    assert quant(lib, res=fake) == INVALID
    assert quant(lib, block=16) == UNSUPPORTED and quant(lib, block=0) == UNSUPPORTED
    assert quant(lib, block=128) == INVALID                    # H = 64
    assert quant(lib, H=65536, block=128) == UNSUPPORTED
    for bad in (dict(x=P(0x1008)), dict(w=P(0x1004)), dict(q=P(0x1004)), dict(sc=P(0x1002)),
                dict(res=P(0x1008), ho=fake), dict(res=fake, ho=P(0x1008))):
        assert quant(lib, **bad) == INVALID
    assert quant(lib, x=None, w=None, q=None, sc=None, T=0) == OK


def test_backward(lib):
    n = moe.moe_rmsnorm_backward_workspace_size(4, 64)
    assert n % 256 == 0 and n >= 4 * 64 * 4
    assert moe.moe_rmsnorm_backward_workspace_size(0, 0) >= 0
    for name in ("g", "h", "gx", "gw"):
        assert back(lib, **{name: None}) == INVALID
    assert back(lib, ws=None) == WORKSPACE and back(lib, ws=P(0x1010)) == WORKSPACE
    assert back(lib, n=n - 1) == WORKSPACE
    assert back(lib, g=None, h=None, w=None, gx=None, gw=None, ws=None, H=0) == OK
    assert lib.moe_rmsnorm_backward_workspace_size(4, 64, None) == INVALID
