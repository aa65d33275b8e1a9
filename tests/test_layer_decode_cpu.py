"""Host-side validation of moe_layer_decode*: refused before anything is launched."""
import ctypes

import pytest

import unpermute_combine_gb300 as moe
from unpermute_combine_gb300 import build as libbuild

P = ctypes.c_void_p
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
fake = P(0x1000)                 # never dereferenced: validation fails first
other = P(0x8000)


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return moe.load_library()


def logits(lib, x=fake, xs=None, lg=fake, T=4, E=8, k=2, H=256, I=128, up=fake, down=fake, idx=fake,
           w=fake, out=other, ws=fake, n=1 << 30):
    return lib.moe_layer_decode(x, xs, lg, T, E, k, H, I, up, down, idx, w, out, ws, n, None)


def choices(lib, x=fake, xs=None, idx=fake, w=fake, T=4, E=8, k=2, H=256, I=128, up=fake, down=fake,
            out=other, ws=fake, n=1 << 30):
    return lib.moe_layer_decode_indices(x, xs, idx, w, T, E, k, H, I, up, down, out, ws, n, None)


@pytest.mark.parametrize("call", [logits, choices])
def test_refusals(lib, call):
    for kw in (dict(T=-1), dict(E=0), dict(k=0), dict(H=0), dict(I=0), dict(x=None), dict(up=None),
               dict(down=None), dict(out=None), dict(idx=None), dict(w=None), dict(x=P(0x1008)),
               dict(up=P(0x1008)), dict(down=P(0x1004)), dict(out=P(0x1002)),
               dict(x=P(0x2000), out=P(0x2000))):
        assert call(lib, **kw) == INVALID, kw
    for kw in (dict(T=65), dict(E=1025, k=2), dict(k=9), dict(E=64, k=33), dict(H=128), dict(H=300),
               dict(I=64), dict(I=130), dict(E=1024, I=1 << 20),
               dict(E=1, k=1, H=1 << 21), dict(E=1, k=1, I=1 << 21)):
        assert call(lib, **kw) == UNSUPPORTED, kw
    n = moe.moe_layer_decode_workspace_size(4, 8, 2, 256, 128)
    assert call(lib, n=n - 1) == WORKSPACE
    assert call(lib, ws=None) == WORKSPACE and call(lib, ws=P(0x1080)) == WORKSPACE


def test_logits_and_scales(lib):
    assert logits(lib, lg=None) == INVALID
    assert logits(lib, lg=P(0x1002)) == INVALID and choices(lib, idx=P(0x1001)) == INVALID
    assert logits(lib, xs=P(0x1002)) == INVALID and choices(lib, xs=P(0x1003)) == INVALID
    assert logits(lib, w=P(0x1002)) == INVALID and choices(lib, w=P(0x1002)) == INVALID


def test_workspace_size(lib):
    sz = ctypes.c_size_t()
    assert lib.moe_layer_decode_workspace_size(4, 8, 2, 256, 128, None) == INVALID
    assert lib.moe_layer_decode_workspace_size(65, 8, 2, 256, 128, ctypes.byref(sz)) == UNSUPPORTED
    small = moe.moe_layer_decode_workspace_size(1, 8, 2, 256, 128)
    assert small % 256 == 0 and moe.moe_layer_decode_workspace_size(0, 8, 2, 256, 128) >= 256
    assert moe.moe_layer_decode_workspace_size(64, 8, 2, 256, 128) > small
    assert moe.MOE_LAYER_DECODE_MAX_TOKENS == 64
