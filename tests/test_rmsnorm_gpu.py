"""moe_rmsnorm, moe_rmsnorm_quantize_fp8 and moe_rmsnorm_backward against a plain
implementation in float64 (written here from the formulas, on the host).

Tolerances, u = 2^-24 (half a float32 step), b = half a step of the output type:
  r = 1/sqrt(mean h^2 + eps): the sum of H squares has at most D additions on
  the way of one term (D <= 64 + H / 256 in the longest thread loop here), so
  mean is off by (D + 3) u, its root by half of that, rsqrt by 2 more ulp (4 u).
  y: two products more.  rel(y) <= (D / 2 + 8) u + b."""
import ctypes

import numpy as np
import pytest

import workloads as wl
from moe_testutil import to_dev, to_host

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import unpermute_combine_gb300 as moe  # noqa: E402

U = 2.0 ** -24
HALF = {"f32": U, "bf16": 2.0 ** -8}
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from unpermute_combine_gb300 import build
    build.build()
    moe.load_library()


def _f64(a):
    return wl.activation_to_f64(a)


def _act(rng, shape, dtype, std=1.0):
    return wl.as_activation((rng.standard_normal(shape) * std).astype(np.float32), dtype)


def _sum(x, res):
    """x + residual rounded to the activation type."""
    if res is None:
        return x
    if x.dtype == np.uint16:
        s = wl.bf16_bits_to_f32(x) + wl.bf16_bits_to_f32(res)     # round to float first:
        return wl.f32_to_bf16_bits(s)                             # the kernel's own rounding
    return x + res


def _norm64(h, w, eps):
    h = _f64(h)
    r = 1.0 / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps)
    return h * r * _f64(w)[None, :], r


def _depth(H):
    return 64 + H / 256


def _val(t):
    a = to_host(t)
    return wl.bf16_bits_to_f32(a).astype(np.float64) if a.dtype == np.uint16 else a.astype(np.float64)


def _inputs(T, H, dtype, wdtype, residual, seed):
    rng = np.random.default_rng(seed)
    x = _act(rng, (T, H), dtype)
    res = _act(rng, (T, H), dtype, 3.0) if residual else None
    w = wl.as_activation((1.0 + 0.1 * rng.standard_normal(H)).astype(np.float32), wdtype)
    return x, res, w


SHAPES = [(1, 8), (3, 1), (1, 2048), (5, 7), (33, 136), (2, 1001), (700, 256), (17, 4096),
          (3, 7168), (2, 8200), (2, 20000), (1, 32768), (1, 40000), (1, 33001), (400, 2048),
          (311, 4104), (320, 520), (500, 88), (400, 8184), (330, 130), (3, 8191), (2, 8193)]


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("dtype,wdtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"),
                                          ("f32", "bf16")])
@pytest.mark.parametrize("residual", [False, True])
def test_norm(T, H, dtype, wdtype, residual):
    x, res, w = _inputs(T, H, dtype, wdtype, residual, T * 100003 + H)
    xd, rd, wd = to_dev(x), None if res is None else to_dev(res), to_dev(w)
    y, h = moe.moe_rmsnorm(xd, wd, residual=rd, eps=EPS)
    torch.cuda.synchronize()
    h_o = _sum(x, res)
    assert (to_host(h) == h_o).all()
    y64, _ = _norm64(h_o, w, EPS)
    tol = (_depth(H) / 2 + 8) * U + HALF[dtype]
    assert (np.abs(_val(y) - y64) <= tol * np.abs(y64)).all()
    if residual:
        assert (to_host(xd) == x).all() and (to_host(rd) == res).all()
    else:
        assert h is xd


@pytest.mark.parametrize("T,H", [(4, 64), (9, 77), (3, 7168)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_in_place(T, H, dtype):
    x, res, w = _inputs(T, H, dtype, dtype, True, T + H)
    y0, h0 = moe.moe_rmsnorm(to_dev(x), to_dev(w), residual=to_dev(res))
    for swap in (False, True):
        xd, rd = to_dev(x), to_dev(res)
        out, stream_ = (rd, xd) if swap else (xd, rd)
        y, h = moe.moe_rmsnorm(xd, to_dev(w), residual=rd, out=out, residual_out=stream_)
        assert torch.equal(y, y0) and torch.equal(h, h0)
    xd = to_dev(x)
    y1, _ = moe.moe_rmsnorm(to_dev(x), to_dev(w))
    y, _ = moe.moe_rmsnorm(xd, to_dev(w), out=xd)
    assert torch.equal(y, y1)


@pytest.mark.parametrize("off", [1, 2, 4])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_of_unaligned_rows(off, dtype):
    """Rows that start off a 16-byte boundary give what aligned ones give."""
    T, H = 6, 520
    x, res, w = _inputs(T, H, dtype, dtype, True, off)
    flat = torch.zeros(T * H + off, dtype=to_dev(x).dtype, device="cuda")
    flat[off:] = to_dev(x).view(-1)
    xu = flat[off:].view(T, H)
    y, h = moe.moe_rmsnorm(xu, to_dev(w), residual=to_dev(res))
    h_o = _sum(x, res)
    assert (to_host(h) == h_o).all()
    y64, _ = _norm64(h_o, w, 1e-6)
    assert (np.abs(_val(y) - y64) <= ((_depth(H) / 2 + 8) * U + HALF[dtype]) * np.abs(y64)).all()


@pytest.mark.parametrize("T,H", [(1, 1), (3, 1), (9, 3), (5, 7), (20, 5), (6, 13), (2, 1001), (40, 33)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_between_others(T, H, dtype):
    """What lies before and behind the tensors, NaN here, is neither used nor
    changed, forward and backward; rows shorter than a chunk among them."""
    x, res, w = _inputs(T, H, dtype, dtype, True, T * 5 + H)

    def between(a):
        t = to_dev(a) if a is not None else torch.zeros((T, H), dtype=to_dev(x).dtype, device="cuda")
        big = torch.full((64 + t.numel() + 64,), float("nan"), dtype=t.dtype, device="cuda")
        big[64:64 + t.numel()] = t.view(-1)
        return big, big[64:64 + t.numel()].view(t.shape)
    bufs = [between(a) for a in (x, res, None, None, None)]
    (_, xd), (_, rd), (_, ho), (_, out), (_, gx) = bufs
    wd = to_dev(w)
    y, h = moe.moe_rmsnorm(xd, wd, residual=rd, out=out, residual_out=ho)
    h_o = _sum(x, res)
    assert (to_host(h) == h_o).all()
    y64, _ = _norm64(h_o, w, 1e-6)
    assert (np.abs(_val(y) - y64) <= ((_depth(H) / 2 + 8) * U + HALF[dtype]) * np.abs(y64)).all()
    g, gw = moe.moe_rmsnorm_backward(xd, h, wd, grad_h=rd, grad_x=gx)
    gx64, size, gw64, gw_size = _backward64(x, h_o, w, res, 1e-6)
    D = _depth(H)
    assert (np.abs(_val(g) - gx64) <= (2.5 * D + 24) * U * size + HALF[dtype] * np.abs(gx64)).all()
    assert (np.abs(_val(gw) - gw64) <= (D / 2 + 10 + T) * U * gw_size).all()
    for big, t in bufs:
        assert torch.isnan(big[:64]).all() and torch.isnan(big[64 + t.numel():]).all()


def test_norm_leaves_what_lies_behind():
    T, H = 5, 333
    x, res, w = _inputs(T, H, "bf16", "f32", True, 3)
    out = torch.full((T + 2, H), 7.0, dtype=torch.bfloat16, device="cuda")
    ho = torch.full((T + 2, H), 7.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_rmsnorm(to_dev(x), to_dev(w), residual=to_dev(res), out=out[:T], residual_out=ho[:T])
    assert (out[T:] == 7).all() and (ho[T:] == 7).all()


def test_more_rows_than_blocks():
    """Over a million rows: the blocks go round.  Rows are computed alike wherever
    they are, so parts of the tensor by themselves give the same bits."""
    T, H = (1 << 20) + 7, 1048
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((T, H), generator=g, device="cuda", dtype=torch.bfloat16)
    w = torch.rand((H,), generator=g, device="cuda").bfloat16()
    y, _ = moe.moe_rmsnorm(x, w)
    for a in (0, (1 << 20) - 500, T - 400):
        assert torch.equal(y[a:a + 400], moe.moe_rmsnorm(x[a:a + 400], w)[0])
    h64 = x[-3:].double()
    ref = h64 / ((h64 * h64).mean(1, keepdim=True) + 1e-6).sqrt() * w.double()
    assert ((y[-3:].double() - ref).abs() <= ((_depth(H) / 2 + 8) * U + HALF["bf16"]) * ref.abs()).all()


def test_special_rows():
    """A zero row gives zeros; a NaN makes its own row NaN and no other; eps = 0."""
    T, H = 4, 512
    x, _, w = _inputs(T, H, "bf16", "bf16", False, 9)
    x[1] = 0
    x[2, 100] = 0x7FC0
    y, _ = moe.moe_rmsnorm(to_dev(x), to_dev(w))
    v = _val(y)
    assert (v[1] == 0).all() and np.isnan(v[2]).all() and np.isfinite(v[[0, 3]]).all()
    y, _ = moe.moe_rmsnorm(to_dev(x[:1].copy()), to_dev(w), eps=0.0)
    y64, _ = _norm64(x[:1], w, 0.0)
    assert (np.abs(_val(y) - y64) <= ((_depth(H) / 2 + 8) * U + HALF["bf16"]) * np.abs(y64)).all()


def test_empty():
    w = torch.ones(16, device="cuda")
    y, h = moe.moe_rmsnorm(torch.empty((0, 16), device="cuda"), w)
    assert y.shape == (0, 16) and h.shape == (0, 16)
    y, _ = moe.moe_rmsnorm(torch.empty((3, 0), device="cuda"), torch.ones(0, device="cuda"))
    assert y.shape == (3, 0)
    q, sc, _ = moe.moe_rmsnorm_quantize_fp8(torch.empty((0, 64), device="cuda"),
                                            torch.ones(64, device="cuda"), block=32)
    assert q.shape == (0, 64) and sc.shape == (0, 2)
    gx, gw = moe.moe_rmsnorm_backward(torch.empty((0, 16), device="cuda"),
                                      torch.empty((0, 16), device="cuda"), w)
    assert gx.shape == (0, 16) and (gw == 0).all()


# ------------------------------------------------------------------- e4m3

def _e4m3_values(q):
    return q.view(torch.uint8).view(torch.float8_e4m3fn).float().cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("T,H,block", [(1, 32, 32), (5, 64, 32), (3, 192, 64), (700, 256, 128),
                                       (2, 256, 256), (33, 1280, 256), (4, 7168, 128),
                                       (2, 8192, 256), (2, 16384, 128), (1, 32768, 64),
                                       (400, 2048, 128), (333, 96, 32), (310, 8448, 256)])
@pytest.mark.parametrize("dtype,wdtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"),
                                          ("f32", "bf16")])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_quantize(T, H, block, dtype, wdtype, residual):
    x, res, w = _inputs(T, H, dtype, wdtype, residual, T * 7 + H + block)
    q, sc, h = moe.moe_rmsnorm_quantize_fp8(to_dev(x), to_dev(w), eps=EPS, block=block,
                                            residual=None if res is None else to_dev(res))
    torch.cuda.synchronize()
    h_o = _sum(x, res)
    assert (to_host(h) == h_o).all()
    y64, _ = _norm64(h_o, w, EPS)
    b64 = y64.reshape(T, H // block, block)
    s64 = np.abs(b64).max(2) / 448.0
    rel = (_depth(H) / 2 + 8) * U
    s = to_host(sc).astype(np.float64)
    assert (np.abs(s - s64) <= (rel + 2 * U) * s64).all()
    # half an e4m3 step of the quotient: 2^-4 of a normal value, 2^-10 below 2^-6;
    # the quotient itself is off by rel of y, and rounded once or twice more
    got = _e4m3_values(q).reshape(b64.shape)
    quot = b64 / s[:, :, None]
    step = np.maximum(np.abs(quot) * 2.0 ** -4, 2.0 ** -10)
    assert (np.abs(got - quot) <= step + 4 * rel * np.abs(quot)).all()
    assert (np.abs(got).max(2) == 448).all()


@pytest.mark.parametrize("block", [32, 128])
def test_norm_quantize_zero_and_tiny_blocks(block):
    """A block of zeros has scale 1; a block whose scale is a subnormal float
    keeps its values; neither touches its neighbours."""
    T, H = 3, 512
    rng = np.random.default_rng(block)
    x = rng.standard_normal((T, H)).astype(np.float32)
    w = np.ones(H, np.float32)
    w[:block] = 0.0
    w[block:2 * block] = 1e-38                    # amax / 448 < 2^-126
    q, sc, _ = moe.moe_rmsnorm_quantize_fp8(to_dev(x), to_dev(w), block=block)
    s, got = to_host(sc).astype(np.float64), _e4m3_values(q)
    assert (s[:, 0] == 1).all() and (got[:, :block] == 0).all()
    y64, _ = _norm64(x, w, 1e-6)
    assert np.isfinite(got).all()
    # a subnormal scale has a whole step of 2^-149; both it and y are rounded to that grid
    tiny = got[:, block:2 * block] * s[:, 1:2]
    err = np.abs(tiny - y64[:, block:2 * block])
    amax = np.abs(y64[:, block:2 * block]).max(1, keepdims=True)
    rel_scale = 2.0 ** -150 / s[:, 1:2]
    assert (err <= (2.0 ** -4 + 2 * rel_scale) * np.abs(y64[:, block:2 * block])
            + amax * 2.0 ** -10 / 448 + amax * rel_scale).all()
    rest = got[:, 2 * block:].reshape(T, -1, block) * s[:, 2:, None]
    r64 = y64[:, 2 * block:].reshape(T, -1, block)
    assert (np.abs(rest - r64) <= 2.0 ** -4 * np.abs(r64) * 1.001 + 2.0 ** -10 * s[:, 2:, None]).all()


# --------------------------------------------------------------- backward

def _backward64(g, h, w, gh, eps):
    g, h, w = _f64(g), _f64(h), _f64(w)
    H = h.shape[1]
    r = 1.0 / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps)
    gw = g * w[None]
    gx = r * gw - h * r ** 3 * np.sum(gw * h, axis=1, keepdims=True) / H
    # sizes of the terms: what a rounding on the way is relative to
    size = np.abs(r * gw) + np.abs(h) * r ** 3 * np.sum(np.abs(gw * h), axis=1, keepdims=True) / H
    if gh is not None:
        gx = gx + _f64(gh)
        size = size + np.abs(_f64(gh))
    return gx, size, np.sum(g * h * r, axis=0), np.sum(np.abs(g * h * r), axis=0)


BWD = [(1, 8), (3, 1), (5, 7), (33, 136), (700, 256), (17, 4096), (2, 1001), (3, 7168), (2, 20000),
       (1, 33001), (1300, 72), (615, 31), (5, 12000), (900, 512), (3, 8191), (2, 8193), (2500, 24),
       (400, 2048), (700, 1001)]


@pytest.mark.parametrize("T,H", BWD)
@pytest.mark.parametrize("dtype,wdtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"),
                                          ("f32", "bf16")])
@pytest.mark.parametrize("residual", [False, True])
def test_backward(T, H, dtype, wdtype, residual):
    h, _, w = _inputs(T, H, dtype, wdtype, False, T * 31 + H)
    rng = np.random.default_rng(T + H)
    g = _act(rng, (T, H), dtype)
    gh = _act(rng, (T, H), dtype) if residual else None
    gx, gw = moe.moe_rmsnorm_backward(to_dev(g), to_dev(h), to_dev(w), eps=EPS,
                                      grad_h=None if gh is None else to_dev(gh))
    torch.cuda.synchronize()
    gx64, size, gw64, gw_size = _backward64(g, h, w, gh, EPS)
    D = _depth(H)
    # r^3: three times r's error; the dot product's D additions; six products
    assert (np.abs(_val(gx) - gx64) <= (2.5 * D + 24) * U * size + HALF[dtype] * np.abs(gx64)).all()
    # rows of one block one after the other, then the blocks: at most T additions
    assert (np.abs(_val(gw) - gw64) <= (D / 2 + 10 + T) * U * gw_size).all()


def test_backward_in_place_and_the_same_twice():
    T, H = 40, 264
    h, _, w = _inputs(T, H, "bf16", "bf16", False, 5)
    rng = np.random.default_rng(6)
    g, gh = _act(rng, (T, H), "bf16"), _act(rng, (T, H), "bf16")
    ref = moe.moe_rmsnorm_backward(to_dev(g), to_dev(h), to_dev(w), grad_h=to_dev(gh))
    ws = torch.randint(0, 255, (moe.moe_rmsnorm_backward_workspace_size(T, H),),
                       dtype=torch.uint8, device="cuda")
    for k in range(3):
        gd, hd, ghd = to_dev(g), to_dev(h), to_dev(gh)
        gx, gw = moe.moe_rmsnorm_backward(gd, hd, to_dev(w), grad_h=ghd, grad_x=(gd, hd, ghd)[k],
                                          workspace=ws)
        assert torch.equal(gx, ref[0]) and torch.equal(gw, ref[1])


def test_backward_is_the_difference_quotient():
    """Along random directions, of the function that moe_rmsnorm computes in
    float32.  Central difference, step d: truncation d^2/6 f''' with f''' of
    order one here, and 2 * 2e-7 * |f| / (2 d) from the rounding of f; at d = 1e-2
    both stay below 1e-3 of |f'|."""
    T, H = 8, 96
    rng = np.random.default_rng(11)
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).cuda()
    w = torch.from_numpy((1 + 0.1 * rng.standard_normal(H)).astype(np.float32)).cuda()
    c = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).cuda()
    gx, gw = moe.moe_rmsnorm_backward(c, x, w)

    def f(xv, wv):
        return (moe.moe_rmsnorm(xv, wv)[0].double() * c.double()).sum().item()
    d = 1e-2
    for k in range(4):
        dx = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).cuda()
        dw = torch.from_numpy(rng.standard_normal(H).astype(np.float32)).cuda()
        scale = c.norm().item()
        got = (gx * dx).sum().item()
        assert abs((f(x + d * dx, w) - f(x - d * dx, w)) / (2 * d) - got) <= 1e-2 * scale
        got = (gw * dw).sum().item()
        assert abs((f(x, w + d * dw) - f(x, w - d * dw)) / (2 * d) - got) <= 1e-2 * scale


# ------------------------------------------------- streams, graphs, together

def test_on_another_stream_and_captured():
    T, H = 64, 2048
    x, res, w = _inputs(T, H, "bf16", "bf16", True, 21)
    xd, rd, wd = to_dev(x), to_dev(res), to_dev(w)
    y0, h0 = moe.moe_rmsnorm(xd, wd, residual=rd)
    g0 = moe.moe_rmsnorm_backward(y0, h0, wd, grad_h=xd)
    q0 = moe.moe_rmsnorm_quantize_fp8(xd, wd, residual=rd)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y, h = moe.moe_rmsnorm(xd, wd, residual=rd, stream=s)
    g = moe.moe_rmsnorm_backward(y, h, wd, grad_h=xd, stream=s)
    q = moe.moe_rmsnorm_quantize_fp8(xd, wd, residual=rd, stream=s)
    s.synchronize()
    for a, b in ((y, y0), (h, h0), (g[0], g0[0]), (g[1], g0[1]), (q[1], q0[1])):
        assert torch.equal(a, b)
    assert torch.equal(q[0].view(torch.uint8), q0[0].view(torch.uint8))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, h = moe.moe_rmsnorm(xd, wd, residual=rd)
        g = moe.moe_rmsnorm_backward(y, h, wd, grad_h=xd)
    for _ in range(2):
        y.zero_(), g[0].zero_(), g[1].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, y0) and torch.equal(g[0], g0[0]) and torch.equal(g[1], g0[1])


def test_norm_into_the_fp8_dispatch():
    """norm + quantize, then moe_permute_fp8 of its rows: the same bytes as
    quantizing a float32 norm's rows at each slot."""
    T, H, E, k = 50, 512, 8, 2
    x, res, w = _inputs(T, H, "bf16", "f32", True, 33)
    logits = torch.from_numpy(np.random.default_rng(1).standard_normal((T, E)).astype(np.float32)).cuda()
    r = moe.moe_route(logits, k)
    q, sc, _ = moe.moe_rmsnorm_quantize_fp8(to_dev(x), to_dev(w), residual=to_dev(res))
    oq, osc = moe.moe_permute_fp8(q, sc, r.slot_pos)
    src = r.sorted_indices.long()
    assert torch.equal(oq.view(torch.uint8), q.view(torch.uint8)[src])
    assert torch.equal(osc, sc[src])


# ----------------------------------------------------------------- refusals

def test_refusals():
    x = torch.zeros((4, 64), device="cuda")
    w = torch.ones(64, device="cuda")
    bad = [dict(x=x.t()[:64], weight=w), dict(x=x.half(), weight=w), dict(x=x, weight=w[:32]),
           dict(x=x, weight=w.half()), dict(x=x.cpu(), weight=w), dict(x=x, weight=w.cpu()),
           dict(x=x, weight=w, residual=x[:2]), dict(x=x, weight=w, residual=x.bfloat16()),
           dict(x=x, weight=w, residual_out=x), dict(x=x[:, :32], weight=w[:32]),
           dict(x=x, weight=w, out=x[:2])]
    for kw in bad:
        with pytest.raises(ValueError):
            moe.moe_rmsnorm(**kw)
    with pytest.raises(moe.MoeError):
        moe.moe_rmsnorm(x, w, eps=-1.0)
    with pytest.raises(moe.MoeError):
        moe.moe_rmsnorm(x, w, eps=float("nan"))
    with pytest.raises(ValueError):
        moe.moe_rmsnorm_quantize_fp8(x, w, block=128)
    with pytest.raises(moe.MoeError):
        moe.moe_rmsnorm_quantize_fp8(x, w, block=16)
    with pytest.raises(moe.MoeError):
        moe.moe_rmsnorm_quantize_fp8(torch.zeros((1, 65536), device="cuda"),
                                     torch.ones(65536, device="cuda"))
    flat = torch.zeros(4 * 64 + 1, device="cuda")
    with pytest.raises(moe.MoeError):
        moe.moe_rmsnorm_quantize_fp8(flat[1:].view(4, 64), w, block=64)
    with pytest.raises(ValueError):
        moe.moe_rmsnorm_backward(x, x[:2], w)
    with pytest.raises(ValueError):
        moe.moe_rmsnorm_backward(x, x, w, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


# ------------------------------------------------ rows far from one in size

@pytest.mark.parametrize("T,H,off", [(6, 256, 0), (400, 2048, 0), (5, 77, 0), (3, 1001, 0), (4, 520, 1),
                                     (2, 20000, 0), (2, 33001, 0)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rms,eps", [(1e15, EPS), (1e-14, 0.0)])
@pytest.mark.parametrize("residual", [False, True])
def test_backward_of_large_and_small_rows(T, H, off, dtype, rms, eps, residual):
    """Rows of 1e15 and 1e-14: their norm and its gradient are ordinary numbers, though
    r^3 is none in float32.  grad_y leans on h, so that the term of the mean counts.  off:
    rows that start so many elements off a 16-byte boundary.  The error is that of the
    backward's other tests: r three times, the mean's D additions, and products."""
    rng = np.random.default_rng(T + H)
    unit = rng.standard_normal((T, H)).astype(np.float32)
    h = wl.as_activation((unit * rms).astype(np.float32), dtype)
    g = wl.as_activation((unit + 0.3 * rng.standard_normal((T, H))).astype(np.float32), dtype)
    gh = wl.as_activation((rng.standard_normal((T, H)) / rms).astype(np.float32), dtype) if residual else None
    w = wl.as_activation((1.0 + 0.1 * rng.standard_normal(H)).astype(np.float32), dtype)

    def put(a):
        t = to_dev(a)
        flat = torch.zeros(t.numel() + off, dtype=t.dtype, device="cuda")
        flat[off:] = t.view(-1)
        return flat[off:].view(t.shape)
    gx, gw = moe.moe_rmsnorm_backward(put(g), put(h), to_dev(w), eps=eps,
                                      grad_h=None if gh is None else put(gh))
    gx64, size, gw64, gw_size = _backward64(g, h, w, gh, eps)
    D = _depth(H)
    assert (np.abs(_val(gx) - gx64) <= (2.5 * D + 24) * U * size + HALF[dtype] * np.abs(gx64)).all()
    assert (np.abs(_val(gw) - gw64) <= (D / 2 + 10 + T) * U * gw_size).all()
    y, _ = moe.moe_rmsnorm(put(h), to_dev(w), eps=eps)
    y64, _ = _norm64(h, w, eps)
    assert (np.abs(_val(y) - y64) <= ((D / 2 + 8) * U + HALF[dtype]) * np.abs(y64)).all()


@pytest.mark.parametrize("T,H,block", [(2048, 4096, 128), (3, 512, 32), (40, 8192, 256), (700, 1024, 64)])
@pytest.mark.parametrize("residual", [False, True])
def test_codes_are_those_of_the_quotient(T, H, block, residual):
    """scale = amax / 448 and code = e4m3(y / scale), each quotient rounded as float32's
    division rounds it, bit for bit, from the float32 y that moe_rmsnorm gives (a row's
    sum has the same order in both).  Blocks of scales below 2^-90 and above 2^60, of
    zeros of both signs and of an infinite y among them."""
    rng = np.random.default_rng(T + H)
    x = rng.standard_normal((T, H)).astype(np.float32)
    res = rng.standard_normal((T, H)).astype(np.float32) if residual else None
    w = (1.0 + 0.1 * rng.standard_normal(H)).astype(np.float32)
    w[:block] *= np.float32(2.0 ** -87)
    w[block:2 * block] *= np.float32(2.0 ** -100)
    w[2 * block:3 * block] *= np.float32(2.0 ** 70)
    w[3 * block:4 * block:2] = 0.0                       # y = 0 or -0 beside others
    w[4 * block:5 * block] = 0.0
    if H // block > 6:
        w[5 * block + 3] = np.inf
    xd, rd, wd = to_dev(x), None if res is None else to_dev(res), to_dev(w)
    y, _ = moe.moe_rmsnorm(xd, wd, residual=rd)
    q, sc, _ = moe.moe_rmsnorm_quantize_fp8(xd, wd, residual=rd, block=block)
    y = y.cpu().view(T, H // block, block)
    amax = y.abs().amax(2)
    s = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
    assert torch.equal(sc.cpu(), s)
    quot = y / s[:, :, None]
    want = quot.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(T, H)
    got, want = q.cpu().view(torch.uint8), want.view(torch.uint8)
    nan = torch.isnan(quot).view(T, H)
    assert ((got & 0x7F) == 0x7F)[nan].all()
    assert torch.equal(got[~nan], want[~nan])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("block", [32, 256])
def test_codes_next_to_a_boundary(dtype, block):
    """Rows of ones with eps = 0 have y = weight, so that a block's scale and quotients can
    be chosen: every scale has values one or two float steps around midpoints of
    neighbouring e4m3 values, where the last bit of the quotient decides."""
    T, H = 2, 32768
    rng = np.random.default_rng(block)
    mids = np.concatenate([(1 + (2 * np.arange(8) + 1) / 16)[None, :] * 2.0 ** np.arange(-6, 9)[:, None],
                           ((np.arange(8) + 0.5) * 2.0 ** -9)[None, :]]).ravel()
    mids = mids[mids < 448]
    for turn in range(8):
        n = H // block
        s = (1.0 + rng.integers(0, 1 << 23, n) * 2.0 ** -23).astype(np.float32)
        s[:4] = np.float32(2.0) - np.float32(2.0 ** -23) * np.arange(1, 5, dtype=np.float32)
        s *= (2.0 ** rng.integers(-95, 100, n)).astype(np.float32)
        amax = s * np.float32(448)
        s = amax / np.float32(448)                        # the scale that the kernel finds
        w = (rng.choice(mids, (n, block)) * s.astype(np.float64)[:, None]).astype(np.float32)
        w = (w.view(np.int32) + rng.integers(-2, 3, w.shape).astype(np.int32)).view(np.float32)
        w *= rng.choice(np.array([-1, 1], np.float32), w.shape)
        w[:, turn] = amax
        ones = to_dev(wl.as_activation(np.ones((T, H), np.float32), dtype))
        q, sc, _ = moe.moe_rmsnorm_quantize_fp8(ones, to_dev(w.ravel()), eps=0.0, block=block)
        assert (to_host(sc) == s[None, :]).all()
        want = torch.from_numpy(w / s[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        got = q.cpu().view(torch.uint8)
        assert (got == want.view(torch.uint8).view(1, H)).all()


@pytest.mark.parametrize("T,H", [(4000, 2048), (700, 1001), (900, 4096), (400, 8528), (300, 8544),
                                 (310, 9001), (200, 12792), (160, 12800), (40, 20000), (3, 8), (2500, 24)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_grad_weight_does_not_depend_on_grad_h(T, H, dtype):
    """grad_h is not in grad_weight's formula, and changes no bit of it; wide float32
    rows, of which a ring has only two tensors', among them."""
    rng = np.random.default_rng(T + H)
    g, h, gh = (_act(rng, (T, H), dtype) for _ in range(3))
    w = wl.as_activation((1.0 + 0.1 * rng.standard_normal(H)).astype(np.float32), dtype)
    gd, hd, ghd, wd = to_dev(g), to_dev(h), to_dev(gh), to_dev(w)
    gx0, gw0 = moe.moe_rmsnorm_backward(gd, hd, wd)
    gx1, gw1 = moe.moe_rmsnorm_backward(gd, hd, wd, grad_h=ghd)
    assert torch.equal(gw0, gw1)
    for k, extra in ((0, None), (1, gh)):
        gx64, size, gw64, gw_size = _backward64(g, h, w, extra, EPS)
        D = _depth(H)
        got = (gx0, gx1)[k]
        assert (np.abs(_val(got) - gx64) <= (2.5 * D + 24) * U * size + HALF[dtype] * np.abs(gx64)).all()
    assert (np.abs(_val(gw0) - gw64) <= (D / 2 + 10 + T) * U * gw_size).all()
    for k in range(3):                                     # in place
        t = [gd.clone(), hd.clone(), ghd.clone()]
        gx, gw = moe.moe_rmsnorm_backward(t[0], t[1], wd, grad_h=t[2], grad_x=t[k])
        assert torch.equal(gx, gx1) and torch.equal(gw, gw1)


@pytest.mark.parametrize("T,H", [(5, 8600), (3, 12790), (2, 12792), (1, 9001)])
def test_wide_float32_rows_between_others(T, H):
    """What lies before and behind wide rows and their grad_h, NaN here, is neither used
    nor changed."""
    rng = np.random.default_rng(H)
    a = [_act(rng, (T, H), "f32") for _ in range(3)]
    w = (1.0 + 0.1 * rng.standard_normal(H)).astype(np.float32)
    big = [torch.full((64 + T * H + 64,), float("nan"), device="cuda") for _ in range(4)]
    rows = [b[64:64 + T * H].view(T, H) for b in big]
    for r, v in zip(rows, a):
        r.copy_(to_dev(v))
    gx, gw = moe.moe_rmsnorm_backward(rows[0], rows[1], to_dev(w), grad_h=rows[2], grad_x=rows[3])
    gx64, size, gw64, gw_size = _backward64(a[0], a[1], w, a[2], EPS)
    D = _depth(H)
    assert (np.abs(_val(gx) - gx64) <= (2.5 * D + 24) * U * size + U * np.abs(gx64)).all()
    assert (np.abs(_val(gw) - gw64) <= (D / 2 + 10 + T) * U * gw_size).all()
    for b in big:
        assert torch.isnan(b[:64]).all() and torch.isnan(b[64 + T * H:]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_codes_of_the_smallest_floats(dtype):
    """Blocks whose largest value is below 448 times the smallest float: the scale is the
    smallest float, not 0, and a 0 in them stays 0."""
    H, block = 256, 32
    k = np.arange(H) % block
    w = (k * np.repeat([1, 2, 4, 7, 1, 3, 5, 7], block)).astype(np.float64)      # at most 217
    w[4 * block:5 * block] = 0.0
    w[4 * block] = 1.0
    w[1::2] *= -1
    ones = to_dev(wl.as_activation(np.ones((3, H), np.float32), dtype))
    q, sc, _ = moe.moe_rmsnorm_quantize_fp8(ones, to_dev((w * 2.0 ** -149).astype(np.float32)), eps=0.0,
                                            block=block)
    assert (to_host(sc) == np.float32(2.0 ** -149)).all()
    assert torch.equal(q.float().cpu(), torch.from_numpy(w).to(torch.float8_e4m3fn).float().expand(3, H))
