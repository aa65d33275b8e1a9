"""moe_layer_decode and moe_layer_decode_indices against a plain implementation
in float64 (written here from the formulas, on the host).

Tolerance, u = 2^-24, for sums of K terms done 16 (a tensor-core step) or 32
(a warp) at a time, each step's rounding at most 2u of the sum of magnitudes:
  |d gate| <= cH S_g with cH = 2 (H/16 + 6) u, S_g = sum |x||w|; the same for up
  |d hidden| <= 1.1 |d gate| |up| + |silu| |d up| + (2^-17 + 8u) |hidden|
     (|silu'| <= 1.1; 2^-17: the hidden rows are kept in two bf16 parts; e4m3
     rows in two parts as well: 2^-17 more in S_g and S_u)
  |d out| <= sum p (|d hidden| |wd| + cI |hidden| |wd|) + 2^-8 |out|, cI with I,
     and k + 2 more roundings of the sum over slots."""
import numpy as np
import pytest

import workloads as wl
from moe_testutil import to_dev, to_host

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import unpermute_combine_gb300 as moe  # noqa: E402

U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from unpermute_combine_gb300 import build
    build.build()
    moe.load_library()


class Layer:
    def __init__(self, E, H, I, seed):
        rng = np.random.default_rng(seed)
        self.E, self.H, self.I = E, H, I
        self.up = wl.f32_to_bf16_bits((rng.standard_normal((E, H, 2 * I)) * H ** -0.5).astype(np.float32))
        self.down = wl.f32_to_bf16_bits((rng.standard_normal((E, I, H)) * I ** -0.5).astype(np.float32))
        self.up_p, self.down_p = moe.moe_grouped_swiglu_pack(to_dev(self.up), to_dev(self.down))

    def expert(self, e):
        return (wl.bf16_bits_to_f32(self.up[e]).astype(np.float64),
                wl.bf16_bits_to_f32(self.down[e]).astype(np.float64))


def _reference(layer, x64, idx, w, parts):
    """(out, tolerance) in float64; parts: whether x is kept in two bf16 parts."""
    T, k = idx.shape
    I = layer.I
    cH = 2 * (layer.H / 16 + 6) * U + (2.0 ** -17 if parts else 0.0)
    cI = 2 * (I / 16 + 6) * U
    out, tol = np.zeros((T, layer.H)), np.zeros((T, layer.H))
    for e in np.unique(idx[idx >= 0]):
        t, j = np.nonzero(idx == e)
        up, down = layer.expert(e)
        g, u = x64[t] @ up[:, :I], x64[t] @ up[:, I:]
        size = np.abs(x64[t]) @ np.abs(up) * cH
        silu = g / (1 + np.exp(-g))
        hid = silu * u
        dh = 1.1 * size[:, :I] * np.abs(u) + np.abs(silu) * size[:, I:] + \
            1.1 * size[:, :I] * size[:, I:] + (2.0 ** -17 + 8 * U) * np.abs(hid)
        p = w[t, j].astype(np.float64)[:, None]
        np.add.at(out, t, p * (hid @ down))
        np.add.at(tol, t, np.abs(p) * ((dh + (cI + (k + 2) * U) * (np.abs(hid) + dh)) @ np.abs(down)))
    return out, tol + 2.0 ** -8 * (np.abs(out) + tol)


def _x(rng, T, H, fp8):
    """(arguments of a call, x in float64)"""
    x = rng.standard_normal((T, H)).astype(np.float32)
    if not fp8:
        b = wl.f32_to_bf16_bits(x)
        return dict(x=to_dev(b)), wl.bf16_bits_to_f32(b).astype(np.float64)
    q, sc = moe.moe_quantize_fp8(to_dev(wl.f32_to_bf16_bits(x)), 128)
    v = q.float().cpu().numpy().astype(np.float64) * np.repeat(to_host(sc).astype(np.float64), 128, axis=1)
    return dict(x=q, x_scales=sc), v


def _route64(logits, k):
    idx = np.argsort(-logits.astype(np.float64), axis=1, kind="stable")[:, :k].astype(np.int32)
    v = np.take_along_axis(logits.astype(np.float64), idx, axis=1)
    p = np.exp(v - v[:, :1])
    return idx, p / p.sum(1, keepdims=True)


def _out64(t):
    return wl.bf16_bits_to_f32(to_host(t)).astype(np.float64)


def _check(out, ref, tol):
    torch.cuda.synchronize()
    assert moe.moe_workspace_status(out._moe_workspace) == 0
    err = np.abs(_out64(out) - ref)
    assert (err <= tol).all(), (err / np.maximum(tol, 1e-30)).max()


SHAPES = [(1, 1, 1, 256, 128), (1, 8, 2, 256, 128), (3, 5, 1, 256, 256), (7, 16, 4, 512, 128),
          (16, 8, 2, 768, 256), (17, 33, 8, 256, 384), (64, 8, 8, 256, 128), (64, 300, 32, 256, 128),
          (33, 1024, 6, 256, 128), (2, 64, 6, 2048, 1408), (48, 4, 2, 1280, 256), (64, 6, 1, 512, 640),
          (5, 40, 32, 256, 128), (1, 12, 3, 4096, 128), (1, 9, 2, 256, 2048)]


@pytest.mark.parametrize("T,E,k,H,I", SHAPES)
@pytest.mark.parametrize("fp8", [False, True])
def test_layer_from_logits(T, E, k, H, I, fp8):
    layer = Layer(E, H, I, T + E + H)
    rng = np.random.default_rng(T * 7 + E)
    args, x64 = _x(rng, T, H, fp8)
    logits = rng.standard_normal((T, E)).astype(np.float32)
    logits = wl.bf16_bits_to_f32(wl.f32_to_bf16_bits(logits))          # equal logits occur
    out, idx, w = moe.moe_layer_decode(logits=to_dev(logits), k=k, w_up_packed=layer.up_p,
                                       w_down_packed=layer.down_p, **args)
    idx_o, w_o = _route64(logits, k)
    assert (to_host(idx) == idx_o).all()
    # exp: 2 ulp, the sum of k terms, a division, all in float32
    assert (np.abs(to_host(w) - w_o) <= (k + 8) * 2 * U * w_o).all()
    _check(out, *_reference(layer, x64, idx_o, w_o, fp8))
    r = moe.moe_route(to_dev(logits), k)
    assert torch.equal(r.topk_idx, idx) and (r.topk_w - w).abs().max() <= 1e-6


@pytest.mark.parametrize("T,E,k,H,I", SHAPES)
@pytest.mark.parametrize("fp8", [False, True])
def test_layer_from_choices(T, E, k, H, I, fp8):
    layer = Layer(E, H, I, T + E + I)
    rng = np.random.default_rng(T * 11 + E)
    args, x64 = _x(rng, T, H, fp8)
    idx, w = wl.random_routing(T + k, T, E, k, empty_frac=0.3)
    idx[T // 2] = -1                                                   # a row with no expert
    out = moe.moe_layer_decode_indices(topk_idx=to_dev(idx), topk_w=to_dev(w), **args,
                                       w_up_packed=layer.up_p, w_down_packed=layer.down_p)
    _check(out, *_reference(layer, x64, idx, w, fp8))
    assert (to_host(out)[T // 2] == 0).all()


def test_everyone_to_one_expert():
    layer = Layer(16, 512, 256, 1)
    rng = np.random.default_rng(2)
    args, x64 = _x(rng, 64, 512, False)
    idx, w = np.full((64, 1), 11, np.int32), rng.uniform(0.1, 1, (64, 1)).astype(np.float32)
    out = moe.moe_layer_decode_indices(topk_idx=to_dev(idx), topk_w=to_dev(w), **args,
                                       w_up_packed=layer.up_p, w_down_packed=layer.down_p)
    _check(out, *_reference(layer, x64, idx, w, False))


def test_equal_logits_go_to_the_lower_id():
    layer = Layer(70, 256, 128, 3)
    args, _ = _x(np.random.default_rng(4), 4, 256, False)
    logits = np.zeros((4, 70), np.float32)
    logits[1, ::2] = -0.0                                              # as floats they are equal
    logits[2] = -5.0
    logits[3, 60:] = 1.0
    _, idx, w = moe.moe_layer_decode(logits=to_dev(logits), k=5, w_up_packed=layer.up_p,
                                     w_down_packed=layer.down_p, **args)
    assert to_host(idx).tolist() == [list(range(5))] * 3 + [list(range(60, 65))]
    assert (to_host(w) == np.float32(0.2)).all()


def test_no_expert_at_all_and_no_token():
    layer = Layer(4, 512, 128, 5)
    args, _ = _x(np.random.default_rng(6), 9, 512, False)
    out = torch.full((9, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_layer_decode_indices(topk_idx=torch.full((9, 2), -1, dtype=torch.int32, device="cuda"),
                                 topk_w=torch.ones((9, 2), device="cuda"), out=out, **args,
                                 w_up_packed=layer.up_p, w_down_packed=layer.down_p)
    assert (out == 0).all() and moe.moe_workspace_status(out._moe_workspace) == 0
    out, idx, _ = moe.moe_layer_decode(torch.empty((0, 512), dtype=torch.bfloat16, device="cuda"),
                                       torch.empty((0, 4), device="cuda"), 2, layer.up_p, layer.down_p)
    assert out.shape == (0, 512) and idx.shape == (0, 2)
    assert moe.moe_workspace_status(out._moe_workspace) == 0


def test_bad_choices_are_reported_and_empty():
    layer = Layer(6, 256, 128, 7)
    rng = np.random.default_rng(8)
    args, x64 = _x(rng, 4, 256, False)
    w = rng.uniform(0.1, 1, (4, 3)).astype(np.float32)
    idx = np.array([[0, 6, 2], [3, 3, 1], [-2, 5, 4], [2, 1, 0]], np.int32)
    good = np.array([[0, -1, 2], [3, -1, 1], [-1, 5, 4], [2, 1, 0]], np.int32)
    kw = dict(topk_w=to_dev(w), w_up_packed=layer.up_p, w_down_packed=layer.down_p, **args)
    out = moe.moe_layer_decode_indices(topk_idx=to_dev(idx), **kw)
    assert moe.moe_workspace_status(out._moe_workspace) == 6
    ref = moe.moe_layer_decode_indices(topk_idx=to_dev(good), **kw)
    _check(ref, *_reference(layer, x64, good, w, False))
    assert torch.equal(out, ref)


def test_nan_and_inf_stay_in_their_token():
    layer = Layer(4, 256, 128, 9)
    rng = np.random.default_rng(10)
    x = wl.f32_to_bf16_bits(rng.standard_normal((6, 256)).astype(np.float32))
    idx, w = wl.random_routing(3, 6, 4, 2)
    kw = dict(topk_idx=to_dev(idx), topk_w=to_dev(w), w_up_packed=layer.up_p,
              w_down_packed=layer.down_p)
    clean = moe.moe_layer_decode_indices(to_dev(x), **kw)
    x[2, 7], x[4, 9] = 0x7FC0, 0x7F80
    out = moe.moe_layer_decode_indices(to_dev(x), **kw)
    keep = [0, 1, 3, 5]
    assert torch.equal(out[keep], clean[keep])
    assert torch.isnan(out[2]).all()
    assert not torch.isfinite(out[4].float()).any()


def test_rows_behind_and_any_workspace_contents():
    layer = Layer(10, 512, 256, 11)
    rng = np.random.default_rng(12)
    T, k = 13, 3
    args, x64 = _x(rng, T, 512, False)
    logits = rng.standard_normal((T, 10)).astype(np.float32)
    n = moe.moe_layer_decode_workspace_size(T, 10, k, 512, 256)
    first = None
    for fill in (0, 255, 0x7F, 1):
        ws = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
        buf = torch.full((T + 3, 512), 9.0, dtype=torch.bfloat16, device="cuda")
        for _ in range(2):
            out, _, _ = moe.moe_layer_decode(logits=to_dev(logits), k=k, w_up_packed=layer.up_p,
                                             w_down_packed=layer.down_p, workspace=ws, out=buf[:T],
                                             **args)
            first = out.clone() if first is None else first
            assert torch.equal(out, first)
        assert (buf[T:] == 9).all()
    # in the rows of a larger batch of which T are used
    idx_o, w_o = _route64(logits, k)
    _check(out, *_reference(layer, x64, idx_o, w_o, False))


def test_graphs_that_share_a_workspace_and_another_stream():
    layer = Layer(32, 512, 256, 13)
    rng = np.random.default_rng(14)
    n = moe.moe_layer_decode_workspace_size(16, 32, 4, 512, 256)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    sets = []
    for T in (16, 5):
        args, _ = _x(rng, T, 512, T == 5)
        logits = to_dev(rng.standard_normal((T, 32)).astype(np.float32))
        kw = dict(logits=logits, k=4, w_up_packed=layer.up_p, w_down_packed=layer.down_p, **args)
        sets.append((kw, moe.moe_layer_decode(**kw)[0].clone()))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for kw, ref in sets:
        out, _, _ = moe.moe_layer_decode(**kw, stream=s)
        s.synchronize()
        assert torch.equal(out, ref)
    graphs = []
    for kw, _ in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = moe.moe_layer_decode(**kw, workspace=ws)[0]
        graphs.append((g, out))
    for _ in range(3):
        for (g, out), (_, ref) in zip(graphs, sets):
            out.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, ref)
    for _ in range(20):                                   # back to back, nothing waited for
        for g, out in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(out, ref) for (_, out), (_, ref) in zip(graphs, sets))


def test_two_calls_at_once():
    """On two streams with a workspace each, one behind the other on the GPU."""
    layer = Layer(32, 512, 256, 21)
    rng = np.random.default_rng(22)
    sets = []
    for T, fp8 in ((9, False), (40, True)):
        args, _ = _x(rng, T, 512, fp8)
        logits = to_dev(rng.standard_normal((T, 32)).astype(np.float32))
        sets.append(dict(logits=logits, k=4, w_up_packed=layer.up_p, w_down_packed=layer.down_p, **args))
    refs = [moe.moe_layer_decode(**kw)[0] for kw in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    outs = [[], []]
    for _ in range(10):
        for kw, s, o in zip(sets, streams, outs):
            o.append(moe.moe_layer_decode(**kw, stream=s)[0])
    torch.cuda.synchronize()
    for o, ref in zip(outs, refs):
        assert all(torch.equal(v, ref) for v in o)
        assert all(moe.moe_workspace_status(v._moe_workspace) == 0 for v in o)


def test_a_workspace_that_another_call_wrote():
    """The norm's backward and the router leave their data in a workspace; the
    layer takes it as it is, and the other way round."""
    layer = Layer(16, 512, 256, 23)
    rng = np.random.default_rng(24)
    args, _ = _x(rng, 20, 512, False)
    logits = to_dev(rng.standard_normal((20, 16)).astype(np.float32))
    kw = dict(logits=logits, k=3, w_up_packed=layer.up_p, w_down_packed=layer.down_p, **args)
    ref = moe.moe_layer_decode(**kw)[0]
    n = max(moe.moe_layer_decode_workspace_size(20, 16, 3, 512, 256),
            moe.moe_rmsnorm_backward_workspace_size(700, 512), moe.moe_route_workspace_size(20, 16, 3))
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    g = torch.randn((700, 512), device="cuda")
    w = torch.ones(512, device="cuda")
    gw = moe.moe_rmsnorm_backward(g, g, w)[1]
    idx = moe.moe_route(logits, 3).topk_idx
    for _ in range(3):
        assert torch.equal(moe.moe_layer_decode(**kw, workspace=ws)[0], ref)
        assert torch.equal(moe.moe_rmsnorm_backward(g, g, w, workspace=ws)[1], gw)
        assert torch.equal(moe.moe_layer_decode(**kw, workspace=ws)[0], ref)
        assert torch.equal(moe.moe_route(logits, 3, workspace=ws).topk_idx, idx)


def test_logits_that_are_no_numbers():
    """NaN and infinite logits (which the header excludes) touch no other token,
    and every chosen id is one of the experts, or -1."""
    layer = Layer(12, 256, 128, 25)
    args, _ = _x(np.random.default_rng(26), 20, 256, False)
    for T in (3, 20):
        logits = np.random.default_rng(27).standard_normal((T, 12)).astype(np.float32)
        kw = dict(k=4, w_up_packed=layer.up_p, w_down_packed=layer.down_p, x=args["x"][:T])
        clean, cidx, _ = moe.moe_layer_decode(logits=to_dev(logits), **kw)
        logits.view(np.uint32)[1] = 0xFFFFFFFF                 # the lowest of all bit patterns
        logits[2] = -np.inf
        out, idx, _ = moe.moe_layer_decode(logits=to_dev(logits), **kw)
        keep = [t for t in range(T) if t not in (1, 2)]
        assert torch.equal(idx[keep], cidx[keep])
        assert ((idx >= -1) & (idx < 12)).all()
        # another grouping of the experts' tokens sums in another order: 2^-8 and a bit
        a, b = out[keep].float(), clean[keep].float()
        assert torch.isfinite(a).all() and (a - b).abs().max() <= 2.0 ** -7 * b.abs().max()


def test_agrees_with_the_dispatch_path():
    """route, permute, moe_grouped_swiglu and combine of the same tokens.  There
    the hidden rows and the experts' outputs are rounded to bf16: half a step of
    2^-8 each on their magnitudes, on top of this call's tolerance."""
    T, E, k, H, I = 40, 16, 4, 512, 256
    layer = Layer(E, H, I, 15)
    rng = np.random.default_rng(16)
    args, x64 = _x(rng, T, H, False)
    logits = rng.standard_normal((T, E)).astype(np.float32)
    out, idx, w = moe.moe_layer_decode(logits=to_dev(logits), k=k, w_up_packed=layer.up_p,
                                       w_down_packed=layer.down_p, **args)
    r = moe.moe_route(to_dev(logits), k)
    y = moe.moe_grouped_swiglu(moe.moe_permute(args["x"], r.slot_pos), layer.up_p, layer.down_p,
                               r.offsets)
    ref = moe.moe_combine(y, r.slot_pos, r.topk_w)
    idx_o, w_o = _route64(logits, k)
    _, tol = _reference(layer, x64, idx_o, w_o, False)
    size = np.zeros((T, H))
    for t in range(T):
        for j in range(k):
            up, down = layer.expert(idx_o[t, j])
            g, u = x64[t] @ up[:, :I], x64[t] @ up[:, I:]
            hid = g / (1 + np.exp(-g)) * u
            size[t] += w_o[t, j] * (np.abs(hid) @ np.abs(down) + np.abs(hid @ down))
    assert (np.abs(_out64(out) - _out64(ref)) <= 2 * tol + 2.0 ** -8 * size).all()


def test_a_whole_block_of_a_decode_step():
    """norm + quantize of the residual stream, the layer from its codes, and the
    next norm with the layer's output added to the stream."""
    T, E, k, H, I = 6, 16, 4, 512, 256
    layer = Layer(E, H, I, 17)
    rng = np.random.default_rng(18)
    bf = lambda a: to_dev(wl.f32_to_bf16_bits(a.astype(np.float32)))
    attn, stream = bf(rng.standard_normal((T, H))), bf(3 * rng.standard_normal((T, H)))
    w1, w2 = bf(1 + 0.1 * rng.standard_normal(H)), bf(1 + 0.1 * rng.standard_normal(H))
    logits = to_dev(rng.standard_normal((T, E)).astype(np.float32))
    q, sc, h = moe.moe_rmsnorm_quantize_fp8(attn, w1, residual=stream)
    out, idx, w = moe.moe_layer_decode(q, logits, k, layer.up_p, layer.down_p, x_scales=sc)
    y, h2 = moe.moe_rmsnorm(out, w2, residual=h)
    torch.cuda.synchronize()
    x64 = q.float().cpu().numpy().astype(np.float64) * np.repeat(to_host(sc).astype(np.float64), 128, axis=1)
    idx_o, w_o = _route64(to_host(logits), k)
    ref, tol = _reference(layer, x64, idx_o, w_o, True)
    assert (np.abs(_out64(out) - ref) <= tol).all()
    # the last norm, of the stream that the kernels left
    s64 = _out64(h) + _out64(out)
    assert (np.abs(_out64(h2) - s64) <= (2.0 ** -8 + U) * np.abs(s64)).all()
    v = _out64(h2)
    n = v / np.sqrt((v * v).mean(1, keepdims=True) + 1e-6) * _out64(w2)
    assert (np.abs(_out64(y) - n) <= (2.0 ** -8 + 200 * U) * np.abs(n)).all()


def test_refusals():
    layer = Layer(4, 256, 128, 19)
    x = torch.zeros((3, 256), dtype=torch.bfloat16, device="cuda")
    lg = torch.zeros((3, 4), device="cuda")
    call = lambda **kw: moe.moe_layer_decode(**{**dict(x=x, logits=lg, k=2, w_up_packed=layer.up_p,
                                                       w_down_packed=layer.down_p), **kw})
    for kw in (dict(x=x.float()), dict(logits=lg[:2]), dict(logits=lg.double()), dict(x=x.cpu()),
               dict(w_down_packed=layer.up_p), dict(x_scales=torch.ones((3, 2), device="cuda")),
               dict(out=torch.empty((2, 256), dtype=torch.bfloat16, device="cuda")),
               dict(workspace=torch.empty(64, dtype=torch.uint8, device="cuda")),
               dict(x=x.t().contiguous().t()), dict(logits=lg.cpu())):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(k=0), dict(k=5),
               dict(x=torch.zeros((65, 256), dtype=torch.bfloat16, device="cuda"),
                    logits=torch.zeros((65, 4), device="cuda"))):
        with pytest.raises(moe.MoeError):
            call(**kw)
    q = x.to(torch.float8_e4m3fn)
    with pytest.raises(ValueError):
        call(x=q)                                          # codes without scales
    with pytest.raises(ValueError):
        call(x=q, x_scales=torch.ones((3, 4), device="cuda"))


def _fill(byte, first, last):
    return lambda ws: ws[first:last].fill_(byte)


def _small_backward(ws):
    moe.moe_rmsnorm_backward(torch.ones((1, 128), device="cuda"), torch.ones((1, 128), device="cuda"),
                             torch.ones(128, device="cuda"), workspace=ws)


def _router(ws):
    moe.moe_route(torch.eye(16, device="cuda"), 2, workspace=ws)


def _chunks(ws):
    moe.moe_sort_chunks(torch.ones((8, 3), device="cuda"),
                        torch.full((4,), 2, dtype=torch.int32, device="cuda"),
                        torch.arange(4, dtype=torch.int32, device="cuda"), workspace=ws)


WRITERS = {"nobody": lambda ws: None, "head": _fill(0, 0, 512), "epoch": _fill(0x5A, 256, 264),
           "second flags": _fill(0, 512 + 160 * 8, 512 + 320 * 8), "everything": _fill(0xFF, 0, None),
           "backward": _small_backward, "router": _router, "chunks": _chunks}


@pytest.mark.parametrize("writer", WRITERS)
@pytest.mark.parametrize("T,E,k,H,I", [(16, 32, 4, 512, 256), (1, 8, 2, 256, 128), (9, 64, 6, 2048, 1408)])
def test_replays_between_which_others_write_the_workspace(writer, T, E, k, H, I):
    """A captured layer repeats its call; what another node of the graph leaves in the
    workspace is the same after every replay.  Every replay has other tokens and other
    choices, and the bits of a call by itself."""
    layer = Layer(E, H, I, 31)
    rng = np.random.default_rng(32)
    sets = []
    for _ in range(6):
        x = to_dev(wl.f32_to_bf16_bits(rng.standard_normal((T, H)).astype(np.float32)))
        lg = to_dev(rng.standard_normal((T, E)).astype(np.float32))
        sets.append((x, lg, moe.moe_layer_decode(x, lg, k, layer.up_p, layer.down_p)[0]))
    n = max(moe.moe_layer_decode_workspace_size(T, E, k, H, I), moe.moe_rmsnorm_backward_workspace_size(1, 128),
            moe.moe_route_workspace_size(16, 16, 2), moe.moe_sort_chunks_workspace_size(4))
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    x, lg = sets[0][0].clone(), sets[0][1].clone()
    WRITERS[writer](ws)                                   # (their first call outside the capture)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = moe.moe_layer_decode(x, lg, k, layer.up_p, layer.down_p, workspace=ws)[0]
        status = ws[:4].clone()
        WRITERS[writer](ws)
    for xs, ls, ref in sets + sets[::-1]:
        x.copy_(xs)
        lg.copy_(ls)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert (status == 0).all()
        assert torch.equal(out, ref)


def test_a_call_leaves_no_flag_of_its_first_meeting():
    """Where a later call with the same token would take it: bytes 512 to 1791.  The
    second meeting's, behind them, are cleared by the blocks that set them."""
    layer = Layer(8, 256, 128, 33)
    x = to_dev(wl.f32_to_bf16_bits(np.random.default_rng(34).standard_normal((3, 256)).astype(np.float32)))
    ws = torch.full((moe.moe_layer_decode_workspace_size(3, 8, 2, 256, 128),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    moe.moe_layer_decode(x, torch.zeros((3, 8), device="cuda"), 2, layer.up_p, layer.down_p, workspace=ws)
    assert (ws[512:512 + 160 * 8] == 0).all()
    assert moe.moe_workspace_status(ws) == 0


@pytest.mark.parametrize("T,E,k,H,I", [(6, 8, 2, 256, 128), (40, 4, 2, 512, 256)])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("where", ["up", "gate", "down"])
def test_infinite_weights(T, E, k, H, I, fp8, where):
    """An infinite weight makes of the outputs it enters what it makes of them in float64,
    infinities and NaN at the same places, and touches no other output: rows are kept in
    two parts, of which a part of 0 or of the other sign must not turn it into NaN."""
    layer = Layer(E, H, I, 41)
    if where == "down":
        layer.down[1, 5, 17], layer.down[2, 70, 200] = 0x7F80, 0xFF80
    else:                                                 # one row of expert 1's gate or up weights
        layer.up[1, 9, 33 + (I if where == "up" else 0)] = 0x7F80
    layer.up_p, layer.down_p = moe.moe_grouped_swiglu_pack(to_dev(layer.up), to_dev(layer.down))
    rng = np.random.default_rng(42)
    args, x64 = _x(rng, T, H, fp8)
    idx, w = wl.random_routing(43, T, E, k)
    out = moe.moe_layer_decode_indices(topk_idx=to_dev(idx), topk_w=to_dev(w), **args,
                                       w_up_packed=layer.up_p, w_down_packed=layer.down_p)
    with np.errstate(all="ignore"):
        ref, tol = _reference(layer, x64, idx, w, fp8)
    got = _out64(out)
    assert not np.isfinite(ref).all()
    assert (np.isnan(got) == np.isnan(ref)).all()
    assert (got[np.isinf(ref)] == ref[np.isinf(ref)]).all()
    fine = np.isfinite(ref)
    assert (np.abs(got[fine] - ref[fine]) <= tol[fine]).all()


@pytest.mark.parametrize("T", [1, 24])
def test_a_block_with_its_router(T):
    """The norm's rows go to a router and to the layer, in bf16 and quantized to e4m3; the
    next norm adds the layer's rows to the stream.  Each step against float64 from what
    the step before left."""
    E, k, H, I = 12, 3, 512, 256
    layer = Layer(E, H, I, 51)
    rng = np.random.default_rng(52)
    bf = lambda a: to_dev(wl.f32_to_bf16_bits(a.astype(np.float32)))
    attn, stream = bf(rng.standard_normal((T, H))), bf(3 * rng.standard_normal((T, H)))
    w1, w2 = bf(1 + 0.1 * rng.standard_normal(H)), bf(1 + 0.1 * rng.standard_normal(H))
    w_router = to_dev((rng.standard_normal((E, H)) * H ** -0.5).astype(np.float32))
    y, h = moe.moe_rmsnorm(attn, w1, residual=stream)
    logits = y.float() @ w_router.t()
    q, sc = moe.moe_quantize_fp8(y, 128)
    outs = [moe.moe_layer_decode(y, logits, k, layer.up_p, layer.down_p),
            moe.moe_layer_decode(q, logits, k, layer.up_p, layer.down_p, x_scales=sc)]
    idx_o, w_o = _route64(to_host(logits), k)
    q64 = q.float().cpu().numpy().astype(np.float64) * np.repeat(to_host(sc).astype(np.float64), 128, axis=1)
    for (out, idx, _), x64, fp8 in zip(outs, (_out64(y), q64), (False, True)):
        assert (to_host(idx) == idx_o).all()
        _check(out, *_reference(layer, x64, idx_o, w_o, fp8))
        y2, h2 = moe.moe_rmsnorm(out, w2, residual=h)
        s64 = _out64(h) + _out64(out)
        assert (np.abs(_out64(h2) - s64) <= (2.0 ** -8 + U) * np.abs(s64)).all()
        v = _out64(h2)
        n = v / np.sqrt((v * v).mean(1, keepdims=True) + 1e-6) * _out64(w2)
        assert (np.abs(_out64(y2) - n) <= (2.0 ** -8 + 200 * U) * np.abs(n)).all()
