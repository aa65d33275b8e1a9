"""Rows, weights and products in e2m1 against float64."""
import os
import subprocess
import sys

import pytest
import torch

import fp4_testutil as f4
import unpermute_combine_gb300 as moe

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rows(T, H, seed, dtype=BF16, scale=1.0):
    x = torch.randn((T, H), generator=gen(seed), device="cuda") * scale
    x[:, ::37] *= 16.0
    return x.to(dtype)


def scalar(v):
    return None if v is None else torch.full((1,), v, device="cuda")


# ------------------------------------------------------------- quantizers

@pytest.mark.parametrize("block,g", [(16, None), (16, 0.0237), (16, 3.0), (32, None)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,H", [(1, 32), (3, 96), (1, 7168), (33, 1440), (257, 2048), (1000, 160)])
def test_quantize_matches_definition(T, H, dtype, block, g):
    x = rows(T, H, T + H, dtype)
    q, sc = moe.moe_quantize_fp4(x, block, global_scale=scalar(g))
    codes, byte, _ = f4.quantize(x, block, 1.0 if g is None else g)
    assert torch.equal(sc, byte)
    assert torch.equal(q, f4.pairs(codes))
    out = moe.moe_dequantize_fp4(q, sc, block, global_scale=scalar(g))
    gf = 1.0 if g is None else torch.tensor(g, dtype=F32).double().item()
    # the product of a value of 6 bits and g of 24 is exact in float64: one rounding
    assert torch.equal(out, (f4.values(codes, byte, block) * gf).to(BF16))


@pytest.mark.parametrize("block", [16, 32])
def test_quantize_ties_and_special_values(block):
    step = 0.75 if block == 16 else 0.5
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], device="cuda") * step
    x = torch.zeros((12, 64), device="cuda")
    x[0, :8], x[0, 8:16], x[0, 16] = ties, -ties, 6 * step          # every tie, both signs
    x[1] = 0.0                                                      # nothing
    x[2, 5] = float("nan")
    x[3, 40] = float("inf")
    x[4, 3] = -float("inf")
    x[5] = 3e38                                                     # past e4m3's largest scale
    x[5, 1::2] = -3e38
    x[6] = 1e-40                                                    # subnormal floats
    x[7, ::2], x[7, 1::2] = 2.0 ** -126, -2.0 ** -149
    x[8] = torch.linspace(-1, 1, 64, device="cuda") * 2.0 ** -9     # the smallest e4m3 scales
    x[9, 0] = -0.0
    x[10] = torch.linspace(-448 * 6, 448 * 6, 64, device="cuda")
    x[11] = torch.linspace(-5000, 5000, 64, device="cuda")
    q, sc = moe.moe_quantize_fp4(x, block)
    codes, byte, _ = f4.quantize(x, block)
    assert torch.equal(sc, byte)
    assert torch.equal(f4.unpairs(q), codes)
    out = moe.moe_dequantize_fp4(q, sc, block)
    bad = ~torch.isfinite(x.unflatten(1, (-1, block))).all(-1).repeat_interleave(block, dim=1)
    assert torch.equal(torch.isnan(out), bad)


@pytest.mark.parametrize("g", [1e-38, 1e-33, 1e30, 3e37])
def test_quantize_far_global_scales(g):
    x = rows(7, 256, 3, F32) * g * 100
    x = torch.where(torch.isfinite(x), x, 0.0)
    q, sc = moe.moe_quantize_fp4(x, 16, global_scale=scalar(g))
    codes, byte, _ = f4.quantize(x, 16, g)
    assert torch.equal(sc, byte) and torch.equal(f4.unpairs(q), codes)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_quantize_rows_on_16_byte_boundaries(dtype):
    whole = rows(1, 4096 + 64, 11, dtype).view(-1)
    off = 16 // whole.element_size()
    x = whole[off:off + 2048].view(2, 1024)
    assert x.data_ptr() % 32 == 16
    for block in (16, 32):
        q, sc = moe.moe_quantize_fp4(x, block)
        p, sp = moe.moe_quantize_fp4(x.clone(), block)
        assert torch.equal(q, p) and torch.equal(sc, sp)


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,H,k", [(1, 32, 1), (5, 96, 3), (64, 7168, 8), (777, 1440, 2), (9, 2080, 32)])
def test_permute_quantize(T, H, k, dtype, block):
    x = rows(T, H, H + k, dtype)
    n = T * k + 3
    slot = torch.randperm(n, generator=gen(5), device="cuda")[:T * k].to(torch.int32).view(T, k)
    drop = torch.rand((T, k), generator=gen(6), device="cuda")
    slot = torch.where(drop < 0.2, -1, torch.where(drop > 0.95, n + 7, slot.long())).to(torch.int32)
    out = (torch.full((n, H // 2), 0xA5, dtype=torch.uint8, device="cuda"),
           torch.full((n, H // block), 0x5A, dtype=torch.uint8, device="cuda"))
    g = scalar(0.02) if block == 16 else None
    moe.moe_permute_quantize_fp4(x, slot, block, global_scale=g, n_rows=n, out=out)
    q, sc = moe.moe_quantize_fp4(x, block, global_scale=g)
    want = (torch.full_like(out[0], 0xA5), torch.full_like(out[1], 0x5A))
    for j in range(k):
        ok = (slot[:, j] >= 0) & (slot[:, j] < n)
        want[0][slot[ok, j].long()], want[1][slot[ok, j].long()] = q[ok], sc[ok]
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_rows_move_as_bytes():
    x = rows(50, 512, 1)
    r = moe.moe_route(torch.randn((50, 8), generator=gen(2), device="cuda"), 2)
    q, sc = moe.moe_quantize_fp4(x, 32)
    e4 = torch.float8_e4m3fn
    moved = moe.moe_permute(q.view(e4), r.slot_pos).view(torch.uint8)
    moved_s = moe.moe_permute(sc.view(e4), r.slot_pos).view(torch.uint8)
    p, sp = moe.moe_permute_quantize_fp4(x, r.slot_pos, 32)
    assert torch.equal(moved, p) and torch.equal(moved_s, sp)


# ---------------------------------------------------------------- weights

@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("E,N,K,gate_up", [(1, 8, 32, False), (3, 200, 288, False),
                                           (2, 128, 256, True), (2, 384, 1440, True)])
def test_pack(E, N, K, gate_up, block):
    w = rows(E * N, K, N + K).view(E, N, K)
    g = torch.rand((E,), generator=gen(1), device="cuda") * 0.01 + 0.001 if block == 16 else None
    q, sc = moe.moe_pack_fp4(w, block, global_scale=g, gate_up=gate_up)
    assert q.shape == (E, N, K // 2)
    assert sc.numel() == moe.moe_pack_fp4_scales_size(E, N, K, block)
    src = f4.in_turn(N // 2).cuda() if gate_up else torch.arange(N, device="cuda")
    at = f4.packed_at(N, K, block, "cuda")
    for e in range(E):
        codes, byte, _ = f4.quantize(w[e], block, 1.0 if g is None else g[e].item())
        assert torch.equal(q[e], f4.pairs(codes[src]))
        mine = sc.view(E, -1)[e]
        assert torch.equal(mine[at], byte[src])
        rest = torch.ones_like(mine, dtype=torch.bool)
        rest[at.reshape(-1)] = False
        assert not mine[rest].any()


# --------------------------------------------------------------- products

def segments(kind, M, E, seed):
    if kind == "even":
        cuts = torch.linspace(0, M, E + 1).long()
    elif kind == "one":                             # all rows are one expert's
        cuts = torch.zeros(E + 1, dtype=torch.long)
        cuts[E // 2 + 1:] = M
    elif kind == "short":                           # rows in front of and behind the segments
        cuts = torch.sort(torch.randint(min(3, M), max(M - 2, min(3, M)) + 1, (E + 1,),
                                        generator=torch.Generator().manual_seed(seed))).values
    else:
        cuts = torch.sort(torch.randint(0, M + 1, (E + 1,),
                                        generator=torch.Generator().manual_seed(seed))).values
        cuts[0], cuts[-1] = 0, M
    return cuts.to(torch.int32).cuda()


def fp4_rows(M, K, block, seed):
    q, sc = moe.moe_quantize_fp4(rows(M, K, seed), block)
    return q, sc, f4.values(f4.unpairs(q), sc, block)


def fp4_weights(E, N, K, block, seed, gate_up=False):
    w = rows(E * N, K, seed, scale=K ** -0.5).view(E, N, K)
    g = (w.float().abs().amax((1, 2)) / (448 * 6)).contiguous() if block == 16 else None
    q, sc = moe.moe_pack_fp4(w, block, global_scale=g, gate_up=gate_up)
    at = f4.packed_at(N, K, block, "cuda")
    v = torch.stack([f4.values(f4.unpairs(q[e]), sc.view(E, -1)[e][at], block) for e in range(E)])
    return q, sc, g, v


def product_error(x, w, K):
    """Bound of a float32 sum on the tensor cores: of K/64 steps, each of which may drop
    the bits below its largest term's (one step of float32, 2^-23), and alpha's rounding."""
    return (x.abs() @ w.abs().t()) * ((K / 64 + 4) * 2.0 ** -23)


MATMUL = [(1, 1, 256, 256, "even"), (1, 1, 8, 32, "even"), (5, 2, 40, 96, "even"),
          (128, 1, 128, 64, "even"), (129, 1, 136, 320, "even"), (300, 3, 264, 512, "ragged"),
          (1003, 24, 1000, 1440, "ragged"), (70, 8, 512, 2048, "one"), (64, 40, 384, 1408, "ragged"),
          (200, 5, 256, 288, "short"), (4096, 4, 2048, 1024, "ragged"), (700, 2, 6000, 544, "ragged"),
          # tiles of 128 rows, more experts than pairs take, pairs over odd sizes
          (9000, 6, 520, 1440, "ragged"), (40000, 300, 264, 288, "ragged"), (6000, 300, 384, 288, "one"),
          (3100, 3, 3000, 1440, "short"), (2600, 2, 2056, 544, "one"), (1500, 3, 2000, 480, "ragged"),
          (30000, 4, 1000, 1440, "ragged"), (9000, 5, 3000, 2080, "short"), (20000, 3, 2056, 544, "one")]


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("M,E,N,K,kind", MATMUL)
def test_matmul(M, E, N, K, kind, block):
    xq, xs, x = fp4_rows(M, K, block, M + K)
    wq, ws, g, w = fp4_weights(E, N, K, block, N)
    off = segments(kind, M, E, M)
    out = torch.full((M, N), 7.0, dtype=BF16, device="cuda")
    moe.moe_grouped_matmul_fp4(xq, xs, wq, ws, off, block, alpha=g, out=out)
    assert moe.moe_workspace_status(out._moe_workspace) == 0
    cuts = off.tolist()
    want = torch.full((M, N), 7.0, dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(want)
    for e in range(E):
        a, b = cuts[e], cuts[e + 1]
        if a < b:
            al = 1.0 if g is None else g[e].double()
            want[a:b] = x[a:b] @ w[e].t() * al
            tol[a:b] = product_error(x[a:b], w[e], K) * al
    # and the rounding to bf16
    assert ((out.double() - want).abs() <= want.abs() * 2.0 ** -8 + tol).all()
    again = torch.full_like(out, 7.0)
    moe.moe_grouped_matmul_fp4(xq, xs, wq, ws, off, block, alpha=g, out=again)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))


def hidden_reference(gate, up, gate_tol, up_tol, block, g):
    """(values that the quantized hidden rows stand for, without g; how far the kernel's
    may be from them): errors of gate and up move a value past a code's border, or a
    block's largest past a scale's, only near these."""
    sig = torch.sigmoid(gate)
    h = gate * sig * up
    # |d silu / d gate| <= 1.1; __expf is off by (2 + 1.2 |x|) steps of 2^-23, the division and
    # the products by 5 more
    tol = 1.1 * up.abs() * gate_tol + (gate * sig).abs() * up_tol + gate_tol * up_tol
    tol = tol + h.abs() * (7 + 1.2 * gate.abs()) * 2.0 ** -23
    _, byte, _ = f4.quantize(h.float(), block, g)
    blocks, tb = h.unflatten(-1, (-1, block)), tol.unflatten(-1, (-1, block))
    mid = None
    ends = []
    gf = torch.tensor(g, dtype=F32).double().item()
    for amax in ((blocks.abs()).amax(-1), (blocks.abs() - tb).clamp(min=0).amax(-1),
                 (blocks.abs() + tb).amax(-1)):
        _, s = f4.scales(amax.float().double(), block, g)
        step = (s * gf).float().double()[..., None]
        for v in ((blocks,) if mid is None else (blocks - tb, blocks + tb)):
            q = torch.where(step > 0, v / step, 0.0).float().abs()
            code = torch.zeros(q.shape, dtype=torch.long, device=h.device)
            for i, edge in enumerate(f4.EDGES):
                code += (q > edge) if i % 2 == 0 else (q >= edge)
            val = torch.tensor(f4.VALUES, dtype=torch.float64, device=h.device)[code]
            val = torch.where(v < 0, -val, val) * s[..., None]
            if mid is None:
                mid = val
            else:
                ends.append((val - mid).abs())
    far = torch.stack(ends).amax(0)
    return mid.flatten(-2), far.flatten(-2)


LAYERS = [(1, 1, 64, 64, "even"), (6, 64, 2048, 1408, "ragged"), (130, 3, 320, 192, "ragged"),
          (64, 8, 1024, 512, "one"), (513, 16, 512, 704, "ragged"), (40, 4, 256, 128, "short"),
          (3000, 4, 1024, 2048, "ragged"), (9000, 6, 512, 256, "ragged"), (20000, 300, 64, 64, "ragged"),
          (5000, 3, 2240, 1472, "short"), (2100, 5, 1024, 320, "one")]


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("M,E,H,I,kind", LAYERS)
def test_swiglu(M, E, H, I, kind, block):
    xq, xs, x = fp4_rows(M, H, block, M)
    uq, us, ug, u = fp4_weights(E, 2 * I, H, block, I, gate_up=True)
    dq, ds, dg, d = fp4_weights(E, H, I, block, H)
    off = segments(kind, M, E, I)
    g = 0.004 if block == 16 else 1.0
    hs = scalar(g) if block == 16 else None
    ad = None if dg is None else dg * hs
    out = torch.full((M, H), 7.0, dtype=BF16, device="cuda")
    moe.moe_grouped_swiglu_fp4(xq, xs, uq, us, dq, ds, off, block, alpha_up=ug, alpha_down=ad,
                               hidden_scale=hs, out=out)
    assert moe.moe_workspace_status(out._moe_workspace) == 0
    cuts = off.tolist()
    want = torch.full((M, H), 7.0, dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(want)
    place = torch.arange(2 * I, device="cuda").view(-1, 2, 64)
    gr, ur = place[:, 0].reshape(-1), place[:, 1].reshape(-1)
    for e in range(E):
        a, b = cuts[e], cuts[e + 1]
        if a == b:
            continue
        au = 1.0 if ug is None else ug[e].double()
        al = 1.0 if ad is None else ad[e].double()
        both, err = x[a:b] @ u[e].t() * au, product_error(x[a:b], u[e], H) * au
        h, far = hidden_reference(both[:, gr], both[:, ur], err[:, gr], err[:, ur], block, g)
        want[a:b] = h @ d[e].t() * al
        tol[a:b] = (product_error(h.abs() + far, d[e], I) + far @ d[e].abs().t()) * al
    off_by = (out.double() - want).abs()
    assert (off_by <= want.abs() * 2.0 ** -8 + tol).all()
    # what a border may move is little of the whole
    live = torch.zeros((M,), dtype=torch.bool, device="cuda")
    live[cuts[0]:cuts[-1]] = True
    assert tol[live].norm() < 0.02 * want[live].norm() or M < 8
    again = torch.full_like(out, 7.0)
    moe.moe_grouped_swiglu_fp4(xq, xs, uq, us, dq, ds, off, block, alpha_up=ug, alpha_down=ad,
                               hidden_scale=hs, out=again)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))


# --------------------------------- tiles of 32, 128 and 256 rows: what they share

# (M, E, N, K): one of each, by the library's rule
EACH_TILE = [(40, 4, 256, 512), (9000, 6, 520, 1440), (4096, 4, 2048, 1024)]


def matmul_inputs(M, E, N, K, block, seed=0):
    xq, xs, x = fp4_rows(M, K, block, seed + M)
    wq, ws, g, w = fp4_weights(E, N, K, block, seed + N)
    return (xq, xs, wq, ws), g, x, w


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("M,E,N,K", EACH_TILE)
def test_any_workspace_and_graphs_and_streams(M, E, N, K, block):
    args, g, _, _ = matmul_inputs(M, E, N, K, block)
    off = segments("ragged", M, E, 3)
    want = moe.moe_grouped_matmul_fp4(*args, off, block, alpha=g)
    n = moe.moe_grouped_matmul_fp4_workspace_size(M, E, N, K, block)
    for fill in (0xFF, 0x7F, 0):                    # NaN scales of both kinds among them
        ws = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
        out = moe.moe_grouped_matmul_fp4(*args, off, block, alpha=g, workspace=ws)
        assert torch.equal(out.view(torch.int16), want.view(torch.int16))
        assert moe.moe_workspace_status(ws) == 0
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = moe.moe_grouped_matmul_fp4(*args, off, block, alpha=g, stream=side)
    again = moe.moe_grouped_matmul_fp4(*args, off, block, alpha=g)    # at the same time
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(again, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = moe.moe_grouped_matmul_fp4(*args, off, block, alpha=g)
    for _ in range(3):
        out.zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("M,E,N,K", EACH_TILE)
def test_nan_rows_and_columns_stay_where_they_are(M, E, N, K, block):
    x = rows(M, K, 1)
    w = rows(E * N, K, 2, scale=K ** -0.5).view(E, N, K)
    off = segments("even", M, E, 0)
    out = []
    for spoil in (False, True):
        if spoil:
            x[M // 2, 5], x[M - 1, K - 1], w[1, 7, 40] = float("inf"), float("nan"), float("nan")
        q, s = moe.moe_quantize_fp4(x, block)
        wq, ws = moe.moe_pack_fp4(w, block)
        out.append(moe.moe_grouped_matmul_fp4(q, s, wq, ws, off, block))
    bad = torch.zeros((M, N), dtype=torch.bool, device="cuda")
    bad[M // 2], bad[M - 1] = True, True
    bad[off[1]:off[2], 7] = True
    assert torch.equal(torch.isnan(out[1]), bad)
    assert torch.equal(out[0][~bad], out[1][~bad])


@pytest.mark.parametrize("M,E,N,K", EACH_TILE)
def test_bad_offsets_are_reported(M, E, N, K):
    args, _, _, _ = matmul_inputs(M, E, N, K, 32)
    good = segments("even", M, E, 0)
    want = moe.moe_grouped_matmul_fp4(*args, good, 32)
    for at, v in ((E, M + 1), (0, -3), (E, -1), (2, int(good[1]) - 5)):
        off = good.clone()
        off[at] = v
        out = torch.full_like(want, 5.0)
        moe.moe_grouped_matmul_fp4(*args, off, 32, out=out)
        assert moe.moe_workspace_status(out._moe_workspace) == 6 and (out == 5.0).all()
    out = moe.moe_grouped_matmul_fp4(*args, good, 32, workspace=out._moe_workspace)
    assert moe.moe_workspace_status(out._moe_workspace) == 0 and torch.equal(out, want)


def test_most_experts():
    M, E, N, K = 500, 1024, 136, 96
    args, g, x, w = matmul_inputs(M, E, N, K, 16)
    e = torch.randint(0, E, (M,), generator=gen(4), device="cuda").sort().values
    off = torch.searchsorted(e, torch.arange(E + 1, device="cuda")).to(torch.int32)
    out = moe.moe_grouped_matmul_fp4(*args, off, 16, alpha=g)
    want = torch.einsum("mk,mnk->mn", x, w[e]) * g[e, None].double()
    tol = torch.einsum("mk,mnk->mn", x.abs(), w[e].abs()) * g[e, None] * ((K / 64 + 4) * 2.0 ** -23)
    assert ((out.double() - want).abs() <= want.abs() * 2.0 ** -8 + tol).all()


def test_no_rows():
    args, g, _, _ = matmul_inputs(4, 2, 64, 64, 16)
    off = torch.zeros((3,), dtype=torch.int32, device="cuda")
    out = moe.moe_grouped_matmul_fp4(args[0][:0], args[1][:0], args[2], args[3], off, 16, alpha=g)
    assert out.shape == (0, 64) and moe.moe_workspace_status(out._moe_workspace) == 0
    y = torch.full((4, 64), 3.0, dtype=BF16, device="cuda")
    moe.moe_grouped_matmul_fp4(*args, off, 16, alpha=g, out=y)
    assert (y == 3.0).all()
    q, s = moe.moe_quantize_fp4(torch.empty((0, 64), device="cuda"))
    assert q.shape == (0, 32) and s.shape == (0, 4)
    assert moe.moe_dequantize_fp4(q, s).shape == (0, 64)


def test_binding_refuses():
    args, g, _, _ = matmul_inputs(4, 2, 64, 64, 16)
    off = torch.zeros((3,), dtype=torch.int32, device="cuda")
    xq, xs, wq, ws = args
    bad = [(xq[:, :16], xs, wq, ws, off), (xq, xs[:, :2], wq, ws, off), (xq, xs, wq[:, :, :16], ws, off),
           (xq, xs, wq, ws[:-1], off), (xq, xs, wq, ws, off[:2]), (xq.cpu(), xs, wq, ws, off),
           (xq, xs, wq, ws, off.long()), (xq.t(), xs, wq, ws, off)]
    for b in bad:
        with pytest.raises(ValueError):
            moe.moe_grouped_matmul_fp4(*b, 16)
    for kw in (dict(block=8), dict(alpha=g[:1]), dict(alpha=g.double()),
               dict(out=torch.empty((4, 32), dtype=BF16, device="cuda")),
               dict(workspace=torch.empty((8,), dtype=torch.uint8, device="cuda"))):
        with pytest.raises(ValueError):
            moe.moe_grouped_matmul_fp4(*args, off, **{"block": 16, **kw})
    x = rows(4, 64, 0)
    for call in (lambda: moe.moe_quantize_fp4(x, 64), lambda: moe.moe_quantize_fp4(x[:, :48]),
                 lambda: moe.moe_quantize_fp4(x.half()), lambda: moe.moe_quantize_fp4(x.t()),
                 lambda: moe.moe_permute_quantize_fp4(x, off[None]),
                 lambda: moe.moe_pack_fp4(x), lambda: moe.moe_pack_fp4(x[None].float())):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(moe.MoeError):               # a power of two needs no g
        moe.moe_quantize_fp4(x, 32, global_scale=torch.ones((1,), device="cuda"))
    with pytest.raises(moe.MoeError):               # 64 rows of the gate and 64 of up in turn
        moe.moe_pack_fp4(rows(96, 64, 0)[None], gate_up=True)


# ------------------------------------------------------- together, as in a model

@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("T,E,k,H,I", [(5, 16, 4, 512, 256), (700, 8, 2, 1024, 512)])
def test_layer_from_router_to_combine(T, E, k, H, I, block):
    """Norm, route, dispatch in e2m1, experts and combine, captured as one graph."""
    x = rows(T, H, 1)
    logits = torch.randn((T, E), generator=gen(2), device="cuda")
    w_norm = torch.ones((H,), dtype=BF16, device="cuda")
    w_up = torch.randn((E, 2 * I, H), generator=gen(3), device="cuda") * H ** -0.5
    w_down = torch.randn((E, H, I), generator=gen(4), device="cuda") * I ** -0.5
    g = scalar(0.004) if block == 16 else None
    ug = dg = None
    if block == 16:
        ug = (w_up.abs().amax((1, 2)) / (448 * 6)).contiguous()
        dg = (w_down.abs().amax((1, 2)) / (448 * 6)).contiguous()
    uq, us = moe.moe_pack_fp4(w_up.to(BF16), block, global_scale=ug, gate_up=True)
    dq, ds = moe.moe_pack_fp4(w_down.to(BF16), block, global_scale=dg)
    kw = {} if block == 32 else dict(alpha_up=ug * g, alpha_down=dg * g, hidden_scale=g)

    def step():
        y, _ = moe.moe_rmsnorm(x, w_norm)
        r = moe.moe_route(logits, k)
        q, s = moe.moe_permute_quantize_fp4(y, r.slot_pos, block, global_scale=g)
        z = moe.moe_grouped_swiglu_fp4(q, s, uq, us, dq, ds, r.offsets, block, **kw)
        return moe.moe_combine(z, r.slot_pos, r.topk_w), r, z

    out, r, z = step()
    # the experts' rows by way of the token order, and the weighted sum of their outputs (each
    # call is held to float64 above)
    y, _ = moe.moe_rmsnorm(x, w_norm)
    q, s = moe.moe_quantize_fp4(y, block, global_scale=g)
    src = r.sorted_indices.long()
    again = moe.moe_grouped_swiglu_fp4(q[src], s[src], uq, us, dq, ds, r.offsets, block, **kw)
    assert torch.equal(again, z)
    want = (z.double()[r.slot_pos.long()] * r.topk_w[..., None].double()).sum(1)
    assert ((out.double() - want).abs() <= want.abs() * 2.0 ** -8).all()       # one rounding to bf16
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got, _, _ = step()
    got.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, out)


def test_elements_past_32_bits():
    """More than 2^31 elements of rows and of y: the last rows as a call of their own gives them."""
    T, H, k = 300007, 7168, 64
    x = torch.empty((T, H), dtype=BF16, device="cuda").normal_(generator=gen(1))
    q, s = moe.moe_quantize_fp4(x, 16)
    back = moe.moe_dequantize_fp4(q, s, 16)
    tail = slice(T - 300, T)
    qt, st = moe.moe_quantize_fp4(x[tail].contiguous(), 16)
    assert torch.equal(q[tail], qt) and torch.equal(s[tail], st)
    assert torch.equal(back[tail], moe.moe_dequantize_fp4(qt, st, 16))
    slot = torch.arange(T - 1, -1, -1, dtype=torch.int32, device="cuda").view(T, 1)
    p, sp = moe.moe_permute_quantize_fp4(x, slot, 16)
    assert torch.equal(p[:300], qt.flip(0)) and torch.equal(sp[:300], st.flip(0))
    del x, back, p, sp
    w = rows(H, k, 2).view(1, H, k)
    wq, ws = moe.moe_pack_fp4(w, 16)
    qk, sk = q[:, :k // 2].contiguous(), s[:, :k // 16].contiguous()
    y = moe.moe_grouped_matmul_fp4(qk, sk, wq, ws, torch.tensor([0, T], dtype=torch.int32, device="cuda"), 16)
    yt = moe.moe_grouped_matmul_fp4(qk[tail].contiguous(), sk[tail].contiguous(), wq, ws,
                                    torch.tensor([0, 300], dtype=torch.int32, device="cuda"), 16)
    # one step of 64 columns: the same sum, rounded once
    assert torch.equal(y[tail], yt)


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("K", [32, 256, 512, 1024, 1280, 1536, 2592])
def test_pairs_with_fewer_and_more_stages_than_the_ring(K, block):
    """One to eleven stages a tile: which stages' last arrivals no next stage waits for differs.
    Calls in a row end and begin on the same SMs."""
    M, E, N = 20000, 2, 4096
    xq, xs, x = fp4_rows(M, K, block, K)
    wq, ws, g, w = fp4_weights(E, N, K, block, K + 1)
    off = torch.tensor([0, 9001, M], dtype=torch.int32, device="cuda")
    out = [moe.moe_grouped_matmul_fp4(xq, xs, wq, ws, off, block, alpha=g) for _ in range(20)]
    for y in out:
        assert moe.moe_workspace_status(y._moe_workspace) == 0
        assert torch.equal(y.view(torch.int16), out[0].view(torch.int16))
    for e, (a, b) in enumerate(((0, 9001), (9001, M))):
        al = 1.0 if g is None else g[e].double()
        want, tol = x[a:b] @ w[e].t() * al, product_error(x[a:b], w[e], K) * al
        assert ((out[0][a:b].double() - want).abs() <= want.abs() * 2.0 ** -8 + tol).all()


# --------------------------------------------- zeros, and the g that they give

@pytest.mark.parametrize("dtype", [BF16, F32])
def test_zeros_without_a_global_scale(dtype):
    """g = largest / (448 * 6) of a tensor of zeros is 0: its blocks are 0, not NaN."""
    x = torch.zeros((3, 96), dtype=dtype, device="cuda")
    g = scalar(0.0)
    q, sc = moe.moe_quantize_fp4(x, 16, global_scale=g)
    assert not q.any() and not sc.any()
    assert not moe.moe_dequantize_fp4(q, sc, 16, global_scale=g).any()
    slot = torch.arange(6, dtype=torch.int32, device="cuda").view(3, 2)
    q, sc = moe.moe_permute_quantize_fp4(x, slot, 16, global_scale=g)
    assert not q.any() and not sc.any()
    x[1, 40], x[2, 3] = float("nan"), 2.0           # NaN stays NaN; scale g is 0: code 0
    q, sc = moe.moe_quantize_fp4(x, 16, global_scale=g)
    want = torch.zeros_like(sc)
    want[1, 2], want[2, 0] = 0x7F, 0x7E
    assert torch.equal(sc, want) and not q.any()


def test_an_expert_of_zeros():
    """Packed with one g an expert, its rows' products are 0 and the others' as without it."""
    M, E, N, K = 30, 3, 128, 96
    w = rows(E * N, K, 1, scale=K ** -0.5).view(E, N, K)
    w[1] = 0.0
    g = w.float().abs().amax((1, 2)) / (448 * 6)
    assert g[1].item() == 0.0
    wq, ws = moe.moe_pack_fp4(w, 16, global_scale=g)
    assert not wq[1].any() and not ws.view(E, -1)[1].any()
    xq, xs, _ = fp4_rows(M, K, 16, 2)
    off = torch.tensor([0, 10, 20, 30], dtype=torch.int32, device="cuda")
    y = moe.moe_grouped_matmul_fp4(xq, xs, wq, ws, off, 16, alpha=g)
    assert not y[10:20].any() and torch.isfinite(y).all()
    for e in (0, 2):
        cut = slice(10 * e, 10 * e + 10)
        alone = moe.moe_grouped_matmul_fp4(
            xq[cut].contiguous(), xs[cut].contiguous(), wq[e:e + 1], ws.view(E, -1)[e].contiguous(),
            torch.tensor([0, 10], dtype=torch.int32, device="cuda"), 16, alpha=g[e:e + 1])
        assert torch.equal(y[cut], alone) and alone.any()


@pytest.mark.parametrize("zero", ["up", "down", "both"])
def test_a_network_of_zeros(zero):
    M, E, H, I = 20, 2, 128, 64
    w_up, w_down = rows(E * 2 * I, H, 3).view(E, 2 * I, H), rows(E * H, I, 4).view(E, H, I)
    if zero != "down":
        w_up[0] = 0.0
    if zero != "up":
        w_down[0] = 0.0
    gu, gd = (w.float().abs().amax((1, 2)) / (448 * 6) for w in (w_up, w_down))
    up, down = moe.moe_pack_fp4(w_up, 16, global_scale=gu, gate_up=True), \
        moe.moe_pack_fp4(w_down, 16, global_scale=gd)
    xq, xs, _ = fp4_rows(M, H, 16, 5)
    off = torch.tensor([0, 10, 20], dtype=torch.int32, device="cuda")
    # hidden rows of zeros alone, and their g, which is 0 then
    for hs in (scalar(0.01), None) if zero == "down" else (scalar(0.01), scalar(0.0), None):
        y = moe.moe_grouped_swiglu_fp4(xq, xs, *up, *down, off, 16, alpha_up=gu, alpha_down=gd,
                                       hidden_scale=hs)
        assert not y[:10].any() and torch.isfinite(y).all()
        assert y[10:].any() or (hs is not None and hs.item() == 0.0)


@pytest.mark.parametrize("block,g", [(16, None), (16, 0.0237), (16, 1e-33), (32, None)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_negative_zeros_keep_their_sign(dtype, block, g):
    """The code of -0 / step is that of -0, as is that of what lies below 1/4 of a step."""
    x = rows(5, 96, 17, dtype).float() * (1.0 if g is None else g * 100)
    x[:, 1::4], x[:, 3::8] = -0.0, 0.0
    x[1, 5::8], x[2, 5::8] = -1e-45, -1e-40
    x = x.to(dtype)
    codes, byte, _ = f4.quantize(x, block, 1.0 if g is None else g)
    assert (codes == 8).any()
    q, sc = moe.moe_quantize_fp4(x, block, global_scale=scalar(g))
    assert torch.equal(sc, byte) and torch.equal(f4.unpairs(q), codes)
    w = x.to(BF16).view(1, 5, 96)
    codes, _, _ = f4.quantize(w[0], block, 1.0 if g is None else g)
    q, _ = moe.moe_pack_fp4(w, block, global_scale=scalar(g))
    assert torch.equal(f4.unpairs(q[0]), codes)


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("E,H,I", [(1, 512, 512), (4, 1024, 2048)])
def test_one_workspace_for_calls_of_fewer_rows(E, H, I, block):
    """That of 4096 rows, through tiles of 256, 128 and 32 rows."""
    most = 4096
    xq, xs, _ = fp4_rows(most, H, block, 1)
    up, us, ug, _ = fp4_weights(E, 2 * I, H, block, 2, gate_up=True)
    down, ds, dg, _ = fp4_weights(E, H, I, block, 3)
    n = moe.moe_grouped_swiglu_fp4_workspace_size(most, E, H, I, block)
    n2 = moe.moe_grouped_matmul_fp4_workspace_size(most, E, 2 * I, H, block)
    ws, ws2 = (torch.full((v,), 0xFF, dtype=torch.uint8, device="cuda") for v in (n, n2))
    for M in (4096, 2048, 2047, 1025, 1024, 513, 300, 129, 128, 65, 64, 33, 7, 1, 0):
        off = segments("ragged", M, E, M)
        args = (xq[:M], xs[:M], up, us, down, ds, off, block)
        want = moe.moe_grouped_swiglu_fp4(*args, alpha_up=ug, alpha_down=dg)
        got = moe.moe_grouped_swiglu_fp4(*args, alpha_up=ug, alpha_down=dg, workspace=ws)
        assert torch.equal(want.view(torch.int16), got.view(torch.int16))
        assert moe.moe_workspace_status(ws) == 0
        args = (xq[:M], xs[:M], up, us, off, block)
        want = moe.moe_grouped_matmul_fp4(*args, alpha=ug)
        got = moe.moe_grouped_matmul_fp4(*args, alpha=ug, workspace=ws2)
        assert torch.equal(want.view(torch.int16), got.view(torch.int16))
        assert moe.moe_workspace_status(ws2) == 0


@pytest.mark.parametrize("block", [16, 32])
def test_first_calls_of_a_process_are_captured(block):
    """What is looked up once, for each kernel by itself, is looked up under a capture."""
    code = f"""
import torch, test_fp4_gpu as t, unpermute_combine_gb300 as moe
M, E, H, I = 8000, 2, 512, 1024
block = {block}
xq, xs, _ = t.fp4_rows(M, H, block, 1)
up, us, ug, _ = t.fp4_weights(E, 2 * I, H, block, 2, gate_up=True)
down, ds, dg, _ = t.fp4_weights(E, H, I, block, 3)
off = t.segments("ragged", M, E, 4)
def step():
    return (moe.moe_grouped_swiglu_fp4(xq, xs, up, us, down, ds, off, block, alpha_up=ug, alpha_down=dg),
            moe.moe_grouped_matmul_fp4(xq, xs, up, us, off, block, alpha=ug))
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = step()
graph.replay()
want = step()
torch.cuda.synchronize()
assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(got, want))
assert all(moe.moe_workspace_status(a._moe_workspace) == 0 for a in (*got, *want))
"""
    here = os.path.dirname(os.path.abspath(__file__))
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([here, os.path.dirname(here)]))
    r = subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
