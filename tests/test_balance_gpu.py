"""moe_balance_loss and its gradient against float64."""
import math

import pytest
import torch

import unpermute_combine_gb300 as moe

pytestmark = pytest.mark.gpu
INF = float("inf")


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def choices(x, k, seed, empty=0.05):
    idx = torch.argsort(x, dim=1, descending=True, stable=True)[:, :k]
    drop = torch.rand(idx.shape, generator=gen(seed), device="cuda") < empty
    return torch.where(drop, -1, idx).to(torch.int32).contiguous()


def offsets(kind, T, S):
    if kind == "none":
        return None
    if kind == "even":
        cuts = torch.linspace(0, T, S + 1).long()
    else:                                           # empty ones, tokens in front and behind
        cuts = torch.sort(torch.randint(T // 10, T - T // 10 + 1, (S + 1,),
                                        generator=torch.Generator().manual_seed(T + S))).values
    return cuts.to(torch.int32).cuda()


def reference(x, idx, off, score, bc, zc, E):
    """(loss, counts, mean scores, gradient for ones) in float64."""
    T, k = idx.shape
    cuts = [0, T] if off is None else off.tolist()
    S = len(cuts) - 1
    tokens = max(1, cuts[-1] - cuts[0])
    x = x.double()
    loss = torch.zeros(2, dtype=torch.float64, device="cuda")
    counts = torch.zeros((S, E), dtype=torch.int32, device="cuda")
    mean = torch.zeros((S, E), dtype=torch.float64, device="cuda")
    grad = torch.zeros((2, T, E), dtype=torch.float64, device="cuda")
    for s in range(S):
        a, b = cuts[s], cuts[s + 1]
        if a >= b:
            continue
        v = x[a:b]
        off_row = (v == -INF).all(1, keepdim=True)
        soft = torch.where(off_row, 0.0, torch.softmax(v, 1))
        lse = torch.where(off_row, 0.0, torch.logsumexp(v, 1, keepdim=True))
        p = soft
        if score == "sigmoid":
            p = torch.where(off_row, 0.0, torch.softmax(torch.nn.functional.logsigmoid(v), 1))
        ids = idx[a:b].reshape(-1).long()
        counts[s] = torch.bincount(ids[ids >= 0], minlength=E).int()
        mean[s] = p.mean(0)
        f = counts[s].double() * E / (k * (b - a))
        loss[0] += bc / S * (f * mean[s]).sum()
        loss[1] += zc / tokens * (lse * lse).sum()
        d = p * ((f - f.mean()) - (p * (f - f.mean())).sum(1, keepdim=True)) * (bc / S / (b - a))
        grad[0, a:b] = d * torch.sigmoid(-v) if score == "sigmoid" else d
        grad[1, a:b] = 2 * zc / tokens * lse * soft
    return loss, counts, mean, grad


def spread(x):
    """Logits less their row's largest, without the ones that are off."""
    d = x - x.amax(1, keepdim=True)
    return d[torch.isfinite(d)].abs().max().item() if torch.isfinite(d).any() else 0.0


def relative(x):
    """Bound of a score's relative error: __expf is off by 2 + 1.2 |v| steps of 2^-23 at v,
    its argument by half a step of v; the sum over the experts averages the same errors, with
    log2 E + E/32 + 5 roundings of its own, and two divisions and products follow."""
    E = x.shape[1]
    v = max(spread(x), x[torch.isfinite(x)].abs().max().item() if torch.isfinite(x).any() else 0.0)
    return (2 * (2 + 1.8 * v) + 12 + math.log2(E) + E / 32) * 2.0 ** -23


def check(x, idx, off, score, bc=0.01, zc=0.001, seed=0):
    T, E = x.shape
    k = idx.shape[1]
    how = dict(seq_offsets=off, score=score, balance_coef=bc, z_coef=zc)
    loss, counts, mean = moe.moe_balance_loss(x, idx, **how)
    assert moe.moe_workspace_status(loss._moe_workspace) == 0
    want, wc, wm, wg = reference(x, idx, off, score, bc, zc, E)
    rel = relative(x)
    n = T if off is None else int((off[1:] - off[:-1]).max())
    sums = rel + (n / 8 + 40) * 2.0 ** -24          # a group's sum in float, at most all of a chunk's rows
    assert torch.equal(counts, wc)
    assert ((mean.double() - wm).abs() <= wm * sums + 1e-30).all()
    assert abs(loss[0].item() - want[0].item()) <= want[0].item() * sums
    top = max(1.0, x[torch.isfinite(x)].abs().max().item()) if torch.isfinite(x).any() else 1.0
    # lse = m + log(sum): absolute error of rel and of a few steps at the size of m
    lse_err = rel + (top + math.log(E)) * 2.0 ** -22
    assert abs(loss[1].item() - want[1].item()) <= zc * 2 * (top + math.log(E)) * lse_err + \
        want[1].item() * sums
    gl = torch.tensor([0.75, -1.25], device="cuda")
    gin = torch.randn((T, E), generator=gen(seed + 9), device="cuda") * wg[0].abs().max().float()
    for add in (None, gin):
        got = moe.moe_balance_loss_backward(x, counts, k, gl, grad_in=add, **how)
        assert moe.moe_device_status() == 0
        full = 0.75 * wg[0] - 1.25 * wg[1] + (0 if add is None else add.double())
        # p (a - dot): the error of dot is that of the p it sums, at the largest |a| met
        cut = [0, T] if off is None else off.tolist()
        bound = torch.zeros((T, E), dtype=torch.float64, device="cuda")
        for s in range(len(cut) - 1):
            a, b = cut[s], cut[s + 1]
            if a < b:
                f = wc[s].double() * E / (k * (b - a))
                most = (f - f.mean()).abs().max() * bc / (len(cut) - 1) / (b - a)
                v = x[a:b].double()
                p = torch.softmax(torch.nn.functional.logsigmoid(v) if score == "sigmoid" else v, 1)
                bound[a:b] = torch.nan_to_num(p) * most * 4 * rel
        bound += 1.25 * wg[1].abs() * (2 * rel) + 1.25 * 2 * zc / max(1, cut[-1] - cut[0]) * lse_err
        bound += full.abs() * 2.0 ** -22
        assert ((got.double() - full).abs() <= bound + 1e-38).all()
    # in place of what is added, and the same bits again
    here = gin.clone()
    moe.moe_balance_loss_backward(x, counts, k, gl, grad_in=here, grad_logits=here, **how)
    assert torch.equal(here, got)
    again = moe.moe_balance_loss(x, idx, **how)
    assert all(torch.equal(p, q) for p, q in zip(again, (loss, counts, mean)))
    return loss, counts, mean, got


CASES = [(1, 1, 1, 1, "none"), (1, 8, 2, 1, "none"), (3, 5, 5, 2, "even"), (97, 8, 2, 3, "cut"),
         (200, 12, 3, 7, "cut"), (1000, 24, 4, 1, "none"), (513, 33, 4, 5, "cut"),
         (4096, 64, 6, 1, "none"), (777, 62, 6, 9, "cut"), (640, 100, 8, 4, "cut"),
         (300, 130, 8, 2, "even"), (2000, 256, 8, 6, "cut"), (501, 255, 8, 3, "cut"),
         (64, 512, 16, 2, "even"), (129, 1024, 32, 3, "cut"), (60, 1021, 4, 1, "none"),
         (20000, 16, 2, 1, "none"), (3000, 64, 4, 700, "cut")]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,S,kind", CASES)
def test_matches_float64(T, E, k, S, kind, score):
    x = torch.randn((T, E), generator=gen(T + E), device="cuda") * 2.0
    check(x, choices(x, k, T), offsets(kind, T, S), score, seed=T)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_without_z_loss(score):
    x = torch.randn((300, 64), generator=gen(1), device="cuda")
    loss, _, _, _ = check(x, choices(x, 4, 2), offsets("cut", 300, 4), score, zc=0.0)
    assert loss[1].item() == 0.0


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_experts_that_are_off(score):
    x = torch.randn((200, 40), generator=gen(3), device="cuda")
    x[:, 5], x[20:30, ::2] = -INF, -INF
    x[40:50, 1:] = -INF                             # one expert is left
    idx = choices(x, 4, 4)
    check(x, idx, offsets("even", 200, 5), score)
    x[60:64] = -INF                                 # nothing is left
    _, _, mean, grad = check(x, idx, offsets("even", 200, 5), score)
    assert torch.isfinite(mean).all() and torch.isfinite(grad).all()
    x[:] = -INF
    idx[:] = -1
    loss, counts, mean, grad = check(x, idx, None, score)
    assert loss.tolist() == [0.0, 0.0] and not counts.any() and not mean.any()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_large_logits(score):
    x = torch.randn((128, 64), generator=gen(5), device="cuda")
    for shift in (80.0, -80.0, -2000.0, 3000.0):
        check(x + shift, choices(x, 2, 6), None, score)
    check(x * 40.0, choices(x, 2, 6), None, score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_padding_may_hold_anything(score):
    x = torch.randn((150, 40), generator=gen(12), device="cuda")
    idx = choices(x, 4, 1)
    off = torch.tensor([10, 60, 61, 130], dtype=torch.int32, device="cuda")
    want = moe.moe_balance_loss(x, idx, off, score, z_coef=0.1)
    wg = moe.moe_balance_loss_backward(x, want[1], 4, seq_offsets=off, score=score, z_coef=0.1)
    for v in (float("nan"), INF, 3e38):
        x[:10], x[130:] = v, v
        got = moe.moe_balance_loss(x, idx, off, score, z_coef=0.1)
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        g = moe.moe_balance_loss_backward(x, got[1], 4, seq_offsets=off, score=score, z_coef=0.1)
        assert torch.equal(g, wg) and not g[:10].any() and not g[130:].any()


def test_nan_stays_visible():
    x = torch.randn((64, 16), generator=gen(7), device="cuda")
    idx = choices(x, 2, 1)
    x[10, 3] = float("nan")
    off = torch.tensor([0, 32, 64], dtype=torch.int32, device="cuda")
    for score in ("softmax", "sigmoid"):
        loss, counts, mean = moe.moe_balance_loss(x, idx, off, score, z_coef=0.1)
        assert torch.isnan(loss).all() and torch.isnan(mean[0]).any()
        assert torch.isfinite(mean[1]).all()
        g = moe.moe_balance_loss_backward(x, counts, 2, seq_offsets=off, score=score, z_coef=0.1)
        assert torch.isnan(g[10]).any() and torch.isfinite(g[11:]).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gradient_against_differences(score):
    """Central differences of the forward definition in float64, counts held."""
    T, E, k = 12, 9, 3
    x = torch.randn((T, E), generator=gen(8), device="cuda")
    idx, off = choices(x, k, 3), torch.tensor([0, 5, 12], dtype=torch.int32, device="cuda")
    _, counts, _ = moe.moe_balance_loss(x, idx, off, score, 0.5, 0.25)
    got = moe.moe_balance_loss_backward(x, counts, k, seq_offsets=off, score=score, balance_coef=0.5,
                                        z_coef=0.25)
    h = 1e-4
    for t in range(T):
        for e in range(E):
            ends = []
            for sign in (1, -1):
                v = x.double().clone()
                v[t, e] += sign * h
                ends.append(reference(v, idx, off, score, 0.5, 0.25, E)[0].sum().item())
            # the difference's error: h^2 / 6 times a third derivative of order 1
            assert abs((ends[0] - ends[1]) / (2 * h) - got[t, e].item()) < 1e-6


def test_bad_choices_and_offsets_are_reported():
    x = torch.randn((100, 16), generator=gen(9), device="cuda")
    idx = choices(x, 2, 1, empty=0.0)
    good = moe.moe_balance_loss(x, idx)
    bad = idx.clone()
    bad[7, 1], bad[90, 0] = 16, -2
    loss, counts, _ = moe.moe_balance_loss(x, bad)
    assert moe.moe_workspace_status(loss._moe_workspace) == 6
    assert counts.sum().item() == good[1].sum().item() - 2
    for cuts in ([0, 50, 101], [-1, 50, 100], [0, 60, 40]):
        off = torch.tensor(cuts, dtype=torch.int32, device="cuda")
        loss, counts, _ = moe.moe_balance_loss(x, idx, off)
        assert moe.moe_workspace_status(loss._moe_workspace) == 6
        moe.moe_balance_loss_backward(x, counts, 2, seq_offsets=off)
        assert moe.moe_device_status() == 6
    loss, _, _ = moe.moe_balance_loss(x, idx, workspace=loss._moe_workspace)
    assert moe.moe_workspace_status(loss._moe_workspace) == 0


def test_no_tokens():
    x, idx = torch.empty((0, 8), device="cuda"), torch.empty((0, 2), dtype=torch.int32, device="cuda")
    loss, counts, mean = moe.moe_balance_loss(x, idx, z_coef=1.0)
    assert loss.tolist() == [0.0, 0.0] and not counts.any() and not mean.any()
    assert moe.moe_balance_loss_backward(x, counts, 2).shape == (0, 8)


def test_unaligned_logits():
    x = torch.randn((100 * 64 + 1,), generator=gen(10), device="cuda")[1:].view(100, 64)
    check(x, choices(x, 4, 1), None, "softmax")


def test_graph_and_other_stream():
    x = torch.randn((500, 64), generator=gen(11), device="cuda")
    idx = choices(x, 4, 1)
    want = moe.moe_balance_loss(x, idx, z_coef=0.1)
    wg = moe.moe_balance_loss_backward(x, want[1], 4, z_coef=0.1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        here = moe.moe_balance_loss(x, idx, z_coef=0.1)
    there = moe.moe_balance_loss(x, idx, z_coef=0.1, stream=side)
    torch.cuda.synchronize()
    for got in (here, there):
        assert all(torch.equal(p, q) for p, q in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = moe.moe_balance_loss(x, idx, z_coef=0.1)
        g = moe.moe_balance_loss_backward(x, out[1], 4, z_coef=0.1)
    for t in (*out, g):
        t.zero_()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(out, want)) and torch.equal(g, wg)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_training_step_of_a_router(score):
    """Route, the routing weights' gradient and the balance loss's on top, against float64."""
    T, E, k = 300, 16, 3
    x = torch.randn((T, E), generator=gen(13), device="cuda")
    off = torch.tensor([0, 120, 290], dtype=torch.int32, device="cuda")
    r = moe.moe_route(x, k)
    gp = torch.randn((T, k), generator=gen(14), device="cuda") * 1e-3
    _, counts, _ = moe.moe_balance_loss(x, r.topk_idx, off, score, 0.01, 0.001)
    first = moe.moe_route_backward(r.topk_idx, r.topk_w, gp, E)
    grad = moe.moe_balance_loss_backward(x, counts, k, seq_offsets=off, score=score, balance_coef=0.01,
                                         z_coef=0.001, grad_in=first, grad_logits=first)
    assert grad is first
    v = x.double().requires_grad_()
    top = torch.gather(v, 1, r.topk_idx.long())
    loss = (torch.softmax(top, 1) * gp.double()).sum()
    for a, b in ((0, 120), (120, 290)):
        p = torch.softmax(v[a:b], 1) if score == "softmax" else \
            torch.sigmoid(v[a:b]) / torch.sigmoid(v[a:b]).sum(1, keepdim=True)
        f = torch.bincount(r.topk_idx[a:b].reshape(-1).long(), minlength=E).double() * E / (k * (b - a))
        loss = loss + 0.01 / 2 * (f * p.mean(0)).sum()
    loss = loss + 0.001 / 290 * torch.logsumexp(v[:290], 1).square().sum()
    loss.backward()
    # every term is a few float32 roundings of values below 1e-3
    assert (grad.double() - v.grad).abs().max() < 1e-3 * 2.0 ** -18


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_sequences_of_one_token(score):
    T, E, k = 5000, 12, 2
    x = torch.randn((T, E), generator=gen(15), device="cuda")
    idx = choices(x, k, 1)
    off = torch.arange(T + 1, dtype=torch.int32, device="cuda")
    loss, counts, mean = moe.moe_balance_loss(x, idx, off, score, 0.5, 0.25)
    v = x.double()
    p = torch.softmax(torch.nn.functional.logsigmoid(v) if score == "sigmoid" else v, 1)
    want = torch.zeros((T, E + 1), dtype=torch.int32, device="cuda")
    want.scatter_add_(1, torch.where(idx < 0, E, idx).long(), torch.ones_like(idx))
    assert torch.equal(counts, want[:, :E])
    f = counts.double() * E / k
    rel = relative(x)
    assert ((mean.double() - p).abs() <= p * rel).all()
    assert abs(loss[0].item() - 0.5 / T * (f * p).sum().item()) <= loss[0].item() * (rel + 2.0 ** -18)
    grad = moe.moe_balance_loss_backward(x, counts, k, torch.tensor([1.0, 0.0], device="cuda"),
                                         seq_offsets=off, score=score, balance_coef=0.5)
    d = 0.5 / T * p * (f - (p * f).sum(1, keepdim=True))
    if score == "sigmoid":
        d = d * torch.sigmoid(-v)
    assert ((grad.double() - d).abs() <= 0.5 / T * p * E * 8 * rel).all()


def test_infinite_logits_of_sigmoids():
    """sigmoid(inf) is 1: without a z loss nothing of the row is NaN, and without weight for it."""
    T, E, k = 70, 12, 2
    x = torch.randn((T, E), generator=gen(23), device="cuda")
    idx = choices(x, k, 1)
    x[3, 5], x[40, 2:4], x[41] = INF, INF, INF
    x[40, 7] = -INF
    off = torch.tensor([0, 30, 70], dtype=torch.int32, device="cuda")
    loss, counts, mean = moe.moe_balance_loss(x, idx, off, "sigmoid", 0.5, 0.0)
    v = x.double()
    p = torch.sigmoid(v) / torch.sigmoid(v).sum(1, keepdim=True)
    rel = relative(x)
    ones = torch.tensor([1.0, 0.0], device="cuda")
    total = 0.0
    for s, (a, b) in enumerate(((0, 30), (30, 70))):
        f = counts[s].double() * E / (k * (b - a))
        wm = p[a:b].mean(0)
        assert ((mean[s].double() - wm).abs() <= wm * (rel + 45 * 2.0 ** -24)).all()
        total += 0.5 / 2 * (f * wm).sum().item()
        c = f - f.mean()
        d = 0.5 / 2 / (b - a) * p[a:b] * (c - (p[a:b] * c).sum(1, keepdim=True)) * torch.sigmoid(-v[a:b])
        bound = 0.5 / 2 / (b - a) * p[a:b] * c.abs().max() * 4 * rel + d.abs() * 2.0 ** -22
        for gl, zc in ((None, 0.0), (ones, 0.25)):
            g = moe.moe_balance_loss_backward(x, counts, k, gl, seq_offsets=off, score="sigmoid",
                                              balance_coef=0.5, z_coef=zc)
            assert ((g[a:b].double() - d).abs() <= bound).all()
    assert abs(loss[0].item() - total) <= total * (rel + 2.0 ** -18) and loss[1].item() == 0.0


@pytest.mark.parametrize("T,E,cuts", [
    (100, 16, [0, 50, 30, 100]), (100, 16, [0, 10, 5, 100]), (100, 16, [0, 100, 40]),
    (128, 256, [0, 128, 200]), (128, 256, [0, 128, -1]), (128, 256, [-7, 0, 0, 128]),
    (1, 1, [0, 1, 0, 1]), (3000, 64, [0, 1500, 1499, 1500, 3000])])
def test_backward_reports_every_bad_offset(T, E, cuts):
    """Also those of sequences that no token is in."""
    x = torch.randn((T, E), generator=gen(21), device="cuda")
    off = torch.tensor(cuts, dtype=torch.int32, device="cuda")
    counts = torch.zeros((len(cuts) - 1, E), dtype=torch.int32, device="cuda")
    assert moe.moe_device_status() == 0
    moe.moe_balance_loss_backward(x, counts, 1, seq_offsets=off)
    assert moe.moe_device_status() == 6
    good = off.clamp(0, T).cummax(0).values.to(torch.int32)
    moe.moe_balance_loss_backward(x, counts, 1, seq_offsets=good)
    assert moe.moe_device_status() == 0


def test_backward_reports_one_of_many_offsets():
    T, E, S = 2000, 8, 300000
    x = torch.randn((T, E), generator=gen(22), device="cuda")
    off = torch.full((S + 1,), T, dtype=torch.int32, device="cuda")
    off[:T] = torch.arange(T, device="cuda")
    counts = torch.ones((S, E), dtype=torch.int32, device="cuda")
    want = moe.moe_balance_loss_backward(x, counts, 1, seq_offsets=off)
    assert moe.moe_device_status() == 0
    for at in (S, S - 1, S // 2, T + 1):
        bad = off.clone()
        bad[at] = T + 1
        got = moe.moe_balance_loss_backward(x, counts, 1, seq_offsets=bad)
        assert moe.moe_device_status() == 6
        assert got.shape == want.shape


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("shift", [80.0, -80.0, -2000.0, 3000.0])
def test_shifted_rows_are_as_exact_as_near_ones(shift, score):
    """Rows whose exponentials' sum leaves float's middle are shifted by their largest: the
    scores' error goes by how far a row's logits lie from one another, not from 0."""
    T, E, k = 128, 64, 2
    x = torch.randn((T, E), generator=gen(24), device="cuda") + shift
    idx = choices(x, k, 6)
    how = dict(score=score, balance_coef=0.5, z_coef=0.0)
    loss, counts, mean = moe.moe_balance_loss(x, idx, **how)
    want, wc, wm, wg = reference(x, idx, None, score, 0.5, 0.0, E)
    assert torch.equal(counts, wc)
    # With v = x less the row's largest, in steps of 2^-24: v is off by |v|, v log2 e by
    # 2 |v| (log2 e itself and the product, of which ln 2 reaches the exponential), 2^x by 4,
    # twice: the element's and the sum's; the sum by log2 64 + 2 additions, 1/x and the product
    # by 2 + 1.  A sigmoid of x > 0 adds 2 |x| e^-x, its exponential's error, and 3.
    v = spread(x)
    rel = (2 * (3 * v + 4) + 8 + 3 + 6) * 2.0 ** -24
    # sums: eight rows of a chunk of 32 side by side, then warps, chunks
    sums = rel + (4 + 8 + 8 + 2) * 2.0 ** -24
    assert ((mean.double() - wm).abs() <= wm * sums).all()
    assert abs(loss[0].item() - want[0].item()) <= want[0].item() * (sums + 10 * 2.0 ** -24)
    got = moe.moe_balance_loss_backward(x, counts, k, **how)
    f = wc[0].double() * E / (k * T)
    most = (f - f.mean()).abs().max()
    p = torch.softmax(torch.nn.functional.logsigmoid(x.double()) if score == "sigmoid" else x.double(), 1)
    bound = p * most * (0.5 / T) * (4 * rel)
    if score == "sigmoid":                          # times 1 - sigmoid, an exponential of x itself
        keep = torch.sigmoid(-x.double())
        bound = bound * keep + wg[0].abs() * (3 * abs(shift) + 20) * 2.0 ** -24 + 1e-37
    assert ((got.double() - wg[0]).abs() <= bound + wg[0].abs() * 2.0 ** -22).all()


def padded(kind, T, S):
    """Offsets of few sequences among S, the others without tokens."""
    cuts = torch.sort(torch.randint(1, T - 9, (9,), generator=torch.Generator().manual_seed(S))).values
    if kind == "behind":                            # a buffer for the most sequences of a batch
        off = torch.full((S + 1,), int(cuts[-1]), dtype=torch.int32)
        off[:9] = cuts
    elif kind == "front":
        off = torch.full((S + 1,), int(cuts[0]), dtype=torch.int32)
        off[-9:] = cuts
    else:                                           # at every place that a sequence begins
        off = cuts.repeat_interleave((S + 1 + 8) // 9)[:S + 1].to(torch.int32)
    return off.cuda()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("kind", ["behind", "front", "between"])
@pytest.mark.parametrize("T,E,S", [(700, 16, 40), (5000, 64, 300), (300, 256, 1024)])
def test_sequences_without_tokens(T, E, S, kind, score):
    x = torch.randn((T, E), generator=gen(T), device="cuda")
    check(x, choices(x, 2, S), padded(kind, T, S), score)


@pytest.mark.parametrize("kind", ["behind", "front", "between"])
def test_many_sequences_without_tokens_take_no_walk(kind):
    """They are searched past, not read one by one: 200 000 of them in one place took 37 ms."""
    T, E, S = 20000, 8, 200000
    x = torch.randn((T, E), generator=gen(31), device="cuda")
    idx, off = choices(x, 2, 1), padded(kind, T, S)
    times = []
    for _ in range(5):
        ends = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
        ends[0].record()
        _, counts, _ = moe.moe_balance_loss(x, idx, off)
        moe.moe_balance_loss_backward(x, counts, 2, seq_offsets=off)
        ends[1].record()
        torch.cuda.synchronize()
        times.append(ends[0].elapsed_time(ends[1]))
    assert min(times) < 12.0, times
    assert counts.sum().item() == int((idx[off[0]:off[-1]] >= 0).sum())
