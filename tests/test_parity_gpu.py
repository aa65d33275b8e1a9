"""GPU (sm_103a) vs CPU oracle parity through the C ABI.

Integer, index and row-movement outputs must be bit-exact.  The combine is
bit-exact too (it reaches the double slot-order sum rounded once); the
routing softmax must be within 1e-6 absolute; grad_probs within one bf16 ulp
of the oracle's double dot.  Inputs are seeded and synthetic (workloads/);
the oracle never sees anything the GPU produced, except where a test says it
feeds both sides the same bytes."""
import numpy as np
import pytest

import oracle
import workloads as wl
from moe_testutil import (bf16_ulp_diff, bf16_ulp_of, f32_ulp_diff, to_dev, to_host,
                          within_one_bf16_ulp)

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import unpermute_combine_gb300 as moe  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from unpermute_combine_gb300 import build
    build.build()
    moe.load_library()


def _route_both(logits, k, routing_map=True):
    r = moe.moe_route(to_dev(logits), k, routing_map=routing_map)
    torch.cuda.synchronize()
    o = oracle.route(logits, k)
    return r, o


def _assert_route_equal(r, o, E):
    assert (to_host(r.topk_idx) == o["topk_idx"]).all()
    assert np.abs(to_host(r.topk_w) - o["topk_w"]).max(initial=0) <= 1e-6
    for name in ("counts", "offsets", "group_list", "sorted_indices", "slot_pos"):
        got = to_host(getattr(r, name))
        assert (got == o[name]).all(), name
    if r.routing_map is not None:
        assert (to_host(r.routing_map) == o["routing_map"]).all()
    # permuted probabilities: the GPU's own weights, moved bit-exactly
    n = int(o["offsets"][E])
    pp = to_host(r.permuted_probs)
    w = to_host(r.topk_w)
    sp = o["slot_pos"]
    valid = sp >= 0
    assert (pp[sp[valid]] == w[valid]).all()
    assert (pp[n:] == 0).all()
    assert np.abs(pp - o["permuted_probs"]).max(initial=0) <= 1e-6


# ---------------------------------------------------------------------- route

@pytest.mark.parametrize("name", ["tiny", "mid", "skewed", "vep8", "layer"])
def test_route_full_workloads(name):
    d = wl.make(name)
    w_ = d["workload"]
    r, o = _route_both(d["logits"], w_.k)
    _assert_route_equal(r, o, w_.E)
    assert moe.moe_workspace_status(r.workspace) == 0


def test_route_barrier_with_any_workspace_state():
    """The fused route's grid barrier needs no cleared workspace: a workspace
    of random bytes, the same one reused (the count left at zero by the
    previous call), its barrier area overwritten by other data, only its
    count overwritten, and two workspaces taking turns all give the oracle's
    routing."""
    d = wl.make("skewed", T=4096)
    W = d["workload"]
    lg = to_dev(d["logits"])
    o = oracle.route(d["logits"], W.k)
    nbytes = moe.moe_route_workspace_size(4096, W.E, W.k)
    gen = torch.Generator(device="cuda").manual_seed(5)

    def noise():
        return torch.randint(0, 256, (nbytes,), dtype=torch.uint8, device="cuda", generator=gen)

    moe.moe_device_status()                 # start from a clear status word
    ws_a, ws_b = noise(), noise()
    # the barrier count sits after the 256-byte header and 128 rows of 256
    # 16-bit counts (T = 4096: blocks of 32 tokens); poking it alone leaves the
    # marker saying the workspace is clean
    count_at = 256 + 128 * 256 * 2
    order = [ws_a, ws_a, ws_a, ws_b, ws_a, ws_b, ws_b, ws_b, ws_b]
    # the way each call takes: the count where the previous call on this
    # workspace left it clean, else the flags (a workspace not seen before,
    # or written over since)
    ways = ["flags", "count", "count", "flags", "count", "flags", "count", "flags", "count"]
    for i, ws in enumerate(order):
        if i == 5:
            ws.copy_(noise())               # another user's data lands in the workspace
        if i == 7:
            ws[count_at:count_at + 4] = torch.tensor([3, 0, 0, 0], dtype=torch.uint8)
        r = moe.moe_route(lg, W.k, workspace=ws, routing_map=True)
        torch.cuda.synchronize()
        _assert_route_equal(r, o, W.E)
        assert moe.moe_workspace_status(ws) == 0
        assert moe.moe_device_status() == 0
        # after the call: the count back at zero, the marker holding the
        # call's tag and `go` the tag (count) or the tag ^ 1 (flags)
        words = ws[count_at:count_at + 24].cpu().numpy().view("<u8")
        assert int(words[0]) & 0xFFFFFFFF == 0
        go, marker = int(words[1]), int(words[2])
        assert go ^ marker == (0 if ways[i] == "count" else 1), (i, ways[i])


@pytest.mark.parametrize("T,E,k", [(1, 64, 6), (127, 256, 8), (129, 64, 6), (1000, 256, 8),
                                   (333, 9, 3), (77, 33, 5)])
def test_route_forced_ties(T, E, k):
    logits = wl.tie_logits(T * 7 + E, T, E)
    r, o = _route_both(logits, k)
    _assert_route_equal(r, o, E)


@pytest.mark.parametrize("T,E,k", [(0, 8, 2), (1, 1, 1), (5, 4, 4), (260, 1024, 32), (40000, 64, 4),
                                   (33000, 300, 6),
                                   (300, 100, 7), (513, 32, 32), (64, 2, 1)])
def test_route_edge_shapes(T, E, k):
    rng = np.random.default_rng(T + 31 * E + k)
    logits = rng.standard_normal((T, E)).astype(np.float32)
    r, o = _route_both(logits, k)
    _assert_route_equal(r, o, E)


@pytest.mark.parametrize("T,E,hot", [(1000, 64, [37]),
                                     (40000, 256, [3, 17, 42, 99, 100, 200, 201, 255])])
def test_route_all_tokens_on_the_same_experts(T, E, hot):
    """Every token picks the same k experts: k segments of T rows each and
    every other expert empty (T = 40000 is beyond the fused scan)."""
    k = len(hot)
    logits = np.random.default_rng(T + E).standard_normal((T, E)).astype(np.float32)
    logits[:, hot] += 100.0
    r, o = _route_both(logits, k)
    _assert_route_equal(r, o, E)
    c = to_host(r.counts)
    assert (c[hot] == T).all() and c.sum() == T * k
    # the permute and the combine on this layout, bit-exact
    x = wl.random_activation(E + k, (T, 64), "bf16")
    xp = moe.moe_permute(to_dev(x), r.slot_pos)
    out = to_host(moe.moe_combine(xp, r.slot_pos, to_dev(o["topk_w"])))
    xp_o = oracle.permute(x, o["sorted_indices"], T * k)
    assert to_host(xp).tobytes() == xp_o.tobytes()
    ref, _ = oracle.combine(xp_o, o["slot_pos"], o["topk_w"])
    assert out.tobytes() == ref.tobytes()


@pytest.mark.parametrize("T,E,k,G,KG,ties", [(16384, 256, 8, 8, 4, False), (3000, 64, 6, 4, 2, False),
                                              (777, 256, 8, 8, 4, True), (500, 96, 4, 32, 3, False),
                                              (300, 40, 5, 5, 5, False), (129, 1024, 16, 16, 2, False),
                                              (64, 8, 2, 2, 1, True)])
def test_route_grouped(T, E, k, G, KG, ties):
    if ties:
        logits = wl.tie_logits(T + E, T, E)
    else:
        logits = np.random.default_rng(T + G).standard_normal((T, E)).astype(np.float32)
    r = moe.moe_route_grouped(to_dev(logits), k, G, KG, routing_map=True)
    torch.cuda.synchronize()
    idx, w, w64 = oracle.topk_softmax_grouped(logits, k, G, KG)
    o = oracle.route_indices(idx, w, E)
    o.update(topk_idx=idx, topk_w=w)
    _assert_route_equal(r, o, E)


def test_route_grouped_rejects_bad_groups():
    x = to_dev(np.zeros((4, 12), np.float32))
    for args in [(2, 5, 2), (7, 4, 2), (2, 3, 4), (2, 0, 1)]:
        with pytest.raises(moe.MoeError):
            moe.moe_route_grouped(x, *args)


def test_route_indices_dispatcher_worked_example(golden):
    g = golden("dispatcher_permute_example.json")
    idx = np.array(g["topk_idx_k2"], np.int32)
    r = moe.moe_route_indices(to_dev(idx), None, g["num_experts"], routing_map=True)
    torch.cuda.synchronize()
    n = int(to_host(r.offsets)[-1])
    assert to_host(r.routing_map).tolist() == g["routing_map"]
    assert to_host(r.sorted_indices)[:n].tolist() == g["sorted_indices"]
    assert (to_host(r.sorted_indices)[n:] == -1).all()
    assert to_host(r.group_list).tolist() == [2, 5, 7]
    tokens = np.repeat(np.arange(4, dtype=np.float32)[:, None], 8, axis=1)
    xp = to_host(moe.moe_permute(to_dev(tokens), r.slot_pos))
    assert xp[:n, 0].astype(int).tolist() == g["permuted_input_token_rows"]


def test_route_indices_group_list_example(golden):
    g = golden("moe_ops_group_list.json")
    experts = np.concatenate([np.full(c, e) for e, c in enumerate(g["tokens_per_expert"])])
    np.random.default_rng(3).shuffle(experts)
    r = moe.moe_route_indices(to_dev(experts[:, None].astype(np.int32)), None, 3)
    assert to_host(r.group_list).tolist() == g["group_list"]


@pytest.mark.parametrize("T,E,k,drop", [(1000, 64, 4, 0.2), (257, 256, 8, 0.5), (31, 5, 5, 0.0)])
def test_route_indices_with_empty_slots(T, E, k, drop):
    idx, w = wl.random_routing(T + E, T, E, k, empty_frac=drop)
    r = moe.moe_route_indices(to_dev(idx), to_dev(w), E, routing_map=True)
    torch.cuda.synchronize()
    o = oracle.route_indices(idx, w, E)
    for name in ("counts", "offsets", "group_list", "sorted_indices", "slot_pos",
                 "routing_map", "permuted_probs"):
        assert (to_host(getattr(r, name)) == o[name]).all(), name
    assert moe.moe_workspace_status(r.workspace) == 0


def test_route_indices_flags_invalid_ids():
    idx = np.array([[0, 1], [1, 1], [2, 9], [-3, 0], [1, -1]], np.int32)
    r = moe.moe_route_indices(to_dev(idx), None, 4)
    assert moe.moe_workspace_status(r.workspace) == 6
    clean = np.array([[0, 1], [1, -1], [2, -1], [-1, 0], [1, -1]], np.int32)
    o = oracle.route_indices(clean, None, 4)
    for name in ("counts", "offsets", "sorted_indices", "slot_pos"):
        assert (to_host(getattr(r, name)) == o[name]).all(), name
    # a clean call on the same workspace resets the status
    moe.moe_route_indices(to_dev(clean), None, 4, workspace=r.workspace)
    assert moe.moe_workspace_status(r.workspace) == 0


# -------------------------------------------------------------------- permute

@pytest.mark.parametrize("dtype,T,H,E,k", [("bf16", 1000, 4096, 64, 2), ("bf16", 257, 7168, 256, 8),
                                           ("f32", 256, 128, 8, 2), ("bf16", 100, 13, 8, 3),
                                           ("f32", 129, 7, 16, 4), ("bf16", 64, 8, 4, 4),
                                           ("bf16", 300, 12000, 32, 4),   # 24000-byte rows: 2 pieces
                                           ("f32", 200, 9000, 16, 3)])    # 36000-byte rows: 3 pieces
def test_permute_bit_exact(dtype, T, H, E, k):
    x = wl.random_activation(T + H, (T, H), dtype)
    idx, _ = wl.random_routing(T * 3 + k, T, E, k, empty_frac=0.1)
    o = oracle.route_indices(idx, None, E)
    n = int(o["offsets"][E])
    r = moe.moe_route_indices(to_dev(idx), None, E)
    got = to_host(moe.moe_permute(to_dev(x), r.slot_pos))
    assert got[:n].tobytes() == oracle.permute(x, o["sorted_indices"], n).tobytes()
    assert moe.moe_device_status() == 0          # no bounded copy wait gave up


def test_permute_then_unweighted_combine_k1_identity():
    for dtype in ("bf16", "f32"):
        T, H, E = 777, 1024, 16
        x = wl.random_activation(5, (T, H), dtype)
        idx, _ = wl.random_routing(6, T, E, 1)
        r = moe.moe_route_indices(to_dev(idx), None, E)
        xp = moe.moe_permute(to_dev(x), r.slot_pos)
        back = moe.moe_combine(xp, r.slot_pos, None)
        ones = moe.moe_combine(xp, r.slot_pos, torch.ones((T, 1), device="cuda"))
        assert to_host(back).tobytes() == x.tobytes()
        assert to_host(ones).tobytes() == x.tobytes()


# -------------------------------------------------------------------- combine

@pytest.mark.parametrize("dtype,T,H,E,k,drop,weighted",
                         [("bf16", 1000, 4096, 64, 2, 0.0, True),
                          ("bf16", 300, 7168, 256, 8, 0.1, True),
                          ("bf16", 500, 1000, 32, 6, 0.2, False),
                          ("bf16", 700, 2048, 64, 6, 0.1, True),   # the layer shape's k
                          ("bf16", 200, 4104, 64, 8, 0.2, True),   # rows in 2 column parts, ragged
                          ("bf16", 150, 5000, 32, 7, 0.0, False),
                          ("bf16", 1, 7168, 16, 8, 0.0, True),     # one token in 4 parts
                          ("bf16", 3, 4104, 16, 8, 0.5, False),
                          ("bf16", 333, 512, 16, 5, 0.0, True),
                          ("bf16", 129, 36, 8, 3, 0.0, True),    # 72-byte rows: element path
                          ("f32", 256, 128, 8, 2, 0.0, True),
                          ("f32", 99, 33, 8, 5, 0.3, True),
                          ("bf16", 64, 256, 40, 32, 0.1, True)])
def test_combine_bit_exact(dtype, T, H, E, k, drop, weighted):
    idx, w = wl.random_routing(T + 5 * k, T, E, k, empty_frac=drop)
    if not weighted:
        w = None
    r = moe.moe_route_indices(to_dev(idx), None, E)
    o = oracle.route_indices(idx, None, E)
    y = wl.random_activation(H + k, (T * k, H), dtype)     # random signs: cancellation
    out = to_host(moe.moe_combine(to_dev(y), r.slot_pos, None if w is None else to_dev(w)))
    ref, ref64 = oracle.combine(y, o["slot_pos"], w)
    if dtype == "bf16":
        d = bf16_ulp_diff(out, ref)
    else:
        d = f32_ulp_diff(out, ref)
    assert d.max() == 0, f"max ulp {d.max()}, {np.count_nonzero(d)} mismatches"


@pytest.mark.parametrize("k,weighted", [(2, True), (4, True), (5, True), (6, True), (8, True),
                                        (2, False), (5, False), (6, False), (8, False)])
def test_combine_bit_exact_under_cancellation(k, weighted):
    """Rows built to cancel (exactly, or down to a few ulps): every tier of
    the combine -- float fast path (or, unweighted, the exact TwoSum chain),
    double-float middle tier, double last resort -- must still give the
    oracle's double slot-order sum rounded once."""
    T, H, E = 700, 512, 16
    rng = np.random.default_rng(100 + k)
    idx, _ = wl.random_routing(200 + k, T, E, k)
    r = moe.moe_route_indices(to_dev(idx), None, E)
    o = oracle.route_indices(idx, None, E)
    w = np.full((T, k), 0.5, np.float32)
    w[:, 1::2] = rng.choice([0.5, 0.25, 0.375], size=(T, k // 2)).astype(np.float32)
    if not weighted:
        w[:] = 1.0
    base = rng.standard_normal((T, H)).astype(np.float32)
    y32 = np.zeros((T * k, H), np.float32)
    for t in range(T):
        for j in range(k):
            p = o["slot_pos"][t, j]
            sign = 1.0 if j % 2 == 0 else -1.0
            wiggle = 1.0 + (rng.integers(-3, 4) * 2.0 ** -8 if t % 3 else 0.0)
            y32[p] = sign * base[t] * (0.5 / w[t, j]) * wiggle
    y = wl.f32_to_bf16_bits(y32)
    if not weighted:                                  # very different magnitudes too
        y[::5] = wl.f32_to_bf16_bits(y32[::5] * np.float32(2.0 ** 20))
    out = to_host(moe.moe_combine(to_dev(y), r.slot_pos, to_dev(w) if weighted else None))
    ref, _ = oracle.combine(y, o["slot_pos"], w if weighted else None)
    d = bf16_ulp_diff(out, ref)
    assert d.max() == 0, f"max ulp {d.max()}, {np.count_nonzero(d)} mismatches"


def test_combine_all_slots_empty_gives_positive_zero_rows():
    T, H, E, k = 300, 1024, 8, 4
    idx, w = wl.random_routing(77, T, E, k, empty_frac=0.0)
    idx[::2] = -1                                   # every other token routes nowhere
    r = moe.moe_route_indices(to_dev(idx), None, E)
    y = wl.random_activation(78, (T * k, H), "bf16")
    zero_rows = np.zeros((4, H), np.uint16)
    y[:4] = zero_rows
    y[4:8] = 0x8000                                 # negative zeros
    out = to_host(moe.moe_combine(to_dev(y), r.slot_pos, to_dev(w)))
    o = oracle.route_indices(idx, None, E)
    ref, _ = oracle.combine(y, o["slot_pos"], w)
    assert (out[::2] == 0).all()
    assert bf16_ulp_diff(out, ref).max() == 0 and (out == ref).all()


@pytest.mark.parametrize("weighted", [True, False])
def test_combine_and_backward_with_mostly_empty_slots(weighted):
    """Tokens with zero or one live slot take their own paths (capacity
    drops make them common): bit-exact combine including the +0 a zero
    product gives, and the backward's grad_y / grad_probs."""
    T, H, E, k = 900, 7168, 64, 8
    idx, w = wl.random_routing(31, T, E, k, empty_frac=0.85)
    w = np.random.default_rng(32).uniform(-1.5, 1.5, (T, k)).astype(np.float32)   # signed
    if not weighted:
        w = None
    r = moe.moe_route_indices(to_dev(idx), None, E)
    o = oracle.route_indices(idx, None, E)
    live = (idx >= 0).sum(axis=1)
    assert (live == 0).any() and (live == 1).sum() > T // 4
    y = wl.random_activation(33, (T * k, H), "bf16")
    y[:, ::97] = 0x8000                                    # negative zeros
    y[:, 1::89] = 0
    wd = None if w is None else to_dev(w)
    out = to_host(moe.moe_combine(to_dev(y), r.slot_pos, wd))
    ref, _ = oracle.combine(y, o["slot_pos"], w)
    assert (out == ref).all(), f"{np.count_nonzero(out != ref)} mismatches"
    g = wl.random_activation(34, (T, H), "bf16")
    gy, gp = moe.moe_combine_backward(to_dev(g), to_dev(y), r.slot_pos, wd)
    gy, gp = to_host(gy), to_host(gp)
    gy_o, gp_o, gp64 = oracle.combine_backward(g, y, o["slot_pos"], w)
    n = int(o["offsets"][E])
    assert gy[:n].tobytes() == gy_o[:n].tobytes()
    assert within_one_bf16_ulp(gp, gp64).all()
    assert (gp[o["slot_pos"] < 0] == 0).all()


def test_combine_deterministic_and_stable_across_calls():
    T, H, E, k = 2000, 2048, 64, 8
    idx, w = wl.random_routing(1, T, E, k)
    r = moe.moe_route_indices(to_dev(idx), None, E)
    y = to_dev(wl.random_activation(2, (T * k, H), "bf16"))
    a = moe.moe_combine(y, r.slot_pos, to_dev(w))
    b = moe.moe_combine(y, r.slot_pos, to_dev(w))
    g = to_dev(wl.random_activation(3, (T, H), "bf16"))
    ga, pa = moe.moe_combine_backward(g, y, r.slot_pos, to_dev(w))
    gb, pb = moe.moe_combine_backward(g, y, r.slot_pos, to_dev(w))
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    assert torch.equal(ga.view(torch.int16), gb.view(torch.int16))
    assert torch.equal(pa.view(torch.int32), pb.view(torch.int32))


@pytest.mark.parametrize("dtype,T,H,E,k,drop,weighted",
                         [("bf16", 600, 4096, 64, 2, 0.0, True),
                          ("bf16", 300, 7168, 256, 8, 0.1, True),
                          ("bf16", 300, 4104, 64, 8, 0.3, True),   # rows in 2 ragged column parts
                          ("bf16", 129, 7168, 32, 6, 0.0, False),  # 4 parts, unweighted
                          ("bf16", 400, 7168, 64, 5, 0.6, True),   # 4 parts, mostly 0-1 live slots
                          ("bf16", 1, 7168, 16, 8, 0.0, True),     # one token, one part pair
                          ("bf16", 3, 4104, 16, 8, 0.5, False),
                          ("bf16", 200, 1000, 16, 4, 0.0, False),
                          ("bf16", 77, 20, 8, 3, 0.2, True),     # element path
                          ("f32", 256, 128, 8, 2, 0.0, True),
                          ("f32", 50, 45, 6, 3, 0.2, True),
                          ("bf16", 40, 512, 64, 32, 0.0, True)])
def test_combine_backward(dtype, T, H, E, k, drop, weighted):
    idx, w = wl.random_routing(T + k, T, E, k, empty_frac=drop)
    if not weighted:
        w = None
    r = moe.moe_route_indices(to_dev(idx), None, E)
    o = oracle.route_indices(idx, None, E)
    n = int(o["offsets"][E])
    y = wl.random_activation(11, (T * k, H), dtype)
    g = wl.random_activation(12, (T, H), dtype)
    gy, gp = moe.moe_combine_backward(to_dev(g), to_dev(y), r.slot_pos,
                                      None if w is None else to_dev(w))
    gy, gp = to_host(gy), to_host(gp)
    gy_o, gp_o, gp64 = oracle.combine_backward(g, y, o["slot_pos"], w)
    assert gy[:n].tobytes() == gy_o[:n].tobytes()
    assert within_one_bf16_ulp(gp, gp64).all()
    assert (gp[o["slot_pos"] < 0] == 0).all()
    # in practice the compensated dot lands within a few float32 ulps
    assert f32_ulp_diff(gp, gp_o).max() <= 64


def test_expert_scale_bit_exact():
    # 16-byte-multiple bf16 rows (vector kernel, one with a ragged last batch
    # of vectors), an odd bf16 row (element kernel) and float32 rows
    for dtype, H in (("bf16", 520), ("bf16", 4104), ("bf16", 13), ("f32", 520)):
        T, E, k = 300, 16, 4
        idx, _ = wl.random_routing(4, T, E, k, empty_frac=0.1)
        o = oracle.route_indices(idx, None, E)
        r = moe.moe_route_indices(to_dev(idx), None, E)
        x = wl.random_activation(5, (T * k, H), dtype)
        scale = np.random.default_rng(6).uniform(-2, 2, E).astype(np.float32)
        got = to_host(moe.moe_expert_scale(to_dev(x), r.offsets, to_dev(scale)))
        ref = oracle.expert_scale(x, o["offsets"], scale)
        n = int(o["offsets"][E])
        assert got[:n].tobytes() == ref[:n].tobytes()


# ---------------------------------------------------------------- sort_chunks

def _virtual_rank_buffers(d, R=8, L=8):
    """Rank-major receive buffers of each virtual rank from the oracle's
    routing of 8 source slices (test infrastructure)."""
    w_ = d["workload"]
    T, k = w_.T, w_.k
    per = T // R
    idx, _, _ = oracle.topk_softmax(d["logits"], k)
    bufs = []
    for r_ in range(R):
        M = np.zeros((R, L), np.int32)
        rows = []
        for src in range(R):
            toks = np.arange(src * per, (src + 1) * per)
            for le in range(L):
                e = r_ * L + le
                sel = toks[(idx[toks] == e).any(axis=1)]
                M[src, le] = sel.size
                rows.append(sel)
        order = np.concatenate(rows)
        bufs.append((M, np.ascontiguousarray(d["x"][order])))
    return bufs


def test_sort_chunks_virtual_ep8_round_trip():
    d = wl.make("vep8")
    R = L = 8
    fwd = np.array(moe.moe_chunk_idxs(R, L, False), np.int32)
    inv = np.array(moe.moe_chunk_idxs(R, L, True), np.int32)
    for M, buf in _virtual_rank_buffers(d, R, L):
        xd = to_dev(buf)
        em = moe.moe_sort_chunks(xd, to_dev(M.ravel().copy()), to_dev(fwd))
        back = moe.moe_sort_chunks(em, to_dev(M.T.ravel().copy()), to_dev(inv))
        torch.cuda.synchronize()
        assert moe.moe_workspace_status(em._moe_workspace) == 0
        ref = oracle.sort_chunks(buf, M.ravel(), oracle.chunk_idxs(R, L, False))
        assert to_host(em).tobytes() == ref.tobytes()
        assert to_host(back).tobytes() == buf.tobytes()


def test_sort_chunks_virtual_ranks_concurrently_in_a_cuda_graph():
    """The 8 virtual ranks' reorders forked over 4 streams and captured in
    CUDA graphs (as the virtual-EP benchmark runs them): every rank's output
    is still the oracle's, byte for byte, after repeated replays."""
    d = wl.make("vep8")
    R = L = 8
    fwd = to_dev(np.array(moe.moe_chunk_idxs(R, L, False), np.int32))
    inv = to_dev(np.array(moe.moe_chunk_idxs(R, L, True), np.int32))
    ranks = []
    for M, buf in _virtual_rank_buffers(d, R, L):
        xd = to_dev(buf)
        ranks.append(dict(M=M, buf=buf, x=xd, em=torch.empty_like(xd), back=torch.empty_like(xd),
                          sp=to_dev(M.ravel().copy()), spt=to_dev(M.T.ravel().copy()),
                          wf=torch.empty(moe.moe_sort_chunks_workspace_size(R * L),
                                         dtype=torch.uint8, device="cuda"),
                          wb=torch.empty(moe.moe_sort_chunks_workspace_size(R * L),
                                         dtype=torch.uint8, device="cuda")))
    main = torch.cuda.Stream()
    side = [torch.cuda.Stream() for _ in range(4)]

    def both():
        for st in side:
            st.wait_stream(main)
        for i, q in enumerate(ranks):
            moe.moe_sort_chunks(q["x"], q["sp"], fwd, out=q["em"], workspace=q["wf"],
                                stream=side[i % 4])
        for st in side:
            main.wait_stream(st)
        for st in side:
            st.wait_stream(main)
        for i, q in enumerate(ranks):
            moe.moe_sort_chunks(q["em"], q["spt"], inv, out=q["back"], workspace=q["wb"],
                                stream=side[i % 4])
        for st in side:
            main.wait_stream(st)

    with torch.cuda.stream(main):
        both()                                   # eager, then captured
    main.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=main):
        both()
    for q in ranks:
        q["em"].zero_()
        q["back"].zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(main):
        for _ in range(3):
            g.replay()
    main.synchronize()
    fwd_o = oracle.chunk_idxs(R, L, False)
    for q in ranks:
        assert moe.moe_workspace_status(q["wf"]) == 0
        assert moe.moe_workspace_status(q["wb"]) == 0
        ref = oracle.sort_chunks(q["buf"], q["M"].ravel(), fwd_o)
        assert to_host(q["em"]).tobytes() == ref.tobytes()
        assert to_host(q["back"]).tobytes() == q["buf"].tobytes()


@pytest.mark.parametrize("R,L,H,dtype", [(3, 5, 100, "bf16"), (2, 2, 16, "f32"), (1, 9, 64, "bf16"),
                                         (16, 16, 1024, "bf16"),
                                         (40, 40, 64, "bf16"),       # C > 1024: plan kernel path
                                         (8, 8, 12000, "bf16")])     # rows of 24000 B: 2 pieces
def test_sort_chunks_asymmetric(R, L, H, dtype):
    rng = np.random.default_rng(R * 100 + L)
    M = rng.integers(0, 40, (R, L)).astype(np.int32)
    M[0, -1] = 0
    N = int(M.sum())
    x = wl.random_activation(R + L, (N, H), dtype)
    fwd = oracle.chunk_idxs(R, L, False)
    em = moe.moe_sort_chunks(to_dev(x), to_dev(M.ravel().copy()), to_dev(fwd))
    ref = oracle.sort_chunks(x, M.ravel(), fwd)
    assert to_host(em).tobytes() == ref.tobytes()
    back = moe.moe_sort_chunks(em, to_dev(M.T.ravel().copy()),
                               to_dev(oracle.chunk_idxs(R, L, True)))
    assert to_host(back).tobytes() == x.tobytes()


def test_sort_chunks_rejects_bad_splits_on_device():
    x = to_dev(wl.random_activation(1, (10, 64), "bf16"))
    sentinel = torch.full_like(x, 3.0)
    out = moe.moe_sort_chunks(x, to_dev(np.array([4, 4], np.int32)),
                              to_dev(np.array([1, 0], np.int32)), out=sentinel.clone())
    assert moe.moe_workspace_status(out._moe_workspace) == 6
    assert torch.equal(out, sentinel)
    out = moe.moe_sort_chunks(x, to_dev(np.array([4, 6], np.int32)),
                              to_dev(np.array([1, 1], np.int32)), out=sentinel.clone())
    assert moe.moe_workspace_status(out._moe_workspace) == 6


# ------------------------------------------------------------------ pipelines

def _pipeline_gpu(d, with_grad, weights=None):
    """The GPU chain; `weights` (host, [T,k]) replaces the route's own topk_w
    in the combine and backward, so they see the same inputs as the oracle."""
    w_ = d["workload"]
    r = moe.moe_route(to_dev(d["logits"]), w_.k)
    w = r.topk_w if weights is None else to_dev(weights)
    xp = moe.moe_permute(to_dev(d["x"]), r.slot_pos)
    y = moe.moe_expert_scale(xp, r.offsets, to_dev(d["scale"]))
    out = moe.moe_combine(y, r.slot_pos, w)
    res = {"r": r, "xp": xp, "y": y, "out": out}
    if with_grad:
        res["gy"], res["gp"] = moe.moe_combine_backward(to_dev(d["grad_out"]), y, r.slot_pos, w)
    torch.cuda.synchronize()
    return res


@pytest.mark.parametrize("name", ["tiny", "mid"])
def test_pipeline_full_compare(name):
    d = wl.make(name)
    w_ = d["workload"]
    g = _pipeline_gpu(d, with_grad=False)
    o = oracle.route(d["logits"], w_.k)
    _assert_route_equal(g["r"], o, w_.E)
    n = int(o["offsets"][w_.E])
    xp_o = oracle.permute(d["x"], o["sorted_indices"], n)
    assert to_host(g["xp"])[:n].tobytes() == xp_o.tobytes()
    y_o = oracle.expert_scale(xp_o, o["offsets"], d["scale"])
    assert to_host(g["y"])[:n].tobytes() == y_o.tobytes()
    out_o, out64 = oracle.combine(y_o, o["slot_pos"], o["topk_w"])
    got = to_host(g["out"])
    # the two sides used their own softmax weights (within 1e-6): 1 ulp
    if got.dtype == np.uint16:
        assert bf16_ulp_diff(got, out_o).max() <= 1
    else:
        assert within_one_bf16_ulp(got, out64).all()
    # round trip: the stand-in closed form out[t] = x[t] * sum_j w_j (e_j+1)/E.
    # Each stand-in row is rounded once (relative 2^-9 in bf16, 2^-24 in f32)
    # and the sum once more, so allow 2 ulps of the exact value.
    factor = (o["topk_w_f64"] * (o["topk_idx"] + 1) / w_.E).sum(axis=1)
    exact = wl.activation_to_f64(d["x"]) * factor[:, None]
    err = np.abs(wl.activation_to_f64(got) - exact)
    assert (err <= 2 * bf16_ulp_of(exact)).all()


def test_pipeline_skewed_sampled():
    """The DeepSeek-shaped workload at full size in the benchmark's launch
    configuration; the oracle checks every routing output and a seeded sample
    of tokens for the row outputs."""
    d = wl.make("skewed", with_grad=True)
    w_ = d["workload"]
    o = oracle.route(d["logits"], w_.k)
    # the combine and backward take the oracle's weights: identical inputs on
    # both sides (the route's own weights are checked within 1e-6 above)
    g = _pipeline_gpu(d, with_grad=True, weights=o["topk_w"])
    _assert_route_equal(g["r"], o, w_.E)
    counts = o["counts"]
    assert (counts == 0).sum() > 0 and counts.max() > 4 * w_.N / w_.E   # skewed as intended
    rng = np.random.default_rng(2024)
    toks = np.sort(rng.choice(w_.T, 256, replace=False))
    toks[-1] = w_.T - 1
    sp = o["slot_pos"][toks]
    rows = sp.ravel()
    xp = to_host(g["xp"][torch.from_numpy(rows).long().cuda()])
    assert (xp == d["x"][np.repeat(toks, w_.k)]).all()
    # the oracle's stand-in rows for the sample: each row its own segment,
    # scaled by its expert's factor
    experts = np.searchsorted(o["offsets"], rows, side="right") - 1
    y_o = oracle.expert_scale(np.ascontiguousarray(d["x"][np.repeat(toks, w_.k)]),
                              np.arange(rows.size + 1, dtype=np.int32),
                              np.ascontiguousarray(d["scale"][experts]))
    assert (to_host(g["y"][torch.from_numpy(rows).long().cuda()]) == y_o).all()
    w_o = np.ascontiguousarray(o["topk_w"][toks])
    sp_local = np.arange(toks.size * w_.k, dtype=np.int32).reshape(toks.size, w_.k)
    out_o, _ = oracle.combine(y_o, sp_local, w_o)
    assert (to_host(g["out"])[toks] == out_o).all()
    gy_o, gp_o, gp64 = oracle.combine_backward(np.ascontiguousarray(d["grad_out"][toks]), y_o,
                                               sp_local, w_o)
    assert (to_host(g["gy"][torch.from_numpy(rows).long().cuda()]) == gy_o).all()
    assert within_one_bf16_ulp(to_host(g["gp"])[toks], gp64).all()


@pytest.mark.parametrize("warm", [True, False])
@pytest.mark.parametrize("between", ["nothing", "zeros", "noise", "the same image", "an eager call",
                                     "the layer's meeting"])
@pytest.mark.parametrize("T,E,k", [(4096, 256, 8), (300, 64, 6)])
def test_route_replayed_with_other_logits(T, E, k, between, warm):
    """A captured route repeats its barrier's tag: what a replay leaves in the workspace,
    or what another writer puts there after every replay, must not let the next one
    through before all blocks have counted.  Every replay has other logits."""
    rng = np.random.default_rng(T)
    hot = rng.permutation(E)
    sets = []
    for i in range(6):                                     # the experts' shares move about
        lg = (rng.standard_normal((T, E)) + 3.0 * (hot == 0)[None, :] * (i % 2)
              + np.roll(np.linspace(0, 2, E), 40 * i)[None, :]).astype(np.float32)
        sets.append((to_dev(lg), oracle.route(lg, k)))
    nbytes = moe.moe_route_workspace_size(T, E, k)
    gen = torch.Generator(device="cuda").manual_seed(3)
    ws = torch.randint(0, 256, (nbytes,), dtype=torch.uint8, device="cuda", generator=gen)
    image = ws.clone()
    lg = sets[0][0].clone()
    moe.moe_device_status()
    if warm:
        moe.moe_route(lg, k, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = moe.moe_route(lg, k, workspace=ws, routing_map=True)
    for turn, (logits, o) in enumerate(sets + sets[::-1]):
        lg.copy_(logits)
        for t in (r.counts, r.offsets, r.sorted_indices, r.slot_pos):
            t.fill_(-7)
        graph.replay()
        torch.cuda.synchronize()
        _assert_route_equal(r, o, E)
        assert moe.moe_workspace_status(ws) == 0 and moe.moe_device_status() == 0
        if between == "zeros":
            ws.zero_()
        elif between == "noise":
            ws.copy_(torch.randint(0, 256, (nbytes,), dtype=torch.uint8, device="cuda", generator=gen))
        elif between == "the same image":
            ws.copy_(image)
        elif between == "an eager call":
            e = moe.moe_route(sets[turn % 6][0], k, workspace=ws, routing_map=True)
            _assert_route_equal(e, sets[turn % 6][1], E)
        elif between == "the layer's meeting":
            ws[:4096].fill_(turn & 1)


def test_route_replays_back_to_back():
    """Replays of two graphs over one workspace with nothing waited for in between: the
    last ones' results are the oracle's."""
    T, E, k = 2000, 128, 8
    rng = np.random.default_rng(9)
    ws = torch.zeros(moe.moe_route_workspace_size(T, E, k), dtype=torch.uint8, device="cuda")
    pairs = []
    for i in range(2):
        lg = (rng.standard_normal((T, E)) + np.roll(np.linspace(0, 3, E), 60 * i)[None, :]).astype(np.float32)
        d = to_dev(lg)
        moe.moe_route(d, k, workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            r = moe.moe_route(d, k, workspace=ws, routing_map=True)
        pairs.append((graph, r, oracle.route(lg, k), d))       # (a graph reads d where it is)
    moe.moe_device_status()
    for _ in range(50):
        for graph, _, _, _ in pairs:
            graph.replay()
    torch.cuda.synchronize()
    for _, r, o, _ in pairs:
        _assert_route_equal(r, o, E)
    assert moe.moe_device_status() == 0
