"""The operators around a mixture-of-experts layer, as they are measured.

Four operators: the root-mean-square norm in front of the layer, with the
residual's addition (`norm`), the same norm with its output in e4m3 with a scale
for each block (`norm_fp8`), the norm's gradient (`norm_backward`), and the
whole layer for a few tokens, from the router's logits or its choices to the
combined rows (`layer`).  Every case is a dict of plain values; `own` selects
the framework's calls instead of the plain form.

  h = round(x + residual)          (as it is stored: h = x without a residual)
  y = h * r * weight,              r = 1 / sqrt(mean(h^2) + eps)
  e4m3: scale = max|y| / 448 over a block (1 for a block of zeros), code = e4m3(y / scale)
  gradient, with g = dL/dy and gh = dL/dh from the residual stream:
    grad_x = r * (g * weight) - h * r^3 * mean(g * weight * h) + gh
    grad_weight = sum over rows of g * h * r
  layer: out[t] = sum_j p[t,j] * (silu(x_t Wg[e]) * (x_t Wu[e])) Wd[e],  e = idx[t,j]
    idx = the k largest logits (equal ones: the lower id first), p = softmax over those k
"""
import math

import torch

own = False

EPS = 1e-6
_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f32": 4}

# The largest sizes that listed() has and draw() stays within.
_MOST_T, _MOST_H = 16384, 7168
_MOST_LAYER_T = 64


# ---------------------------------------------------------------- cases

def listed():
    bf = {"dtype": "bf16", "weight_dtype": "bf16"}
    return [
        # one token of a decode step: latency alone counts
        {"name": "norm token", "op": "norm", "T": 1, "H": 2048, "residual": True, **bf},
        # a long prefill of the widest rows
        {"name": "norm prefill", "op": "norm", "T": 16384, "H": 7168, "residual": True, **bf},
        # odd rows in float32 that no vector load fits, and no residual: a first layer's norm
        {"name": "norm odd f32", "op": "norm", "T": 777, "H": 1001, "residual": False,
         "dtype": "f32", "weight_dtype": "f32"},
        # a decode batch in front of an e4m3 dispatch
        {"name": "norm fp8 step", "op": "norm_fp8", "T": 32, "H": 7168, "block": 128,
         "residual": True, **bf},
        # a prefill in front of an e4m3 dispatch
        {"name": "norm fp8 prefill", "op": "norm_fp8", "T": 8192, "H": 4096, "block": 128,
         "residual": True, **bf},
        # a training step's norm with the gradient of the residual stream
        {"name": "norm backward", "op": "norm_backward", "T": 4096, "H": 2048, "residual": True,
         **bf},
        # the same for a long batch of the widest rows, weight kept in float32
        {"name": "norm backward long", "op": "norm_backward", "T": 16384, "H": 7168,
         "residual": True, "dtype": "bf16", "weight_dtype": "f32"},
        # short odd rows in float32
        {"name": "norm backward odd", "op": "norm_backward", "T": 300, "H": 137,
         "residual": False, "dtype": "f32", "weight_dtype": "f32"},
        # one token through a layer of 64 experts: six experts' weights are read
        {"name": "layer token", "op": "layer", "T": 1, "E": 64, "k": 6, "H": 2048, "I": 1408,
         "fp8": False, "given": False},
        # a decode batch whose choices come from a router of the user's, with padded slots
        {"name": "layer given", "op": "layer", "T": 16, "E": 64, "k": 6, "H": 2048, "I": 1408,
         "fp8": False, "given": True},
        # a few tokens in e4m3 (speculative steps) over wider rows, two experts each
        {"name": "layer fp8", "op": "layer", "T": 7, "E": 64, "k": 2, "H": 4096, "I": 2048,
         "fp8": True, "given": False},
        # the most tokens over 256 experts of the widest rows
        {"name": "layer wide", "op": "layer", "T": 64, "E": 256, "k": 8, "H": 7168, "I": 2048,
         "fp8": False, "given": False},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "norm_fp8", "norm_backward", "layer", "layer"))
    if op == "layer":
        E = rng.choice((8, 16, 24, 64, 128, 256))
        return {"op": op, "T": _log(rng, 1, _MOST_LAYER_T), "E": E, "k": rng.randint(1, 8),
                "H": 256 * _log(rng, 1, _MOST_H // 256), "I": 128 * _log(rng, 1, 16),
                "fp8": rng.random() < 0.4, "given": rng.random() < 0.4}
    case = {"op": op, "T": _log(rng, 1, _MOST_T), "H": _log(rng, 8, _MOST_H),
            "residual": rng.random() < 0.6, "dtype": rng.choice(("bf16", "bf16", "f32")),
            "weight_dtype": rng.choice(("bf16", "f32"))}
    if case["dtype"] == "f32":                      # the bytes of the largest listed case
        case["T"] = min(case["T"], _MOST_T // 2)
    if op == "norm_fp8":
        case["block"] = rng.choice((32, 64, 128, 256))
        case["H"] = case["block"] * _log(rng, 1, _MOST_H // case["block"])
    elif rng.random() < 0.5:                        # half of the rows fit 16-byte vectors
        case["H"] = max(8, case["H"] // 8 * 8)
    return case


def _active(case):
    """Experts that the tokens' random choices reach, on average."""
    T, k = case["T"], case["k"]
    if case["given"]:                               # a tenth of the slots is empty, and the last row
        T, k = max(1, T - 1), 0.9 * k
    return case["E"] * (1.0 - (1.0 - k / case["E"]) ** T)


def work(case):
    T, H = case["T"], case["H"]
    if case["op"] == "layer":
        E, k, I = case["E"], case["k"], case["I"]
        slots = T * k
        bytes_ = _active(case) * 3 * H * I * 2 + T * H * (1 + 2)
        bytes_ += T * H / 128 * 4 if case["fp8"] else T * H
        bytes_ += slots * 8 + (0 if case["given"] else T * E * 4)
        return {"bytes": bytes_, "flops": 2.0 * slots * 3 * H * I}
    el, wel = _BYTES[case["dtype"]], _BYTES[case["weight_dtype"]]
    if case["op"] == "norm_backward":
        rows = 3 + int(case["residual"])            # g, h (and gh) in, grad_x out
        return {"bytes": T * H * rows * el + H * (wel + 4), "flops": 12.0 * T * H}
    bytes_ = T * H * el * (3 if case["residual"] else 1) + H * wel
    bytes_ += T * H * (1 + 4.0 / case["block"]) if case["op"] == "norm_fp8" else T * H * el
    return {"bytes": bytes_, "flops": 5.0 * T * H}


# --------------------------------------------------------------- inputs

def _rows(g, T, H, dtype):
    """Rows of a residual stream: unit normals with a few channels far larger."""
    x = torch.randn((T, H), generator=g, device="cuda")
    x[:, torch.randint(0, H, (max(1, H // 256),), generator=g, device="cuda")] *= 16.0
    return x.to(_TYPES[dtype])


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T, H = case["T"], case["H"]
    s = {"case": dict(case)}
    if case["op"] == "layer":
        E, k, I = case["E"], case["k"], case["I"]
        x = torch.randn((T, H), generator=g, device="cuda")
        if case["fp8"]:                             # as a quantizing norm or a dispatch leaves it
            blocks = x.view(T, H // 128, 128)
            scales = blocks.abs().amax(-1) / 448.0
            s["x"] = (blocks / scales[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(T, H)
            s["x_scales"] = scales.contiguous()
        else:
            s["x"] = x.to(torch.bfloat16)
        # packed once when the model is loaded: [E,2I,H] with rows in blocks of
        # 128 gate rows and the matching 128 up rows, and [E,H,I]
        s["w_up"] = torch.empty((E, 2 * I, H), dtype=torch.bfloat16, device="cuda")
        s["w_up"].normal_(0.0, H ** -0.5, generator=g)
        s["w_down"] = torch.empty((E, H, I), dtype=torch.bfloat16, device="cuda")
        s["w_down"].normal_(0.0, I ** -0.5, generator=g)
        # a router in bf16: equal logits occur
        logits = torch.randn((T, E), generator=g, device="cuda").to(torch.bfloat16).float()
        if case["given"]:
            idx = torch.argsort(logits, dim=1, descending=True, stable=True)[:, :k].contiguous()
            p = torch.rand((T, k), generator=g, device="cuda") + 0.05
            empty = torch.rand((T, k), generator=g, device="cuda") < 0.1
            if T > 1:
                empty[T - 1] = True                 # a padded row of the batch
            empty[0, 0] = False
            s["topk_idx"] = torch.where(empty, -1, idx).to(torch.int32)
            s["topk_w"] = p / p.sum(1, keepdim=True)
        else:
            s["logits"] = logits
        return s
    s["weight"] = (1.0 + 0.1 * torch.randn((H,), generator=g, device="cuda")).to(
        _TYPES[case["weight_dtype"]])
    s["x"] = _rows(g, T, H, case["dtype"])
    if case["op"] == "norm_backward":
        s["grad"] = torch.randn((T, H), generator=g, device="cuda").to(_TYPES[case["dtype"]])
        if case["residual"]:
            s["grad_h"] = torch.randn((T, H), generator=g, device="cuda").to(_TYPES[case["dtype"]])
    elif case["residual"]:
        s["residual"] = _rows(g, T, H, case["dtype"])
    return s


# --------------------------------------------------------- the operators

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    import unpermute_combine_gb300 as moe
    case = s["case"]
    if case["op"] == "norm":
        return moe.moe_rmsnorm(s["x"], s["weight"], residual=s.get("residual"), eps=EPS)
    if case["op"] == "norm_fp8":
        return moe.moe_rmsnorm_quantize_fp8(s["x"], s["weight"], residual=s.get("residual"),
                                            eps=EPS, block=case["block"])
    if case["op"] == "norm_backward":
        return moe.moe_rmsnorm_backward(s["grad"], s["x"], s["weight"], grad_h=s.get("grad_h"),
                                        eps=EPS)
    if case["given"]:
        return moe.moe_layer_decode_indices(s["x"], s["topk_idx"], s["topk_w"], s["w_up"],
                                            s["w_down"], x_scales=s.get("x_scales"))
    return moe.moe_layer_decode(s["x"], s["logits"], case["k"], s["w_up"], s["w_down"],
                                x_scales=s.get("x_scales"))


def _run_plain(s):
    case = s["case"]
    return {"norm": _norm, "norm_fp8": _norm_fp8, "norm_backward": _norm_backward,
            "layer": _layer}[case["op"]](s)


def _normed(s):
    x, res = s["x"], s.get("residual")
    h = x if res is None else (x.float() + res.float()).to(x.dtype)
    hf = h.float()
    return hf * torch.rsqrt(hf.square().mean(1, keepdim=True) + EPS) * s["weight"].float(), h


def _norm(s):
    y, h = _normed(s)
    return y.to(s["x"].dtype), h


def _norm_fp8(s):
    y, h = _normed(s)
    blocks = y.view(y.shape[0], -1, s["case"]["block"])
    amax = blocks.abs().amax(-1)
    scales = torch.where(amax > 0, amax / 448.0, 1.0)
    q = (blocks / scales[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q.view(y.shape), scales, h


def _norm_backward(s):
    g, h, w = s["grad"].float(), s["x"].float(), s["weight"].float()
    r = torch.rsqrt(h.square().mean(1, keepdim=True) + EPS)
    gw = g * w
    grad = r * gw - h * (r * r * r * (gw * h).mean(1, keepdim=True))
    if "grad_h" in s:
        grad = grad + s["grad_h"].float()
    return grad.to(s["x"].dtype), (g * (h * r)).sum(0)


def _layer(s):
    case, x = s["case"], s["x"]
    T, E, k, H, I = (case[n] for n in ("T", "E", "k", "H", "I"))
    xf = x.float()
    if case["fp8"]:
        xf = (xf.view(T, -1, 128) * s["x_scales"][..., None]).view(T, -1)
    if case["given"]:
        idx, p = s["topk_idx"].long(), s["topk_w"]
    else:
        top, idx = torch.sort(s["logits"], dim=1, descending=True, stable=True)
        idx, e = idx[:, :k], torch.exp(top[:, :k] - top[:, :1])
        p = e / e.sum(1, keepdim=True)
    # share[t, e]: the weight that token t gives expert e; only experts that a token chose are read
    share = torch.zeros((T, E), device=x.device)
    share.scatter_add_(1, idx.clamp(min=0), torch.where(idx < 0, 0.0, p))
    active = torch.unique(idx[idx >= 0])
    up = s["w_up"][active].float().view(len(active), I // 128, 2, 128, H)
    gate, up = up[:, :, 0].reshape(len(active), I, H), up[:, :, 1].reshape(len(active), I, H)
    a, b = xf @ gate.transpose(1, 2), xf @ up.transpose(1, 2)       # [active, T, I]
    hidden = a / (1.0 + torch.exp(-a)) * b
    hidden = hidden * share[:, active].t()[:, :, None]
    out = (hidden @ s["w_down"][active].float().transpose(1, 2)).sum(0).to(torch.bfloat16)
    return out if case["given"] else (out, idx.to(torch.int32), p)


# ----------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "layer":
        return _exact_layer(case, s)
    w, x = s["weight"].double(), s["x"]
    T, H = x.shape
    if case["op"] == "norm_backward":
        gx = torch.empty((T, H), dtype=torch.float64, device="cuda")
        gw = torch.zeros((H,), dtype=torch.float64, device="cuda")
        for a in range(0, T, 1024):
            h, g = x[a:a + 1024].double(), s["grad"][a:a + 1024].double()
            ms = (h * h).sum(1, keepdim=True) / H + EPS
            n = h / ms.sqrt()                                       # the normed row
            gw += (g * n).sum(0)
            v = g * w
            gx[a:a + 1024] = (v - n * (v * n).sum(1, keepdim=True) / H) / ms.sqrt()
            if case["residual"]:
                gx[a:a + 1024] += s["grad_h"][a:a + 1024].double()
        return gx, gw
    h = torch.empty_like(x)
    y = torch.empty((T, H), dtype=torch.float64, device="cuda")
    for a in range(0, T, 1024):
        v = x[a:a + 1024].double()
        if case["residual"]:
            v = (v + s["residual"][a:a + 1024].double()).to(x.dtype).double()
        h[a:a + 1024] = v.to(x.dtype)
        y[a:a + 1024] = v / ((v * v).sum(1, keepdim=True) / H + EPS).sqrt() * w
    if case["op"] == "norm":
        return y, h.double()
    b = y.view(T, H // case["block"], case["block"])
    top = b.abs().amax(2)
    scales = torch.where(top == 0, torch.ones_like(top), top / 448.0)
    return (b / scales[:, :, None]).view(T, H), scales, h.double()


def _exact_layer(case, s):
    T, E, k, H, I = (case[n] for n in ("T", "E", "k", "H", "I"))
    x = s["x"].float().double()
    if case["fp8"]:
        x = x * s["x_scales"].double().repeat_interleave(128, dim=1)
    if case["given"]:
        idx, p = s["topk_idx"].long().cpu(), s["topk_w"].double()
    else:
        # one choice after another, the largest first; argmax on the host keeps the first of equals
        left = s["logits"].double().cpu().numpy().copy()
        idx = torch.empty((T, k), dtype=torch.long)
        for j in range(k):
            best = left.argmax(1)
            idx[:, j] = torch.from_numpy(best)
            left[range(T), best] = -math.inf
        p = torch.softmax(torch.gather(s["logits"].double(), 1, idx.cuda()), dim=1)
    out = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    for e in range(E):
        t, j = (idx == e).nonzero(as_tuple=True)
        if not len(t):
            continue
        t, j = t.cuda(), j.cuda()
        rows = s["w_up"][e].view(I // 128, 2, 128, H)
        g = x[t] @ rows[:, 0].reshape(I, H).double().t()
        u = x[t] @ rows[:, 1].reshape(I, H).double().t()
        y = (g * torch.sigmoid(g) * u) @ s["w_down"][e].double().t()
        out.index_add_(0, t, y * p[t, j][:, None])
    return out if case["given"] else (out, idx.to(torch.int32).cuda(), p)
