"""A feed-forward block of many experts, as measured: the routing of tokens to experts and the
experts' gated products, each forward and backward.

``run`` computes them in plain torch operations in fp32 (rounded once at the end; the order in which
experts are chosen in fp64, where two scores may lie closer than fp32 tells apart), or, where ``own``
is true, through the package's entry points. ``exact`` gives the same results in fp64 from the
definitions, the gradients by automatic differentiation.

Routing, for a token's logits l over E experts: scores s = softmax(l) or the logistic function of
l; experts are ranked by s + bias (ties: the lowest index first). With groups, E is cut into equal
runs, a run's score is the sum of its two largest s + bias, and only the best ``top_groups`` runs'
experts take part. The first ``top_k`` are chosen; their weights are s (without the bias),
divided by their sum where renormalised, times ``scale``. A padding token has index -1 and weight 0
everywhere.

Experts: y_t = sum_j weight_tj (a(x_t Wgate) * (x_t Wup)) Wdown with the matrices of expert
index_tj, stored as [E, d, 2f] (gate columns first) and [E, f, d].
"""
import math

import torch

own = False

BLOCK = 128  # columns that share one power of two in an 8-bit checkpoint


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # one token of a decoding step: launch latency
        _route("route_one", 1, 64, 6),
        # a full micro-step, fine-grained experts in groups, logistic scores with a bias for balance
        _route("route_groups", 8192, 256, 8, score="sigmoid", bias=True, groups=8, top_groups=4, scale=2.5),
        # several sequences at once, logits as a bf16 product leaves them (many exact ties)
        _route("route_bf16", 32768, 128, 8, type="bf16"),
        # both directions of a padded batch, an odd number of experts, plain softmax weights (a dense gradient)
        _route("route_step_ragged", 4099, 60, 4, step=True, renorm=False, padding=True),
        # both directions of a large micro-step with a bias for balance
        _route("route_step_bias", 16384, 256, 8, step=True, score="sigmoid", bias=True),
        # one token through six of 64 experts: the chosen weights' bytes bound it
        _experts("experts_fwd_one", 1, 2048, 1408, 64, 6),
        # a decoding batch: nearly every expert is read for a few rows
        _experts("experts_fwd_batch", 48, 2048, 1408, 64, 6),
        # a full micro-step forward, gate and up kept in bf16
        _experts("experts_fwd_2048", 8192, 2048, 1408, 64, 6, keep="bf16"),
        # eight experts of the dense block's own width
        _experts("experts_fwd_wide", 4096, 2048, 5632, 8, 2),
        # the tiny decoder's widths, backward, gate and up kept in 8 bits
        _experts("experts_bwd_256", 1023, 256, 768, 8, 2, step=True, keep="e4m3"),
        # backward at widths that no tile divides, the other activation, a padded batch, kept in bf16
        _experts("experts_bwd_ragged", 1537, 1000, 683, 12, 3, step=True, keep="bf16", act="gelu", padding=True),
        # a full micro-step backward, gate and up kept in 8 bits
        _experts("experts_bwd_2048", 8192, 2048, 1408, 64, 6, step=True, keep="e4m3"),
    ]


def _route(name, tokens, experts, top_k, step=False, score="softmax", bias=False, groups=1, top_groups=1, renorm=True,
           scale=1.0, type="f32", padding=False):
    c = {"op": "route_step" if step else "route", "tokens": tokens, "experts": experts, "top_k": top_k, "score": score,
         "bias": bias, "groups": groups, "top_groups": top_groups, "renorm": renorm, "scale": scale, "type": type,
         "padding": padding}
    return c if name is None else {"name": name, **c}


def _experts(name, tokens, dim, hidden, experts, top_k, step=False, keep="none", act="silu", padding=False):
    c = {"op": "experts_bwd" if step else "experts_fwd", "tokens": tokens, "dim": dim, "hidden": hidden,
         "experts": experts, "top_k": top_k, "keep": keep, "act": act, "padding": padding}
    return c if name is None else {"name": name, **c}


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    padding = rng.random() < 0.3
    if rng.random() < 0.5:
        tokens, groups, top_groups = _log(rng, 1, 32768), 1, 1
        experts = rng.choice([_log(rng, 4, 512), rng.choice([8, 16, 64, 128, 256])])
        if rng.random() < 0.4:
            groups = rng.choice([2, 4, 8])
            top_groups = rng.randint(1, groups)
            experts = groups * max(2, experts // groups)
        experts, tokens = max(2, experts), max(1, min(tokens, (1 << 23) // experts))
        top_k = rng.randint(1, min(8, experts // groups * top_groups))
        return _route(None, tokens, experts, top_k, rng.random() < 0.5, rng.choice(["softmax", "sigmoid"]),
                      rng.random() < 0.5, groups, top_groups, top_k > 1 and rng.random() < 0.7, rng.choice([1.0, 2.5]),
                      rng.choice(["f32", "bf16"]), padding)
    step = rng.random() < 0.5
    dim = rng.choice([256, 768, 2048, 8 * _log(rng, 8, 256), _log(rng, 64, 2048)])
    hidden = rng.choice([768, 1408, 8 * _log(rng, 8, 704), _log(rng, 64, 5632)])
    experts = _log(rng, 2, 128)
    experts = max(2, min(experts, (64 * 2048 * 1408) // (dim * hidden)))
    top_k = rng.randint(1, min(8, experts))
    tokens = max(1, min(_log(rng, 1, 8192), 8192 * 6 * 2048 // (max(dim, hidden) * top_k), 8192 * 6 * 2048 * 1408 // (dim * hidden * top_k)))
    keep = rng.choice(["bf16", "e4m3"] if step else ["none", "bf16", "e4m3"])
    return _experts(None, tokens, dim, hidden, experts, top_k, step, keep, rng.choice(["silu", "gelu"]), padding)


def work(case):
    op, t, e, k = case["op"], case["tokens"], case["experts"], case["top_k"]
    if op in ("route", "route_step"):
        size = 2 if case["type"] == "bf16" else 4
        n = t * e * size + 8 * t * k + 4 * e + (4 * e if case["bias"] else 0) + (t if case["padding"] else 0)
        if op == "route":
            return {"bytes": n, "flops": 0}
        return {"bytes": n + 4 * t * k + t * e * size, "flops": 0}
    d, f = case["dim"], case["hidden"]
    used = e * (1.0 - (1.0 - k / e) ** t)  # experts that some token chooses
    weights = int(used * 2 * 3 * d * f)
    kept = {"none": 0, "bf16": 4 * t * k * f, "e4m3": 2 * t * k * f}[case["keep"]]
    fwd = 2 * 2 * t * d + 8 * t * k + weights + kept
    if op == "experts_fwd":
        return {"bytes": fwd, "flops": 6 * t * k * d * f}
    # x, dy, the routing, the weights and what was kept come in, dx, dweight and the gradients go out (an
    # expert that nobody chose has a gradient too: zeros)
    grads = 2 * 3 * e * d * f
    return {"bytes": 2 * 3 * t * d + 12 * t * k + weights + grads + kept, "flops": 12 * t * k * d * f}


# --------------------------------------------------------------------------- inputs

def _normal(g, shape, sigma=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * sigma).bfloat16()


def _live(case):
    """Which tokens are not padding: a batch padded at its end by a twentieth."""
    t = case["tokens"]
    return torch.arange(t, device="cuda") < t - (t // 20 if case["padding"] else 0)


def _inputs(case, seed):
    """The inputs alone (prepare adds the outputs and workspaces)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, t, e, k = case["op"], case["tokens"], case["experts"], case["top_k"]
    # a router part way through training: some experts are liked more than others
    logits = torch.randn((t, e), generator=g, device="cuda") + 0.3 * torch.randn((e,), generator=g, device="cuda")
    live = _live(case)
    if op in ("route", "route_step"):
        s = {"logits": logits.bfloat16() if case["type"] == "bf16" else logits,
             "bias": 0.02 * torch.randn((e,), generator=g, device="cuda") if case["bias"] else None,
             "live": live if case["padding"] else None}
        if op == "route_step":
            s["dweight"] = torch.randn((t, k), generator=g, device="cuda")
        return s
    d, f = case["dim"], case["hidden"]
    top, index = logits.topk(k, dim=1)
    s = {"x": _normal(g, (t, d)), "index": torch.where(live[:, None], index, -1).int(),
         "weight": torch.where(live[:, None], torch.softmax(top, dim=1), 0.0),
         "w_gate_up": _normal(g, (e, d, 2 * f), 1.0 / math.sqrt(d)), "w_down": _normal(g, (e, f, d), 1.0 / math.sqrt(f))}
    if op == "experts_bwd":
        s["dy"] = _normal(g, (t, d), 1e-3)
        s["gate_up"] = _normal(g, (t * k, 2 * f))  # the forward's, slot by slot (a token's j-th choice)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if "gate_up" in s:  # as the forward kept it
        gate_up = s.pop("gate_up")
        s["kept"] = _pack_8_bits(gate_up) if case["keep"] == "e4m3" else gate_up
    if not own:
        return s
    import zero_sharded_optimizer_flat_gb300 as Z
    op, t, e, k = case["op"], case["tokens"], case["experts"], case["top_k"]
    if op in ("route", "route_step"):
        s["index"] = torch.empty((t, k), dtype=torch.int32, device="cuda")
        s["weight"] = torch.empty((t, k), device="cuda")
        s["counts"] = torch.empty((e,), dtype=torch.int32, device="cuda")
        if op == "route_step":
            s["dlogits"] = torch.empty_like(s["logits"])
        return s
    rows, cols = t * k, 2 * case["hidden"]
    s["ws"] = Z.new_experts_workspace(s["x"], s["index"], s["w_gate_up"], s["w_down"], backward=op == "experts_bwd")
    if op == "experts_bwd":
        s["kept_own"] = Z.Act8(*s["kept"], parts=2) if case["keep"] == "e4m3" else s["kept"]
        s["dx"], s["dweight"] = torch.empty_like(s["x"]), torch.empty_like(s["weight"])
        s["dw_gate_up"], s["dw_down"] = torch.empty_like(s["w_gate_up"]), torch.empty_like(s["w_down"])
        return s
    s["y"] = torch.empty_like(s["x"])
    s["kept_own"] = None
    if case["keep"] != "none":  # (rows of padding tokens stay as they are)
        s["kept_values"] = s["kept_own"] = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    if case["keep"] == "e4m3":
        s["kept_own"] = Z.new_act8(rows, cols, parts=2)
        s["kept_own"].q.zero_()
        s["kept_own"].scale.zero_()
    return s


# --------------------------------------------------------------------------- one pass

def run(s):
    case = s["case"]
    if case["op"] in ("route", "route_step"):
        return (_route_own if own else _route_plain)(s, case)
    return (_experts_own if own else _experts_plain)(s, case)


def _route_own(s, case):
    import zero_sharded_optimizer_flat_gb300 as Z
    how = dict(score=case["score"], renormalise=case["renorm"], scale=case["scale"])
    Z.route_forward(s["logits"], s["index"], s["weight"], s["counts"], bias=s["bias"], live=s["live"], groups=case["groups"],
                    top_groups=case["top_groups"], **how)
    out = {"index": s["index"], "weight": s["weight"], "counts": s["counts"]}
    if case["op"] == "route_step":
        Z.route_backward(s["logits"], s["index"], s["weight"], s["dweight"], s["dlogits"], **how)
        out["dlogits"] = s["dlogits"]
    return out


def _experts_own(s, case):
    import zero_sharded_optimizer_flat_gb300 as Z
    if case["op"] == "experts_bwd":
        Z.experts_backward(s["dy"], s["x"], s["index"], s["weight"], s["kept_own"], s["w_gate_up"], s["w_down"], s["dx"],
                           s["dweight"], s["dw_gate_up"], s["dw_down"], s["ws"], act=case["act"])
        return {k: s[k] for k in ("dx", "dweight", "dw_gate_up", "dw_down")}
    Z.experts_forward(s["x"], s["index"], s["weight"], s["w_gate_up"], s["w_down"], s["y"], s["ws"], kept=s["kept_own"],
                      act=case["act"])
    if case["keep"] == "none":
        return {"y": s["y"]}
    if case["keep"] == "e4m3":
        Z.act_unpack(s["kept_own"], s["kept_values"])
    return {"y": s["y"], "kept": s["kept_values"]}


def _scores(l, score):
    if score == "sigmoid":
        return 1.0 / (1.0 + (-l).exp())
    p = (l - l.amax(dim=1, keepdim=True)).exp()
    return p / p.sum(dim=1, keepdim=True)


def _chosen(logits, bias, case):
    """The chosen experts of every row, best first, from scores in 64 bits."""
    c = _scores(logits.double(), case["score"])
    if bias is not None:
        c = c + bias.double()
    t, e, n = c.shape[0], case["experts"], case["groups"]
    if n > 1:
        runs = c.view(t, n, e // n)
        best = runs.sort(dim=2, descending=True, stable=True).values[:, :, :2].sum(dim=2)
        keep = best.sort(dim=1, descending=True, stable=True).indices[:, :case["top_groups"]]
        on = torch.zeros((t, n), dtype=torch.bool, device=c.device).scatter_(1, keep, True)
        c = runs.masked_fill(~on[:, :, None], -math.inf).view(t, e)
    return c.sort(dim=1, descending=True, stable=True).indices[:, :case["top_k"]]


def _route_plain(s, case):
    logits, live = s["logits"], s["live"]
    index = _chosen(logits, s["bias"], case)
    score = _scores(logits.float(), case["score"])
    weight = score.gather(1, index)
    total = weight.sum(dim=1, keepdim=True)
    if case["renorm"]:
        weight = weight / total
    out_weight = weight * case["scale"]
    out_index = index.int()
    if live is not None:
        out_weight = torch.where(live[:, None], out_weight, 0.0)
        out_index = torch.where(live[:, None], out_index, -1)
    counts = (out_index.reshape(-1, 1) == torch.arange(case["experts"], device="cuda")).sum(dim=0).int()
    out = {"index": out_index, "weight": out_weight, "counts": counts}
    if case["op"] == "route":
        return out
    g = s["dweight"] * case["scale"]
    if live is not None:
        g = torch.where(live[:, None], g, 0.0)
    if case["renorm"]:  # the gradient of the chosen scores
        g = (g - (g * weight).sum(dim=1, keepdim=True)) / total
    ds = torch.zeros_like(score).scatter_(1, index, g)
    if case["score"] == "sigmoid":
        dl = ds * score * (1.0 - score)
    else:
        dl = score * (ds - (ds * score).sum(dim=1, keepdim=True))
    out["dlogits"] = dl.to(logits.dtype)
    return out


def _pack_8_bits(x):
    """The 8-bit checkpoint of gate beside up: e4m3 bytes, and a power of two's byte for every block."""
    rows, cols = x.shape
    width = cols // 2
    blocks = -(-width // BLOCK)
    p = torch.nn.functional.pad(x.float().reshape(rows, 2, width), (0, blocks * BLOCK - width))
    p = p.reshape(rows, 2, blocks, BLOCK)
    m, k = torch.frexp(p.abs().amax(dim=3, keepdim=True))  # amax = m 2^k, 0.5 <= m < 1
    e = (k - 9 + (m > 0.875).to(k.dtype)).clamp(min=-126)
    q = torch.ldexp(p, -e).to(torch.float8_e4m3fn).reshape(rows, 2, -1)[:, :, :width].reshape(rows, cols)
    return q.contiguous().view(torch.uint8), (e + 127).to(torch.uint8).reshape(rows, 2 * blocks)


def _unpack_8_bits(q, scale):
    """The fp32 values that it stands for."""
    rows, cols = q.shape
    power = torch.ldexp(torch.ones((), device="cuda"), scale.int() - 127).reshape(rows, 2, -1)
    power = power.repeat_interleave(BLOCK, dim=2)[:, :, :cols // 2].reshape(rows, cols)
    return q.view(torch.float8_e4m3fn).float() * power


def _gate(z, act):
    """(a, a') of the activation a(z) = z sigmoid(phi(z))."""
    if act == "silu":
        phi, dphi = z, 1.0
    else:
        c = 2.0 * math.sqrt(2.0 / math.pi)
        phi, dphi = c * (z + 0.044715 * z * z * z), c * (1.0 + 3 * 0.044715 * z * z)
    s = torch.sigmoid(phi)
    return z * s, s + z * s * (1.0 - s) * dphi


def _experts_plain(s, case):
    t, k, e, d, f, act = (case[n] for n in ("tokens", "top_k", "experts", "dim", "hidden", "act"))
    # the slots (a token's j-th choice) expert by expert, each expert's row of them filled up with an empty one
    index = s["index"].reshape(-1)
    order = index.argsort(stable=True)
    order = order[(index < 0).sum():]
    used, which, count = index[order].unique(return_inverse=True, return_counts=True)
    slots = torch.full((used.numel(), int(count.max())), t * k, device="cuda")
    slots[which, torch.arange(order.numel(), device="cuda") - (count.cumsum(0) - count)[which]] = order

    def per_expert(rows, share):  # the rows of the slots, `share` slots to one row
        return torch.cat((rows.float(), torch.zeros_like(rows[:1], dtype=torch.float32)))[slots // share]

    def per_slot(rows):
        out = torch.zeros((t * k + 1, rows.shape[2]), device="cuda")
        out[slots] = rows
        return out[:-1]

    used = used.long()
    wgu, wd = s["w_gate_up"][used].float(), s["w_down"][used].float()
    x, w = per_expert(s["x"], k), per_expert(s["weight"].reshape(-1, 1), 1)
    if case["op"] == "experts_fwd":
        gu = x @ wgu
        h = _gate(gu[:, :, :f], act)[0] * gu[:, :, f:]
        out = {"y": per_slot(w * (h @ wd)).view(t, k, d).sum(dim=1).bfloat16()}
        if case["keep"] == "bf16":
            out["kept"] = per_slot(gu).bfloat16()
        elif case["keep"] == "e4m3":
            out["kept"] = _unpack_8_bits(*_pack_8_bits(per_slot(gu))).bfloat16()
        return out
    kept = s["kept"] if case["keep"] == "bf16" else _unpack_8_bits(*s["kept"])
    gu, dy = per_expert(kept, 1), per_expert(s["dy"], k)
    (a, da), u = _gate(gu[:, :, :f], act), gu[:, :, f:]
    dh = dy @ wd.transpose(1, 2)
    dweight = per_slot((dh * a * u).sum(dim=2, keepdim=True)).view(t, k)
    dgu = w * torch.cat((dh * u * da, dh * a), dim=2)
    dx = per_slot(dgu @ wgu.transpose(1, 2)).view(t, k, d).sum(dim=1).bfloat16()
    dw_gate_up, dw_down = torch.zeros_like(s["w_gate_up"]), torch.zeros_like(s["w_down"])
    dw_gate_up[used] = (x.transpose(1, 2) @ dgu).bfloat16()
    dw_down[used] = ((w * a * u).transpose(1, 2) @ dy).bfloat16()
    return {"dx": dx, "dweight": dweight, "dw_gate_up": dw_gate_up, "dw_down": dw_down}


# --------------------------------------------------------------------------- in 64 bits

def _exact_route(case, s):
    l, bias, live = s["logits"].double().requires_grad_(), s["bias"], s["live"]
    t, e, k = case["tokens"], case["experts"], case["top_k"]
    score = torch.softmax(l, dim=1) if case["score"] == "softmax" else torch.sigmoid(l)
    with torch.no_grad():
        rank = score if bias is None else score + bias.double()
        taken = torch.zeros((t, e), dtype=torch.bool, device="cuda")
        if case["groups"] > 1:  # the runs one after another, then the experts, each the best one left
            runs = rank.view(t, case["groups"], -1)
            first = runs.amax(dim=2)
            at = runs.argmax(dim=2, keepdim=True)
            second = runs.scatter(2, at, -math.inf).amax(dim=2)
            total = first + torch.where(second == -math.inf, 0.0, second)
            allowed = torch.zeros_like(total, dtype=torch.bool)
            for _ in range(case["top_groups"]):
                allowed.scatter_(1, _first_best(total.masked_fill(allowed, -math.inf)), True)
            taken |= ~allowed.repeat_interleave(e // case["groups"], dim=1)
        picks = []
        for _ in range(k):
            picks.append(_first_best(rank.masked_fill(taken, -math.inf)))
            taken.scatter_(1, picks[-1], True)
        index = torch.cat(picks, dim=1)
    weight = score.gather(1, index)
    if case["renorm"]:
        weight = weight / weight.sum(dim=1, keepdim=True)
    weight = weight * case["scale"]
    if live is not None:
        weight = weight * live[:, None]
        index = torch.where(live[:, None], index, -1)
    counts = torch.bincount(index.flatten() + 1, minlength=e + 1)[1:]
    out = {"index": index.int(), "weight": weight.detach(), "counts": counts.int()}
    if case["op"] == "route_step":
        out["dlogits"], = torch.autograd.grad((weight * s["dweight"].double()).sum(), l)
    return out


def _first_best(c):
    """The lowest column of every row's largest entry."""
    n = torch.arange(c.shape[1], device=c.device)
    return torch.where(c == c.amax(dim=1, keepdim=True), n, c.shape[1]).amin(dim=1, keepdim=True)


def _round_8_bits(x):
    """The 8-bit checkpoint's values of gate beside up, from the format: 3 mantissa bits, exponents
    down to 2^-6 (then a fixed step of 2^-9), the largest magnitude 448, times the block's power of two."""
    out = torch.empty_like(x)
    width = x.shape[1] // 2
    for p in range(2):
        for c in range(p * width, (p + 1) * width, BLOCK):
            b = x[:, c:min(c + BLOCK, (p + 1) * width)]
            top = b.abs().amax(dim=1, keepdim=True)
            e = torch.ceil(torch.log2(top / 448.0)).clamp(min=-126.0)
            e = torch.where(top > 0, e, 0.0)
            z = b / torch.exp2(e)
            step = torch.exp2(torch.floor(torch.log2(z.abs().clamp(min=2.0 ** -6))) - 3)
            out[:, c:c + b.shape[1]] = torch.round(z / step) * step * torch.exp2(e)
    return out


def _act64(z, act):
    if act == "silu":
        return torch.nn.functional.silu(z)
    return torch.nn.functional.gelu(z, approximate="tanh")


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] in ("route", "route_step"):
        return _exact_route(case, s)
    f, act, step, keep = case["hidden"], case["act"], case["op"] == "experts_bwd", case["keep"]
    x, index, weight = s["x"].double(), s["index"], s["weight"].double()
    zeros = lambda *shape: torch.zeros(shape, dtype=torch.float64, device="cuda")  # noqa: E731
    if step:
        dy, gu = s["dy"].double(), s["gate_up"].double()
        if keep == "e4m3":
            gu = _round_8_bits(gu)
        out = {"dx": zeros(*x.shape), "dweight": zeros(*weight.shape), "dw_gate_up": zeros(*s["w_gate_up"].shape),
               "dw_down": zeros(*s["w_down"].shape)}
    else:
        out = {"y": zeros(*x.shape)}
        if keep != "none":
            out["kept"] = zeros(weight.numel(), 2 * f)
    for i in range(case["experts"]):
        hit = index == i  # an expert is chosen at most once by a token
        rows = hit.any(dim=1).nonzero()[:, 0]
        if rows.numel() == 0:
            continue
        w, xi = weight[hit][:, None], x[rows]
        up, down = s["w_gate_up"][i].double(), s["w_down"][i].double()
        if not step:
            g = xi @ up
            out["y"][rows] += w * ((_act64(g[:, :f], act) * g[:, f:]) @ down)
            if keep != "none":
                out["kept"][hit.reshape(-1)] = g if keep == "bf16" else _round_8_bits(g)
            continue
        g = gu[hit.reshape(-1)].requires_grad_()
        w.requires_grad_()
        down.requires_grad_()
        loss = (w * ((_act64(g[:, :f], act) * g[:, f:]) @ down) * dy[rows]).sum()
        dgu, dw, dd = torch.autograd.grad(loss, (g, w, down))
        out["dx"][rows] += dgu @ up.t()
        out["dweight"][hit] = dw[:, 0]
        out["dw_gate_up"][i] = xi.t() @ dgu
        out["dw_down"][i] = dd
    return out
