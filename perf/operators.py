"""The training operators next to the optimizer step, as measured: the linear cross entropy over a
vocabulary, the gated feed-forward block and the 8-bit activation checkpoints.

``run`` computes them in plain torch operations in fp32 (rounded once at the end), or, where ``own``
is true, through the package's entry points. ``exact`` gives the same results in fp64 from the
definitions, the gradients by automatic differentiation.

A linear layer's weight is stored as the optimizer's parameter sets store it: the vocabulary matrix
[V, D], ``gate_up`` [d, 2f] (gate columns first), ``down`` [f, d]. Activations are bf16 rows.
"""
import math

import torch

own = False

BLOCK = 128  # columns that share one power of two in an 8-bit checkpoint


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # one token of a tiny decoder: launch latency
        {"name": "ce_fwd_one", "op": "ce_fwd", "tokens": 1, "dim": 256, "vocab": 4096},
        # a micro-step's loss under the 768-wide tied embedding
        {"name": "ce_fwd_768", "op": "ce_fwd", "tokens": 4096, "dim": 768, "vocab": 50304},
        # a short ragged batch, a vocabulary that no tile divides
        {"name": "ce_bwd_ragged", "op": "ce_bwd", "tokens": 777, "dim": 768, "vocab": 50177},
        # a full micro-step under the 2048-wide head
        {"name": "ce_bwd_2048", "op": "ce_bwd", "tokens": 8192, "dim": 2048, "vocab": 32000},
        # one token through the block: the weights' bytes bound it
        {"name": "ffn_fwd_one", "op": "ffn_fwd", "tokens": 1, "dim": 2048, "hidden": 5632, "act": "silu", "keep": "none"},
        # a full micro-step forward, gate and up kept in bf16
        {"name": "ffn_fwd_2048", "op": "ffn_fwd", "tokens": 8192, "dim": 2048, "hidden": 5632, "act": "silu", "keep": "bf16"},
        # the tiny decoder's block, both directions, everything kept in 8 bits
        {"name": "ffn_step_256", "op": "ffn_step", "tokens": 1023, "dim": 256, "hidden": 768, "act": "silu", "keep": "e4m3"},
        # widths that no tile divides, the other activation, kept in bf16
        {"name": "ffn_step_ragged", "op": "ffn_step", "tokens": 1537, "dim": 1000, "hidden": 2732, "act": "gelu", "keep": "bf16"},
        # a full micro-step, both directions, everything kept in 8 bits
        {"name": "ffn_step_2048", "op": "ffn_step", "tokens": 8192, "dim": 2048, "hidden": 5632, "act": "silu", "keep": "e4m3"},
        # a few rows: launch latency of pack and unpack
        {"name": "act8_small", "op": "act8", "tokens": 33, "cols": 256, "parts": 1},
        # the block inputs of a full micro-step
        {"name": "act8_2048", "op": "act8", "tokens": 16384, "cols": 2048, "parts": 1},
        # gate and up of an odd number of tokens, each half with blocks of its own, ragged widths
        {"name": "act8_pair", "op": "act8", "tokens": 4099, "cols": 11240, "parts": 2},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ce_fwd", "ce_bwd", "ffn_fwd", "ffn_step", "act8"])
    tokens = _log(rng, 1, 8192)
    if op in ("ce_fwd", "ce_bwd"):
        dim = rng.choice([256, 768, 2048, 8 * _log(rng, 8, 256), _log(rng, 64, 2048)])
        return {"op": op, "tokens": tokens, "dim": dim, "vocab": min(_log(rng, 1000, 50304), 65536000 // dim)}
    if op == "act8":
        parts = rng.choice([1, 2])
        return {"op": op, "tokens": tokens, "cols": parts * _log(rng, 64, 5632), "parts": parts}
    dim = rng.choice([256, 2048, 8 * _log(rng, 8, 256), _log(rng, 64, 2048)])
    hidden = rng.choice([768, 5632, 8 * _log(rng, 8, 704), _log(rng, 64, 5632)])
    keep = rng.choice(["none", "bf16"] if op == "ffn_fwd" else ["bf16", "e4m3"])
    return {"op": op, "tokens": tokens, "dim": dim, "hidden": hidden, "act": rng.choice(["silu", "gelu"]), "keep": keep}


def work(case):
    op, t = case["op"], case["tokens"]
    if op == "act8":  # pack reads 2 bytes and writes 1, unpack reads 1 and writes 2; and the scales
        n = t * case["cols"]
        s = t * case["parts"] * -(-(case["cols"] // case["parts"]) // BLOCK)
        return {"bytes": 6 * n + 2 * s, "flops": 0}
    d = case["dim"]
    if op in ("ce_fwd", "ce_bwd"):
        v = case["vocab"]
        read = 2 * t * d + 2 * v * d + 8 * t
        if op == "ce_fwd":
            return {"bytes": read + 8 * t, "flops": 2 * t * v * d}
        return {"bytes": read + 8 * t + 2 * t * d + 2 * v * d, "flops": 6 * t * v * d}
    f = case["hidden"]
    weights = 2 * 3 * d * f
    kept = {"none": 0, "bf16": 4 * t * f, "e4m3": 2 * t * f}[case["keep"]]
    fwd = {"bytes": 2 * 2 * t * d + weights + kept, "flops": 6 * t * d * f}
    if op == "ffn_fwd":
        return fwd
    # both directions: x, dy, the weights and what was kept come in, y, dx and the gradients go out
    return {"bytes": 2 * 4 * t * d + 2 * weights + 2 * kept, "flops": 18 * t * d * f}


# --------------------------------------------------------------------------- inputs

def _normal(g, shape, sigma=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * sigma).bfloat16()


def _bf16(*shape):
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda")


def _u8(*shape):
    return torch.empty(shape, dtype=torch.uint8, device="cuda")


def _inputs(case, seed):
    """The inputs alone (prepare adds the outputs and workspaces)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, t = case["op"], case["tokens"]
    if op == "act8":
        # activations: heavy-tailed rows, a few columns much larger than the others
        x = torch.randn((t, case["cols"]), generator=g, device="cuda")
        x *= torch.exp(torch.randn((t, 1), generator=g, device="cuda"))
        x[:, :: 97] *= 30.0
        return {"x": x.bfloat16()}
    d = case["dim"]
    if op in ("ce_fwd", "ce_bwd"):
        v = case["vocab"]
        w = _normal(g, (v, d), 0.04)
        target = torch.randint(0, v, (t,), generator=g, device="cuda")
        # a model part way through training: each token's state leans towards its target by up to a few nats
        wt = w[target].float()
        lean = 8.0 * torch.rand((t, 1), generator=g, device="cuda") / wt.square().sum(1, keepdim=True)
        x = (torch.randn((t, d), generator=g, device="cuda") + lean * wt).bfloat16()
        drop = torch.rand((t,), generator=g, device="cuda") < 0.05  # prompt and padding tokens carry no loss
        if t > 1:
            target = torch.where(drop, -100, target)
        s = {"x": x, "w": w, "target": target}
        if op == "ce_bwd":
            valid = target >= 0
            s["lse"] = torch.where(valid, torch.logsumexp(x.float() @ w.float().t(), dim=1), 0.0)
            s["dloss"] = valid.float() / valid.sum().clamp(min=1)
        return s
    f = case["hidden"]
    s = {"x": _normal(g, (t, d)), "w_gate_up": _normal(g, (d, 2 * f), 1.0 / math.sqrt(d)),
         "w_down": _normal(g, (f, d), 1.0 / math.sqrt(f))}
    if op == "ffn_step":
        s["dy"] = _normal(g, (t, d), 1e-3)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    op, t = case["op"], case["tokens"]
    if own:
        import zero_sharded_optimizer_flat_gb300 as Z
    if op == "act8":
        if own:
            s["packed"] = Z.new_act8(t, case["cols"], parts=case["parts"])
            s["out"] = _bf16(t, case["cols"])
        return s
    d = case["dim"]
    if op in ("ce_fwd", "ce_bwd"):
        if own:
            s["ws"] = Z.new_linear_ce_workspace(s["x"], s["w"], backward=op == "ce_bwd")
            if op == "ce_fwd":
                s["loss"] = torch.empty(t, device="cuda")
                s["lse"] = torch.empty(t, device="cuda")
            else:
                s["dx"], s["dw"] = _bf16(t, d), _bf16(case["vocab"], d)
        return s
    f = case["hidden"]
    if own:
        s["y"] = _bf16(t, d)
        s["kept"] = {"none": lambda: None, "bf16": lambda: _bf16(t, 2 * f),
                     "e4m3": lambda: Z.new_act8(t, 2 * f, parts=2)}[case["keep"]]()
        s["x8"] = Z.new_act8(t, d) if case["keep"] == "e4m3" else None
        s["ws"] = Z.new_ffn_workspace(s["x"] if s["x8"] is None else s["x8"], s["w_gate_up"], s["w_down"],
                                      backward=op == "ffn_step")
        if op == "ffn_step":
            s["dx"], s["dw_gate_up"], s["dw_down"] = _bf16(t, d), _bf16(d, 2 * f), _bf16(f, d)
    return s


# --------------------------------------------------------------------------- one pass

def run(s):
    case = s["case"]
    return (_run_own if own else _run_plain)(s, case, case["op"])


def _run_own(s, case, op):
    import zero_sharded_optimizer_flat_gb300 as Z
    if op == "act8":
        Z.act_pack(s["x"], s["packed"])
        Z.act_unpack(s["packed"], s["out"])
        return s["out"]
    if op == "ce_fwd":
        Z.linear_ce_forward(s["x"], s["w"], s["target"], s["loss"], s["lse"], s["ws"])
        return {"loss": s["loss"], "lse": s["lse"]}
    if op == "ce_bwd":
        Z.linear_ce_backward(s["x"], s["w"], s["target"], s["lse"], s["dloss"], s["dx"], s["dw"], s["ws"])
        return {"dx": s["dx"], "dw": s["dw"]}
    act, x8, kept = case["act"], s["x8"], s["kept"]
    Z.ffn_forward(s["x"], s["w_gate_up"], s["w_down"], s["y"], s["ws"], kept=kept, act=act)
    if op == "ffn_fwd":
        return {"y": s["y"]} if kept is None else {"y": s["y"], "kept": kept}
    if x8 is not None:
        Z.act_pack(s["x"], x8)
    Z.ffn_backward(s["dy"], s["x"] if x8 is None else x8, kept, s["w_gate_up"], s["w_down"], s["dx"],
                   s["dw_gate_up"], s["dw_down"], s["ws"], act=act)
    return {"y": s["y"], "dx": s["dx"], "dw_gate_up": s["dw_gate_up"], "dw_down": s["dw_down"]}


def _through_8_bits(x, parts=1):
    """The fp32 values that the 8-bit checkpoint of x stands for."""
    rows, cols = x.shape
    width = cols // parts
    blocks = -(-width // BLOCK)
    p = torch.nn.functional.pad(x.reshape(rows * parts, width), (0, blocks * BLOCK - width))
    p = p.reshape(rows * parts, blocks, BLOCK)
    m, k = torch.frexp(p.abs().amax(dim=2, keepdim=True))  # amax = m 2^k, 0.5 <= m < 1
    e = (k - 9 + (m > 0.875).to(k.dtype)).clamp(min=-126)
    q = torch.ldexp(p, -e).to(torch.float8_e4m3fn).float()
    return torch.ldexp(q, e).reshape(rows * parts, blocks * BLOCK)[:, :width].reshape(rows, cols)


def _gate(z, act):
    """(a, a') of the activation a(z) = z sigmoid(phi(z))."""
    if act == "silu":
        phi, dphi = z, 1.0
    else:
        c = 2.0 * math.sqrt(2.0 / math.pi)
        phi, dphi = c * (z + 0.044715 * z * z * z), c * (1.0 + 3 * 0.044715 * z * z)
    s = torch.sigmoid(phi)
    return z * s, s + z * s * (1.0 - s) * dphi


def _run_plain(s, case, op):
    x = s["x"].float()
    if op == "act8":
        return _through_8_bits(x, case["parts"]).bfloat16()
    if op in ("ce_fwd", "ce_bwd"):
        w, target = s["w"].float(), s["target"]
        valid = target >= 0
        at = target.clamp(min=0)[:, None]
        logits = x @ w.t()
        if op == "ce_fwd":
            top = logits.amax(dim=1)
            lse = top + (logits - top[:, None]).exp().sum(dim=1).log()
            loss = lse - logits.gather(1, at)[:, 0]
            return {"loss": torch.where(valid, loss, 0.0), "lse": torch.where(valid, lse, 0.0)}
        g = (logits - s["lse"][:, None]).exp()
        g.scatter_add_(1, at, torch.full_like(at, -1, dtype=torch.float32))
        g *= s["dloss"][:, None]
        g[~valid] = 0.0
        return {"dx": (g @ w).bfloat16(), "dw": (g.t() @ x).bfloat16()}
    wgu, wd, f, act = s["w_gate_up"].float(), s["w_down"].float(), case["hidden"], case["act"]
    gu = x @ wgu
    a, _ = _gate(gu[:, :f], act)
    y = ((a * gu[:, f:]) @ wd).bfloat16()
    if op == "ffn_fwd":
        return {"y": y} if case["keep"] == "none" else {"y": y, "kept": gu.bfloat16()}
    if case["keep"] == "e4m3":
        gu, x = _through_8_bits(gu, 2), _through_8_bits(x)
    else:
        gu = gu.bfloat16().float()
    g, u = gu[:, :f], gu[:, f:]
    a, da = _gate(g, act)
    dy = s["dy"].float()
    dh = dy @ wd.t()
    dgu = torch.cat((dh * u * da, dh * a), dim=1)
    return {"y": y, "dx": (dgu @ wgu.t()).bfloat16(), "dw_gate_up": (x.t() @ dgu).bfloat16(),
            "dw_down": ((a * u).t() @ dy).bfloat16()}


# --------------------------------------------------------------------------- in 64 bits

def _round_8_bits(x, parts=1):
    """The 8-bit checkpoint's values of a 64-bit matrix, from the format: 3 mantissa bits, exponents
    down to 2^-6 (then a fixed step of 2^-9), the largest magnitude 448, times the block's power of two."""
    out = torch.empty_like(x)
    width = x.shape[1] // parts
    for p in range(parts):
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
    op = case["op"]
    x = s["x"].double()
    if op == "act8":
        return _round_8_bits(x, case["parts"])
    if op in ("ce_fwd", "ce_bwd"):
        w, target = s["w"].double(), s["target"]
        valid = target >= 0
        if op == "ce_fwd":
            logp, lse = [], []
            for c in range(0, x.shape[0], 1024):
                l = x[c:c + 1024] @ w.t()
                lse.append(torch.logsumexp(l, dim=1))
                logp.append(torch.nn.functional.cross_entropy(l, target[c:c + 1024], reduction="none"))
            zero = torch.zeros((), dtype=torch.float64, device="cuda")
            return {"loss": torch.cat(logp), "lse": torch.where(valid, torch.cat(lse), zero)}
        dx, dw = torch.empty_like(x), torch.zeros_like(w)
        for c in range(0, x.shape[0], 2048):
            xc = x[c:c + 2048].requires_grad_()
            wc = w.detach().requires_grad_()
            loss = torch.nn.functional.cross_entropy(xc @ wc.t(), target[c:c + 2048], reduction="none")
            gx, gw = torch.autograd.grad((loss * s["dloss"][c:c + 2048].double()).sum(), (xc, wc))
            dx[c:c + 2048] = gx
            dw += gw
        return {"dx": dx, "dw": dw}
    f, act = case["hidden"], case["act"]
    wgu, wd = s["w_gate_up"].double(), s["w_down"].double()
    gu = x @ wgu
    y = (_act64(gu[:, :f], act) * gu[:, f:]) @ wd
    if op == "ffn_fwd":
        return {"y": y} if case["keep"] == "none" else {"y": y, "kept": gu}
    if case["keep"] == "e4m3":
        gu, xk = _round_8_bits(gu, 2), _round_8_bits(x)
    else:
        gu, xk = gu.bfloat16().double(), x
    gu.requires_grad_()
    wd.requires_grad_()
    dgu, dwd = torch.autograd.grad(((_act64(gu[:, :f], act) * gu[:, f:]) @ wd * s["dy"].double()).sum(), (gu, wd))
    return {"y": y, "dx": dgu @ wgu.t(), "dw_gate_up": xk.t() @ dgu, "dw_down": dwd}
