"""Routing tokens to experts and the experts' feed-forward block in fp64, token by token from their
definitions.

* Routing: scores s = softmax(l) or the logistic function of l; ranked by s + bias (ties: the lowest
  index), in groups by the sum of a group's two largest; weights s, over their sum where renormalised,
  times scale. Index -1: no expert (a padding token, or all that are left have logits of -inf).
* Experts: a slot's g | u = x gate_up_e, h = w a(g) u, its part of y h down_e; gradients from the kept
  g | u.
"""
from __future__ import annotations

import numpy as np

from .lm import gate


def scores(l, kind):
    """The scores of a row of logits (fp64)."""
    l = np.asarray(l, np.float64)
    if kind == "sigmoid":
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-l))
    top = l.max()
    if top == -np.inf:
        return np.zeros_like(l)
    e = np.exp(l - top)
    return e / e.sum()


def _best(values, names, most):
    """The names of the `most` largest values, best first, the lowest name first among equal ones."""
    return [n for _, n in sorted(zip((-v for v in values), names))][:most]


def route_forward(logits, top_k, kind="softmax", bias=None, groups=1, top_groups=1, renormalise=True, scale=1.0, live=None):
    """(index, weight, counts); logits finite or -inf."""
    logits = np.asarray(logits, np.float64)
    t, e = logits.shape
    index, weight = np.full((t, top_k), -1, np.int32), np.zeros((t, top_k))
    for r in range(t):
        if live is not None and not live[r]:
            continue
        s = scores(logits[r], kind)
        c = s if bias is None else s + np.asarray(bias, np.float64)
        names = [i for i in range(e) if logits[r, i] > -np.inf]
        if groups > 1:
            per = e // groups
            runs = [[i for i in names if i // per == g] for g in range(groups)]
            total = {g: sum(sorted((c[i] for i in m), reverse=True)[:2]) for g, m in enumerate(runs) if m}
            on = _best(total.values(), total.keys(), top_groups)
            names = [i for i in names if i // per in on]
        # without a bias the order is the logits' own: distinct logits may have one and the same score in fp64
        taken = _best([(logits[r] if bias is None else c)[i] for i in names], names, top_k)
        w = s[taken]
        if renormalise and len(taken):
            if kind == "sigmoid" and not w.sum() > 1e-290:  # e^l in place of it, where all are that small
                w = np.exp(logits[r, taken] - logits[r, taken].max())
            w = w / w.sum()
        index[r, :len(taken)], weight[r, :len(taken)] = taken, w * scale
    return index, weight, np.bincount(index[index >= 0], minlength=e).astype(np.int32)


def route_backward(logits, index, dweight, kind="softmax", renormalise=True, scale=1.0):
    """dlogits by the chain rule through the whole row's scores."""
    logits = np.asarray(logits, np.float64)
    out = np.zeros_like(logits)
    for r in range(len(logits)):
        on = index[r] >= 0
        if not on.any():
            continue
        taken, g = index[r][on], np.asarray(dweight, np.float64)[r][on] * scale
        s = scores(logits[r], kind)
        ds = np.zeros_like(s)
        w = s[taken]
        np.add.at(ds, taken, (g - (g * w).sum() / w.sum()) / w.sum() if renormalise else g)
        if kind == "sigmoid":
            out[r] = ds * s * (1.0 - s)
        else:  # renormalised weights do not change with a factor common to all scores: sum ds s is 0 exactly
            out[r] = s * (ds if renormalise else ds - (ds * s).sum())
    return out


def experts_forward(x, index, weight, w_gate_up, w_down, act):
    """(y, g | u by slots, sums of magnitudes): the parts' absolute values added up, and those of
    their products' terms."""
    x, wgu, wd = (np.asarray(a, np.float64) for a in (x, w_gate_up, w_down))
    t, k = index.shape
    f = wd.shape[1]
    y, gu = np.zeros((t, wd.shape[2])), np.zeros((t * k, 2 * f))
    size = np.zeros_like(y)
    for r in range(t):
        for j in range(k):
            e = index[r, j]
            if e < 0:
                continue
            z = x[r] @ wgu[e]
            h = float(weight[r, j]) * gate(z[:f], act)[0] * z[f:]
            part = h @ wd[e]
            gu[r * k + j] = z
            y[r] += part
            size[r] += np.abs(part) + np.abs(h) @ np.abs(wd[e])
    return y, gu, size


def experts_backward(dy, x, index, weight, kept, w_gate_up, w_down, act):
    """{name: (gradient, sums of its terms' magnitudes)} from the kept g | u."""
    dy, x, kept, wgu, wd = (np.asarray(a, np.float64) for a in (dy, x, kept, w_gate_up, w_down))
    t, k = index.shape
    f = wd.shape[1]
    out = {"dx": np.zeros_like(x), "dweight": np.zeros((t, k)), "dw_gate_up": np.zeros_like(wgu), "dw_down": np.zeros_like(wd)}
    size = {n: np.zeros_like(v) for n, v in out.items()}
    for r in range(t):
        for j in range(k):
            e = index[r, j]
            if e < 0:
                continue
            w, g, u = float(weight[r, j]), kept[r * k + j, :f], kept[r * k + j, f:]
            a, da = gate(g, act)
            dh = wd[e] @ dy[r]
            out["dweight"][r, j] = dh @ (a * u)
            size["dweight"][r, j] = (np.abs(wd[e]) @ np.abs(dy[r])) @ np.abs(a * u)
            dgu = w * np.concatenate((dh * u * da, dh * a))
            part = wgu[e] @ dgu
            out["dx"][r] += part
            size["dx"][r] += np.abs(part) + np.abs(wgu[e]) @ np.abs(dgu)
            for name, p, q in (("dw_gate_up", x[r], dgu), ("dw_down", w * a * u, dy[r])):
                out[name][e] += np.outer(p, q)
                size[name][e] += np.outer(np.abs(p), np.abs(q))
    return {n: (out[n], size[n]) for n in out}


# --------------------------------------------------------------------------- error bounds

def weight_bound(ref):
    """An fp32 weight or score's error: exponentials and divisions of 2^-22 each, their arguments'
    rounding (|l| below 64: 2^-18) and a sum of at most 1024 terms over 32 chains (37 roundings of 2^-24)."""
    return 2.0 ** -16 * np.abs(ref) + 1e-37


def block_bound(ref, size):
    """A bf16 result's error: its own rounding and, of each part's or term's magnitude, one more to
    bf16 (2^-8 each), an eighth of the two on top for the second order and the fp32 sums, as
    oracle.lm.product_bound has it."""
    return 1.125 * 2.0 ** -8 * (np.abs(ref) + size) + 1e-30


def dweight_bound(size, dim, hidden):
    """dweight is a sum over hidden of sums over dim in fp32, adds that may truncate (2^-23 each) over terms of
    `size` in all, with activations 64 units of 2^-24 off."""
    return (2 * dim + 2 * hidden + 64) * 2.0 ** -24 * size + 1e-30
