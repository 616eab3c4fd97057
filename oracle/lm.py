"""The training operators in fp64: linear cross entropy, the gated feed-forward block and the 8-bit
activation checkpoint, from their definitions, plus the bound on a bf16 product's error that the
GPU tests hold the kernels to.

* Cross entropy: l = x w'; lse = log sum exp l; loss = lse - l[target]; gradient
  dl = (softmax(l) - onehot(target)) dloss; an ignored row's loss, lse and dl are zero and its x
  adds nothing to dw.
* Block: g | u = x gate_up, h = a(g) u, y = h down, with the gate's columns first
  (bluscript_zero_ckpt.cpp, model config: a gated SwiGLU block).
* Checkpoint: blocks of 128 columns, a power of two per block, e4m3 (3 mantissa bits, bias 7, no
  infinities, largest value 448, subnormals below 2^-6).
"""
from __future__ import annotations

import math

import numpy as np

# --------------------------------------------------------------------------- cross entropy


def ce_forward(x, w, target, ignore=-100):
    """(loss, lse) per row in fp64; 0 for ignored rows, NaN loss for a target out of range."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    loss, lse = np.zeros(len(x)), np.zeros(len(x))
    for t in range(len(x)):
        if target[t] == ignore:
            continue
        l = w @ x[t]
        top = l.max()
        lse[t] = top + math.log(np.exp(l - top).sum()) if np.isfinite(top) else top
        loss[t] = lse[t] - l[target[t]] if 0 <= target[t] < len(w) else np.nan
    return loss, lse


def ce_dlogits(x, w, target, lse, dloss, ignore=-100):
    """dl [T, V] in fp64 from the given lse."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    live = np.asarray(target) != ignore
    l = np.where(live[:, None], x, 0.0) @ w.T
    dl = np.exp(l - np.where(live, np.asarray(lse, np.float64), 0.0)[:, None])
    rows = np.nonzero(live)[0]
    dl[rows, np.asarray(target)[rows]] -= 1.0
    return dl * np.where(live, np.asarray(dloss, np.float64), 0.0)[:, None]


def ce_backward(x, w, target, lse, dloss, ignore=-100):
    """(dx, dw) in fp64."""
    dl = ce_dlogits(x, w, target, lse, dloss, ignore)
    xm = np.where((np.asarray(target) != ignore)[:, None], np.asarray(x, np.float64), 0.0)
    return dl @ np.asarray(w, np.float64), dl.T @ xm


# --------------------------------------------------------------------------- feed-forward block

def _logistic(z):
    return np.where(z >= 0, 1.0 / (1.0 + np.exp(-np.abs(z))), np.exp(-np.abs(z)) / (1.0 + np.exp(-np.abs(z))))


def gate(z, act):
    """(a(z), a'(z)) in fp64: "silu" z s(z), "gelu" z (1 + tanh(c (z + 0.044715 z^3))) / 2."""
    z = np.asarray(z, np.float64)
    if act == "silu":
        s = _logistic(z)
        return z * s, s * (1.0 + z * (1.0 - s))
    c = math.sqrt(2.0 / math.pi)
    t = np.tanh(c * (z + 0.044715 * z ** 3))
    return 0.5 * z * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)


def ffn_forward(x, w_gate_up, w_down, act):
    """(y, g | u, h) in fp64."""
    f = len(w_down)
    gu = np.asarray(x, np.float64) @ np.asarray(w_gate_up, np.float64)
    h = gate(gu[:, :f], act)[0] * gu[:, f:]
    return h @ np.asarray(w_down, np.float64), gu, h


def ffn_dgu(dy, kept, w_down, act):
    """(dg | du, h, dh) in fp64 from the kept g | u."""
    f = len(w_down)
    kept = np.asarray(kept, np.float64)
    g, u = kept[:, :f], kept[:, f:]
    a, da = gate(g, act)
    dh = np.asarray(dy, np.float64) @ np.asarray(w_down, np.float64).T
    return np.concatenate((dh * u * da, dh * a), axis=1), a * u, dh


def ffn_backward(dy, x, kept, w_gate_up, w_down, act):
    """(dx, dw_gate_up, dw_down) in fp64."""
    dgu, h, _ = ffn_dgu(dy, kept, w_down, act)
    return (dgu @ np.asarray(w_gate_up, np.float64).T, np.asarray(x, np.float64).T @ dgu,
            h.T @ np.asarray(dy, np.float64))


# --------------------------------------------------------------------------- 8-bit checkpoint

BLOCK = 128


def e4m3_values() -> np.ndarray:
    """What each of the 256 bytes stands for."""
    out = np.zeros(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        v = math.nan if (e, m) == (15, 7) else (m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
        out[b] = -v if b & 128 else v
    return out


def e4m3_bytes(z) -> np.ndarray:
    """The nearest finite e4m3 value's byte (ties to the even byte), by search over the format's
    values; NaN for what is not finite. |z| <= 448."""
    pos = e4m3_values()[:127]
    z = np.asarray(z, np.float64)
    a = np.minimum(np.abs(np.where(np.isfinite(z), z, 0.0)), 448.0)
    hi = np.clip(np.searchsorted(pos, a), 1, 126)
    lo = hi - 1
    dlo, dhi = a - pos[lo], pos[hi] - a
    pick = np.where((dlo < dhi) | ((dlo == dhi) & (lo % 2 == 0)), lo, hi)
    out = pick.astype(np.uint8) | (np.signbit(z).astype(np.uint8) << 7)
    return np.where(np.isfinite(z), out, 127).astype(np.uint8)


def act8_pack(x, parts=1):
    """(q, scale) bytes of a matrix, as zopt_act8 lays them out."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    width = cols // parts
    q, scale = np.zeros((rows, cols), np.uint8), []
    for p in range(parts):
        for c in range(p * width, (p + 1) * width, BLOCK):
            b = x[:, c:min(c + BLOCK, (p + 1) * width)]
            top = np.where(np.isfinite(b), np.abs(b), 0.0).max(axis=1)
            m, k = np.frexp(top)  # top = m 2^k, 1/2 <= m < 1: 2 m 2^(k-1)
            e = np.maximum(np.where(top > 0, k - 9 + (m > 0.875), -126), -126)
            q[:, c:c + b.shape[1]] = e4m3_bytes(b * 2.0 ** -e[:, None])
            scale.append((e + 127).astype(np.uint8))
    return q, np.stack(scale, axis=1) if scale else np.zeros((rows, 0), np.uint8)


def act8_unpack(q, scale, parts=1):
    """The fp64 values that (q, scale) stands for."""
    rows, cols = q.shape
    width = cols // parts
    nb = -(-width // BLOCK)
    s = 2.0 ** (np.asarray(scale).reshape(rows, parts, nb).astype(np.float64) - 127)
    s = np.repeat(s, BLOCK, axis=2)[:, :, :width].reshape(rows, cols)
    return e4m3_values()[q] * s


# --------------------------------------------------------------------------- error bounds

def product_bound(ref, abs_product):
    """What a bf16 result of a product may be off, entry by entry: its own rounding (bf16's
    unit roundoff, 2^-8 of the result) and the rounding of one operand to bf16 (2^-8 of each term,
    sum |p||q| = abs_product), with 1/8 on top of the two for the second order and for the fp32 sums
    and exponentials (K terms of 2^-24 each, adding as a random walk: below 2^-14 of abs_product up
    to K = 2^20, and operand errors of a few 2^-22)."""
    return 1.125 * 2.0 ** -8 * (np.abs(ref) + abs_product) + 1e-30
