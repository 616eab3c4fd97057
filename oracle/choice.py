"""The experts that a row of logits chooses, in exact order: sums of scores and biases as decimal numbers of
140 digits, in which neither a score of e^-200 beside a bias of 3e38 nor the distance of two logistic scores
from 1 is lost."""
from __future__ import annotations

import decimal

import numpy as np

_DIGITS = decimal.Context(prec=140, Emin=-10 ** 6, Emax=10 ** 6)


def choose(logits, top_k, kind="softmax", bias=None, groups=1, top_groups=1):
    """index [rows, top_k], the best first, the lowest index (of experts, of runs) first among equal ones; logits
    finite, at most 100 in size where there are biases."""
    with decimal.localcontext(_DIGITS):
        return np.array([_row([float(x) for x in row], top_k, kind, bias, groups, top_groups) for row in logits], np.int32)


def _row(l, top_k, kind, bias, groups, top_groups):
    x = [decimal.Decimal(v) for v in l]
    if kind == "softmax":
        top = max(x)
        s = [(v - top).exp() for v in x]
        z = sum(s)
        s = [v / z for v in s]
    else:
        s = [1 / (1 + (-v).exp()) for v in x]
    c = s if bias is None else [v + decimal.Decimal(float(b)) for v, b in zip(s, bias)]
    names, per = range(len(c)), len(c) // groups
    if groups > 1:
        total = [sum(sorted(c[g * per:(g + 1) * per], reverse=True)[:2]) for g in range(groups)]
        on = sorted(range(groups), key=lambda g: (-total[g], g))[:top_groups]
        names = [i for i in names if i // per in on]
    return sorted(names, key=lambda i: (-c[i], i))[:top_k]
