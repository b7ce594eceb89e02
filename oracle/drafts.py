"""CPU oracle for the verification of drafted tokens: whole numbers where it decides, one step per definition.

TEST INFRASTRUCTURE ONLY, like the rest of this package.
"""
from __future__ import annotations

import math
from fractions import Fraction

import numpy as np

UNIT = 149  # every fp32 and bf16 number, and every difference of two, is a whole multiple of 2^-149


def weight(x):
    """A number as a weight, in units of 2^-149: itself if it is positive and finite, else 0."""
    return int(math.ldexp(x, UNIT)) if math.isfinite(x) and x > 0 else 0


def verify(target, ids, u, cu, draft=None):
    """target, draft [tokens][vocab] float64 arrays of what the stored numbers stand for -> (accepted, next)."""
    accepted, after = [], []
    vocab = target.shape[1]
    for first, end in zip(cu[:-1], cu[1:]):
        if end <= first:
            accepted.append(0)
            after.append(-1)
            continue
        t = first
        while t + 1 < end:
            x = int(ids[t + 1])
            if not 0 <= x < vocab:
                break
            p, q, v = float(target[t, x]), 1.0 if draft is None else float(draft[t, x]), float(u[t])
            if not np.isfinite([p, q, v]).all():
                with np.errstate(invalid="ignore"):
                    if not np.float64(v) * np.float64(q) < np.float64(p):
                        break
            elif not Fraction(v) * Fraction(q) < Fraction(p):
                break
            t += 1
        with np.errstate(invalid="ignore"):
            w = np.array(target[t], dtype=np.float64)
            if t + 1 < end:
                if draft is None:
                    if 0 <= ids[t + 1] < vocab:
                        w[ids[t + 1]] = 0.0
                else:
                    w = w - draft[t]
        w = [weight(x) for x in w.tolist()]
        if not any(w):
            w = [weight(x) for x in target[t].tolist()]
        v = float(u[end - 1])
        v = Fraction(min(max(v, 0.0), 1.0)) if v == v else Fraction(0)
        goal, total, pick = v.numerator * sum(w), 0, -1
        for i, x in enumerate(w):
            total += x
            if x:
                pick = i
                if total * v.denominator > goal:
                    break
        accepted.append(t - first)
        after.append(pick)
    return accepted, after
