"""A check of attention that every slot counts, and counts once.

All keys are 0, so every slot that a token sees has the same weight; a slot's value is 1 in one dim and 0 in the
others, or 0 in all.  A dim of the result is then the number of the token's slots that have their 1 there, over all that it sees:
a slot (a run of slots) left out or counted twice changes its dim by as much as there is in it, however many slots there are.
"""
import numpy as np


def wanted(dims, dim, sees):
    """dims [slots]: each slot's dim, or -1 -> what a token that sees the first `sees` slots gets."""
    d = np.asarray(dims)[:max(sees, 0)]
    return np.bincount(d[d >= 0], minlength=dim) / max(sees, 1)


def wrong(got, want, sees):
    """Dims that are off by more than the result's rounding to bf16 (2^-8) and the sums of up to `sees` equal numbers in
    fp32, for numerator and denominator (2^-24 each time)."""
    return np.flatnonzero(~(np.abs(np.asarray(got) - want) <= (2.0**-8 + 2 * max(sees, 0) * 2.0**-24) * want))


def runs(slots, length, dim, first=0):
    """dims of slots in runs of `length`: run number first + d has dim d."""
    d = np.arange(slots) // length - first
    return np.where((d >= 0) & (d < dim), d, -1)
