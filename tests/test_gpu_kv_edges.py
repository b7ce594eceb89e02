"""GPU checks of the key-value cache's operators at the edges of what they promise: weights to their last bits, values
near the largest finite one, infinities, lengths and totals out of the ordinary, tables wider than their rows.

Tolerances are derived beside each test; what only moves is compared bit for bit.
"""
import math

import numpy as np
import pytest
import torch

from test_gpu_kv import BF16, f64, nbw  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


def to_bf16(x):
    """The nearest bf16 of fp64 numbers, as fp64."""
    return torch.from_numpy(np.asarray(x, dtype=np.float64)).to(torch.float32).to(BF16).double().numpy()


def cut_bf16(x):
    """x cut off to bf16's 8 significant bits."""
    m, e = np.frexp(x)
    return np.ldexp(np.trunc(np.ldexp(m, 8)), e - 8)


@pytest.mark.parametrize("group,dim,page", [(1, 64, 16), (8, 128, 4), (12, 128, 16), (3, 256, 16)])
def test_attend_weights_keep_their_24_bits(nbw, group, dim, page):  # noqa: F811
    """Three slots of weights 1, 1 and p and values -c1, -c2 and 1, where c1 + c2 are p's first 16 bits: the result is
    what is left of p, (p - c1 - c2) / (2 + p).  A score here is one product and exact; times log2(e) it is off by 2 units of
    2^-24 of less than 1, which moves p by 1.4 of them; the exponential by 1 unit of p below 1; the sums of products by 8.
    That is below 2^-20, and 2^-21 after the division by 2 + p > 2."""
    rows, heads = 64, 8
    rng = np.random.default_rng(group)
    s = to_bf16(-rng.uniform(0.02, 0.69, (rows, heads)))
    p = np.exp(s)
    c1 = cut_bf16(p)
    c2 = to_bf16(p - c1)
    k, v = np.zeros((rows, heads, page, dim)), np.zeros((rows, heads, page, dim))
    k[:, :, 2, 0] = s
    v[:, :, 0], v[:, :, 1], v[:, :, 2] = -c1[..., None], -c2[..., None], 1.0
    q = np.zeros((rows, heads * group, dim))
    q[:, :, 0] = 1.0
    k, v, q = (torch.from_numpy(x).to(torch.float32).to(BF16).cuda() for x in (k, v, q))
    cache = nbw.KVCache(k, v, torch.arange(rows, dtype=torch.int32, device="cuda")[:, None])
    out = f64(nbw.kv_attend(cache, q, torch.full((rows,), 3, dtype=torch.int32, device="cuda"), scale=1.0))
    want = ((p - c1 - c2) / (2 + p)).repeat(group, axis=1)[..., None]
    assert np.abs(want).max() > 2.0**-19.5  # what two parts would lose is there to be seen
    assert np.all(np.abs(out - want) <= 2.0**-8 * 1.01 * np.abs(want) + 2.0**-21), float(np.abs(out - want).max() * 2.0**21)
