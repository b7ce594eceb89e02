"""GPU checks of the weights' bits in kv_attend_shared: all 24 where lines are few, and everywhere if asked for."""
import math

import numpy as np
import pytest
import torch

from oracle import kv as okv
from test_gpu_drafts import BF16, FP8, GROUPS, Shared, f64, nbw  # noqa: F401

pytestmark = pytest.mark.gpu


def check_all_bits(s, out, scale=None):
    """As Shared.check, but for the weights' rounding.  What is left: scores in fp32, off by the sum of dim products, each off
    by 2^-24 of what is summed (16 times allowed, and twice that, for numerator and sum); a weight's exponential, its
    parts' last rounding and the division, at most 8 * 2^-24 of each weight; sums over n slots in fp32, n * 2^-24 of all that is
    summed at most, for numerator and sum; and the result's own rounding to bf16, 2^-8 of itself."""
    k, v = s.pools()
    q = f64(s.q)
    scale = s.dim ** -0.5 if scale is None else scale
    want = okv.attend_tokens(q, k, v, s.table_np, s.lens, s.cu, scale)
    mean = okv.attend_tokens(q, k, np.abs(v), s.table_np, s.lens, s.cu, scale)
    size = np.abs(q).sum(axis=2).max() * np.nanmax(np.abs(k)) * abs(scale)
    bound = 2.0**-8 * np.abs(want) + 2.0**-24 * (2 * 16 * size + 2 * max(s.lens) + 16) * mean + 1e-30
    got = f64(out)
    ok = np.abs(got - want) <= bound
    assert ok.all(), (float(np.nanmax(np.abs(got - want) / bound)), int((~ok).sum()), ok.size)


@pytest.mark.parametrize("which", list(GROUPS))
@pytest.mark.parametrize("q_heads,kv,dim,page,dtype", [(8, 2, 128, 16, BF16), (3, 3, 64, 8, BF16), (12, 1, 64, 1, FP8),
                                                        (10, 2, 256, 32, BF16), (8, 1, 128, 128, FP8), (40, 2, 256, 4, FP8)])
def test_all_bits(nbw, which, q_heads, kv, dim, page, dtype):  # noqa: F811
    print(which, q_heads, kv, dim, page, dtype, flush=True)
    s = Shared(nbw, GROUPS[which], q_heads, kv, dim, page, dtype, seed=len(which), spread=q_heads == 8)
    out = s.call(all_bits=True)
    check_all_bits(s, out)
    assert torch.equal(out, s.call(all_bits=True))


@pytest.mark.parametrize("dim,dtype", [(64, BF16), (128, BF16), (128, FP8), (256, BF16)])
def test_few_lines_keep_all_bits_unasked(nbw, dim, dtype):  # noqa: F811
    """Single tokens and drafts, as far as 32 lines on average share slots: as kv_attend, which keeps them too."""
    for groups in ([(0, [(900, 1), (40, 1), (3, 1)])], [(700, [(60, 2), (9, 1)]), (300, [(5, 3), (8, 1)])], [(0, [(500, 8), (610, 7)])]):
        s = Shared(nbw, groups, 8, 2, dim, 16, dtype, seed=dim)
        out = s.call()
        check_all_bits(s, out)
        assert torch.equal(out, s.call(all_bits=True))


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_infinite_values_that_all_see_stay_so_with_all_bits(nbw, bad):  # noqa: F811
    s = Shared(nbw, [(600, [(3, 2), (50, 1)])], 8, 2)
    s.v[(int(s.table_np[0, 300 // s.page]), slice(None), 300 % s.page)][..., 3] = bad
    last = s.lens[1] - 1
    s.v[(int(s.table_np[1, last // s.page]), slice(None), last % s.page)][..., 7] = -bad
    out = f64(s.call(all_bits=True))
    assert np.array_equal(out[:, :, 3], np.full(out.shape[:2], bad), equal_nan=True)
    assert np.array_equal(out[2, :, 7], np.full(8, -bad), equal_nan=True) and np.isfinite(out[:2, :, 7]).all()


def test_many_lines_with_all_bits_at_the_ends_of_numbers(nbw):  # noqa: F811
    """Values near the largest finite one, and equal ones, whose average is exact."""
    s = Shared(nbw, [(700, [(9, 3), (200, 30)]), (0, [(1, 1)])], 8, 2)
    s.v[~s.v.isnan()] = 3.3e38
    s.check(s.call(all_bits=True))
    s.v[..., ::2] *= -1
    s.check(s.call(all_bits=True))
    s.v[~s.v.isnan()] = 1.3359375
    assert bool((s.call(all_bits=True) == 1.3359375).all())


def test_all_bits_in_the_scratch_that_is_asked_for(nbw):  # noqa: F811
    """One size serves both forms."""
    s = Shared(nbw, [(300, [(90, 40), (200, 1)]), (0, [(50, 2)])], 8, 2)
    need = s.cache.attend_shared_workspace_bytes(8, s.cu[-1], 2)
    ws = torch.full((need + 512,), 255, dtype=torch.uint8, device="cuda")
    for bits in (False, True):
        out = s.call(workspace=ws[:need], all_bits=bits)
        assert torch.equal(out, s.call(all_bits=bits)) and bool((ws[need:] == 255).all())
