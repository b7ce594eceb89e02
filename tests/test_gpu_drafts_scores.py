"""GPU checks of scores of any size in kv_attend_shared.

Queries and keys are powers of two in one dim each, so scores are exact, and so far apart that a weight is 0 or that of
the largest: the result is a value, or an average of two, which fp32 holds exactly.
"""
import math

import pytest
import torch

from test_gpu_drafts import BF16, FP8, Shared, nbw  # noqa: F401

pytestmark = pytest.mark.gpu
SIZES = [20, 24, 28, 31, 34, 40, 64, 100, 120]


def fill(s, exponent, sign, winners):
    """Scores (scale 1) of +-2^exponent for the winners, one more or less step of a quarter for all others; values whole numbers."""
    q, k = 2.0 ** (exponent // 2), 2.0 ** (exponent - exponent // 2)
    s.q.zero_()
    s.q[..., 0] = sign * q
    s.k[~s.k.isnan()] = 0
    g = torch.Generator(device="cuda").manual_seed(exponent)
    whole = torch.randint(-8, 9, s.v.shape, generator=g, device="cuda").to(torch.float32)
    s.v.copy_(torch.where(s.v.isnan(), math.nan, whole).to(s.v.dtype))
    live = ~s.k[..., 0].isnan()
    s.k[..., 0] = torch.where(live, k * (0.75 if sign > 0 else 1.25), s.k[..., 0].float()).to(s.k.dtype)
    for row, slot in winners:
        s.k[int(s.table_np[row, slot // s.page]), :, slot % s.page, 0] = k


def value(s, row, slot):
    """[q_heads][dim]: what a row's query heads get from a slot."""
    v = s.v[int(s.table_np[row, slot // s.page]), :, slot % s.page].float()
    return v.repeat_interleave(s.q.shape[1] // v.shape[0], dim=0)


@pytest.mark.parametrize("exponent", SIZES)
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("dim,page", [(64, 8), (128, 16), (256, 32)])
def test_the_largest_score_wins(nbw, exponent, sign, new, dim, page):  # noqa: F811
    """In the prefix for one row, among its own slots for another."""
    s = Shared(nbw, [(300, [(200, new), (150, new), (90, new)])], 8, 2, dim, page, seed=exponent)
    fill(s, exponent, sign, [(1, 300 + 20), (2, 300 + 44)])
    for row, slot in ((1, 320), (2, 344)):
        out = s.call(scale=1.0)[s.cu[row]:s.cu[row + 1]].float()
        assert torch.equal(out, value(s, row, slot).expand_as(out)), (row, out[0, 0, :4])
    fill(s, exponent, sign, [(0, 133)])  # of the prefix: all rows
    out = s.call(scale=1.0).float()
    assert torch.equal(out, value(s, 0, 133).expand_as(out))


@pytest.mark.parametrize("exponent", SIZES)
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("new", [1, 40])
def test_equal_scores_on_both_sides(nbw, exponent, sign, new):  # noqa: F811
    """A slot of a long prefix and one of a few own ones, which are summed under different factors: an average of two whole numbers."""
    s = Shared(nbw, [(2000, [(50, new), (41, new), (45, new)])], 8, 2, 128, 16, seed=exponent)
    for slot in (0, 31, 129, 1983):
        fill(s, exponent, sign, [(0, slot), (1, 2000 + 1)])
        out = s.call(scale=1.0)[s.cu[1]:s.cu[2]].float()
        want = (value(s, 0, slot) + value(s, 1, 2001)) / 2
        assert torch.equal(out, want.expand_as(out)), slot


@pytest.mark.parametrize("exponent", [0, 10, 20, 30, 40, 60])
def test_scales_and_8_bit_keys(nbw, exponent):  # noqa: F811
    s = Shared(nbw, [(300, [(200, 1), (150, 20), (90, 3)])], 8, 2, 128, 16, FP8, seed=exponent)
    for by in s.scales:
        by.fill_(0.5)
    live = ~s.k.float()[..., 0].isnan()
    s.q.zero_()
    s.q[..., 0] = 16.0
    s.v.copy_(torch.randint(-8, 9, s.v.shape, device="cuda").to(torch.float32).to(FP8))
    k = torch.where(live, 192.0, math.nan)
    k[int(s.table_np[0, 133 // 16]), :, 133 % 16] = 256.0
    s.k.copy_(torch.where(torch.arange(128, device="cuda") == 0, k[..., None], 0.0).to(FP8))
    out = s.call(scale=2.0 ** exponent).float()
    assert torch.equal(out, (value(s, 0, 133) * 0.5).expand_as(out))


@pytest.mark.parametrize("exponent", [0, 12, 16, 22, 24, 26])
def test_values_near_the_largest_finite_one_under_large_scores(nbw, exponent):  # noqa: F811
    """All scores equal: the average of equal values, which are as large as they come."""
    s = Shared(nbw, [(700, [(9, 3), (200, 30)]), (0, [(1, 1)])], 8, 2)
    s.q.zero_()
    s.q[..., 0] = 2.0 ** (exponent // 2)
    s.k[~s.k.isnan()] = 2.0 ** (exponent - exponent // 2)
    s.v[~s.v.isnan()] = 3.3895e38
    big = torch.tensor(3.3895e38).to(BF16)
    for bits in (False, True):
        for sign in (1.0, -1.0):
            assert bool((s.call(scale=sign, all_bits=bits) == big.cuda()).all())


@pytest.mark.parametrize("step", [1.0, 40.0, 4096.0, 2.0 ** 20, 2.0 ** 33])
def test_scores_that_rise_from_slot_to_slot(nbw, step):  # noqa: F811
    """Each slot's score passes the last one's: only a token's own slot counts."""
    s = Shared(nbw, [(90, [(60, 20), (33, 1)])], 4, 2, 64, 8, seed=2)
    s.q.zero_()
    s.q[..., 0] = 1.0
    s.k[~s.k.isnan()] = 0
    for row in range(2):
        for j in range(s.lens[row]):
            s.k[int(s.table_np[row, j // 8]), :, j % 8, 0] = float(j)
    out = s.call(scale=step * 30).float()
    for row in range(2):
        for t in range(s.cu[row], s.cu[row + 1]):
            sees = s.lens[row] - s.cu[row + 1] + 1 + t
            want = value(s, row, sees - 1)
            assert torch.allclose(out[t], want, rtol=2.0 ** -8, atol=2.0 ** -30), (row, t)


@pytest.mark.parametrize("by", [1e-36, 1e-20, 1e20, 1e31, 1e34, 7e35])
@pytest.mark.parametrize("groups", [[(0, [(5, 1), (40, 2)])], [(0, [(900, 40)])], [(300, [(60, 2), (50, 30)])], [(0, [(9000, 1)])]])
def test_factors_of_values_of_any_size(nbw, by, groups):  # noqa: F811
    """Equal values of 256: their average is 256 times the factor, whatever the weights add up to."""
    s = Shared(nbw, groups, 8, 2, 128, 16, FP8, seed=1)
    s.scales[1].fill_(by)
    s.v.copy_(torch.where(s.v.float().isnan(), math.nan, 256.0).to(FP8))
    want = torch.tensor(by, dtype=torch.float32) * 256
    for bits in (False, True):
        out = s.call(all_bits=bits).float().cpu()
        # the division, the factor's product and the sums (2^-24 each for up to 9000 slots), and the result's own rounding
        assert bool(((out - want).abs() <= want * (2.0**-8 + 2.0**-10)).all()), (bits, out.flatten()[:3], want)
