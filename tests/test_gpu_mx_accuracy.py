"""How the products of libfusedmx.so add up: every step of 64 elements is added with the
running sum on a common exponent and cut once, toward zero, to 24 bits."""
import math

import pytest
import torch

from tests import mx_ref
from tests.test_gpu_mx_gemm import fx  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu

ONE, MINUS_ONE = 0x2, 0xA  # E2M1 codes


def product(fx, M, first, small, n, j, apart):
    """fp32 sum of the codes `first` (times 1) and n terms of 2^-j, in the same
    64-element step or (apart) in the next one."""
    K, at = (128, 64) if apart else (64, 32)
    a, b = torch.zeros((2, K), dtype=torch.uint8)
    a[:len(first)], b[:len(first)] = ONE, torch.tensor(first, dtype=torch.uint8)
    a[at:at + n], b[at:at + n] = ONE, small
    sa, sb = torch.full((2, K // 32), 127, dtype=torch.uint8)
    sa[at // 32:], sb[at // 32:] = 127 - j // 2, 127 - (j - j // 2)
    pack = lambda v: v[0::2] | v[1::2] << 4  # noqa: E731
    rep = lambda v, m: v.repeat(m, 1).cuda()  # noqa: E731
    out = fx.gemm(rep(pack(a), M), rep(sa, M), rep(pack(b), 40), rep(sb, 40),
                  out_dtype=torch.float32)
    assert bool((out == out[0, 0]).all())
    return float(out[0, 0])


@pytest.mark.parametrize("M", [8, 100])
@pytest.mark.parametrize("apart", [False, True])
def test_a_step_is_cut_once(fx, M, apart):  # noqa: F811
    """1 + n 2^-j, all positive or all negative: the sum of the small terms counts
    as a whole, its part below 2^-23 (of a sum in [1, 2)) is cut off."""
    for n in (1, 2, 5, 32):
        for j in range(18, 35):
            want = 1 + math.floor(n * 2.0 ** (23 - j)) * 2.0 ** -23
            assert product(fx, M, [ONE], ONE, n, j, apart) == want, (n, j)
            assert product(fx, M, [MINUS_ONE], MINUS_ONE, n, j, apart) == -want, (n, j)


@pytest.mark.parametrize("M", [8, 100])
def test_small_terms_next_to_cancelling_ones(fx, M):  # noqa: F811
    """1 - 1 + n 2^-j is exact down to 2^-35 of the largest term."""
    for n in (1, 3, 32):
        for j in range(20, 36):
            assert product(fx, M, [ONE, MINUS_ONE], ONE, n, j, False) == n * 2.0 ** -j, (n, j)


@pytest.mark.parametrize("M", [40, 1000])
@pytest.mark.parametrize("K", [64, 96, 256, 4096])
@pytest.mark.parametrize("lo,hi", [(100, 160), (116, 138)])
def test_error_of_wide_scales(fx, M, K, lo, hi):  # noqa: F811
    """Scales over up to 60 binades: 2^-23 of the terms' magnitudes a step, 65 terms
    that can each lose 2^-35 of the largest, and up to seven roundings where a split
    along K joins its parts."""
    N = 1024
    aq, as_ = mx_ref.codes(M, K, K), mx_ref.scales(M, K, K, lo, hi)
    bq, bs = mx_ref.codes(N, K, K + 1), mx_ref.scales(N, K, K + 1, lo, hi)
    exact, mass = mx_ref.product(mx_ref.values(aq, as_), mx_ref.values(bq, bs))
    got = fx.gemm(aq, as_, bq, bs, out_dtype=torch.float32).double()
    steps = -(-K // 64)
    bound = (steps * (2.0 ** -23 + 65 * 2.0 ** -35) + 7 * 2.0 ** -24) * mass
    # (no sum leaves the normal range: 2^(2 (100 - 127)) and 36 * 4096 * 2^(2 (160 - 127)))
    assert bool(((got - exact).abs() <= bound).all())
