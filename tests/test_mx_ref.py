"""The 64-bit forms that judge libfusedmx.so, checked on the CPU: against the
oracle, library conversions and exact fractions, and with mistakes planted in
copies of their inputs that the comparison has to see."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle
from tests import mx_ref

BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


def operands(M, N, K, seed=1):
    return (mx_ref.codes(M, K, seed, "cpu"), mx_ref.scales(M, K, seed, device="cpu"),
            mx_ref.codes(N, K, seed + 1, "cpu"), mx_ref.scales(N, K, seed + 1, device="cpu"))


def test_values_against_the_oracle_formats():
    q = torch.arange(256, dtype=torch.uint8).view(1, 256)  # 512 codes, 16 groups
    s = torch.tensor([[0, 1, 2, 100, 126, 127, 128, 129, 130, 200, 253, 254, 255, 64, 31, 7]],
                     dtype=torch.uint8)
    v = mx_ref.values(q, s)[0].numpy()
    for i in range(512):
        byte, scale = i // 2, int(s[0, i // 32])
        code = byte & 15 if i % 2 == 0 else byte >> 4
        if scale == 255:
            assert np.isnan(v[i])
            continue
        want = Fraction(float(oracle.e2m1_decode(code))) * Fraction(2) ** (scale - 127)
        assert Fraction(float(v[i])) == want, (i, code, scale)


def test_tile_is_the_oracles_placement():
    for rows, groups in ((1, 1), (128, 4), (130, 5), (300, 81)):
        s = mx_ref.scales(rows, 32 * groups, rows, 1, 254, "cpu")
        want = oracle.place_scales(s.numpy(), oracle.SCALE_SWIZZLE_32_4_4)
        assert np.array_equal(mx_ref.tile(s).numpy(), np.asarray(want).reshape(-1))


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
def test_round16_is_nearest_even(dtype):
    """Every 16-bit value, the midpoints between neighbours and one float64 step to
    either side of them."""
    b = np.arange(0x7F80 if dtype == BF else 0x7C00, dtype=np.int16)
    v = torch.from_numpy(b).view(dtype).double().numpy()
    assert (mx_ref.round16(v, dtype) == v).all() and (mx_ref.round16(-v, dtype) == -v).all()
    mid = (v[1:] + v[:-1]) / 2
    even = np.where(b[:-1] % 2 == 0, v[:-1], v[1:])
    assert (mx_ref.round16(mid, dtype) == even).all()
    assert (mx_ref.round16(np.nextafter(mid, np.inf), dtype) == v[1:]).all()
    assert (mx_ref.round16(np.nextafter(mid, -np.inf), dtype) == v[:-1]).all()
    top = v[-1] + (v[-1] - v[-2]) / 2
    assert mx_ref.round16(np.float64(top), dtype) == np.inf
    assert mx_ref.round16(np.nextafter(top, 0), dtype) == v[-1]


def test_product_against_exact_fractions():
    aq, as_, bq, bs = operands(3, 4, 96)
    a, b = mx_ref.values(aq, as_), mx_ref.values(bq, bs)
    exact, mass = mx_ref.product(a, b)
    for m in range(3):
        for n in range(4):
            terms = [Fraction(x) * Fraction(y) for x, y in zip(a[m].tolist(), b[n].tolist())]
            assert Fraction(float(exact[m, n])) == sum(terms)
            assert Fraction(float(mass[m, n])) == sum(abs(t) for t in terms)


@pytest.mark.parametrize("dtype", [BF, HF, FP], ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("plant", ["none", "last_group", "scale_step", "nibbles", "neighbour_row",
                                   "shifted_scales", "one_code"])
def test_check_product_sees_planted_mistakes(dtype, plant):
    """A float32 product rounded to the type passes; the product of operands with
    one mistake in them does not."""
    M, N, K = 20, 24, 320
    aq, as_, bq, bs = operands(M, N, K, 7)
    # scales that keep every sum inside binary16
    as_, bs = as_ - 12, bs - 12
    exact, mass = mx_ref.product(mx_ref.values(aq, as_), mx_ref.values(bq, bs))
    q, s = aq.clone(), as_.clone()
    if plant == "last_group":
        q[:, -16:] = 0
    elif plant == "scale_step":
        s[:, 3] += 1
    elif plant == "nibbles":
        q = (q >> 4) | (q << 4)
    elif plant == "neighbour_row":
        q = q.roll(1, 0)
    elif plant == "shifted_scales":
        s = s.roll(1, 1)
    elif plant == "one_code":
        q[4, 33] ^= 0x8  # one sign
        if int(q[4, 33]) & 7 == 0:
            q[4, 33] ^= 0x4
    got = (mx_ref.values(q, s) @ mx_ref.values(bq, bs).T).float().to(dtype)
    if plant == "none":
        mx_ref.check_product(got, exact, mass, K)
    else:
        with pytest.raises(AssertionError):
            mx_ref.check_product(got, exact, mass, K)
