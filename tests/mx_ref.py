"""Plain 64-bit forms of the operators of libfusedmx.so, and inputs for their
tests.  The arithmetic is written from the formats' fields and the header's
formulas; nothing here is shared with the kernels."""
import numpy as np
import torch

# E2M1 values by code
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def round_up(x, m):
    return (x + m - 1) // m * m


def codes(rows, K, seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return torch.randint(0, 256, (rows, K // 2), generator=g, device=device, dtype=torch.uint8)


def scales(rows, K, seed, lo=120, hi=134, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed + 77)
    return torch.randint(lo, hi + 1, (rows, K // 32), generator=g, device=device,
                         dtype=torch.uint8)


def tile(s, fill=0):
    """E8M0 [rows, groups] -> the 32x4x4 tiling, by its index formula; `fill`
    in the padding."""
    rows, groups = s.shape
    tiles = round_up(groups, 4) // 4
    out = torch.full((round_up(rows, 128) * tiles * 4,), fill, dtype=torch.uint8, device=s.device)
    r = torch.arange(rows, device=s.device).unsqueeze(1)
    c = torch.arange(groups, device=s.device).unsqueeze(0)
    at = ((r // 128) * tiles + c // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + c % 4
    out[at.flatten()] = s.flatten()
    return out


def values(q, s):
    """Codes and E8M0 bytes -> float64 [rows, K] (0xFF: NaN)."""
    level = torch.tensor(LEVELS, dtype=torch.float64, device=q.device)
    v = torch.stack([level[(q & 15).long()], level[(q >> 4).long()]], -1).flatten(-2)
    x = torch.ldexp(torch.ones((), dtype=torch.float64, device=q.device), s.double() - 127)
    x = torch.where(s == 255, torch.full_like(x, float("nan")), x)
    return v * x.repeat_interleave(32, -1)


def product(a, b):
    """float64 product, and the sum of the terms' magnitudes."""
    return a @ b.T, a.abs() @ b.abs().T


HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 0.0}
SUBNORMAL = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -149}


def product_tolerance(exact, mass, K, dtype):
    """Per element: the sums run in fp32 over steps of 64 elements.  One step adds
    its 64 exact products and the running sum on a common exponent, wide enough
    that only the cut of the result to 24 bits counts: less than one unit of its
    last place, 2^-23 of a sum that does not exceed `mass`.  Then one rounding to the
    output type, half a step."""
    fp32 = (K + 63) // 64 * 2.0 ** -23 * mass
    return fp32 + HALF_STEP[dtype] * (exact.abs() + fp32) + SUBNORMAL[dtype]


# the largest magnitude that rounds to a finite value, or more
OVERFLOW = {torch.bfloat16: 2.0 ** 128 * (1 - 2.0 ** -9), torch.float16: 65520.0,
            torch.float32: 2.0 ** 128}


def check_product(got, exact, mass, K):
    tol = product_tolerance(exact, mass, K, got.dtype)
    top = OVERFLOW[got.dtype]
    bad = (got.double() - exact).abs() > tol
    # an infinity stands for the magnitudes that the type cannot hold
    inf = got.isinf() & (torch.sign(got.double()) == torch.sign(exact))
    bad = torch.where(inf, exact.abs() + tol < top, bad | (exact.abs() - tol > top))
    bad |= got.isnan() != exact.isnan()
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[:4].tolist(),
                                 got[bad][:4].tolist(), exact[bad][:4].tolist())


def round16(v, dtype):
    """float64 numpy -> the nearest 16-bit value (ties to even), as float64: the
    spacing at |v| is 2^(e - bits), no smaller than the format's subnormal step."""
    bits, low, top = (8, -133, 2.0 ** 128) if dtype == torch.bfloat16 else (11, -24, 65520.0)
    v = np.asarray(v, dtype=np.float64)
    e = np.maximum(np.frexp(v)[1] - bits, low)
    with np.errstate(invalid="ignore", over="ignore"):
        r = np.ldexp(np.rint(np.ldexp(v, -e)), e)
    r = np.where(np.isfinite(v), r, v)
    return np.where(np.isfinite(r) & (np.abs(r) >= top), np.copysign(np.inf, r), r)
