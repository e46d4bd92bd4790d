"""mx_silu_mul_quant on bf16 gates around the smallest normal magnitude, where the
product of gate and reciprocal is subnormal in fp32, with ups that bring the
result back to ordinary sizes: y is still the correctly rounded value."""
import pytest
import torch

from tests.test_gpu_mx_silu import check_codes, check_y, fx  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def bf16(bits):
    return bits.to(torch.int16).view(BF)


# every subnormal gate, and the binades 2^-126 ... 2^-99 (bits 0x0001 ... 0x0E7F), in
# steps that keep all significands of the first four binades
GATES = torch.cat([torch.arange(1, 0x280), torch.arange(0x280, 0xE80, 5)])
SIGNIFICANDS = 1 + torch.arange(128) / 128.0


def rows(exponent, H):
    """[gate | up] rows of H pairs: every gate, both signs, with every significand of
    2^exponent (the last row filled up with ones)."""
    g = bf16(torch.cat([GATES, GATES + 0x8000]).to(torch.int32))
    u = (SIGNIFICANDS * 2.0 ** exponent).to(BF)
    pairs = torch.stack([g[:, None].expand(-1, 128).flatten(), u.repeat(g.numel())])
    n = pairs.shape[1]
    pairs = torch.cat([pairs, torch.ones((2, -n % H), dtype=BF)], 1)
    return torch.cat([pairs[0].view(-1, H), pairs[1].view(-1, H)], 1).cuda().contiguous()


@pytest.mark.parametrize("exponent", [29, 33, 40, 93, 127])
def test_every_tiny_gate(fx, exponent):  # noqa: F811
    """A result of normal size from a gate whose product with 1/2 is subnormal."""
    for sign in (1, -1):
        x = rows(exponent, 2048)
        x[:, 2048:] *= sign
        check_y(x, fx.silu_mul_quant(x, "fp8_per_token", emit_y=True).y)


@pytest.mark.parametrize("M", [3, 1201])
@pytest.mark.parametrize("mode", ["mxfp4", "fp8_per_group128", "fp8_per_token"])
def test_single_elements_in_every_mode(fx, mode, M):  # noqa: F811
    """One such gate among ordinary ones, at every place of a thread's vectors;
    few rows (one vector a thread in the group modes) and many (two)."""
    H = 2048
    g = torch.Generator(device="cuda")
    g.manual_seed(M)
    x = torch.randn((M, 2 * H), generator=g, device="cuda").to(BF)
    at = torch.arange(M, device="cuda")
    # -3 * 2^-133 * 129 * 2^93: just below a midpoint whose even neighbour is the larger
    x[at, at * 17 % H], x[at, H + at * 17 % H] = -3 * 2.0 ** -133, 129 * 2.0 ** 93
    r = fx.silu_mul_quant(x, mode, emit_y=True)
    assert bool((r.y[at, at * 17 % H].double() == -386 * 2.0 ** -41).all())
    check_y(x, r.y)
    check_codes(x, mode, r.q, r.scale, r.y)
