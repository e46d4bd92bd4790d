"""mx_combine on the GPU against the 64-bit weighted sum."""
import pytest
import torch

from tests import gpu_util, mx_ref

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def fx():
    from mxfp4_quantization_b200.build import build_library, build_mx_library
    build_library()
    build_mx_library()
    from mxfp4_quantization_b200 import fusedmx
    return fusedmx


def inputs(T, k, N, R, dtype, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    y = torch.randn((R, N), generator=g, device="cuda").to(dtype)
    pos = torch.randint(0, max(R, 1), (T, k), generator=g, device="cuda", dtype=torch.int32)
    w = torch.randn((T, k), generator=g, device="cuda")
    base = torch.randn((T, N), generator=g, device="cuda").to(dtype)
    return y, pos, w, base


def reference(y, pos, w, base):
    """float64 sum, and the sum of the terms' magnitudes (skipped rows not read)."""
    R = y.shape[0]
    total = torch.zeros((pos.shape[0], y.shape[1]), dtype=torch.float64, device="cuda")
    mass = total.clone()
    if base is not None:
        total, mass = total + base.double(), mass + base.double().abs()
    for j in range(pos.shape[1]):
        p = pos[:, j].long()
        keep = ((p >= 0) & (p < R)).nonzero().flatten()
        term = w[keep, j].double()[:, None] * y[p[keep]].double()
        total[keep] += term
        mass[keep] += term.abs()
    return total, mass


def check(out, y, pos, w, base):
    total, mass = reference(y, pos, w, base)
    # k fused multiply-adds in fp32, each off by half a step (2^-24) of a sum
    # that is at most the mass; then one rounding to 16 bits
    fp32 = pos.shape[1] * 2.0 ** -24 * mass * (1 + 2.0 ** -19)
    tol = fp32 + mx_ref.HALF_STEP[out.dtype] * (total.abs() + fp32) + mx_ref.SUBNORMAL[out.dtype]
    assert bool(((out.double() - total).abs() <= tol).all())


SIZES = [(1, 1, 8), (1, 8, 7168), (4, 8, 7168), (3, 2, 1), (5, 3, 7), (64, 6, 1001), (200, 8, 2048),
         (33, 32, 264), (2, 4, 4100), (1000, 1, 16)]


@pytest.mark.parametrize("T,k,N", SIZES)
@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
@pytest.mark.parametrize("with_base", [False, True])
def test_sizes(fx, T, k, N, dtype, with_base):
    y, pos, w, base = inputs(T, k, N, T * k, dtype, T + N)
    base = base if with_base else None
    g = gpu_util.Guarded((T, N), dtype)
    out = fx.combine(y, pos, w, base=base, out=g.t)
    torch.cuda.synchronize()
    assert g.intact()
    check(out, y, pos, w, base)


def test_dropped_repeated_and_outside_positions(fx):
    """Skipped positions are not read: NaN rows and NaN weights behind them do
    not show; a row whose choices are all dropped is its base, or zero."""
    y, pos, w, base = inputs(50, 4, 264, 30, BF, 1)
    pos[::3, 1], pos[1::3, 2], pos[7], pos[9], pos[11] = -1, 30, -2 ** 31, 2 ** 31 - 1, 5
    w[::3, 1], w[7] = float("nan"), float("inf")
    for b in (None, base):
        out = fx.combine(y, pos, w, base=b)
        assert not bool(out.isnan().any())
        check(out, y, pos, w.nan_to_num(0, 0, 0), b)
        assert bool((out[7] == (0 if b is None else base[7])).all())


def test_in_place_and_misaligned(fx):
    y, pos, w, base = inputs(21, 5, 328, 60, HF, 2)
    want = fx.combine(y, pos, w, base=base)
    assert fx.mx_last_variant() == fx.MX_VARIANT_COMBINE
    held = base.clone()
    assert fx.combine(y, pos, w, base=held, out=held) is held and torch.equal(held, want)
    # rows that start 2 bytes off a vector take the narrow kernel, same bits
    raw = torch.zeros(y.numel() + 1, dtype=HF, device="cuda")
    off = raw[1:].view(y.shape)
    off.copy_(y)
    assert torch.equal(fx.combine(off, pos, w, base=base), want)
    assert fx.mx_last_variant() == fx.MX_VARIANT_COMBINE_NARROW


def test_no_choices_and_empty(fx):
    y, pos, w, base = inputs(6, 2, 40, 9, BF, 3)
    none = torch.empty((6, 0), dtype=torch.int32, device="cuda")
    assert torch.equal(fx.combine(y, none, none.float(), base=base), base)
    assert bool((fx.combine(y, none, none.float()) == 0).all())
    assert torch.equal(fx.combine(y[:0], pos, w, base=base), base)
    assert fx.combine(y, pos[:0], w[:0]).shape == (0, 40)


def test_refused_calls(fx):
    y, pos, w, base = inputs(6, 2, 40, 9, BF, 4)
    with pytest.raises(TypeError):
        fx.combine(y.float(), pos, w)
    with pytest.raises(TypeError):
        fx.combine(y, pos.long(), w)
    with pytest.raises(TypeError):
        fx.combine(y, pos, w, base=base.half())
    with pytest.raises(ValueError):
        fx.combine(y, pos, w[:5])
    with pytest.raises(ValueError):
        fx.combine(y, pos, w, base=base[:5])
    with pytest.raises(fx.FusedMXError):
        fx.combine(y, pos, w, out=y[:6])
    many = torch.zeros((2, 33), dtype=torch.int32, device="cuda")
    with pytest.raises(fx.FusedMXError) as e:
        fx.combine(y, many, many.float())
    assert e.value.status == -3


def test_graph(fx):
    y, pos, w, base = inputs(16, 8, 512, 128, BF, 5)
    want, held = fx.combine(y, pos, w, base=base), torch.zeros_like(base)
    graph = torch.cuda.CUDAGraph()
    with fx.programmatic_launch(True), torch.cuda.graph(graph):
        fx.combine(y, pos, w, base=base, out=held)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(held, want)
