"""mx_grouped_gemm with weights whose scale byte is NaN (0xFF): a row whose index is
outside the operand is a row of zeros all the same, in the kernel for few rows
and in the one for many."""
import pytest
import torch

from tests import gpu_util, mx_ref
from tests.test_gpu_mx_grouped import fx, weights  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu

BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
OUTSIDE = [-1, 2 ** 31 - 1, -2 ** 31]


@pytest.mark.parametrize("counts", [[3, 0, 17, 1], [16, 16], [300, 2, 0, 511], [17, 40, 31],
                                    [240, 241, 64]])
@pytest.mark.parametrize("dtype,tiled", [(BF, True), (HF, False), (FP, True)],
                         ids=["bf16", "fp16", "fp32"])
def test_outside_rows_are_zero(fx, counts, dtype, tiled):  # noqa: F811
    """NaN in single groups, a whole feature and a whole expert; a third of the rows
    outside, runs of them across the tiles' and the stores' boundaries."""
    N, K, E, a_rows = 300, 544, len(counts), 50
    off = torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    R = int(off[-1])
    aq, as_ = mx_ref.codes(a_rows, K, 1), mx_ref.scales(a_rows, K, 1)
    bq, bs, _ = weights(E, N, K, 2, False)
    bs[:, 5, 2], bs[:, 131], bs[:, 290, 16], bs[E - 1] = 255, 255, 255, 255
    g = torch.Generator(device="cuda")
    g.manual_seed(R)
    rows = torch.randint(0, a_rows, (R,), generator=g, device="cuda", dtype=torch.int32)
    bad = torch.tensor([a_rows] + OUTSIDE, device="cuda", dtype=torch.int32)
    rows[::5] = bad.repeat(R)[:rows[::5].numel()]
    rows[R // 4:R // 4 + R // 6] = a_rows
    out = gpu_util.Guarded((R, N), dtype)
    arg = torch.stack([mx_ref.tile(s, 0xFF) for s in bs]) if tiled else bs
    fx.grouped_gemm(aq, as_, bq, arg, off, rows=rows, out=out.t)
    kind = fx.MX_VARIANT_GEMM if R <= fx.MX_SMALL_EXPERT_ROWS * E else fx.MX_VARIANT_GEMM_PAIR
    assert fx.mx_last_variant() == kind
    torch.cuda.synchronize()
    assert out.intact()
    a = mx_ref.values(aq, as_)
    for e in range(E):
        lo, hi = int(off[e]), int(off[e + 1])
        src = rows[lo:hi].long()
        inside = (src >= 0) & (src < a_rows)
        got = out.t[lo:hi]
        exact, mass = mx_ref.product(a[src[inside]], mx_ref.values(bq[e], bs[e]))
        mx_ref.check_product(got[inside], exact, mass, K)
        assert bool((got[~inside] == 0).all()), (e, int((got[~inside] != 0).sum()))


def test_many_tiles_a_pair(fx):  # noqa: F811
    """More tiles of a pair of blocks than it has warps; an expert without NaN between
    two with it, rows outside in some experts alone."""
    E, n, N, K, a_rows = 100, 40, 4096, 64, 50
    off = torch.arange(E + 1, dtype=torch.int32, device="cuda") * n
    aq, as_ = mx_ref.codes(a_rows, K, 1), mx_ref.scales(a_rows, K, 1)
    bq, bs = mx_ref.codes(E * N, K, 2).view(E, N, -1), mx_ref.scales(E * N, K, 2).view(E, N, -1)
    bs[::2, ::129, 1] = 255
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    rows = torch.randint(0, a_rows, (E, n), generator=g, device="cuda", dtype=torch.int32)
    rows[::3, 5::7] = a_rows
    out = torch.full((E * n, N), 7.0, dtype=BF, device="cuda")
    fx.grouped_gemm(aq, as_, bq, bs, off, rows=rows.flatten(), out=out)
    kind, (blocks, _, tok, _) = fx.mx_last_variant(), fx.mx_last_launch()
    assert kind == fx.MX_VARIANT_GEMM_PAIR and E * N // 256 * -(-n // tok) > 12 * blocks // 2
    a = mx_ref.values(aq, as_)
    for e in range(E):
        src = rows[e].long()
        inside = src < a_rows
        got = out[e * n:e * n + n]
        exact, mass = mx_ref.product(a[src[inside]], mx_ref.values(bq[e], bs[e]))
        mx_ref.check_product(got[inside], exact, mass, K)
        assert bool((got[~inside] == 0).all()), e
