"""mx_grouped_gemm on the GPU against the 64-bit products of the decoded
operands: ragged row ranges, gathered rows, empty experts, rows that no expert
owns, offsets and indices that break the contract."""
import pytest
import torch

from tests import gpu_util, mx_ref

pytestmark = pytest.mark.gpu

BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def fx():
    from mxfp4_quantization_b200.build import build_library, build_mx_library
    build_library()
    build_mx_library()
    from mxfp4_quantization_b200 import fusedmx
    return fusedmx


def weights(E, N, K, seed, tiled):
    bq = torch.stack([mx_ref.codes(N, K, seed + 10 * e) for e in range(E)])
    bs = torch.stack([mx_ref.scales(N, K, seed + 10 * e) for e in range(E)])
    arg = torch.stack([mx_ref.tile(s, 0xFF) for s in bs]) if tiled else bs
    return bq, bs, arg


def check(fx, counts, N, K, dtype=BF, rows=None, a_rows=None, tiled=True, first=0, spare=0, seed=1):
    E = len(counts)
    off = torch.tensor([first] + [first + sum(counts[:e + 1]) for e in range(E)],
                       dtype=torch.int32, device="cuda")
    R = int(off[-1]) + spare
    a_rows = R if rows is None else a_rows
    aq, as_ = mx_ref.codes(a_rows, K, seed), mx_ref.scales(a_rows, K, seed)
    bq, bs, arg = weights(E, N, K, seed + 1, tiled)
    g = gpu_util.Guarded((R, N), dtype)
    g.t.fill_(7.0)
    out = fx.grouped_gemm(aq, as_, bq, arg, off, rows=rows, out=g.t)
    torch.cuda.synchronize()
    assert g.intact()
    a = mx_ref.values(aq, as_)
    for e in range(E):
        lo, hi = int(off[e]), int(off[e + 1])
        src = torch.arange(lo, hi, device="cuda") if rows is None else rows[lo:hi].long()
        inside = (src >= 0) & (src < a_rows)
        x = torch.where(inside[:, None], a[src.clamp(0, a_rows - 1)], 0.0)
        exact, mass = mx_ref.product(x, mx_ref.values(bq[e], bs[e]))
        mx_ref.check_product(out[lo:hi], exact, mass, K)
        assert bool((out[lo:hi][~inside] == 0).all())
    assert bool((out[:first] == 7).all()) and bool((out[int(off[-1]):] == 7).all())
    return out


RAGGED = [
    ([1], 128, 256), ([0, 1, 0], 64, 32), ([3, 0, 17, 1], 130, 96), ([0, 0, 0, 5], 256, 288),
    ([16, 15, 17, 0, 33], 100, 512), ([64, 1, 65, 127], 200, 160), ([128, 0, 129, 3], 257, 1056),
    ([300, 2, 0, 256, 511], 384, 320), ([1] * 40, 128, 64), ([0] * 7 + [90] + [0] * 8, 129, 224),
    ([5] * 65, 72, 2080),
    # pairs of blocks: row ranges around the tile height of 240 and its even cuts
    ([240, 241, 0, 480], 256, 256), ([1000, 1, 15, 16, 17], 300, 544), ([239, 700], 513, 96),
]


@pytest.mark.parametrize("counts,N,K", RAGGED)
@pytest.mark.parametrize("dtype", [BF, HF, FP], ids=["bf16", "fp16", "fp32"])
def test_ragged(fx, counts, N, K, dtype):
    check(fx, counts, N, K, dtype)


@pytest.mark.parametrize("counts,N,K", RAGGED)
@pytest.mark.parametrize("tiled", [True, False])
def test_gathered(fx, counts, N, K, tiled):
    """Rows by index: repeated, unused and out-of-range indices among them."""
    R, a_rows = sum(counts) + 3, max(1, sum(counts) // 3)
    g = torch.Generator(device="cuda")
    g.manual_seed(R)
    rows = torch.randint(0, a_rows, (R,), generator=g, device="cuda", dtype=torch.int32)
    rows[::7] = torch.tensor([-1, a_rows, 2 ** 31 - 1, -2 ** 31], device="cuda",
                             dtype=torch.int32).repeat(R)[:rows[::7].numel()]
    check(fx, counts, N, K, BF, rows=rows, a_rows=a_rows, tiled=tiled, spare=3)


def test_rows_without_an_owner_are_left(fx):
    check(fx, [9, 0, 40], 136, 128, FP, first=5, spare=200)
    check(fx, [0, 0], 136, 128, FP, first=3, spare=20)


@pytest.mark.parametrize("R", [40, 700])
def test_offsets_outside_the_contract_stay_in_bounds(fx, R):
    """Offsets that run backwards, overlap or leave the rows: the call ends and
    nothing outside out is written; the next call is right."""
    N, K = 128, 128
    aq, as_ = mx_ref.codes(R, K, 3), mx_ref.scales(R, K, 3)
    bq, bs, arg = weights(4, N, K, 4, True)
    for off in ([-5, 10, 4, 1000, 20], [R, 0, R, 0, R], [2 ** 31 - 1, -2 ** 31, R, R, -1],
                [0, R, 0, R, 0]):
        off = torch.tensor(off, dtype=torch.int32, device="cuda")
        g = gpu_util.Guarded((R, N), FP)
        fx.grouped_gemm(aq, as_, bq, arg, off, out=g.t)
        torch.cuda.synchronize()
        assert g.intact()
    check(fx, [R // 2, 0, R // 4, 3], N, K)


def test_many_experts(fx):
    """The largest number of experts, most of them idle."""
    counts = [0] * 1024
    for e in (0, 31, 32, 500, 1023):
        counts[e] = 2 + e % 5
    check(fx, counts, 16, 32)


def test_equals_gemm(fx):
    """One expert that owns every row gives mx_gemm's bits."""
    M, N, K = 150, 300, 544
    aq, as_ = mx_ref.codes(M, K, 5), mx_ref.scales(M, K, 5)
    bq, bs, _ = weights(1, N, K, 6, False)
    off = torch.tensor([0, M], dtype=torch.int32, device="cuda")
    one = fx.gemm(aq, as_, bq[0], bs[0])
    assert torch.equal(fx.grouped_gemm(aq, as_, bq, bs, off), one)
    every = torch.arange(M, dtype=torch.int32, device="cuda")
    assert torch.equal(fx.grouped_gemm(aq, as_, bq, bs, off, rows=every), one)


def test_refused_calls(fx):
    aq, as_ = mx_ref.codes(6, 64, 1), mx_ref.scales(6, 64, 1)
    bq, bs, arg = weights(3, 40, 64, 2, True)
    off = torch.tensor([0, 2, 2, 6], dtype=torch.int32, device="cuda")
    rows = torch.zeros(6, dtype=torch.int32, device="cuda")
    g = gpu_util.Guarded((6, 40), BF)
    for args, kind in (((aq, as_, bq, bs, off[:3]), ValueError), ((aq, as_, bq, bs, off.long()), TypeError),
                       ((aq, as_, bq[0], bs, off), ValueError), ((aq, as_, bq, bs[:2], off), ValueError),
                       ((aq, as_, bq, bs[0], off), ValueError), ((aq, as_[:5], bq, bs, off), ValueError),
                       ((aq, as_, bq, bs, off.cpu()), ValueError),
                       ((aq, mx_ref.tile(as_), bq, bs, off), ValueError),
                       ((aq, as_, bq[:, :, :16], bs, off), ValueError)):
        with pytest.raises(kind):
            fx.grouped_gemm(*args, out=g.t)
    for r in (rows.long(), rows.cpu(), rows[::2]):
        with pytest.raises((TypeError, ValueError)):
            fx.grouped_gemm(aq, as_, bq, bs, off, rows=r)
    with pytest.raises(ValueError):  # more rows of out than of a, without an index
        fx.grouped_gemm(aq, as_, bq, bs, off, out=torch.empty((7, 40), dtype=BF, device="cuda"))
    torch.cuda.synchronize()
    assert g.untouched()
    # fewer rows of out than of a: the owned rows beyond it are left out
    part = fx.grouped_gemm(aq, as_, bq, bs, off, out=g.t[:4])
    assert torch.equal(part, fx.grouped_gemm(aq, as_, bq, bs, off)[:4])
    assert bool((g.t[4:].view(torch.uint8) == gpu_util.CANARY).all())
