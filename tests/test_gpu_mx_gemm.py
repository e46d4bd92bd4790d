"""mx_gemm on the GPU against the 64-bit product of the decoded operands."""
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


def operands(M, N, K, seed=1, lo=120, hi=134):
    return (mx_ref.codes(M, K, seed), mx_ref.scales(M, K, seed, lo, hi),
            mx_ref.codes(N, K, seed + 1), mx_ref.scales(N, K, seed + 1, lo, hi))


def check(fx, M, N, K, dtype, a_tiled, b_tiled, seed=1, pad=0xFF):
    aq, as_, bq, bs = operands(M, N, K, seed)
    exact, mass = mx_ref.product(mx_ref.values(aq, as_), mx_ref.values(bq, bs))
    g = gpu_util.Guarded((M, N), dtype)
    out = fx.gemm(aq, mx_ref.tile(as_, pad) if a_tiled else as_, bq,
                  mx_ref.tile(bs, pad) if b_tiled else bs, out=g.t)
    torch.cuda.synchronize()
    assert g.intact()
    mx_ref.check_product(out, exact, mass, K)
    return out


SIZES = [  # every token tile, K below, at and past the steps of 32, 64, 128 and 256
    (1, 128, 256), (1, 1, 32), (2, 7, 64), (3, 129, 96), (16, 256, 2048), (17, 200, 288),
    (16, 1000, 4128), (33, 300, 512), (64, 384, 1120), (65, 130, 160), (127, 513, 736),
    (128, 256, 1024), (129, 257, 1056), (255, 100, 224), (256, 512, 512), (300, 640, 2592),
    (513, 1001, 320), (1024, 1024, 256), (2000, 72, 64),
]


@pytest.mark.parametrize("M,N,K", SIZES, ids=[f"M{s[0]}_N{s[1]}_K{s[2]}" for s in SIZES])
@pytest.mark.parametrize("dtype", [BF, HF, FP], ids=["bf16", "fp16", "fp32"])
def test_sizes_row_major(fx, M, N, K, dtype):
    check(fx, M, N, K, dtype, False, False)


@pytest.mark.parametrize("M,N,K", SIZES, ids=[f"M{s[0]}_N{s[1]}_K{s[2]}" for s in SIZES])
@pytest.mark.parametrize("a_tiled,b_tiled", [(True, True), (False, True), (True, False)])
def test_sizes_tiled_scales(fx, M, N, K, a_tiled, b_tiled):
    """The 32x4x4 tiling, its padding filled with the NaN scale."""
    check(fx, M, N, K, FP, a_tiled, b_tiled)


def test_out_with_a_row_stride(fx):
    """out as a slice of a wider tensor: the columns next to it stay."""
    M, N, K = 70, 129, 192
    aq, as_, bq, bs = operands(M, N, K, 4)
    exact, mass = mx_ref.product(mx_ref.values(aq, as_), mx_ref.values(bq, bs))
    for dtype in (BF, FP):
        for first, width in ((0, 200), (1, 131), (64, 256)):
            wide = torch.full((M, width), 3.0, dtype=dtype, device="cuda")
            out = fx.gemm(aq, as_, bq, bs, out=wide[:, first:first + N])
            mx_ref.check_product(out, exact, mass, K)
            assert bool((wide[:, :first] == 3).all()) and bool((wide[:, first + N:] == 3).all())


def test_extreme_scales(fx):
    """Scale bytes 0 and 254 (2^-127, 2^127) and NaN (0xFF): small sums keep
    their accuracy, sums beyond fp32's range are infinite (or NaN), NaN stays in
    its row and its column."""
    M, N, K = 40, 130, 128
    aq, as_, bq, bs = operands(M, N, K, 5)
    as_[3], as_[4], as_[5, 1], bs[7], bs[8, 3] = 0, 254, 255, 254, 255
    aq[3, 0] = 0x77
    out = fx.gemm(aq, as_, bq, bs, out_dtype=FP)
    exact, mass = mx_ref.product(mx_ref.values(aq, as_), mx_ref.values(bq, bs))
    nan = torch.zeros((M, N), dtype=torch.bool, device="cuda")
    nan[5], nan[:, 8] = True, True
    assert bool(out[nan].isnan().all())
    # where no partial sum can leave fp32's range, whatever the order
    safe = ~nan & (mass < 2.0 ** 127)
    assert bool(safe[3].sum() > 100) and bool(safe[:3, :7].all())
    mx_ref.check_product(out[safe], exact[safe], mass[safe], K)
    # beyond it an infinity, or NaN where infinities of both signs met
    over = ~nan & (exact.abs() > 2.0 ** 129)
    assert not bool(out[over].isfinite().any())


def test_rows_do_not_depend_on_their_neighbours(fx):
    """A row's bits are the same in every batch that adds up its products in the
    same order: all batches whose tiles are not split along K, and those with
    the same split."""
    M, N, K = 520, 264, 1312
    aq, as_, bq, bs = operands(M, N, K, 6)
    exact, mass = mx_ref.product(mx_ref.values(aq, as_), mx_ref.values(bq, bs))
    seen = {}
    for m in (M, 1, 5, 16, 17, 64, 100, 129, 300):
        out = fx.gemm(aq[:m], as_[:m], bq, bs, out_dtype=FP)
        mx_ref.check_product(out, exact[:m], mass[:m], K)
        split = fx.mx_last_launch()[3] if fx.mx_last_variant() == fx.MX_VARIANT_GEMM else 1
        first = seen.setdefault(split, out)
        n = min(m, first.shape[0])
        assert torch.equal(out[:n], first[:n]), (m, split)
    assert len(seen) > 1


def test_replays_streams_and_graphs(fx):
    """Repeated calls, programmatic launches, calls on two streams at once and a
    replayed graph all give the first call's bits."""
    sets = [operands(M, 1000, 1056, M) for M in (5, 200)]
    want = [fx.gemm(*s) for s in sets]
    outs = [[fx.gemm(*s) for s in sets] for _ in range(3)]
    with fx.programmatic_launch(True):
        outs += [[fx.gemm(*s) for s in sets] for _ in range(3)]
    streams = [torch.cuda.Stream() for _ in sets]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        got = []
        for st, s in zip(streams, sets):
            with torch.cuda.stream(st):
                got.append(fx.gemm(*s))
        outs.append(got)
    torch.cuda.synchronize()
    graph, held = torch.cuda.CUDAGraph(), [torch.zeros_like(w) for w in want]
    with torch.cuda.graph(graph):
        for s, o in zip(sets, held):
            fx.gemm(*s, out=o)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for got in outs + [held]:
        for o, w in zip(got, want):
            assert torch.equal(o, w)


def test_quantized_tuple_of_the_row_kernels(fx):
    """Activations from rmsnorm_quant, weights from quant, both scale layouts."""
    from mxfp4_quantization_b200 import fusednorm as fn
    M, N, K = 90, 384, 2048
    g = torch.Generator(device="cuda")
    g.manual_seed(8)
    x = torch.randn((M, K), generator=g, device="cuda").to(BF)
    w = (torch.randn((N, K), generator=g, device="cuda") / 40).to(BF)
    one = torch.ones(K, device="cuda", dtype=BF)
    flat, tiled = fn.FN_MXFP4, fn.FN_MXFP4 | fn.FN_SCALE_SWIZZLE_32_4_4
    a = {m: fn.rmsnorm_quant(x, one, 1e-6, m) for m in (flat, tiled)}
    b = {m: fn.quant(w, m) for m in (flat, tiled)}
    exact, mass = mx_ref.product(mx_ref.values(a[flat].q, a[flat].scale), mx_ref.values(*b[flat]))
    first = fx.gemm(a[flat].q, a[flat].scale, *b[flat])
    mx_ref.check_product(first, exact, mass, K)
    for ma in (flat, tiled):
        for mb in (flat, tiled):
            assert torch.equal(fx.gemm(a[ma].q, a[ma].scale, *b[mb]), first)


def test_empty_and_refused_calls(fx):
    aq, as_, bq, bs = operands(4, 8, 64)
    out = fx.gemm(aq[:0], as_[:0], bq, bs)
    assert out.shape == (0, 8) and fx.mx_last_variant() == fx.MX_VARIANT_NONE
    g = gpu_util.Guarded((4, 8), BF)
    for args, kind in (((aq, as_.int(), bq, bs), TypeError), ((aq, as_[:3], bq, bs), ValueError),
                       ((aq, as_, bq[:, :16], bs), ValueError), ((aq.cpu(), as_, bq, bs), ValueError),
                       ((aq.t(), as_, bq, bs), ValueError), ((aq, as_[0, 0], bq, bs), ValueError),
                       ((aq, as_, bq, bs.cpu()), ValueError), ((aq, as_.view(-1), bq, bs), ValueError),
                       ((aq, as_, bq.cpu(), bs), ValueError), ((aq.int(), as_, bq, bs), TypeError),
                       ((aq[None], as_, bq, bs), ValueError), ((aq, as_, bq, bs.t()), ValueError)):
        with pytest.raises(kind):
            fx.gemm(*args, out=g.t)
    with pytest.raises(ValueError):
        fx.gemm(aq, as_, bq, bs, out=torch.empty((4, 8), dtype=BF))
    with pytest.raises(ValueError):  # rows that overlap
        fx.gemm(aq, as_, bq, bs, out=torch.empty(8, dtype=BF, device="cuda").expand(4, 8))
    shifted = torch.empty(4 * 32 + 8, dtype=torch.uint8, device="cuda")[8:].view(4, 32)
    with pytest.raises(fx.FusedMXError) as e:  # codes 8 bytes off
        fx.gemm(shifted, as_, bq, bs, out=g.t)
    assert e.value.status == -2
    with pytest.raises(ValueError):
        fx.gemm(aq, as_, bq, bs, out=g.t[:3])
    with pytest.raises(TypeError):
        fx.gemm(aq, as_, bq, bs, out_dtype=torch.float64)
    with pytest.raises(fx.FusedMXError):  # out over an input
        fx.gemm(aq, as_, bq, bs, out=aq.view(-1)[:64].view(BF).view(4, 8))
    torch.cuda.synchronize()
    assert g.untouched()
