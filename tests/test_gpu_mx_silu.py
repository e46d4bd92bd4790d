"""mx_silu_mul_quant on the GPU: y is the correctly rounded value of the 64-bit
formula, codes and scales are the oracle's quantization of that y, bit for bit."""
import numpy as np
import pytest
import torch

import oracle
from tests import gpu_util, mx_ref

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
MODES = ["fp8_per_token", "fp8_per_group128", "mxfp4"]


@pytest.fixture(scope="module")
def fx():
    from mxfp4_quantization_b200.build import build_library, build_mx_library
    build_library()
    build_mx_library()
    from mxfp4_quantization_b200 import fusedmx
    return fusedmx


def formula(x):
    """float64 g u / (1 + e^-g) of rows [gate | up], for one rounding to 16 bits.
    Where the value is g u / 2 (small g) or g u (large g) up to a factor that
    float64 cannot hold, it is moved one float64 step to the side on which the
    real value lies: above g u / 2 in magnitude for g > 0, below for g < 0, and
    below g u for large g."""
    v = x.double().cpu().numpy()
    H = v.shape[1] // 2
    g, u = v[:, :H], v[:, H:]
    with np.errstate(all="ignore"):
        y = g * u / (1 + np.exp(-g))
        p = np.where(np.abs(g) < 2.0 ** -30, g * u / 2, np.where(g > 30, g * u, np.nan))
        out = np.nextafter(p, p * 2)
        inward = np.nextafter(p, 0.0)
    side = np.where((g > 0) & (g < 1), out, inward)
    near = np.isfinite(p) & (p != 0)
    small = near & (np.abs(g) < 2.0 ** -30)
    # (g / 2 moves the magnitude by more than a step from |g| = 2^-51 on)
    side = np.where(small & (np.abs(g) > 2.0 ** -50), p + p * (g / 2), side)
    return np.where(near, side, y)


def check_y(x, y):
    want = mx_ref.round16(formula(x), x.dtype)
    got = y.double().cpu().numpy()
    same = (got == want) & (np.signbit(got) == np.signbit(want)) | np.isnan(got) & np.isnan(want)
    assert same.all(), (np.argwhere(~same)[:4].tolist(), got[~same][:4], want[~same][:4])


def check_codes(x, mode, q, scale, y):
    io = oracle.IO_FP16 if x.dtype == HF else oracle.IO_BF16
    rq, rs = oracle.quant_rows(gpu_util.bits(y), MODES.index(mode), io=io)
    assert np.array_equal(gpu_util.u8(q).reshape(rq.shape), rq)
    s = gpu_util.scale_np(scale, MODES.index(mode)).reshape(rs.shape)
    assert np.array_equal(s.view(np.uint8), np.asarray(rs).view(np.uint8))


def rows(M, H, dtype, seed, std=2.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn((M, 2 * H), generator=g, device="cuda") * std).to(dtype)


@pytest.mark.parametrize("M,H", [(1, 128), (3, 256), (16, 2048), (33, 384), (5, 8192), (2, 32768),
                                 (700, 640), (1, 32640)])
@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
def test_rows(fx, M, H, mode, dtype):
    x = rows(M, H, dtype, M + H)
    r = fx.silu_mul_quant(x, mode, emit_y=True)
    check_y(x, r.y)
    check_codes(x, mode, r.q, r.scale, r.y)
    plain = fx.silu_mul_quant(x, mode)
    assert plain.y is None and torch.equal(gpu_view(plain.q), gpu_view(r.q))
    assert torch.equal(plain.scale, r.scale)


def gpu_view(t):
    return t.view(torch.uint8)


@pytest.mark.parametrize("M,H,mode", [(1201, 2176, "mxfp4"), (1201, 2176, "fp8_per_group128"),
                                      (76001, 32, "mxfp4"), (25500, 96, "mxfp4"),
                                      (19001, 128, "fp8_per_group128")])
@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
def test_two_vectors_a_thread(fx, M, H, mode, dtype):
    """The group modes' form for many rows: aligned rows, rows on 16-byte boundaries
    only, a row count, codes on a boundary that one store of 16 does not allow."""
    x = rows(M, H, dtype, M + H)
    r = fx.silu_mul_quant(x, mode, emit_y=True)
    assert fx.mx_last_launch()[2] == 2
    check_y(x, r.y)
    check_codes(x, mode, r.q, r.scale, r.y)
    wide = torch.zeros((M, 2 * H + 8), dtype=dtype, device="cuda")
    wide[:, 8:] = x
    s = fx.silu_mul_quant(wide[:, 8:], mode, emit_y=True)
    assert fx.mx_last_launch()[2] == 2
    for a, b in zip(r, s):
        assert torch.equal(gpu_view(a), gpu_view(b))
    q, used = torch.full_like(gpu_view(r.q), 0xA5), M - 3
    count = torch.tensor([used], dtype=torch.int32, device="cuda")
    fx.silu_mul_quant(x, mode, num_rows=count, out_q=q.view(r.q.dtype),
                      out_scale=torch.empty_like(r.scale))
    assert torch.equal(q[:used], gpu_view(r.q)[:used]) and (q[used:] == 0xA5).all()
    step = 4 if mode == "mxfp4" else 8
    flat = torch.empty(r.q.numel() + step, dtype=torch.uint8, device="cuda")
    shifted = flat[step:].view(r.q.dtype).view(r.q.shape)
    t = fx.silu_mul_quant(x, mode, out_q=shifted)
    assert fx.mx_last_launch()[2] == 1
    assert torch.equal(gpu_view(t.q), gpu_view(r.q))
    assert torch.equal(gpu_view(t.scale), gpu_view(r.scale))


@pytest.mark.parametrize("M,H,threads,vecs", [(601, 8, 32, 1), (601, 264, 64, 1), (601, 504, 32, 2),
                                              (601, 520, 96, 1), (601, 1024, 32, 4),
                                              (601, 2048, 64, 4), (601, 2560, 160, 2),
                                              (601, 4104, 288, 2), (601, 16384, 512, 4),
                                              (593, 32768, 512, 8), (3, 4096, 512, 1),
                                              (3, 4104, 288, 2), (3, 32760, 512, 8)])
@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
def test_row_blocks(fx, M, H, threads, vecs, dtype):
    """The per-token mode's blocks: few and many rows, idle lanes in the last vectors."""
    x = rows(M, H, dtype, M + H)
    r = fx.silu_mul_quant(x, "fp8_per_token", emit_y=True)
    assert fx.mx_last_launch()[1:3] == (threads, vecs)
    check_y(x, r.y)
    check_codes(x, "fp8_per_token", r.q, r.scale, r.y)


@pytest.mark.parametrize("H", [8, 24, 32, 40, 96])
def test_short_rows(fx, H):
    for mode in ("fp8_per_token", "mxfp4"):
        if mode == "mxfp4" and H % 32:
            continue
        x = rows(77, H, BF, H)
        r = fx.silu_mul_quant(x, mode, emit_y=True)
        check_y(x, r.y)
        check_codes(x, mode, r.q, r.scale, r.y)


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
def test_midpoints(fx, dtype):
    """g u / 2 of a tiny g, and g u of a large g, on the midpoint of two 16-bit
    values: the factor decides on which side, however near to 1 it is."""
    one = 1 + 2.0 ** -7 if dtype == BF else 1 + 2.0 ** -10  # one step above 1
    ups = torch.tensor([1 + 2.0 ** -7, 1.5, -1.5, 1 + 3 * 2.0 ** -7, -1.75], dtype=dtype)
    gates = [s * one * 2.0 ** e for s in (1, -1) for e in (range(-100, -20) if dtype == BF
                                                          else range(-14, -2))]
    gates += [one * 2.0 ** e for e in range(5, 60 if dtype == BF else 14)]
    g = torch.tensor(gates, dtype=dtype)
    n = g.numel() // 8 * 8
    x = torch.stack([torch.cat([g[:n], u.expand(n)]) for u in ups]).cuda().contiguous()
    check_y(x, fx.silu_mul_quant(x, "fp8_per_token", emit_y=True).y)


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
def test_every_gate_value(fx, dtype):
    """All finite 16-bit gate values, each against several up values: the
    smallest and the largest magnitudes, subnormals and both zeros."""
    g = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(dtype)
    g = g[g.isfinite()]
    top = torch.finfo(dtype).max
    ups = torch.tensor([1.0, -1.0, 0.0, -0.0, 3.1415, 2.0 ** -14, 1e-3, top, -top,
                        torch.finfo(dtype).smallest_normal, 777.0], dtype=dtype)
    n = g.numel() // 8 * 8
    for u in ups:
        x = torch.cat([g[:n].view(-1, 128 if n % 128 == 0 else 8),
                       torch.full((n,), float(u), dtype=dtype).view(
                           -1, 128 if n % 128 == 0 else 8)], 1).cuda().contiguous()
        r = fx.silu_mul_quant(x, "fp8_per_token", emit_y=True)
        check_y(x, r.y)


def test_specials(fx):
    """NaN and infinities in either half; the codes are those of the row kernels
    on that y."""
    from mxfp4_quantization_b200 import fusednorm as fn
    inf, nan = float("inf"), float("nan")
    x = rows(8, 256, BF, 9)
    x[0, 3], x[1, 4], x[2, 5], x[3, 260], x[4, 261], x[5, 262] = nan, inf, -inf, nan, inf, -inf
    x[6, :256], x[7, 256:] = 0.0, 0.0
    for mode in MODES:
        r = fx.silu_mul_quant(x, mode, emit_y=True)
        check_y(x, r.y)
        q, s = fn.quant(r.y, mode)
        assert torch.equal(gpu_view(q), gpu_view(r.q)) and torch.equal(gpu_view(s), gpu_view(r.scale))


@pytest.mark.parametrize("layout", ["swizzle", "mn"])
def test_scale_layouts(fx, layout):
    from mxfp4_quantization_b200 import fusednorm as fn
    mode = fn.FN_MXFP4 | fn.FN_SCALE_SWIZZLE_32_4_4 if layout == "swizzle" else \
        fn.FN_FP8_PER_GROUP128 | fn.FN_SCALE_MN_MAJOR
    x = rows(131, 640, BF, 11)
    r = fx.silu_mul_quant(x, mode, emit_y=True)
    q, s = fn.quant(r.y, mode)
    assert torch.equal(gpu_view(q), gpu_view(r.q)) and torch.equal(s, r.scale)


@pytest.mark.parametrize("mode", MODES)
def test_num_rows_and_strides(fx, mode):
    """A row count that only the device knows (below zero and above M too), a
    row stride wider than the row: the rows behind the last stay."""
    M, H = 50, 256
    wide = rows(M, H + 36, BF, 12)
    x = wide[:, 8:8 + 2 * H]
    full = fx.silu_mul_quant(x.contiguous(), mode, emit_y=True)
    for n in (-3, 0, 1, 17, 50, 99):
        used = min(max(n, 0), M)
        g = [gpu_util.Guarded(t.shape, t.dtype) for t in full]
        for t in g:
            t.t.view(torch.uint8).fill_(0x5A)
        r = fx.silu_mul_quant(x, mode, num_rows=torch.tensor([n], dtype=torch.int32, device="cuda"),
                              out_q=g[0].t, out_scale=g[1].t, out_y=g[2].t)
        torch.cuda.synchronize()
        for got, want, t in zip(r, full, g):
            assert t.intact()
            assert torch.equal(gpu_view(got[:used]), gpu_view(want[:used]))
            assert bool((gpu_view(got[used:]) == 0x5A).all())


def test_graph_and_programmatic_launch(fx):
    x = rows(40, 512, BF, 13)
    want = [fx.silu_mul_quant(x, m) for m in MODES]
    held = [fx.silu_mul_quant(x, m) for m in MODES]
    for h in held:
        gpu_view(h.q).fill_(0)
    graph = torch.cuda.CUDAGraph()
    with fx.programmatic_launch(True):
        with torch.cuda.graph(graph):
            for m, h in zip(MODES, held):
                fx.silu_mul_quant(x, m, out_q=h.q, out_scale=h.scale)
    graph.replay()
    torch.cuda.synchronize()
    for h, w in zip(held, want):
        assert torch.equal(gpu_view(h.q), gpu_view(w.q)) and torch.equal(h.scale, w.scale)


def test_empty_and_refused_calls(fx):
    x = rows(4, 128, BF, 14)
    r = fx.silu_mul_quant(x[:0], "mxfp4", emit_y=True)
    assert r.q.shape == (0, 64) and fx.mx_last_variant() == fx.MX_VARIANT_NONE
    with pytest.raises(TypeError):
        fx.silu_mul_quant(x.float(), "mxfp4")
    with pytest.raises(ValueError):
        fx.silu_mul_quant(x.cpu(), "mxfp4")
    with pytest.raises(ValueError):
        fx.silu_mul_quant(x[:, :-1].contiguous(), "mxfp4")
    with pytest.raises(ValueError):
        fx.silu_mul_quant(x, "mxfp4", num_rows=torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        fx.silu_mul_quant(x, "mxfp4", out_q=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(fx.FusedMXError) as e:  # 48 values a row are no MX blocks
        fx.silu_mul_quant(x[:, :96].contiguous(), "mxfp4")
    assert e.value.status == -1
    with pytest.raises(fx.FusedMXError):  # the row out_y over x
        fx.silu_mul_quant(x, "mxfp4", out_y=x.view(-1)[:512].view(4, 128))
