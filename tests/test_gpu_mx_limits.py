"""The calls of libfusedmx.so that ordinary sizes do not reach: offsets past 32 bits,
threads and streams at once, graphs, a workspace used again and again, zero rows."""
import os
import subprocess
import sys
import threading

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


def operands(M, N, K, seed=1):
    return (mx_ref.codes(M, K, seed), mx_ref.scales(M, K, seed), mx_ref.codes(N, K, seed + 1),
            mx_ref.scales(N, K, seed + 1))


@pytest.mark.parametrize("M", [9, 100])
@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp32"])
def test_output_rows_far_apart(fx, M, dtype):
    """Row offsets of out beyond 2^31 elements (rows 2^28, the most, or 2^25 apart)."""
    N, K = 130, 96
    ldo = (1 << 28) if M == 9 else (1 << 25)
    aq, as_, bq, bs = operands(M, N, K, 3)
    raw = torch.empty((M - 1) * ldo + N, dtype=dtype, device="cuda")
    out = raw.as_strided((M, N), (ldo, 1))
    ends = raw.as_strided((M - 1, 8), (ldo, 1), N)  # what follows each row but the last
    ends.fill_(3.0)
    fx.gemm(aq, as_, bq, bs, out=out)
    exact, mass = mx_ref.product(mx_ref.values(aq, as_), mx_ref.values(bq, bs))
    mx_ref.check_product(out.contiguous(), exact, mass, K)
    assert bool((ends == 3).all())


@pytest.mark.parametrize("R", [24, 400])
def test_source_rows_and_weights_far_away(fx, R):
    """Codes beyond 2^31 bytes on both sides: rows gathered from the end of a
    2.5 GB operand, the last of 40 experts of 4096 x 32768."""
    a_rows, K = 150_000, 32768
    E, N = 40, 4096
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    aq = torch.randint(0, 256, (a_rows, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    as_ = mx_ref.scales(a_rows, K, 2, 124, 130)
    bq = torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    bs = mx_ref.scales(E * N, K, 3, 124, 130)
    bt = torch.stack([mx_ref.tile(s) for s in bs.view(E, N, -1)])
    rows = (a_rows - 1 - torch.arange(R, device="cuda") * 7).int()
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[1:], off[E] = R // 3, R
    out = fx.grouped_gemm(aq, as_, bq, bt, off, rows=rows)
    for e, lo, hi in ((0, 0, R // 3), (E - 1, R // 3, R)):
        src = rows[lo:hi].long()
        exact, mass = mx_ref.product(mx_ref.values(aq[src], as_[src]),
                                     mx_ref.values(bq[e], bs.view(E, N, -1)[e]))
        mx_ref.check_product(out[lo:hi], exact, mass, K)


def test_silu_and_combine_far_rows(fx):
    M, H = 70_000, 16384  # 2.3e9 input elements
    x = torch.zeros((M, 2 * H), dtype=BF, device="cuda")
    x[-3:] = torch.randn((3, 2 * H), device="cuda").to(BF)
    for mode in ("mxfp4", "fp8_per_token"):
        r = fx.silu_mul_quant(x, mode)
        w = fx.silu_mul_quant(x[-3:].contiguous(), mode)
        assert torch.equal(r.q[-3:].view(torch.uint8), w.q.view(torch.uint8))
        assert torch.equal(r.scale[-3:], w.scale)
    del x, r, w
    R, N = 300_000, 8192
    y = torch.zeros((R, N), dtype=BF, device="cuda")
    y[-5:] = torch.randn((5, N), device="cuda").to(BF)
    pos = torch.tensor([[R - 1, R - 3], [R - 5, 0]], dtype=torch.int32, device="cuda")
    weight = torch.tensor([[0.5, 2.0], [1.0, 7.0]], device="cuda")
    out = fx.combine(y, pos, weight)
    want = torch.stack([0.5 * y[-1].double() + 2 * y[-3].double(), y[-5].double()])
    assert bool(((out.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -22 * (
        0.5 * y[-1].double().abs() + 2 * y[-3].double().abs() + y[-5].double().abs())).all())


def test_threads_and_streams_at_once(fx):
    """Four host threads, each with its own stream and its own kind of call, and
    launches recorded per thread."""
    M = (3, 60, 300, 1000)
    sets = [operands(m, 520, 1056, m) for m in M]
    want = [fx.gemm(*s) for s in sets]
    torch.cuda.synchronize()
    got, kinds = [[] for _ in M], [None] * len(M)

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                got[i].append(fx.gemm(*sets[i]))
            kinds[i] = fx.mx_last_variant()
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(M))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i in range(len(M)):
        assert all(torch.equal(o, want[i]) for o in got[i])
    assert kinds == [fx.MX_VARIANT_GEMM] * 2 + [fx.MX_VARIANT_GEMM_PAIR] * 2


def test_one_workspace_for_calls_in_order(fx):
    """Calls of different sizes that take turns on one workspace, plainly and as
    programmatic launches; a workspace that is too small is refused."""
    sets = [operands(m, n, 544, m) for m, n in ((300, 200), (130, 1000), (700, 72))]
    want = [fx.gemm(*s) for s in sets]
    need = [fx.mx_gemm_workspace_bytes(s[0].shape[0], s[2].shape[0], 544, 0) for s in sets]
    ws = torch.empty(max(need), dtype=torch.uint8, device="cuda")
    for pdl in (False, True):
        with fx.programmatic_launch(pdl):
            got = [fx.gemm(*s, workspace=ws) for _ in range(3) for s in sets]
        torch.cuda.synchronize()
        assert all(torch.equal(o, want[i % 3]) for i, o in enumerate(got))
    with pytest.raises(ValueError):
        fx.gemm(*sets[0], workspace=ws[:need[0] - 1])
    with pytest.raises(ValueError):
        fx.gemm(*sets[0], workspace=ws.cpu())


def test_workspace_is_all_a_call_writes_besides_out(fx):
    M, N, K, E = 333, 264, 1056, 3
    aq, as_, bq, bs = operands(M, N, K)
    need = fx.mx_gemm_workspace_bytes(M, N, K, 0)
    g = gpu_util.Guarded((need,), torch.uint8)
    fx.gemm(aq, as_, bq, bs, workspace=g.t)
    torch.cuda.synchronize()
    assert g.intact()
    rows = torch.arange(M, device="cuda", dtype=torch.int32).flip(0).contiguous()
    off = torch.tensor([0, 100, 100, 330], dtype=torch.int32, device="cuda")
    wq, ws = bq.expand(E, N, K // 2).contiguous(), bs.expand(E, N, K // 32).contiguous()
    need = fx.mx_grouped_gemm_workspace_bytes(M, E, N, K, 0, 1)
    g = gpu_util.Guarded((need,), torch.uint8)
    out = fx.grouped_gemm(aq, as_, wq, ws, off, rows=rows, workspace=g.t)
    torch.cuda.synchronize()
    assert g.intact()
    assert torch.equal(out[:330], fx.gemm(aq.flip(0), as_.flip(0), bq, bs)[:330])


def test_zero_rows_and_no_rows(fx):
    """All-zero rows (codes 0, scale byte 0) give exact zeros; a grouped call without
    rows, or whose experts own none, launches or writes nothing."""
    for M in (5, 300):
        aq, as_, bq, bs = operands(M, 136, 192)
        aq[2], as_[2] = 0, 0
        out = fx.gemm(aq, as_, bq, bs, out_dtype=FP)
        assert bool((out[2] == 0).all()) and bool((out[3] != 0).any())
    aq, as_, bq, bs = operands(4, 136, 192)
    wq, ws = bq[None], bs[None]
    off = torch.zeros(2, dtype=torch.int32, device="cuda")
    empty = fx.grouped_gemm(aq[:0], as_[:0], wq, ws, off)
    assert empty.shape == (0, 136) and fx.mx_last_variant() == fx.MX_VARIANT_NONE
    held = torch.full((4, 136), 5.0, dtype=BF, device="cuda")
    fx.grouped_gemm(aq, as_, wq, ws, off, out=held)
    assert bool((held == 5).all())


def test_graphs_that_hold_the_pair_kernels(fx):
    """Two graphs of products of many rows, replayed in turn and over each other's
    inputs: each keeps its own workspace."""
    sets = [operands(m, 520, 1056, m) for m in (200, 700)]
    want = [fx.gemm(*s) for s in sets]
    graphs, outs = [], []
    for s, w in zip(sets, want):
        o = torch.zeros_like(w)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            fx.gemm(*s, out=o)
        graphs.append(gr), outs.append(o)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for st, gr in zip(streams, graphs):
            with torch.cuda.stream(st):
                gr.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))


FIRST_CALL = """
import torch
from tests import mx_ref
from mxfp4_quantization_b200 import fusedmx as fx
sets = [(mx_ref.codes(m, 544, m), mx_ref.scales(m, 544, m), mx_ref.codes(200, 544, 1),
         mx_ref.scales(200, 544, 1)) for m in (3, 40, 300)]
x = torch.randn((5, 512), device="cuda").to(torch.bfloat16)
held = [torch.zeros((s[0].shape[0], 200), dtype=torch.bfloat16, device="cuda") for s in sets]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    for s, o in zip(sets, held):
        fx.gemm(*s, out=o)
    q = fx.silu_mul_quant(x, "mxfp4").q
graph.replay()
torch.cuda.synchronize()
for s, o in zip(sets, held):
    assert torch.equal(fx.gemm(*s), o)
assert torch.equal(fx.silu_mul_quant(x, "mxfp4").q, q)
print("captured first calls: ok")
"""


def test_first_calls_of_a_process_inside_a_capture(fx):
    """Nothing has to run before a capture: the library's one-time look-ups work
    inside it."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "captured first calls: ok" in r.stdout, r.stderr[-2000:]
