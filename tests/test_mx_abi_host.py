"""Host-side checks of libfusedmx.so's C ABI (no GPU): the library loads,
exports every symbol include/fusedmx.h declares, and rejects bad arguments
before any CUDA call.  Pointers here are fake addresses; a call that breaks no
rule gets as far as the CUDA runtime, finds no device and returns FN_ERR_CUDA."""
import os
import re
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "fusedmx.h")
BASE, STEP = 0x7F0000000000, 1 << 36

E, A, U, CUDA = -1, -2, -3, -4

no_device = pytest.mark.skipif(torch.cuda.is_available(),
                               reason="fake addresses must not reach a launch")


@pytest.fixture(scope="module")
def fx():
    from mxfp4_quantization_b200.build import build_library, build_mx_library
    build_library()
    build_mx_library()
    from mxfp4_quantization_b200 import fusedmx
    return fusedmx


def at(i, off=0):
    return BASE + i * STEP + off


def declared_symbols():
    return set(re.findall(r"FN_API\s+[\w\s\*]+?\b(mx_\w+)\s*\(", open(HEADER).read()))


def test_library_exports_the_header(fx):
    out = subprocess.run(["nm", "-D", "--defined-only", fx.LIB_PATH], capture_output=True,
                         text=True, check=True).stdout
    exported = set(re.findall(r"\bT (\w+)", out))
    exported -= {"_init", "_fini"}
    assert exported == declared_symbols() == set(fx.ABI_SYMBOLS)


def test_header_constants_match_binding(fx):
    src = open(HEADER).read()
    for name in re.findall(r"#define (MX_[A-Z0-9_]+) ", src):
        m = re.search(rf"#define {name} (0x[0-9a-fA-F]+|\d+)", src)
        assert int(m.group(1), 0) == getattr(fx, name), name
    names = re.findall(r"\b(MX_VARIANT_\w+)\s*=\s*(\d+)", src)
    assert len(names) >= 6
    for name, value in names:
        assert int(value) == getattr(fx, name), name


def test_status_strings_and_settings(fx):
    assert fx.mx_status_string(0) == "ok" and fx.mx_status_string(9) == "unknown status"
    assert len({fx.mx_status_string(s) for s in (0, -1, -2, -3, -4, 9)}) == 6
    assert fx.mx_version() >= 100
    import threading
    assert fx.mx_programmatic_launch(1) == 0
    seen = []
    t = threading.Thread(target=lambda: seen.append(fx.mx_programmatic_launch(0)))
    t.start()
    t.join()
    assert seen == [0] and fx.mx_programmatic_launch(0) == 1


def gemm(fx, **kw):
    a = dict(aq=at(1), as_=at(2), bq=at(3), bs=at(4), M=8, N=72, K=96, flags=0, out=at(5), ldo=72,
             ws=at(8))
    a.update(kw)
    return fx.mx_gemm(a["aq"], a["as_"], a["bq"], a["bs"], a["M"], a["N"], a["K"], a["flags"],
                      a["out"], a["ldo"], a["ws"], None)


GEMM_RULES = [
    (dict(M=-1), E), (dict(N=0), E), (dict(N=-3), E), (dict(K=0), E), (dict(K=48), E),
    (dict(K=-32), E), (dict(ldo=71), E), (dict(ldo=-1), E), (dict(flags=3), E),
    (dict(flags=0x40), E), (dict(flags=-1), E),
    (dict(M=1 << 31), U), (dict(N=1 << 31, ldo=1 << 31), U), (dict(K=(1 << 24) + 32), U),
    (dict(ldo=(1 << 28) + 1), U),
    (dict(aq=None), E), (dict(as_=None), E), (dict(bq=None), E), (dict(bs=None), E),
    (dict(out=None), E),
    (dict(aq=at(1, 8)), A), (dict(bq=at(3, 4)), A), (dict(out=at(5, 1)), A),
    (dict(out=at(5, 2), flags=2), A), (dict(as_=at(2, 4), flags=0x10), A),
    (dict(bs=at(4, 8), flags=0x20), A),
    (dict(out=at(1)), E), (dict(out=at(1, 8 * 48 - 2)), E), (dict(out=at(2, 22)), E),
    (dict(out=at(3, 72 * 48 - 2)), E), (dict(out=at(4)), E),
    # the tiled scales' padding counts: 128 x 4 bytes for 8 rows of 3 groups
    (dict(out=at(2, 510), flags=0x10), E),
    # an output row stride reaches further: row 7 starts inside the weight
    (dict(out=at(3) - 7 * 2000 * 2, ldo=2000), E),
]


@pytest.mark.parametrize("kw,want", GEMM_RULES)
def test_gemm_rules(fx, kw, want):
    assert gemm(fx, **kw) == want
    assert fx.mx_last_variant() == fx.MX_VARIANT_NONE


def test_gemm_without_rows(fx):
    assert gemm(fx, M=0) == 0
    assert gemm(fx, M=0, aq=None, as_=None, bq=None, bs=None, out=None) == 0
    assert gemm(fx, M=0, N=0) == E


@no_device
@pytest.mark.parametrize("kw", [
    {}, dict(flags=1), dict(flags=0x32), dict(as_=at(2, 1), bs=at(4, 3)), dict(out=at(5, 2)),
    dict(out=at(1, 8 * 48)), dict(out=at(2, 24)), dict(out=at(2, 512), flags=0x10),
    dict(ldo=1 << 28), dict(M=1)])
def test_gemm_accepts(fx, kw):
    assert gemm(fx, **kw) == CUDA


def grouped(fx, **kw):
    a = dict(aq=at(1), as_=at(2), a_rows=8, rows=None, off=at(6), E=3, bq=at(3), bs=at(4), R=8,
             N=72, K=96, flags=0, out=at(5), ldo=72, ws=at(8))
    a.update(kw)
    return fx.mx_grouped_gemm(a["aq"], a["as_"], a["a_rows"], a["rows"], a["off"], a["E"], a["bq"],
                              a["bs"], a["R"], a["N"], a["K"], a["flags"], a["out"], a["ldo"],
                              a["ws"], None)


def test_workspace_rules(fx):
    """A call of many rows takes a workspace: it has to be there, aligned and
    apart from every tensor of the call; a call of few rows needs none."""
    M, N, K = 500, 512, 1024
    need = fx.mx_gemm_workspace_bytes(M, N, K, 0)
    assert need > 0 and need % 16 == 0
    assert 0 < fx.mx_gemm_workspace_bytes(M, N, K, 0x20) < need  # tiled weights stay where they are
    assert fx.mx_gemm_workspace_bytes(8, N, K, 0) == 0 and gemm(fx, M=8, ws=None) in (0, CUDA)
    assert fx.mx_gemm_workspace_bytes(0, N, K, 0) == 0
    for bad in ((-1, N, K, 0), (M, 0, K, 0), (M, N, 48, 0), (M, N, K, 3), (M, N, 1 << 25, 0)):
        assert fx.mx_gemm_workspace_bytes(*bad) == -1
    g = fx.mx_grouped_gemm_workspace_bytes(M, 2, N, K, 0x20, 0)
    assert fx.mx_grouped_gemm_workspace_bytes(M, 2, N, K, 0x20, 1) == g + M * K // 2
    assert fx.mx_grouped_gemm_workspace_bytes(M, 2, N, K, 0x10, 0) == -1
    big = dict(M=M, N=N, K=K, ldo=N)
    for kw, want in ((dict(ws=None), E), (dict(ws=at(8, 8)), A), (dict(ws=at(1)), E),
                     (dict(ws=at(5, 16)), E), (dict(ws=at(4) - need + 16), E),
                     (dict(ws=at(3, N * K // 2 - 16)), E)):
        assert gemm(fx, **big, **kw) == want, kw
    assert grouped(fx, R=M, a_rows=M, E=2, N=N, K=K, ldo=N, ws=at(6, 0)) == E
    assert grouped(fx, R=M, a_rows=5, rows=at(7), E=2, N=N, K=K, ldo=N, ws=at(7, 1984)) == E


GROUPED_RULES = [
    (dict(R=-1), E), (dict(E=0), E), (dict(a_rows=-1), E), (dict(N=0), E), (dict(K=16), E),
    (dict(flags=7), E), (dict(ldo=5), E),
    (dict(flags=0x10), U), (dict(E=1025), U), (dict(a_rows=1 << 31), U),
    (dict(E=1000, N=1 << 22, ldo=1 << 22), U),
    (dict(off=None), E), (dict(bq=None), E), (dict(as_=None), E), (dict(out=None), E),
    (dict(a_rows=7), E), (dict(a_rows=0, rows=at(7)), E),
    (dict(off=at(6, 2)), A), (dict(rows=at(7, 1)), A), (dict(aq=at(1, 2)), A),
    (dict(out=at(5, 1)), A), (dict(bs=at(4, 4), flags=0x20), A),
    (dict(out=at(6, 14)), E), (dict(rows=at(5, 1148)), E), (dict(out=at(3, 3 * 72 * 48 - 2)), E),
    # three experts' tilings of 128 x 4 bytes
    (dict(out=at(4, 3 * 512 - 2), flags=0x20), E),
]


@pytest.mark.parametrize("kw,want", GROUPED_RULES)
def test_grouped_rules(fx, kw, want):
    assert grouped(fx, **kw) == want
    assert fx.mx_last_variant() == fx.MX_VARIANT_NONE


def test_grouped_without_rows(fx):
    assert grouped(fx, R=0) == 0 and grouped(fx, R=0, aq=None, off=None, out=None, a_rows=0) == 0
    assert grouped(fx, R=0, E=0) == E


@no_device
@pytest.mark.parametrize("kw", [{}, dict(rows=at(7), a_rows=1), dict(a_rows=100), dict(E=1024),
                                dict(flags=0x22), dict(out=at(4, 3 * 512), flags=0x20)])
def test_grouped_accepts(fx, kw):
    assert grouped(fx, **kw) == CUDA


def silu(fx, **kw):
    a = dict(x=at(1), ldx=512, mode=0, M=4, H=256, n=None, q=at(2), s=at(3), y=None)
    a.update(kw)
    return fx.mx_silu_mul_quant(a["x"], a["ldx"], a["mode"], a["M"], a["H"], a["n"], a["q"],
                                a["s"], a["y"], None)


SILU_RULES = [
    (dict(M=-1), E), (dict(H=0), E), (dict(H=12, ldx=24), E), (dict(ldx=504), E),
    (dict(mode=3), E), (dict(mode=-1), E), (dict(mode=0x100), E), (dict(mode=0x202), E),
    (dict(mode=0x402), E), (dict(mode=1, H=192), E), (dict(mode=2, H=40), E),
    (dict(H=32776, ldx=65552), U), (dict(M=1 << 29), U), (dict(ldx=(1 << 31) + 8), U),
    (dict(x=None), E), (dict(q=None), E), (dict(s=None), E),
    (dict(x=at(1, 8)), A), (dict(ldx=516), A), (dict(y=at(4, 8)), A), (dict(n=at(5, 2)), A),
    (dict(q=at(2, 4)), A), (dict(s=at(3, 2)), A), (dict(q=at(2, 2), mode=2), A),
    (dict(q=at(1, 1024)), E), (dict(y=at(1, 3 * 1024 + 1008)), E), (dict(s=at(2, 1020)), E),
    (dict(y=at(2, -2032)), E), (dict(n=at(2, 8)), E), (dict(n=at(3, 12)), E),
    (dict(s=at(3), y=at(3, 1008), mode=0x102), E),
]


@pytest.mark.parametrize("kw,want", SILU_RULES)
def test_silu_rules(fx, kw, want):
    assert silu(fx, **kw) == want
    assert fx.mx_last_variant() == fx.MX_VARIANT_NONE


def test_silu_without_rows(fx):
    assert silu(fx, M=0) == 0 and silu(fx, M=0, x=None, q=None, s=None) == 0
    assert silu(fx, M=0, H=4) == E


@no_device
@pytest.mark.parametrize("kw", [{}, dict(mode=0x1102), dict(mode=0x1201), dict(n=at(5)),
                                dict(y=at(4)), dict(q=at(2, 4), s=at(3, 1), mode=2),
                                dict(ldx=1024), dict(H=32768, ldx=65536), dict(H=8, ldx=16)])
def test_silu_accepts(fx, kw):
    assert silu(fx, **kw) == CUDA


def combine(fx, **kw):
    a = dict(y=at(1), R=9, pos=at(2), w=at(3), base=None, T=5, k=4, N=72, flags=0, out=at(4))
    a.update(kw)
    return fx.mx_combine(a["y"], a["R"], a["pos"], a["w"], a["base"], a["T"], a["k"], a["N"],
                         a["flags"], a["out"], None)


COMBINE_RULES = [
    (dict(T=-1), E), (dict(R=-1), E), (dict(k=-1), E), (dict(N=0), E), (dict(flags=1), E),
    (dict(k=33), U), (dict(N=(1 << 24) + 1), U), (dict(T=1 << 31, N=1), U), (dict(R=1 << 31), U),
    (dict(T=1 << 24, N=1 << 20), U),
    (dict(out=None), E), (dict(pos=None), E), (dict(w=None), E), (dict(y=None), E),
    (dict(y=at(1, 1)), A), (dict(base=at(5, 1)), A), (dict(out=at(4, 3)), A),
    (dict(pos=at(2, 2)), A), (dict(w=at(3, 1)), A),
    (dict(out=at(1, 9 * 144 - 2)), E), (dict(out=at(2, 78)), E), (dict(out=at(3)), E),
    (dict(base=at(4, 144)), E),
]


@pytest.mark.parametrize("kw,want", COMBINE_RULES)
def test_combine_rules(fx, kw, want):
    assert combine(fx, **kw) == want
    assert fx.mx_last_variant() == fx.MX_VARIANT_NONE


def test_combine_without_rows(fx):
    assert combine(fx, T=0) == 0 and combine(fx, T=0, y=None, pos=None, w=None, out=None) == 0


@no_device
@pytest.mark.parametrize("kw", [{}, dict(base=at(4)), dict(k=0, pos=None, w=None, y=None),
                                dict(R=0, y=None), dict(flags=0x1000), dict(y=at(1, 2)),
                                dict(N=1), dict(k=32)])
def test_combine_accepts(fx, kw):
    assert combine(fx, **kw) == CUDA


def test_every_device_wait_is_bounded():
    """The kernels spin only through the bounded waits."""
    csrc = os.path.join(ROOT, "mxfp4_quantization_b200", "csrc")
    for name in ("tc_device.cuh", "mg_kernel.cuh", "mgp_kernel.cuh", "mg_common.cuh",
                 "act_kernel.cuh", "combine_kernel.cuh"):
        src = open(os.path.join(csrc, name)).read()
        assert not re.search(r"while\s*\(\s*!\s*mbar|while\s*\(\s*(true|1)\s*\)|for\s*\(\s*;\s*;", src)
