"""The operators of libfusedmx.so as a serving step uses them: rmsnorm_quant,
the experts' two products with the gated activation between them, the weighted
sum, and the next rmsnorm_quant on the result; every stage against its own
64-bit form on the inputs that the stage had."""
import pytest
import torch

from tests import mx_ref

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module")
def libs():
    from mxfp4_quantization_b200.build import build_library, build_mx_library
    build_library()
    build_mx_library()
    from mxfp4_quantization_b200 import fusedmx, fusednorm
    return fusednorm, fusedmx


def route(ids, E):
    """Choices [T, k] in expert order: offsets, source token, row of each choice."""
    T, k = ids.shape
    flat = ids.flatten()
    order = torch.sort(flat, stable=True).indices
    off = torch.zeros(E + 1, dtype=torch.int32, device=ids.device)
    off[1:] = torch.bincount(flat, minlength=E).cumsum(0)
    pos = torch.empty_like(order)
    pos[order] = torch.arange(T * k, device=ids.device)
    return off, (order // k).to(torch.int32), pos.view(T, k).to(torch.int32)


def layer(fn, fx, x, res, st, T):
    """One expert layer on T rows; all intermediate tensors."""
    q, s, h, y0 = fn.rmsnorm_quant(x, st["norm"], 1e-6, "mxfp4", residual=res, emit_y=True)
    gu = fx.grouped_gemm(q, s, st["w1"][0], st["w1"][1], st["off"], rows=st["rows"])
    a = fx.silu_mul_quant(gu, "mxfp4", num_rows=st["off"][-1:], emit_y=True)
    y = fx.grouped_gemm(a.q, a.scale, st["w2"][0], st["w2"][1], st["off"])
    out = fx.combine(y, st["pos"], st["weight"])
    nxt = fn.rmsnorm_quant(out, st["norm"], 1e-6, "mxfp4", residual=h)
    return dict(q=q, s=s, h=h, gu=gu, aq=a.q, as_=a.scale, ay=a.y, y=y, out=out, nq=nxt.q,
                ns=nxt.scale, nh=nxt.residual_out)


def setup(fn, T, k, E, hidden, inter, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    tiled = fn.FN_MXFP4 | fn.FN_SCALE_SWIZZLE_32_4_4

    def weight(n, kk):
        w = (torch.randn((E, n, kk), generator=g, device="cuda") / kk ** 0.5).to(BF)
        pairs = [fn.quant(w[e], tiled) for e in range(E)]
        return torch.stack([p[0] for p in pairs]), torch.stack([p[1] for p in pairs])

    ids = torch.stack([torch.randperm(E, generator=g, device="cuda")[:k] for _ in range(T)])
    ids = torch.where(ids == 1, 2 if k == 1 else ids, ids)  # (with k = 1 expert 1 stays idle)
    off, rows, pos = route(ids, E)
    x = torch.randn((T, hidden), generator=g, device="cuda").to(BF)
    res = torch.randn((T, hidden), generator=g, device="cuda").to(BF)
    norm = (1 + 0.1 * torch.randn(hidden, generator=g, device="cuda")).to(BF)
    return x, res, dict(off=off, rows=rows, pos=pos, norm=norm, w1=weight(2 * inter, hidden),
                        w2=weight(hidden, inter),
                        weight=torch.softmax(torch.randn((T, k), generator=g, device="cuda"), 1))


def from_tiles(t, rows, groups):
    tiles = mx_ref.round_up(groups, 4) // 4
    r = torch.arange(rows, device=t.device).unsqueeze(1)
    c = torch.arange(groups, device=t.device).unsqueeze(0)
    return t[((r // 128) * tiles + c // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + c % 4]


@pytest.mark.parametrize("T,k,E,hidden,inter", [(1, 2, 4, 256, 128), (7, 1, 3, 512, 160),
                                                (130, 4, 8, 384, 192), (33, 3, 5, 2048, 256)])
def test_layer(libs, T, k, E, hidden, inter):
    fn, fx = libs
    x, res, st = setup(fn, T, k, E, hidden, inter, T)
    r = layer(fn, fx, x, res, st, T)
    a = mx_ref.values(r["q"], r["s"])
    mid = mx_ref.values(r["aq"], r["as_"])
    for e in range(E):
        lo, hi = int(st["off"][e]), int(st["off"][e + 1])
        w1 = mx_ref.values(st["w1"][0][e], from_tiles(st["w1"][1][e], 2 * inter, hidden // 32))
        w2 = mx_ref.values(st["w2"][0][e], from_tiles(st["w2"][1][e], hidden, inter // 32))
        mx_ref.check_product(r["gu"][lo:hi], *mx_ref.product(a[st["rows"][lo:hi].long()], w1), hidden)
        mx_ref.check_product(r["y"][lo:hi], *mx_ref.product(mid[lo:hi], w2), inter)
    g, u = r["gu"][:, :inter].double(), r["gu"][:, inter:].double()
    act = mx_ref.round16((g * u / (1 + torch.exp(-g))).cpu().numpy(), BF)
    assert (r["ay"].double().cpu().numpy() == act).all()
    q, s = fn.quant(r["ay"], "mxfp4")
    assert torch.equal(q, r["aq"]) and torch.equal(s, r["as_"])
    terms = st["weight"].double()[..., None] * r["y"][st["pos"].long()].double()
    tol = k * 2.0 ** -23 * terms.abs().sum(1) + 2.0 ** -8 * terms.sum(1).abs()
    assert bool(((r["out"].double() - terms.sum(1)).abs() <= tol).all())


def test_layer_in_a_graph_and_as_programmatic_launches(libs):
    """The whole chain captured once and replayed on new inputs and a new
    routing in the same buffers, with programmatic launches too."""
    fn, fx = libs
    T, k, E, hidden, inter = 24, 2, 6, 512, 256
    x, res, st = setup(fn, T, k, E, hidden, inter, 1)
    for pdl in (False, True):
        with fn.programmatic_launch(pdl), fx.programmatic_launch(pdl):
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                layer(fn, fx, x, res, st, T)
            torch.cuda.current_stream().wait_stream(side)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                held = layer(fn, fx, x, res, st, T)
        for seed in (1, 2, 3):
            nx, nres, new = setup(fn, T, k, E, hidden, inter, seed)
            x.copy_(nx), res.copy_(nres)
            for name in ("off", "rows", "pos", "weight", "norm"):
                st[name].copy_(new[name])
            for name in ("w1", "w2"):
                for i in range(2):
                    st[name][i].copy_(new[name][i])
            graph.replay()
            torch.cuda.synchronize()
            want = layer(fn, fx, nx, nres, new, T)
            for name in held:
                assert torch.equal(held[name], want[name]), name
