"""Cases and plain forms of the operators around an MXFP4 product.

Four operators, as a serving program chains them behind rmsnorm_quant:

  gemm            out = A B^T of two MXFP4 operands (E2M1 codes, one E8M0
                  scale per 32 elements): a linear layer on quantized rows
  grouped_gemm    the same with a weight for each expert and ragged row
                  ranges, the rows gathered by index or already in order
  silu_mul_quant  silu(gate) * up of rows [gate | up], rounded to 16 bits and
                  quantized (MXFP4, or FP8 E4M3 per token or per 128 elements)
  combine         the weighted sum of every token's expert rows

`own` false computes them in elementary torch operations; `own` true makes the
calls of mxfp4_quantization_b200.fusedmx.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
MODES = ("fp8_per_token", "fp8_per_group128", "mxfp4")
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one token through a linear layer that returns to the hidden size
        {"name": "gemm decode M=1", "op": "gemm", "M": 1, "N": 7168, "K": 2048, "out": "bf16",
         "a_swizzled": False},
        # a decode batch through a wide linear layer
        {"name": "gemm decode M=16", "op": "gemm", "M": 16, "N": 8192, "K": 7168, "out": "bf16",
         "a_swizzled": False},
        # a ragged batch, an odd output width (a vocabulary slice), a row that
        # ends inside a 64-element step, full-precision output
        {"name": "gemm odd", "op": "gemm", "M": 333, "N": 1001, "K": 2592, "out": "fp32",
         "a_swizzled": False},
        # prefill of 8192 tokens
        {"name": "gemm prefill", "op": "gemm", "M": 8192, "N": 8192, "K": 7168, "out": "bf16",
         "a_swizzled": True},
        # decode of a few tokens through many experts: most experts are idle
        {"name": "grouped decode T=4", "op": "grouped", "T": 4, "top": 8, "E": 64, "N": 4096,
         "K": 7168, "out": "bf16", "gather": True, "spare": 0, "skew": 0.5},
        # a mixed batch in expert order already, odd sizes, binary16, a
        # capacity above the rows in use
        {"name": "grouped odd", "op": "grouped", "T": 301, "top": 6, "E": 24, "N": 1410, "K": 2080,
         "out": "fp16", "gather": False, "spare": 90, "skew": 1.5},
        # prefill: the first expert product, rows gathered from the tokens
        {"name": "grouped prefill", "op": "grouped", "T": 4096, "top": 8, "E": 32, "N": 4096,
         "K": 7168, "out": "bf16", "gather": True, "spare": 0, "skew": 0.5},
        # the activation between the two expert products: decode, prefill, and
        # the FP8 form of binary16 rows with the 16-bit row kept
        {"name": "silu decode mxfp4", "op": "silu", "M": 32, "H": 2048, "mode": "mxfp4",
         "dtype": "bf16", "spare": 0, "emit_y": False},
        {"name": "silu prefill mxfp4", "op": "silu", "M": 32768, "H": 2048, "mode": "mxfp4",
         "dtype": "bf16", "spare": 512, "emit_y": False},
        {"name": "silu odd group128", "op": "silu", "M": 4097, "H": 2560, "mode": "fp8_per_group128",
         "dtype": "fp16", "spare": 0, "emit_y": True},
        # the expert rows back to token order: a decode step, and a prefill
        # with a shared branch added
        {"name": "combine decode", "op": "combine", "T": 4, "top": 8, "N": 7168, "dtype": "bf16",
         "base": False, "dropped": 0.0},
        {"name": "combine prefill", "op": "combine", "T": 4096, "top": 8, "N": 7168,
         "dtype": "bf16", "base": True, "dropped": 0.02},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("gemm", "gemm", "grouped", "grouped", "silu", "combine"))
    out = rng.choice(("bf16", "bf16", "fp16", "fp32"))
    if op == "gemm":
        n, k = _log(rng, 16, 8192), 32 * _log(rng, 1, 256)
        m = min(_log(rng, 1, 8192), max(1, 8192 * 8192 * 7168 // (n * k)))
        return {"op": op, "M": m, "N": n, "K": k, "out": out, "a_swizzled": rng.random() < 0.5}
    if op == "grouped":
        experts = _log(rng, 2, 64)
        n, k = _log(rng, 64, 4096), 32 * _log(rng, 2, 224)
        tokens = min(_log(rng, 1, 4096), 4096 * 8 * 32 // experts)
        top = min(rng.randint(1, 8), experts)
        return {"op": op, "T": tokens, "top": top, "E": experts, "N": n, "K": k, "out": out,
                "gather": rng.random() < 0.5, "spare": rng.choice((0, 0, 7, 128)),
                "skew": round(rng.uniform(0.0, 2.0), 3)}
    if op == "silu":
        mode = rng.choice(MODES)
        step = 128 if mode == "fp8_per_group128" else 32
        h = step * _log(rng, 1, 8192 // step)
        m = min(_log(rng, 1, 32768), 32768 * 2048 // h)
        return {"op": op, "M": m, "H": h, "mode": mode, "dtype": rng.choice(("bf16", "fp16")),
                "spare": rng.choice((0, 0, 5)), "emit_y": rng.random() < 0.5}
    n = _log(rng, 16, 8192)
    return {"op": op, "T": _log(rng, 1, 4096), "top": rng.randint(1, 8), "N": n,
            "dtype": rng.choice(("bf16", "fp16")), "base": rng.random() < 0.5,
            "dropped": rng.choice((0.0, 0.0, 0.05))}


# ---- inputs -----------------------------------------------------------------------------


def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed((seed * 1_000_003 + salt * 7919) % (1 << 62))
    return g


def _pow2(e):
    """2^e of whole numbers, fp64, from the format's exponent field."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _mxfp4(x):
    """The OCP MX rule on fp32 rows [..., K]: packed codes (element 2i in the
    low nibble of byte i) and E8M0 bytes."""
    b = x.unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1)
    e = (torch.frexp(amax).exponent - 3).clamp(-127, 127)
    e = torch.where(amax == 0, torch.full_like(e, -127), e)
    a = b.abs() * _pow2(-e).float().unsqueeze(-1)
    code = torch.zeros_like(a, dtype=torch.uint8)
    for t, half_up in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False),
                       (3.5, True), (5.0, False)):
        code += (a >= t) if half_up else (a > t)
    code += (b < 0).to(torch.uint8) * 8
    code = code.flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), (e + 127).to(torch.uint8)


def _quantized(rows, k, seed, salt, std, outliers):
    """MXFP4 of normal rows, in pieces; with outliers, 1 % of the entries are
    20 times larger, as activations have them."""
    q = torch.empty((rows, k // 2), dtype=torch.uint8, device="cuda")
    s = torch.empty((rows, k // 32), dtype=torch.uint8, device="cuda")
    g = _gen(seed, salt)
    step = max(1, (1 << 26) // k)
    for i in range(0, rows, step):
        x = torch.randn((min(step, rows - i), k), generator=g, device="cuda") * std
        if outliers:
            x = torch.where(torch.rand(x.shape, generator=g, device="cuda") < 0.01, x * 20, x)
        q[i:i + step], s[i:i + step] = _mxfp4(x)
    return q, s


def _to_tiles(s):
    """E8M0 [..., R, G] in the 32x4x4 tiling of block-scaled products, flat per
    leading index, with zeros in the padding."""
    lead, (r, c) = s.shape[:-2], s.shape[-2:]
    p = torch.zeros((*lead, -(-r // 128) * 128, -(-c // 4) * 4), dtype=torch.uint8, device=s.device)
    p[..., :r, :c] = s
    t = p.unflatten(-1, (-1, 4)).unflatten(-3, (-1, 4, 32))  # [.., R/128, 4, 32, C/4, 4]
    n = len(lead)
    t = t.permute(*range(n), n, n + 3, n + 2, n + 1, n + 4)
    return t.reshape(*lead, -1).contiguous()


def _from_tiles(t, r, c):
    lead, n = t.shape[:-1], t.dim() - 1
    rt, ct = -(-r // 128), -(-c // 4)
    t = t.reshape(*lead, rt, ct, 32, 4, 4)
    t = t.permute(*range(n), n, n + 3, n + 2, n + 1, n + 4)
    return t.reshape(*lead, rt * 128, ct * 4)[..., :r, :c]


def _route(tokens, top, experts, skew, seed):
    """Expert choices of every token (distinct, some experts popular) in expert
    order: offsets [E+1], source token of each row, row of each choice."""
    g = _gen(seed, 3)
    liking = -skew * torch.log(torch.arange(1, experts + 1, device="cuda", dtype=torch.float32))
    liking = liking[torch.randperm(experts, generator=g, device="cuda")]
    noise = torch.rand((tokens, experts), generator=g, device="cuda").clamp_min(1e-9)
    ids = torch.topk(liking - torch.log(-torch.log(noise)), top, dim=1).indices
    flat = ids.flatten()
    order = torch.sort(flat, stable=True).indices
    counts = torch.bincount(flat, minlength=experts)
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0)
    pos = torch.empty_like(order)
    pos[order] = torch.arange(order.numel(), device="cuda")
    return (offsets, (order // top).to(torch.int32), pos.reshape(tokens, top).to(torch.int32),
            int(counts.max()))


def prepare(case, seed):
    op = case["op"]
    if op == "gemm":
        a_q, a_s = _quantized(case["M"], case["K"], seed, 1, 1.0, True)
        b_q, b_s = _quantized(case["N"], case["K"], seed, 2, case["K"] ** -0.5, False)
        return {"case": case, "a_q": a_q, "a_s": _to_tiles(a_s) if case["a_swizzled"] else a_s,
                "b_q": b_q, "b_s": _to_tiles(b_s)}
    if op == "grouped":
        t, e, n, k = case["T"], case["E"], case["N"], case["K"]
        offsets, rows, _, most = _route(t, case["top"], e, case["skew"], seed)
        used = t * case["top"]
        a_q, a_s = _quantized(t if case["gather"] else used + case["spare"], k, seed, 1, 1.0, True)
        b_q, b_s = _quantized(e * n, k, seed, 2, k ** -0.5, False)
        if case["gather"] and case["spare"]:
            rows = torch.cat([rows, rows.new_zeros(case["spare"])])
        out = torch.zeros((used + case["spare"], n), dtype=DT[case["out"]], device="cuda")
        return {"case": case, "a_q": a_q, "a_s": a_s, "b_q": b_q.reshape(e, n, k // 2),
                "b_s": _to_tiles(b_s.reshape(e, n, k // 32)), "offsets": offsets,
                "rows": rows if case["gather"] else None, "most": most, "used": used, "out": out}
    if op == "silu":
        g = _gen(seed, 1)
        m, h = case["M"], case["H"]
        x = torch.randn((m + case["spare"], 2 * h), generator=g, device="cuda")
        x = torch.where(torch.rand(x.shape, generator=g, device="cuda") < 0.01, x * 8, x)
        # four codes a word, for the values that a consumer of the codes sees
        w = torch.arange(1 << 16, device="cuda")
        level = torch.tensor(LEVELS + tuple(-v for v in LEVELS), device="cuda")
        table = torch.stack([level[(w >> (4 * i)) & 15] for i in range(4)], 1)
        return {"case": case, "x": x.to(DT[case["dtype"]]),
                "num_rows": torch.full((1,), m, dtype=torch.int32, device="cuda")
                if case["spare"] else None, "table": table.to(torch.bfloat16).view(torch.int64)[:, 0]}
    t, top, n = case["T"], case["top"], case["N"]
    g = _gen(seed, 1)
    y = torch.randn((t * top, n), generator=g, device="cuda").to(DT[case["dtype"]])
    pos = torch.randperm(t * top, generator=g, device="cuda").reshape(t, top)
    drop = torch.rand((t, top), generator=g, device="cuda") < case["dropped"]
    weight = torch.softmax(torch.randn((t, top), generator=g, device="cuda"), 1)
    base = torch.randn((t, n), generator=g, device="cuda").to(DT[case["dtype"]])
    return {"case": case, "y": y, "pos": torch.where(drop, -1, pos).to(torch.int32),
            "weight": weight, "base": base if case["base"] else None}


# ---- one pass -----------------------------------------------------------------------------


def _decode(q, s):
    """Packed codes and E8M0 bytes -> fp32 values."""
    level = torch.tensor(LEVELS + tuple(-v for v in LEVELS), device=q.device)
    v = torch.stack([level[(q & 15).int()], level[(q >> 4).int()]], -1).flatten(-2)
    return (v.unflatten(-1, (-1, 32)) * _pow2(s.int() - 127).float().unsqueeze(-1)).flatten(-2)


def _round16(v, dtype):
    """fp64 -> 16-bit format, one rounding to nearest even."""
    bits, low = (8, -133) if dtype == torch.bfloat16 else (11, -24)
    e = (torch.frexp(v).exponent - bits).clamp_min(low)
    return (torch.round(v * _pow2(-e)) * _pow2(e)).to(dtype)


def _plain_silu(st):
    case, x = st["case"], st["x"]
    m, h = case["M"], case["H"]
    g, u = x[:m, :h].double(), x[:m, h:].double()
    y = _round16(g / (1 + torch.exp(-g)) * u, x.dtype)
    out = {}
    if case["mode"] == "mxfp4":
        q, s = _mxfp4(y.float())
        codes = _decode(q, torch.full_like(s, 127))
        out["q"], out["scale"] = codes.to(torch.bfloat16), _pow2(s.int() - 127).float()
    else:
        group = 128 if case["mode"] == "fp8_per_group128" else h
        b = y.float().unflatten(-1, (-1, group))
        amax = b.abs().amax(-1)
        s = torch.where(amax == 0, torch.ones_like(amax), amax / torch.full_like(amax, 448))
        out["q"] = (b / s.unsqueeze(-1)).flatten(-2).to(torch.float8_e4m3fn)
        out["scale"] = s
    if case["emit_y"]:
        out["y"] = y
    return out


def _plain(st):
    case = st["case"]
    op = case["op"]
    if op == "gemm":
        a_s = _from_tiles(st["a_s"], case["M"], case["K"] // 32) if case["a_swizzled"] else st["a_s"]
        a = _decode(st["a_q"], a_s)
        b = _decode(st["b_q"], _from_tiles(st["b_s"], case["N"], case["K"] // 32))
        return torch.matmul(a, b.T).to(DT[case["out"]])
    if op == "grouped":
        e, n, k, used, most = case["E"], case["N"], case["K"], st["used"], st["most"]
        a = _decode(st["a_q"], st["a_s"])
        row = torch.arange(used, device=a.device, dtype=torch.int32)
        expert = torch.searchsorted(st["offsets"][1:], row, right=True)
        slot = expert * most + (row - st["offsets"][expert])
        padded = torch.zeros((e * most, k), device=a.device)
        padded[slot] = a[st["rows"][:used].long()] if case["gather"] else a[:used]
        b = _decode(st["b_q"], _from_tiles(st["b_s"], n, k // 32))
        y = torch.bmm(padded.reshape(e, most, k), b.transpose(1, 2))
        out = torch.zeros_like(st["out"])
        out[:used] = y.reshape(e * most, n)[slot].to(out.dtype)
        return out
    if op == "silu":
        return _plain_silu(st)
    pos, dtype = st["pos"].long(), st["y"].dtype
    part = st["y"][pos.clamp_min(0)].float() * (st["weight"] * (pos >= 0)).unsqueeze(-1)
    total = part.sum(1)
    return (total if st["base"] is None else total + st["base"].float()).to(dtype)


def _own(st):
    from mxfp4_quantization_b200 import fusedmx as fx
    case = st["case"]
    op = case["op"]
    if op == "gemm":
        return fx.gemm(st["a_q"], st["a_s"], st["b_q"], st["b_s"], out_dtype=DT[case["out"]])
    if op == "grouped":
        return fx.grouped_gemm(st["a_q"], st["a_s"], st["b_q"], st["b_s"], st["offsets"],
                               rows=st["rows"], out=st["out"])
    if op == "silu":
        m = case["M"]
        r = fx.silu_mul_quant(st["x"], case["mode"], num_rows=st["num_rows"],
                              emit_y=case["emit_y"])
        out = {"q": r.q[:m], "scale": r.scale[:m]}
        if case["mode"] == "mxfp4":  # the values that the codes stand for
            words = r.q[:m].view(torch.int16).int() & 0xFFFF
            out["q"] = st["table"].index_select(0, words.flatten()).view(torch.bfloat16).view(m, -1)
            out["scale"] = r.scale[:m].view(torch.float8_e8m0fnu).float()
        if case["emit_y"]:
            out["y"] = r.y[:m]
        return out
    return fx.combine(st["y"], st["pos"], st["weight"], base=st["base"])


def run(state):
    return _own(state) if own else _plain(state)


# ---- work and the 64-bit definition ----------------------------------------------------------


def work(case):
    op = case["op"]
    if op == "gemm":
        m, n, k = case["M"], case["N"], case["K"]
        return {"bytes": (m + n) * (k // 2 + k // 32) + m * n * BYTES[case["out"]],
                "flops": 2 * m * n * k}
    if op == "grouped":
        used, e, n, k = case["T"] * case["top"], case["E"], case["N"], case["K"]
        # experts in use: all but those that no choice meets, evenly spread
        active = e * (1 - (1 - case["top"] / e) ** case["T"])
        source = case["T"] if case["gather"] else used
        return {"bytes": int((source + active * n) * (k // 2 + k // 32)) +
                used * n * BYTES[case["out"]], "flops": 2 * used * n * k}
    if op == "silu":
        m, h = case["M"], case["H"]
        codes = {"mxfp4": h // 2 + h // 32, "fp8_per_group128": h + h // 32,
                 "fp8_per_token": h + 4}[case["mode"]]
        return {"bytes": m * (4 * h + codes + (2 * h if case["emit_y"] else 0)), "flops": 6 * m * h}
    t, top, n = case["T"], case["top"], case["N"]
    kept = int(t * top * (1 - case["dropped"]))
    return {"bytes": 2 * n * (kept + t * (2 if case["base"] else 1)) + 8 * t * top,
            "flops": 2 * kept * n}


def _values(q, s):
    """Packed codes and E8M0 bytes -> fp64 values, from the format's fields:
    sign, two exponent bits (bias 1), one mantissa bit."""
    n = torch.stack([q & 15, q >> 4], -1).flatten(-2).long()
    sign, ex, man = n >> 3, (n >> 1) & 3, (n & 1).double()
    mag = torch.where(ex == 0, 0.5 * man, (1 + 0.5 * man) * torch.exp2((ex - 1).double()))
    v = torch.where(sign == 1, -mag, mag)
    return v * torch.exp2(s.double() - 127).repeat_interleave(32, -1)


def _rows_of(t, r, c):
    """Scales [r, c] out of the 32x4x4 tiling, entry by entry."""
    i = torch.arange(r, device=t.device).unsqueeze(1)
    j = torch.arange(c, device=t.device).unsqueeze(0)
    tiles = (c + 3) // 4
    return t[((i // 128) * tiles + j // 4) * 512 + (i % 32) * 16 + (i % 128) // 32 * 4 + j % 4]


def _nearest16(v, dtype):
    """fp64 -> 16-bit format by comparing a first guess with its two
    neighbours; ties to the even pattern."""
    bits = v.to(dtype).view(torch.int16).int()
    order = torch.where(bits < 0, -(bits & 0x7FFF), bits)
    best, miss = v.to(dtype), (v.to(dtype).double() - v).abs()
    for step in (1, -1):
        o = order + step
        other = torch.where(o < 0, -o | -0x8000, o).to(torch.int16).view(dtype)
        off = (other.double() - v).abs()
        better = (off < miss) | ((off == miss) & (o % 2 == 0))
        best, miss = torch.where(better, other, best), torch.where(better, off, miss)
    return best


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "gemm":
        m, n, g = case["M"], case["N"], case["K"] // 32
        a = _values(st["a_q"], _rows_of(st["a_s"], m, g) if case["a_swizzled"] else st["a_s"])
        b = _values(st["b_q"], _rows_of(st["b_s"], n, g))
        return a @ b.T
    if op == "grouped":
        n, g = case["N"], case["K"] // 32
        out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
        bounds = st["offsets"].tolist()
        for e in range(case["E"]):
            lo, hi = bounds[e], bounds[e + 1]
            if hi > lo:
                src = st["rows"][lo:hi].long() if case["gather"] else slice(lo, hi)
                b = _values(st["b_q"][e], _rows_of(st["b_s"][e], n, g))
                out[lo:hi] = _values(st["a_q"][src], st["a_s"][src]) @ b.T
        return out
    if op == "silu":
        m, h = case["M"], case["H"]
        x = st["x"][:m].double()
        gate, up = x[:, :h], x[:, h:]
        y = _nearest16(gate * up / (1 + torch.exp(-gate)), st["x"].dtype).double()
        group = {"mxfp4": 32, "fp8_per_group128": 128, "fp8_per_token": h}[case["mode"]]
        b = y.reshape(m, h // group, group)
        amax = b.abs().amax(-1)
        if case["mode"] == "mxfp4":
            scale = torch.where(amax == 0, 2.0 ** -127, 0.25 * torch.exp2(
                (amax.view(torch.int64) >> 52).double() - 1023).clamp_min(2.0 ** -125))
            a = b.abs() / scale.unsqueeze(-1)
            # spacing of E2M1: 0.5 below 2, 1 below 4, 2 above; round() is half-to-even
            # in each and the patterns' parity follows it
            step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
            q = torch.copysign((torch.round(a / step) * step).clamp_max(6.0), b)
        else:
            scale = torch.where(amax == 0, 1.0, (amax / torch.full_like(amax, 448)).float().double())
            quotient = (b / scale.unsqueeze(-1)).float().double()
            ex = (torch.frexp(quotient).exponent - 1).clamp_min(-6).double()
            step = torch.exp2(ex - 3)
            q = (torch.round(quotient / step) * step).clamp(-448, 448)
        out = {"q": q.reshape(m, h), "scale": scale}
        if case["emit_y"]:
            out["y"] = y
        return out
    pos = st["pos"].tolist() if case["T"] * case["top"] <= 64 else None
    if pos is not None:
        rows = [sum((st["weight"][t, j].double() * st["y"][p].double()
                     for j, p in enumerate(row) if p >= 0),
                    torch.zeros(case["N"], dtype=torch.float64, device="cuda"))
                for t, row in enumerate(pos)]
        total = torch.stack(rows)
    else:
        total = torch.zeros((case["T"], case["N"]), dtype=torch.float64, device="cuda")
        for j in range(case["top"]):
            p = st["pos"][:, j].long()
            keep = (p >= 0).nonzero().flatten()
            total[keep] += st["weight"][keep, j].double().unsqueeze(1) * st["y"][p[keep]].double()
    return total if st["base"] is None else total + st["base"].double()
