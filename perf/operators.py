"""What is measured of the microscaled 4-bit operators and of the expert routing around them.

Five kinds of pass: quantising a matrix to e2m1 codes with block scales (read back as the values it stands for); a linear
layer on such weights (its bf16 activations are quantised in the pass); the same with one weight per expert over rows sorted
by expert; sorting tokens by expert and gathering their rows, with the gather's gradient; and bringing the experts' rows back
with the router's weights, with that step's gradients. The plain form of each is elementary torch in 32 bits.

The stored form: `codes` (rows, 16 * ceil(cols / 32)) bytes, column 2i in the low half of byte i; one scale byte for each 32
(mx: a power of two, biased by 127) or 16 columns (nv: e4m3, times one fp32 number for the whole matrix), in tiles of 128 rows x 4
scales: scale b of row r is byte (r % 32) * 16 + (r % 128) / 32 * 4 + b % 4 of tile (r / 128, b / 4), 0 outside the matrix.
"""
import math

import torch

own = False

BLOCK = {"mx": 32, "nv": 16}
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------------- cases

def listed():
    return [
        # the activations of one token, before a linear layer
        {"name": "quantise one token", "op": "quantise", "rows": 1, "cols": 4096, "dtype": "bf16", "format": "mx"},
        # a whole MLP weight, when a checkpoint is converted
        {"name": "quantise a weight", "op": "quantise", "rows": 14336, "cols": 4096, "dtype": "f32", "format": "nv"},
        # a linear layer while one sequence is generated
        {"name": "linear one token", "op": "linear", "tokens": 1, "cols": 4096, "out": 4096, "format": "mx"},
        # a small batch through a layer whose sizes are no multiples of anything
        {"name": "linear ragged", "op": "linear", "tokens": 77, "cols": 1000, "out": 2310, "format": "nv"},
        # the attention projection over one calibration segment
        {"name": "linear segment", "op": "linear", "tokens": 2048, "cols": 4096, "out": 4096, "format": "nv"},
        # the widest MLP layer over eight segments
        {"name": "linear large", "op": "linear", "tokens": 16384, "cols": 4096, "out": 14336, "format": "mx"},
        # expert layer while sixteen sequences are generated
        {"name": "experts decode", "op": "experts", "tokens": 16, "top": 2, "experts": 16, "cols": 4096, "out": 1024, "format": "nv", "drop": 0.0},
        # expert layer over two calibration segments
        {"name": "experts prefill", "op": "experts", "tokens": 4096, "top": 2, "experts": 8, "cols": 4096, "out": 14336, "format": "mx", "drop": 0.01},
        # routing while a few sequences are generated
        {"name": "dispatch decode", "op": "dispatch", "tokens": 5, "top": 2, "experts": 8, "cols": 4096, "dtype": "bf16", "train": False, "drop": 0.0},
        # routing of eight segments, forward and backward
        {"name": "dispatch train", "op": "dispatch", "tokens": 16384, "top": 2, "experts": 8, "cols": 4096, "dtype": "bf16", "train": True, "drop": 0.02},
        # many small experts, fp32 rows
        {"name": "combine decode", "op": "combine", "tokens": 33, "top": 6, "experts": 64, "cols": 1000, "dtype": "f32", "train": False, "drop": 0.1},
        # the way back of eight segments, forward and backward
        {"name": "combine train", "op": "combine", "tokens": 16384, "top": 2, "experts": 8, "cols": 4096, "dtype": "bf16", "train": True, "drop": 0.02},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("quantise", "linear", "linear", "experts", "dispatch", "combine"))
    form = rng.choice(("mx", "nv"))
    if op == "quantise":
        rows = _log(rng, 1, 16384)
        cols = _log(rng, 17, max(18, min(14336, 14336 * 4096 // rows)))
        return {"op": op, "rows": rows, "cols": cols, "dtype": rng.choice(("bf16", "f32")), "format": form}
    if op == "linear":
        tokens = _log(rng, 1, 16384)
        cols, out = _log(rng, 64, 14336), _log(rng, 24, 14336)
        return {"op": op, "tokens": tokens, "cols": cols, "out": min(out, max(1, 16384 * 4096 * 14336 // (tokens * cols))), "format": form}
    top = rng.randint(1, 8)
    experts = max(top, _log(rng, 2, 128))
    drop = rng.choice((0.0, 0.01, 0.3))
    if op == "experts":
        tokens, cols, out = _log(rng, 1, 4096), _log(rng, 64, 4096), _log(rng, 24, 4096)
        top, experts = min(top, 4), min(experts, 32)
        return {"op": op, "tokens": tokens, "top": min(top, experts), "experts": experts, "cols": cols, "out": out, "format": form, "drop": drop}
    tokens = _log(rng, 1, 16384)
    cols = _log(rng, 33, max(34, min(8192, 16384 * 2 * 4096 // (tokens * top))))
    return {"op": op, "tokens": tokens, "top": top, "experts": experts, "cols": cols, "dtype": rng.choice(("bf16", "f32")),
            "train": rng.random() < 0.6, "drop": drop}


# --------------------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _activations(rows, cols, g, dtype=torch.bfloat16):
    """Channels of unlike size, a few of them outliers."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    channel = torch.randn(cols, generator=g, device="cuda").mul_(0.5).exp_()
    at = torch.randint(0, cols, (1 + cols // 512,), generator=g, device="cuda")
    channel[at] *= 20.0
    return (x * channel).to(dtype)


def _routes(case, g):
    """Each token's experts (the best of uneven random scores), some slots dropped, and the router's weights."""
    t, k, e = case["tokens"], case["top"], case["experts"]
    lean = torch.randn(e, generator=g, device="cuda")
    score = torch.randn(t, e, generator=g, device="cuda") + lean
    best, ids = torch.topk(score, k, dim=1)
    lost = torch.rand(t, k, generator=g, device="cuda") < case["drop"]
    ids = torch.where(lost, -1, ids).to(torch.int32)
    return ids.contiguous(), torch.softmax(best, 1).contiguous()


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = {"op": op, "grid": torch.tensor(GRID + tuple(-v for v in GRID), device="cuda")}
    if op == "quantise":
        if case["dtype"] == "f32":
            s["x"] = torch.randn(case["rows"], case["cols"], generator=g, device="cuda") * 0.02
        else:
            s["x"] = _activations(case["rows"], case["cols"], g)
        s |= {"format": case["format"], "scale": _tensor_scale(s["x"], case["format"])}
        return s
    if op in ("linear", "experts"):
        k, n = case["cols"], case["out"]
        e = case.get("experts", 1)
        w = torch.randn(e * n, k, generator=g, device="cuda") * 0.02
        s["w_scale"] = _tensor_scale(w, case["format"])
        codes, scales = _plain_quantise(w, case["format"], s["w_scale"])
        del w
        codes = codes.view(e, n, -1)
        scales = scales.view(e, n, -1)
        s |= {"format": case["format"], "cols": k, "w_codes": _packed(codes), "w_scales": _tiled(scales)}
        if op == "experts":
            ids, _ = _routes(case, g)
            s["offsets"] = _plain_sort(ids, e)[0]
            s["most"] = max(1, int((s["offsets"][1:] - s["offsets"][:-1]).max()))
            s["x"] = _activations(ids.numel(), k, g)
        else:
            s["w_codes"], s["w_scales"] = s["w_codes"][0], s["w_scales"][0]
            s["x"] = _activations(case["tokens"], k, g)
        s["x_scale"] = _tensor_scale(s["x"], case["format"])
        return s
    ids, weights = _routes(case, g)
    t, k, d, dt = case["tokens"], case["top"], case["cols"], DTYPE[case["dtype"]]
    s |= {"experts": case["experts"], "train": case["train"]}
    if op == "dispatch":
        s |= {"ids": ids, "x": _activations(t, d, g, dt)}
        if case["train"]:
            s["dxs"] = torch.randn(t * k, d, generator=g, device="cuda").to(dt)
        return s
    s["offsets"], s["src"], s["pos"] = _plain_sort(ids, case["experts"])
    s |= {"weights": weights, "ys": torch.randn(t * k, d, generator=g, device="cuda").to(dt)}
    if case["train"]:
        s["dy"] = torch.randn(t, d, generator=g, device="cuda").to(dt)
    return s


# ------------------------------------------------------------------------------ plain forms

def _tensor_scale(x, form):
    """nv: the least power of two that brings every block's scale within e4m3 (448); mx has none."""
    if form == "mx":
        return None
    _, e = torch.frexp(x.abs().amax().float() / 2688.0)
    return torch.ldexp(torch.ones((), device=x.device), e).reshape(1)


def _power(byte):
    """2 ** (byte - 127) in fp32, by its bits."""
    return torch.where(byte > 0, byte.int() << 23, 1 << 22).view(torch.float32)


def _plain_quantise(x, form, scale):
    """The 4-bit codes (rows, columns up to whole blocks of 32) and the blocks' scale bytes (rows, blocks)."""
    block = BLOCK[form]
    rows, cols = x.shape
    xb = torch.nn.functional.pad(x.float(), (0, -cols % 32)).view(rows, -1, block)
    most = xb.abs().amax(-1, keepdim=True)
    if form == "mx":
        _, e = torch.frexp(most)
        byte = torch.where(most > 0, (e + 124).clamp(0, 254), 0)
        y = xb / _power(byte)
        byte = byte.to(torch.uint8)
    else:
        s8 = (most / (scale * 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn)
        d = s8.float() * scale
        y = torch.where(d > 0, xb / d, 0.0)
        byte = s8.view(torch.uint8)
    m = y.abs()
    code = (m > 0.25).to(torch.uint8)
    code += m >= 0.75
    code += m > 1.25
    code += m >= 1.75
    code += m > 2.5
    code += m >= 3.5
    code += m > 5.0
    code += 8 * (y < 0).to(torch.uint8)
    return code.view(rows, -1), byte.view(rows, -1)


def _packed(code):
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _tiled(byte):
    """(..., rows, blocks) -> (..., row tiles, block tiles, 512)"""
    rows, blocks = byte.shape[-2:]
    b = torch.nn.functional.pad(byte, (0, -blocks % 4, 0, -rows % 128))
    b = b.view(*byte.shape[:-2], -(-rows // 128), 4, 32, -(-blocks // 4), 4)
    return b.movedim(-2, -4).transpose(-3, -2).reshape(*byte.shape[:-2], -(-rows // 128), -(-blocks // 4), 512)


def _untiled(tiles, rows, blocks):
    b = tiles.view(*tiles.shape[:-1], 32, 4, 4).transpose(-3, -2).movedim(-4, -2)
    return b.reshape(*tiles.shape[:-3], tiles.shape[-3] * 128, tiles.shape[-2] * 4)[..., :rows, :blocks]


def _plain_values(code, byte, form, scale, grid):
    """The values in fp32 of codes (..., rows, columns up to whole blocks of 32) and scale bytes (..., rows, blocks)."""
    v = grid[code.int()].view(*byte.shape, BLOCK[form])
    s = _power(byte) if form == "mx" else byte.view(torch.float8_e4m3fn).float() * scale
    return (v * s.unsqueeze(-1)).view(code.shape)


def _plain_weight(s, rows):
    code = torch.stack((s["w_codes"] & 15, s["w_codes"] >> 4), -1).flatten(-2)
    byte = _untiled(s["w_scales"], rows, code.shape[-1] // BLOCK[s["format"]])
    return _plain_values(code, byte.contiguous(), s["format"], s["w_scale"], s["grid"])


def _plain_sort(ids, experts):
    """Offsets (experts + 1), the slot in each place (-1: none) and each slot's place (-1: dropped)."""
    flat = torch.where(ids.flatten() < 0, experts, ids.flatten())
    count = (flat.unsqueeze(1) == torch.arange(experts, device=ids.device)).sum(0)
    offsets = torch.nn.functional.pad(count.cumsum(0), (1, 0))
    _, order = torch.sort(flat, stable=True)
    place = torch.arange(flat.numel(), device=ids.device)
    live = place < offsets[-1]
    pos = torch.empty_like(place)
    pos[order] = torch.where(live, place, -1)
    return offsets.to(torch.int32), torch.where(live, order, -1).to(torch.int32), pos.view(ids.shape).to(torch.int32)


def _plain_back(rows, pos, weights):
    """sum over a token's slots of weight x the slot's row, in fp32"""
    got = rows.float()[pos.clamp(min=0).long()] * (pos >= 0).unsqueeze(-1)
    return (got * weights.unsqueeze(-1) if weights is not None else got).sum(1)


def _plain_run(s):
    op = s["op"]
    if op == "quantise":
        x, form = s["x"], s["format"]
        code, byte = _plain_quantise(x, form, s["scale"])
        return {"values": _plain_values(code, byte, form, s["scale"], s["grid"])[:, :x.shape[1]].contiguous()}
    if op == "linear":
        code, byte = _plain_quantise(s["x"], s["format"], s["x_scale"])
        x = _plain_values(code, byte, s["format"], s["x_scale"], s["grid"])
        return {"y": (x @ _plain_weight(s, s["w_codes"].shape[0]).T).to(torch.bfloat16)}
    if op == "experts":
        code, byte = _plain_quantise(s["x"], s["format"], s["x_scale"])
        x = _plain_values(code, byte, s["format"], s["x_scale"], s["grid"])
        w = _plain_weight(s, s["w_codes"].shape[1])
        first = s["offsets"].long()
        row = torch.arange(x.shape[0], device=x.device)
        live = row < first[-1]
        e = (row.unsqueeze(1) >= first[1:]).sum(1).clamp(max=w.shape[0] - 1)
        at = torch.where(live, row - first[e], 0)
        padded = torch.zeros(w.shape[0], s["most"], x.shape[1], device=x.device)
        padded.index_put_((e, at), x * live.unsqueeze(1), accumulate=True)
        y = torch.bmm(padded, w.transpose(1, 2))[e, at] * live.unsqueeze(1)
        return {"y": y.to(torch.bfloat16)}
    if op == "dispatch":
        offsets, src, pos = _plain_sort(s["ids"], s["experts"])
        top = s["ids"].shape[1]
        token = (src.clamp(min=0) // top).long()
        out = {"offsets": offsets, "src": src, "pos": pos, "xs": s["x"][token] * (src >= 0).unsqueeze(1)}
        if s["train"]:
            out["dx"] = _plain_back(s["dxs"], pos, None).to(s["x"].dtype)
        return out
    pos, src, w, ys = s["pos"], s["src"].long(), s["weights"], s["ys"]
    out = {"y": _plain_back(ys, pos, w).to(ys.dtype)}
    if s["train"]:
        slot, live = src.clamp(min=0), src >= 0
        dy = s["dy"].float()
        out["dys"] = (dy[slot // pos.shape[1]] * (w.flatten()[slot] * live).unsqueeze(1)).to(ys.dtype)
        got = ys.float()[pos.clamp(min=0).long()]
        out["dw"] = (got * dy.unsqueeze(1)).sum(-1) * (pos >= 0)
    return out


# --------------------------------------------------------------------------------- one pass

_library = None


def _framework():
    """The framework, set as a serving program sets it: errors found on the device are left for status_sync."""
    global _library
    if _library is None:
        import post_weight_quantization_04_gb300 as g
        g.set_status_mode(True)
        _library = g
    return _library


def run(state):
    if not own:
        return _plain_run(state)
    g, s, op = _framework(), state, state["op"]
    if op == "quantise":
        q = g.gptq_fp4_quantize(s["x"], s["format"], s["scale"])
        return {"values": g.gptq_fp4_dequantize(q, torch.float32)}
    if op in ("linear", "experts"):
        w = g.Fp4(s["w_codes"], s["w_scales"], s["cols"], s["format"], s["w_scale"])
        q = g.gptq_fp4_quantize(s["x"], s["format"], s["x_scale"])
        return {"y": g.gptq_fp4_matmul(q, w, offsets=s.get("offsets"), out_dtype=torch.bfloat16)}
    if op == "dispatch":
        route = g.gptq_expert_sort(s["ids"], s["experts"])
        out = {"offsets": route.offsets, "src": route.src, "pos": route.pos, "xs": g.gptq_expert_gather(s["x"], route)}
        if s["train"]:
            out["dx"] = g.gptq_expert_gather_grad(s["dxs"], route)
        return out
    route = g.Route(s["offsets"], s["src"], s["pos"])
    out = {"y": g.gptq_expert_combine(s["ys"], route, s["weights"])}
    if s["train"]:
        out["dys"], out["dw"] = g.gptq_expert_combine_grad(s["dy"], s["ys"], route, s["weights"])
    return out


def work(case):
    op = case["op"]
    if op == "quantise":
        r, c = case["rows"], case["cols"]
        return {"bytes": r * c * ((2 if case["dtype"] == "bf16" else 4) + 4), "flops": 4 * r * c}
    if op in ("linear", "experts"):
        k, n, block = case["cols"], case["out"], BLOCK[case["format"]]
        rows = case["tokens"] * case.get("top", 1)
        weights = min(case.get("experts", 1), rows)
        return {"bytes": 2 * rows * k + weights * n * (k // 2 + k // block) + 2 * rows * n, "flops": 2 * rows * n * k}
    t, k, d = case["tokens"], case["top"], case["cols"]
    size = 2 if case["dtype"] == "bf16" else 4
    if op == "dispatch":
        moved = 12 * t * k + (t + t * k) * d * size
        return {"bytes": moved * (2 if case["train"] else 1), "flops": t * k * d if case["train"] else 0}
    moved, flops = 8 * t * k + (t + t * k) * d * size, 2 * t * k * d
    if case["train"]:
        moved, flops = moved + 4 * t * k + (t + t * k) * d * size, flops + 3 * t * k * d
    return {"bytes": moved, "flops": flops}


# ------------------------------------------------------------------------------------ exact

def _exact_floor(v):
    """The greatest power of two up to v, in fp64."""
    _, e = torch.frexp(v)
    return torch.ldexp(torch.full_like(v, 0.5), e)


def _exact_rounded(x, form, scale):
    """What x stands for once quantised, from the definition in fp64: the nearest e2m1 multiple of its block's scale."""
    rows, cols = x.shape
    block = BLOCK[form]
    x = torch.cat((x.double(), x.new_zeros(rows, -cols % block, dtype=torch.float64)), 1).reshape(-1, block)
    a = x.abs().max(1, keepdim=True).values
    if form == "mx":
        s = _exact_floor(a.clamp(min=1e-300)).div(4).clamp(min=2.0 ** -127)
    else:
        r = (a / (6 * scale.double())).clamp(max=448)
        step = _exact_floor(r.clamp(min=2.0 ** -6)) / 8
        s = torch.round(r / step) * step * scale.double()
    y = x / torch.where(s > 0, s, 1.0)
    m = y.abs()
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))
    v = (torch.round(m / step) * step).clamp(max=6) * torch.sign(y) * s
    return v.reshape(rows, -1)[:, :cols]


def _exact_weight(codes, tiles, cols, form, scale):
    """The values of one stored matrix in fp64, scale by scale from its place in the tiles."""
    rows, block = codes.shape[0], BLOCK[form]
    r = torch.arange(rows, device=codes.device).view(-1, 1)
    b = torch.arange(-(-cols // block), device=codes.device)
    byte = tiles.reshape(-1)[((r // 128) * tiles.shape[1] + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4].long()
    if form == "mx":
        s = torch.pow(2.0, byte.double() - 127)
    else:
        e, f = byte // 8 % 16, (byte % 8).double()
        s = torch.where(e > 0, (1 + f / 8) * torch.pow(2.0, (e - 7).double()), f / 512) * scale.double()
    c = torch.arange(cols, device=codes.device)
    code = (codes[:, c // 2] >> (4 * (c % 2)).to(torch.uint8)) & 15
    e, f = (code // 2 % 4).double(), (code % 2).double()
    v = torch.where(e > 0, (1 + f / 2) * torch.pow(2.0, e - 1), f / 2)
    return torch.where(code > 7, -v, v) * s[:, c // block]


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "quantise":
        return {"values": _exact_rounded(s["x"], s["format"], s["scale"])}
    if op == "linear":
        x = _exact_rounded(s["x"], s["format"], s["x_scale"])
        return {"y": x @ _exact_weight(s["w_codes"], s["w_scales"], s["cols"], s["format"], s["w_scale"]).T}
    if op == "experts":
        x = _exact_rounded(s["x"], s["format"], s["x_scale"])
        y = x.new_zeros(x.shape[0], s["w_codes"].shape[1])
        first = s["offsets"].tolist()
        for e, (a, b) in enumerate(zip(first, first[1:])):
            if b > a:
                y[a:b] = x[a:b] @ _exact_weight(s["w_codes"][e], s["w_scales"][e], s["cols"], s["format"], s["w_scale"]).T
        return {"y": y}
    if op == "dispatch":
        ids, x = s["ids"].cpu(), s["x"].double()
        t, top = ids.shape
        slots = sorted((i for i in range(t * top) if ids.view(-1)[i] >= 0), key=ids.view(-1).tolist().__getitem__)
        at = torch.tensor(slots, dtype=torch.int64, device=x.device)
        xs = x.new_zeros(t * top, x.shape[1])
        xs[:len(slots)] = x[at // top]
        out = {"offsets": None, "src": None, "pos": None, "xs": xs}
        if s["train"]:
            out["dx"] = torch.zeros_like(x).index_add_(0, at // top, s["dxs"].double()[:len(slots)])
        return out
    at, top = s["src"][s["src"] >= 0].long(), s["pos"].shape[1]
    w, ys = s["weights"].double().view(-1), s["ys"].double()
    y = ys.new_zeros(s["pos"].shape[0], ys.shape[1]).index_add_(0, at // top, ys[:len(at)] * w[at].unsqueeze(1))
    out = {"y": y}
    if s["train"]:
        dy = s["dy"].double()[at // top]
        out["dys"] = torch.cat((dy * w[at].unsqueeze(1), ys.new_zeros(len(ys) - len(at), ys.shape[1])))
        out["dw"] = torch.zeros_like(w).index_copy_(0, at, (dy * ys[:len(at)]).sum(1)).view(s["pos"].shape)
    return out
