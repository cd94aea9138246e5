"""What is measured of the 8-bit integer operators and of the router's balance loss.

Four kinds of pass: the root-mean-square norm before a linear layer, with the residual's addition and an output in 8-bit integers
with a scale for each token (read back as the values it stands for), and in training the gradients of its inputs and gain; a linear
layer on 8-bit weights with a scale for each output channel (its bf16 activations are quantised in the pass); the same with one
weight per expert over rows sorted by expert; and the balance loss of a router with the experts' counts, and its gradient. The
plain form of each is elementary torch in 32 bits.

The stored form of a matrix: `codes` (rows, 16 * ceil(cols / 16)) int8, zeros past the columns, and one fp32 scale for each
row: value = code * scale, scale = max|x| / 127, code = the whole number nearest to x / scale, ties to even.
"""
import math

import torch

own = False

DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


# ---------------------------------------------------------------------------------- cases

def listed():
    return [
        # before the attention projections of one token
        {"name": "norm one token", "op": "norm", "rows": 1, "cols": 4096, "dtype": "bf16", "residual": True, "train": False},
        # the first norm of a small model in fp32 (nothing to add yet), sizes that are no multiples of anything
        {"name": "norm ragged", "op": "norm", "rows": 333, "cols": 2310, "dtype": "f32", "residual": False, "train": True},
        # eight calibration segments
        {"name": "norm segments", "op": "norm", "rows": 16384, "cols": 4096, "dtype": "bf16", "residual": True, "train": False},
        # the same while the gains are tuned after quantisation
        {"name": "norm train", "op": "norm", "rows": 16384, "cols": 4096, "dtype": "bf16", "residual": True, "train": True},
        # a linear layer while one sequence is generated
        {"name": "linear one token", "op": "linear", "tokens": 1, "cols": 4096, "out": 4096},
        # a small batch through a layer whose sizes are no multiples of anything
        {"name": "linear ragged", "op": "linear", "tokens": 77, "cols": 1000, "out": 2310},
        # the attention projection over one calibration segment
        {"name": "linear segment", "op": "linear", "tokens": 2048, "cols": 4096, "out": 4096},
        # the widest MLP layer over eight segments
        {"name": "linear large", "op": "linear", "tokens": 16384, "cols": 4096, "out": 14336},
        # expert layer while sixteen sequences are generated
        {"name": "experts decode", "op": "experts", "tokens": 16, "top": 2, "experts": 16, "cols": 4096, "out": 1024, "drop": 0.0},
        # expert layer over two calibration segments
        {"name": "experts prefill", "op": "experts", "tokens": 4096, "top": 2, "experts": 8, "cols": 4096, "out": 14336, "drop": 0.01},
        # the balance of a small padded batch, looked at while it is served
        {"name": "balance small", "op": "balance", "tokens": 33, "top": 6, "experts": 64, "dtype": "bf16", "padded": 0.2, "drop": 0.1, "train": False},
        # the balance loss of eight segments while the router is tuned
        {"name": "balance train", "op": "balance", "tokens": 16384, "top": 6, "experts": 64, "dtype": "f32", "padded": 0.05, "drop": 0.02, "train": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "norm", "linear", "linear", "experts", "balance"))
    if op == "norm":
        rows = _log(rng, 1, 16384)
        cols = _log(rng, 17, max(18, min(16384, 16384 * 4096 // rows)))
        return {"op": op, "rows": rows, "cols": cols, "dtype": rng.choice(("bf16", "f32")), "residual": rng.random() < 0.7, "train": rng.random() < 0.5}
    if op == "linear":
        tokens = _log(rng, 1, 16384)
        cols, out = _log(rng, 64, 14336), _log(rng, 24, 14336)
        return {"op": op, "tokens": tokens, "cols": cols, "out": min(out, max(1, 16384 * 4096 * 14336 // (tokens * cols)))}
    top = rng.randint(1, 8)
    experts = max(top, _log(rng, 2, 256))
    drop = rng.choice((0.0, 0.01, 0.3))
    if op == "experts":
        tokens, cols, out = _log(rng, 1, 4096), _log(rng, 64, 4096), _log(rng, 24, 4096)
        top, experts = min(top, 4), min(experts, 32)
        return {"op": op, "tokens": tokens, "top": min(top, experts), "experts": experts, "cols": cols, "out": out, "drop": drop}
    return {"op": op, "tokens": _log(rng, 1, 16384), "top": top, "experts": experts, "dtype": rng.choice(("bf16", "f32")),
            "padded": rng.choice((0.0, 0.2)), "drop": drop, "train": rng.random() < 0.6}


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


def _chosen(case, g):
    """A router's logits (uneven experts), each token's best experts, some slots dropped."""
    t, k, e = case["tokens"], case["top"], case["experts"]
    lean = torch.randn(e, generator=g, device="cuda")
    logits = torch.randn(t, e, generator=g, device="cuda") + lean
    ids = torch.topk(logits, k, dim=1).indices
    lost = torch.rand(t, k, generator=g, device="cuda") < case["drop"]
    return logits, torch.where(lost, -1, ids).to(torch.int32).contiguous()


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = {"op": op}
    if op == "norm":
        r, c, dt = case["rows"], case["cols"], DTYPE[case["dtype"]]
        s |= {"x": _activations(r, c, g, dt), "gain": 1.0 + 0.2 * torch.randn(c, generator=g, device="cuda"), "train": case["train"],
              "residual": _activations(r, c, g, dt) if case["residual"] else None}
        if case["train"]:
            s |= {"dy": torch.randn(r, c, generator=g, device="cuda").to(dt), "dh": torch.randn(r, c, generator=g, device="cuda").to(dt)}
        return s
    if op in ("linear", "experts"):
        k, n = case["cols"], case["out"]
        e = case.get("experts", 1)
        w = torch.randn(e * n, k, generator=g, device="cuda") * 0.02
        codes, scales = _plain_quantise(w)
        codes = torch.nn.functional.pad(codes.to(torch.int8), (0, -k % 16))
        s |= {"cols": k, "w_codes": codes, "w_scales": scales}
        if op == "experts":
            s |= {"w_codes": codes.view(e, n, -1), "w_scales": scales.view(e, n)}
            ids = _chosen(case, g)[1].flatten()
            count = (ids.unsqueeze(1) == torch.arange(e, device="cuda")).sum(0)
            s["offsets"] = torch.nn.functional.pad(count.cumsum(0), (1, 0)).to(torch.int32)
            s["most"] = max(1, int(count.max()))
            s["x"] = _activations(ids.numel(), k, g)
        else:
            s["x"] = _activations(case["tokens"], k, g)
        return s
    logits, ids = _chosen(case, g)
    s |= {"logits": logits.to(DTYPE[case["dtype"]]), "ids": ids, "train": case["train"], "mask": None}
    if case["padded"]:
        s["mask"] = torch.rand(case["tokens"], generator=g, device="cuda") >= case["padded"]
    if case["train"]:
        s["dloss"] = torch.full((1,), 0.01, device="cuda")
    return s


# ------------------------------------------------------------------------------ plain forms

def _plain_quantise(x):
    """The codes of fp32 rows, as fp32 whole numbers, and the rows' scales."""
    scale = x.abs().amax(1) / 127.0
    d = scale.unsqueeze(1)
    return torch.where(d > 0, torch.round(x / d), 0.0).clamp(-127.0, 127.0), scale


def _plain_norm(s):
    x, gain = s["x"], s["gain"]
    h = x if s["residual"] is None else (x.float() + s["residual"].float()).to(x.dtype)
    hf = h.float()
    rstd = torch.rsqrt((hf * hf).mean(1) + EPS)
    u = hf * rstd.unsqueeze(1)
    code, scale = _plain_quantise(u * gain)
    out = {"values": (code * scale.unsqueeze(1)).to(torch.bfloat16), "scales": scale, "rstd": rstd}
    if s["residual"] is not None:
        out["h"] = h
    if s["train"]:
        dy = s["dy"].float()
        v = dy * gain
        dx = s["dh"].float() + rstd.unsqueeze(1) * (v - u * (u * v).mean(1, keepdim=True))
        out |= {"dx": dx.to(x.dtype), "dgain": (dy * u).sum(0)}
    return out


def _plain_balance(s):
    logits, ids = s["logits"].float(), s["ids"]
    t, e = logits.shape
    live = torch.ones(t, dtype=torch.bool, device=ids.device) if s["mask"] is None else s["mask"]
    p = torch.exp(logits - logits.amax(1, keepdim=True))
    p = p / p.sum(1, keepdim=True) * live.unsqueeze(1)
    hits = (ids.unsqueeze(2) == torch.arange(e, device=ids.device)) & live.view(-1, 1, 1)
    counts, n = hits.sum((0, 1)), live.sum()
    c = counts.float()
    scale = e / (ids.shape[1] * n.clamp(min=1).float() ** 2)
    out = {"loss": (scale * (c * p.sum(0)).sum()).reshape(1), "counts": torch.cat((counts, n.reshape(1))).to(torch.int32)}
    if s["train"]:
        out["dlogits"] = (s["dloss"] * scale * p * (c - (p * c).sum(1, keepdim=True))).to(s["logits"].dtype)
    return out


def _plain_run(s):
    op = s["op"]
    if op == "norm":
        return _plain_norm(s)
    if op == "balance":
        return _plain_balance(s)
    code, scale = _plain_quantise(s["x"].float())
    w = s["w_codes"][..., :s["cols"]].float()
    if op == "linear":
        return {"y": ((code @ w.T) * scale.unsqueeze(1) * s["w_scales"]).to(torch.bfloat16)}
    first = s["offsets"].long()
    row = torch.arange(code.shape[0], device=code.device)
    live = row < first[-1]
    e = (row.unsqueeze(1) >= first[1:]).sum(1).clamp(max=w.shape[0] - 1)
    at = torch.where(live, row - first[e], 0)
    padded = torch.zeros(w.shape[0], s["most"], code.shape[1], device=code.device)
    padded.index_put_((e, at), code * live.unsqueeze(1), accumulate=True)
    y = torch.bmm(padded, w.transpose(1, 2))[e, at] * scale.unsqueeze(1) * s["w_scales"][e] * live.unsqueeze(1)
    return {"y": y.to(torch.bfloat16)}


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
    if op == "norm":
        q, h, rstd = g.gptq_int8_rms_norm(s["x"], s["gain"], EPS, s["residual"])
        out = {"values": g.gptq_int8_dequantize(q, torch.bfloat16), "scales": q.scales, "rstd": rstd}
        if s["residual"] is not None:
            out["h"] = h
        if s["train"]:
            out["dx"], out["dgain"] = g.gptq_int8_rms_norm_grad(s["dy"], h, s["gain"], rstd, s["dh"])
        return out
    if op == "balance":
        b = g.gptq_expert_balance(s["logits"], s["ids"], s["mask"])
        out = {"loss": b.loss, "counts": b.counts}
        if s["train"]:
            out["dlogits"] = g.gptq_expert_balance_grad(s["dloss"], s["logits"], b, s["mask"])
        return out
    w = g.Int8(s["w_codes"], s["w_scales"], s["cols"])
    q = g.gptq_int8_quantize(s["x"])
    return {"y": g.gptq_int8_matmul(q, w, offsets=s.get("offsets"), out_dtype=torch.bfloat16)}


def work(case):
    op = case["op"]
    if op == "norm":
        n, size = case["rows"] * case["cols"], 2 if case["dtype"] == "bf16" else 4
        moved = n * (size * (3 if case["residual"] else 1) + 2) + 8 * case["rows"] + 4 * case["cols"]
        return {"bytes": moved + (3 * n * size + 4 * case["cols"] if case["train"] else 0), "flops": n * (18 if case["train"] else 8)}
    if op in ("linear", "experts"):
        k, n = case["cols"], case["out"]
        rows = case["tokens"] * case.get("top", 1)
        weights = min(case.get("experts", 1), rows)
        return {"bytes": 2 * rows * k + weights * n * (k + 4) + 2 * rows * n, "flops": 2 * rows * n * k}
    t, k, e = case["tokens"], case["top"], case["experts"]
    moved = t * e * (2 if case["dtype"] == "bf16" else 4)
    return {"bytes": moved * (2 if case["train"] else 1) + 4 * t * k + t + 4 * e, "flops": t * e * (12 if case["train"] else 5)}


# ------------------------------------------------------------------------------------ exact

def _exact_rounded(x):
    """fp64 rows as the nearest whole numbers of steps of a 127th of their largest magnitude, and the steps."""
    step = x.abs().max(1, keepdim=True).values / 127
    return torch.round(x / torch.where(step > 0, step, 1.0)), step


def exact(case, seed):
    s = prepare(case, seed)
    op, out = s["op"], {}
    if op == "norm":
        h = s["x"].double()
        if s["residual"] is not None:
            out["h"] = h + s["residual"].double()
            h = out["h"].to(s["x"].dtype).double()
        norm = (h.square().sum(1, keepdim=True) / h.shape[1] + EPS).sqrt()
        steps, step = _exact_rounded(h / norm * s["gain"].double())
        out |= {"values": steps * step, "scales": step.squeeze(1), "rstd": (1 / norm).squeeze(1)}
        if s["train"]:
            # d/dh of <dy, gain h / norm(h)>, and of <dh, h>
            dy, gain = s["dy"].double(), s["gain"].double()
            along = torch.einsum("rc,rc,c->r", dy, h, gain).unsqueeze(1)
            out["dx"] = s["dh"].double() + dy * gain / norm - h * along / (h.shape[1] * norm ** 3)
            out["dgain"] = torch.einsum("rc,rc->c", dy, h / norm)
        return out
    if op == "linear":
        x, step = _exact_rounded(s["x"].double())
        return {"y": x @ s["w_codes"][:, :s["cols"]].double().T * s["w_scales"].double() * step}
    if op == "experts":
        x, step = _exact_rounded(s["x"].double())
        y = x.new_zeros(x.shape[0], s["w_codes"].shape[1])
        first = s["offsets"].tolist()
        for e, (a, b) in enumerate(zip(first, first[1:])):
            if b > a:
                y[a:b] = x[a:b] @ s["w_codes"][e, :, :s["cols"]].double().T * s["w_scales"][e].double() * step[a:b]
        return {"y": y}
    rows = torch.arange(case["tokens"], device="cuda") if s["mask"] is None else torch.nonzero(s["mask"]).squeeze(1)
    z, ids, n, e = s["logits"].double()[rows], s["ids"][rows].long(), len(rows), case["experts"]
    p = torch.softmax(z, 1)
    share = torch.bincount(ids[ids >= 0], minlength=e).double() / max(1, n * case["top"])
    out = {"loss": (e * (share * p.sum(0) / max(1, n)).sum()).reshape(1), "counts": None}
    if s["train"]:
        dp = (s["dloss"].double() * e * share / max(1, n)).expand(n, e)
        out["dlogits"] = torch.zeros(case["tokens"], e, dtype=torch.float64, device="cuda")
        out["dlogits"][rows] = p * dp - p * (p * dp).sum(1, keepdim=True)
    return out
