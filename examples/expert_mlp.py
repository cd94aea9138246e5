"""A layer of experts taken to 4 bits, run, and its router tuned: the microscaled 4-bit operators and the
expert routing as they are used together.

    python examples/expert_mlp.py [--tokens 2048] [--width 1024] [--hidden 4096] [--experts 8] [--top 2]

Quantises an expert MLP (random weights, calibration-like activations with outlier channels) to both
formats, prints each one's output error against the layer in fp32, the Hessians that its calibration
rows give expert by expert, and a few steps of gradient descent on the router's weights that bring the
4-bit layer's output closer to the fp32 layer's.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import post_weight_quantization_04_gb300 as g  # noqa: E402


def stacked(matrices, fmt):
    """One Fp4 of one matrix per expert."""
    q = [g.gptq_fp4_quantize(w, fmt) for w in matrices]
    scale = torch.cat([x.tensor_scale for x in q]) if fmt == "nv" else None
    return g.Fp4(torch.stack([x.codes for x in q]), torch.stack([x.scales for x in q]), q[0].cols, fmt, scale)


def fp32_layer(x, ids, weights, up, down):
    y = torch.zeros_like(x, dtype=torch.float32)
    for e, (u, d) in enumerate(zip(up, down)):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        y.index_add_(0, t, weights[t, j, None] * (torch.relu(x[t].float() @ u.T) @ d.T))
    return y


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 2048), ("width", 1024), ("hidden", 4096), ("experts", 8), ("top", 2), ("steps", 5)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    rng = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *s: torch.randn(*s, generator=rng, device="cuda")  # noqa: E731
    x = rand(a.tokens, a.width)
    x[:, :: a.width // 8] *= 10.0
    x = x.to(torch.bfloat16)
    up = [rand(a.hidden, a.width) / a.width ** 0.5 for _ in range(a.experts)]
    down = [rand(a.width, a.hidden) / a.hidden ** 0.5 for _ in range(a.experts)]
    score, ids = torch.topk(rand(a.tokens, a.experts), a.top, dim=1)
    ids, weights = ids.to(torch.int32), torch.softmax(score, 1)
    want = fp32_layer(x, ids, weights, up, down)

    g.set_status_mode(True)
    for fmt in ("mx", "nv"):
        w_up, w_down = stacked(up, fmt), stacked(down, fmt)
        y, route, ys = g.gptq_expert_mlp(x, ids, weights, w_up, w_down)
        print(f"{fmt}: output error {float((y - want).norm() / want.norm()):.4f}")
        # the router's weights, tuned on the 4-bit layer: loss |y - want|^2 / 2
        w = weights.clone()
        rate = 0.5 / float(ys.float().square().sum(1).mean())
        for _ in range(a.steps):
            y = g.gptq_expert_combine(ys, route, w)
            _, dw = g.gptq_expert_combine_grad((y.float() - want).to(torch.bfloat16), ys, route, w)
            w -= rate * dw
        y = g.gptq_expert_combine(ys, route, w)
        print(f"{fmt}: after {a.steps} steps on the router's weights {float((y - want).norm() / want.norm()):.4f}")

    # one Hessian per expert, from its contiguous rows of the gathered calibration matrix
    xs = g.gptq_expert_gather(x, route)
    first = route.offsets.tolist()
    g.set_status_mode(False)
    for e in range(a.experts):
        if first[e + 1] > first[e]:
            h = g.Hessian(a.width)
            h.accumulate(xs[first[e]:first[e + 1]])
            H, _, n = h.finalize()
            print(f"expert {e}: {n} rows, mean of diag H {float(H.diagonal().mean()):.3f}")
    g.status_sync()


if __name__ == "__main__":
    main()
