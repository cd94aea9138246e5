"""The expert layer on 4-bit weights, all operators together.

Against fp64: the hidden rows are rounded to bf16 from fp32 sums, whose error (K 2^-23 of the sum of
magnitudes) moves about K 2^-15 of them to the neighbouring bf16 number (K = 256: 1 %); one of those in
about 60 then quantises to the neighbouring code, a quarter off. 2e-4 of the hidden values a quarter off
are 0.4 % of the output, so the relative error stays below 1 %; a wrong row, expert, scale or weight is
far above it.
"""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import fp4_oracle as F

pytestmark = pytest.mark.gpu
DEV = "cuda"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _bf16(v):
    return torch.tensor(v.astype(np.float32)).to(torch.bfloat16).double().numpy()


@pytest.mark.parametrize("T,k,E,D,H", [(1, 2, 4, 256, 300), (50, 2, 8, 200, 256), (700, 3, 5, 256, 224)])
@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_expert_mlp_matches_fp64(lib, T, k, E, D, H, fmt):
    rng = np.random.default_rng(T + E)
    x = _bf16(rng.normal(size=(T, D)))
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    ids[rng.random((T, k)) < 0.1] = -1
    w = rng.random((T, k)).astype(np.float32)
    gs = {"up": 2.0 ** -9, "down": 2.0 ** -9, "x": 2.0 ** -8, "h": 2.0 ** -8} if fmt == "nv" else dict.fromkeys(("up", "down", "x", "h"))
    mats, stored = {}, {}
    for name, (r, c) in (("up", (H, D)), ("down", (D, H))):
        q = [F.quantise((rng.normal(size=(r, c)) / c ** 0.5).astype(np.float32), fmt, gs[name]) for _ in range(E)]
        mats[name] = [v for v, _, _ in q]
        stored[name] = lib.Fp4(torch.tensor(np.stack([F.pack_codes(v) for _, v, _ in q]), device=DEV),
                               torch.tensor(np.stack([F.tile_scales(b, c, fmt) for _, _, b in q]), device=DEV), c, fmt,
                               None if fmt == "mx" else torch.tensor([gs[name]], device=DEV))
    scale = lambda n: None if fmt == "mx" else torch.tensor([gs[n]], device=DEV)  # noqa: E731
    X = torch.tensor(x).to(torch.bfloat16).to(DEV)
    idt, wt = torch.tensor(ids, device=DEV), torch.tensor(w, device=DEV)
    y, route, ys = lib.gptq_expert_mlp(X, idt, wt, stored["up"], stored["down"], scale("x"), scale("h"))
    # the same steps in fp64
    xq = F.quantise(x.astype(np.float32), fmt, gs["x"])[0]
    ref = np.zeros((T, D))
    for t in range(T):
        for j in range(k):
            e = ids[t, j]
            if e < 0:
                continue
            h = _bf16(np.maximum(xq[t] @ mats["up"][e].T, 0))[None]
            hq = F.quantise(h.astype(np.float32), fmt, gs["h"])[0]
            ref[t] += w[t, j].astype(np.float64) * (hq[0] @ mats["down"][e].T)
    got = y.double().cpu().numpy()
    assert np.linalg.norm(got - ref) <= 0.01 * np.linalg.norm(ref)
    dropped = (ids < 0).all(1)
    assert (got[dropped] == 0).all()
    # the gathering quantisation and the separate steps are the same bit for bit
    xs = lib.gptq_fp4_quantize(lib.gptq_expert_gather(X, route), fmt, scale("x"))
    h = lib.gptq_fp4_matmul(xs, stored["up"], offsets=route.offsets, relu=True, out_dtype=torch.bfloat16)
    ys2 = lib.gptq_fp4_matmul(lib.gptq_fp4_quantize(h, fmt, scale("h")), stored["down"], offsets=route.offsets,
                              out_dtype=torch.bfloat16)
    assert torch.equal(ys, ys2)


def test_example_runs(lib):
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "expert_mlp.py"), "--tokens", "200", "--width", "256",
                        "--hidden", "512", "--experts", "4"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    lines = r.stdout.splitlines()
    before = [float(v.split()[-1]) for v in lines if "output error" in v]
    after = [float(v.split()[-1]) for v in lines if "after" in v]
    assert len(before) == 2 and all(b < 0.35 for b in before) and all(y < x for x, y in zip(before, after))
