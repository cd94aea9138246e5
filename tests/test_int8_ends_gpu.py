"""The 8-bit integer operators at the ends of their ranges: rows and eps whose squares leave fp32's middle.

Bounds as in test_int8_gpu.py (u = 2^-24): rstd is off by r = (cols / 32 + 24) u / 2 + 4 u of it, and |q - y| <= s (1/2 + 127 (2 r + 8 u)).
"""
import time

import numpy as np
import pytest
import torch

from oracle import int8_oracle as I
from test_int8_gpu import B, DEV, DT, U, _offsets, _operands, _stored, f64, rows_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale,eps", [(1e-13, 1e-30), (4e-13, 1e-30), (9e-13, 1e-30), (4e-13, 1e-45), (1e-18, 1e-40), (1e-21, 1e-45)])
@pytest.mark.parametrize("cols", [40, 1024, 4096, 4099, 16384, 40000])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("even", [False, True])
def test_norm_of_small_rows(lib, scale, eps, cols, dt, even):
    """The mean square and eps are far below 1, the sum of the scaled squares is not past fp32; then the gradient with that rstd."""
    x = torch.full((3, cols), scale, device=DEV).to(DT[dt]) if even else rows_of(3, cols, dt, cols, 0, scale)
    gain = torch.rand(cols, generator=torch.Generator().manual_seed(cols)).to(DEV) + 0.5
    q, h, rstd = lib.gptq_int8_rms_norm(x, gain, eps)
    y, ref = I.rms_norm(f64(x), f64(gain), np.float64(np.float32(eps)))
    off = (cols / 32 + 24) * U / 2 + 4 * U
    assert (np.abs(f64(rstd) - ref) <= off * ref).all()
    s = np.abs(y).max(1) / 127
    assert (np.abs(f64(q.scales) - s) <= (off + 4 * U) * s).all()
    v = q.codes[:, :cols].cpu().numpy() * f64(q.scales)[:, None]
    assert (np.abs(v - y) <= s[:, None] * (0.5 + 127 * (2 * off + 8 * U))).all()
    dy = rows_of(3, cols, dt, 5)
    dx, dg = lib.gptq_int8_rms_norm_grad(dy, h, gain, rstd)
    H, G, R, Y = f64(h), f64(gain), f64(rstd)[:, None], f64(dy)
    ref, refg = I.rms_norm_grad(Y, H, G, R[:, 0], None)
    u, w = H * R, Y * G
    off = (cols / 32 + 24) * U * R * np.abs(u) * np.abs(u * w).mean(1, keepdims=True)
    off = off + 6 * U * R * (np.abs(w) + np.abs(u) * np.abs((u * w).mean(1, keepdims=True))) + (B * np.abs(ref) if dt == "bf16" else 0)
    assert (np.abs(f64(dx) - ref) <= off).all()
    assert (np.abs(f64(dg) - refg) <= 7 * U * np.abs(Y * u).sum(0)).all()


@pytest.mark.parametrize("T,E,N,K", [(2000, 20, 256, 4096), (300, 33, 100, 3000), (900, 70, 300, 200)])
@pytest.mark.parametrize("kind", ["up and down", "one back", "past the rows"])
def test_offsets_out_of_order(lib, T, E, N, K, kind):
    """Ranges that share rows, where the columns are split over a cluster (the first two) and where they are not: reported at once, not
    when a wait of 2 s has given up, and the next call is right."""
    rng = np.random.default_rng(T)
    xc, xs, wc, ws = _operands(rng, T, N, K, E)
    good = _offsets(rng, T, E, "even")
    X, W, o = _stored(lib, xc, xs), _stored(lib, wc, ws), torch.tensor(good, dtype=torch.int32, device=DEV)
    ref = lib.gptq_int8_matmul(X, W, offsets=o)
    bad = good.copy()
    if kind == "up and down":
        bad[1::2], bad[::2] = T, 0
    elif kind == "one back":
        bad[E - 1] = 3
    else:
        bad[1:] += T // 2
    b = torch.tensor(bad, dtype=torch.int32, device=DEV)
    torch.cuda.synchronize()
    t = time.perf_counter()
    with pytest.raises(lib.GptqError) as e:
        lib.gptq_int8_matmul(X, W, offsets=b)
    assert e.value.status == 1 and time.perf_counter() - t < 1
    assert torch.equal(lib.gptq_int8_matmul(X, W, offsets=o), ref)
