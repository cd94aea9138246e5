"""The 8-bit integer operators at the ends of their ranges: rows and eps whose squares leave fp32's middle, scales whose products do,
offsets out of order, codes and gradients of rows at every address.

Bounds as in test_int8_gpu.py (u = 2^-24): rstd is off by r = (cols / 32 + 24) u / 2 + 4 u of it, and |q - y| <= s (1/2 + 127 (2 r + 8 u)).
"""
import time

import numpy as np
import pytest
import torch

from oracle import int8_oracle as I
from test_int8_gpu import B, DEV, DT, U, _check, _offsets, _operands, _stored, f64, rows_of

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


@pytest.mark.parametrize("T,K,experts", [(4, 100, None), (20, 300, None), (40, 1500, None), (64, 1500, None), (120, 2000, None), (250, 4000, None),
                                         (300, 100, None), (100, 100, None), (300, 100, 3), (90, 1500, 3)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_product_of_far_scales_in_every_epilogue(lib, T, K, experts, dt):
    """Few rows, pairs with the columns whole and split, 64 features (packed pairs of bf16 where the type allows it). A weight's scale times
    the sum is exact where it is subnormal, so the bound is _check's and half the last subnormal step: 2^-150 of fp32, 2^-134 of bf16."""
    rng = np.random.default_rng(T)
    xc, _, wc, _ = _operands(rng, T, 64, K, experts)
    o = None if experts is None else _offsets(rng, T, experts, "even")
    off = None if o is None else torch.tensor(o, dtype=torch.int32, device=DEV)
    last = 2.0 ** -149 if dt == "f32" else 2.0 ** -149 + 2.0 ** -134
    for a, b in ((1e-30, 1e30), (1e30, 1e-30), (1e-44, 1e38), (1e38, 1e-44), (1e-20, 1e-22), (1e20, 1e12), (1e12, 1e20), (1e-40, 1.0), (1.0, 1e-40),
                 (1e-45, 1.0), (0.0, 1e38), (1e38, 0.0)):
        xs, ws = np.full(T, a, np.float32), np.full(wc.shape[:-1], b, np.float32)
        y = lib.gptq_int8_matmul(_stored(lib, xc, xs), _stored(lib, wc, ws), offsets=off, out_dtype=DT[dt])
        _check(y, I.matmul(xc, xs, wc, ws, o), dt, last)
    # one feature in nine far above the others, tokens far below
    xs, ws = np.full(T, 1e-36, np.float32), np.ones(wc.shape[:-1], np.float32)
    ws[..., ::9] = 1e37
    y = lib.gptq_int8_matmul(_stored(lib, xc, xs), _stored(lib, wc, ws), offsets=off, out_dtype=DT[dt])
    _check(y, I.matmul(xc, xs, wc, ws, o), dt, last)
    # a row that was not finite
    xs, ws = np.ones(T, np.float32), np.ones(wc.shape[:-1], np.float32)
    xs[-1] = np.nan
    for relu in (False, True):
        y = lib.gptq_int8_matmul(_stored(lib, xc, xs), _stored(lib, wc, ws), offsets=off, relu=relu, out_dtype=DT[dt])
        assert torch.isnan(y[-1]).all() and torch.isfinite(y[:-1]).all()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(9, 333), (5, 2310), (40, 17), (3, 8195), (6, 1001), (4, 17000)])
def test_codes_and_gains_gradient_at_every_address(lib, dt, rows, cols):
    """q of the norm and dgain of its gradient (and plain codes) for inputs that start anywhere within 16 bytes, against 64 bits."""
    x, r, dy = (rows_of(rows, cols, dt, i) for i in (1, 2, 3))
    gain = torch.rand(cols, generator=torch.Generator().manual_seed(cols)).to(DEV) + 0.5
    h = (x.float() + r.float()).to(x.dtype)
    y, _ = I.rms_norm(f64(h), f64(gain), np.float64(np.float32(1e-5)))
    off = (cols / 32 + 24) * U / 2 + 4 * U
    s = np.abs(y).max(1) / 127
    codes, scales = I.quantise(x.float().cpu().numpy())
    _, _, rstd = lib.gptq_int8_rms_norm(x, gain, 1e-5, r)
    u = f64(h) * f64(rstd)[:, None]
    _, refg = I.rms_norm_grad(f64(dy), f64(h), f64(gain), f64(rstd), f64(r))

    def moved(t, start, more):
        flat = torch.full((rows * (cols + more) + start + 40,), 3, dtype=t.dtype, device=DEV)
        m = flat[start:start + rows * (cols + more)].view(rows, cols + more)[:, :cols]
        m.copy_(t)
        return m
    for start in range(16 * 8 // torch.finfo(DT[dt]).bits):
        for more in (0, 1, 3):
            x2, r2 = moved(x, start, more), moved(r, (start + 1) % 8, more + 1)
            gain2 = torch.cat((gain[:start % 4], gain))[start % 4:]
            q, _, _ = lib.gptq_int8_rms_norm(x2, gain2, 1e-5, r2, out=(None, moved(h, (start + 3) % 8, more), None))
            assert (np.abs(f64(q.scales) - s) <= (off + 4 * U) * s).all()
            v = q.codes[:, :cols].cpu().numpy() * f64(q.scales)[:, None]
            assert (np.abs(v - y) <= s[:, None] * (0.5 + 127 * (2 * off + 8 * U))).all() and not q.codes[:, cols:].any()
            p = lib.gptq_int8_quantize(x2)
            np.testing.assert_array_equal(p.codes.cpu().numpy(), I.stored(codes))
            np.testing.assert_array_equal(p.scales.cpu().numpy(), scales)
            _, dg = lib.gptq_int8_rms_norm_grad(moved(dy, start, 0), moved(h, (start + 2) % 8, more + 2), gain2, rstd, r2)
            assert (np.abs(f64(dg) - refg) <= (rows + 4) * U * np.abs(f64(dy) * u).sum(0)).all()
