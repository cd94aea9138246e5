"""The 8-bit integer operators against fp64.

Bounds, with u = 2^-24 (fp32) and b = 2^-8 (bf16):
  codes and scales of plain rows    equal: both sides take the fp32 quotients
  product    the sum is the exact whole number (below 2^24 here, but where a test says otherwise), then two fp32 products:
             |Y - ref| <= 2.1 u |ref|, and b |ref| more for bf16
  rstd       a sum of squares in chains of at most cols / 32 + 16 terms (a thread's own, then trees), each rounded once, the
             mean, eps and rsqrtf (2 units): rstd is off by (cols / 32 + 24) u / 2 + 4 u, called r below
  norm       y = (h rstd) gain: off by (r + 2 u) |y|, so the scale by (r + 4 u) of it, and code * scale is within half a step of
             y and that: |q - y| <= s (1/2 + 127 (2 r + 8 u))
  gradient   with the rstd it is given: u v summed in chains as above, then four roundings of each term:
             |dx - ref| <= (cols / 32 + 24) u rstd |u| mean|u v| + 6 u (|dh| + rstd (|v| + |u| |mean u v|)) (+ b |ref|)
             |dgain - ref| <= (rows + 4) u sum |dy u|
"""
import numpy as np
import pytest
import torch

from oracle import int8_oracle as I

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
U, B = 2.0 ** -24, 2.0 ** -8


def f64(t):
    return t.detach().double().cpu().numpy()


def rows_of(n, cols, dt, seed, pad=0, scale=1.0):
    """rows with a few outlier channels; pad: a row stride and a start that are not the columns'"""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, cols + pad, generator=g) * scale
    x[:, ::7] *= 9
    return x.to(DT[dt]).to(DEV)[:, pad:]


SHAPES = [(1, 1), (1, 16), (3, 17), (5, 100), (2, 1000), (7, 1024), (4, 2310), (3, 4096), (2, 4095), (2, 8200), (1, 14336), (2, 16390),
          (1, 33000), (1, 40004), (130, 96), (257, 33)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("pad", [0, 1, 2, 8])
def test_quantize_and_back(lib, rows, cols, dt, pad):
    x = rows_of(rows, cols, dt, rows + cols, pad)
    if rows > 2:
        x[1] = 0
        x[2] *= 0.125
    q = lib.gptq_int8_quantize(x)
    codes, scales = I.quantise(x.float().cpu().numpy())
    np.testing.assert_array_equal(q.codes.cpu().numpy(), I.stored(codes))
    np.testing.assert_array_equal(q.scales.cpu().numpy(), scales)
    v = codes.astype(np.float32) * scales[:, None]
    np.testing.assert_array_equal(lib.gptq_int8_dequantize(q).cpu().numpy(), v)
    got = lib.gptq_int8_dequantize(q, torch.bfloat16)
    np.testing.assert_array_equal(got.float().cpu().numpy(), torch.tensor(v).to(torch.bfloat16).float().numpy())
    out = torch.full((rows, cols + 3), 7.0, device=DEV)
    lib.gptq_int8_dequantize(q, out=out[:, 1:1 + cols])
    np.testing.assert_array_equal(out[:, 1:1 + cols].cpu().numpy(), v)
    assert (out[:, 0] == 7).all() and (out[:, 1 + cols:] == 7).all()


def test_quantize_ties(lib):
    """x on the middle between two codes, for scales that are powers of two and others"""
    for s in (1.0, 0.5, 3.0, 2.0 ** -40, 0.1, 1.7e-5):
        x = np.concatenate([[127], np.arange(-126.5, 127, 1)]).astype(np.float32) * np.float32(s)
        x[0] = np.float32(127) * np.float32(s)
        q = lib.gptq_int8_quantize(torch.tensor(x, device=DEV)[None])
        codes, scales = I.quantise(x[None])
        np.testing.assert_array_equal(q.codes[0, :x.size].cpu().numpy(), codes[0])


@pytest.mark.parametrize("scale", [1e-45, 1e-43, 1e-40, 3e-38, 1e-30, 1e-20, 1e18, 1e25, 1e36])
def test_quantize_at_the_ends(lib, scale):
    x = (np.random.default_rng(3).normal(size=(4, 70)).clip(-3, 3) * scale).astype(np.float32)
    q = lib.gptq_int8_quantize(torch.tensor(x, device=DEV))
    codes, scales = I.quantise(x)
    np.testing.assert_array_equal(q.scales.cpu().numpy(), scales)
    np.testing.assert_array_equal(q.codes.cpu().numpy(), I.stored(codes))


def test_quantize_many_values_near_ties(lib):
    """fp32 rows whose values are within a few units of the middles, where a quotient rounded wrongly shows"""
    rng = np.random.default_rng(0)
    a = rng.uniform(0.5, 2, 200).astype(np.float32)
    s = (a / np.float32(127)).astype(np.float32)
    k = rng.integers(-126, 126, (200, 300)) + 0.5
    x = (k * s[:, None]).astype(np.float32)
    x = (x.view(np.int32) + rng.integers(-2, 3, x.shape).astype(np.int32)).view(np.float32)
    x[:, 0] = a
    q = lib.gptq_int8_quantize(torch.tensor(x, device=DEV))
    codes, _ = I.quantise(x)
    np.testing.assert_array_equal(q.codes[:, :300].cpu().numpy(), codes)


def test_quantize_gathers(lib):
    x = rows_of(9, 100, "bf16", 5)
    index = torch.tensor([17, 0, -1, 3, -5, 8, 17], dtype=torch.int32, device=DEV)
    q, whole = lib.gptq_int8_quantize(x, index=index, per=2), lib.gptq_int8_quantize(x)
    src = [8, 0, None, 1, None, 4, 8]
    for r, i in enumerate(src):
        assert torch.equal(q.codes[r], whole.codes[i]) if i is not None else not q.codes[r].any()
        assert q.scales[r] == (whole.scales[i] if i is not None else 0)
    with pytest.raises(lib.GptqError) as e:
        lib.gptq_int8_quantize(x, index=torch.tensor([18], dtype=torch.int32, device=DEV), per=2)
    assert e.value.status == 1


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_quantize_reports_what_is_not_finite(lib, bad):
    x = rows_of(3, 50, "f32", 1)
    x[1, 7] = bad
    with pytest.raises(lib.GptqError) as e:
        lib.gptq_int8_quantize(x)
    assert e.value.status == 7
    with lib.deferred_status():
        q = lib.gptq_int8_quantize(x)
        y = lib.gptq_int8_dequantize(q)
    with pytest.raises(lib.GptqError):
        lib.status_sync()
    assert torch.isnan(q.scales).tolist() == [False, True, False] and torch.isnan(y[1]).all() and torch.isfinite(y[[0, 2]]).all()


def test_nothing_to_quantise(lib):
    for rows, cols in ((0, 5), (3, 0), (0, 0)):
        q = lib.gptq_int8_quantize(torch.empty(rows, cols, device=DEV))
        assert q.scales.tolist() == [0] * rows and q.rows == rows and lib.gptq_int8_dequantize(q).shape == (rows, cols)


# ---------------------------------------------------------------------------------------- norm

def _norm(lib, rows, cols, dt, residual, pad, eps=1e-5, scale=1.0):
    x = rows_of(rows, cols, dt, rows + cols, pad, scale)
    r = rows_of(rows, cols, dt, rows + cols + 1, pad, scale) if residual else None
    gain = (1 + 0.3 * torch.randn(cols + pad, generator=torch.Generator().manual_seed(cols))).to(DEV)[pad:]
    h = x if r is None else (x.float() + r.float()).to(x.dtype)
    return x, r, gain, h, lib.gptq_int8_rms_norm(x, gain, eps, r)


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("pad", [0, 1, 8])
def test_norm(lib, rows, cols, dt, residual, pad):
    x, r, gain, h, (q, got_h, rstd) = _norm(lib, rows, cols, dt, residual, pad)
    assert torch.equal(got_h, h)
    y, ref = I.rms_norm(f64(h), f64(gain), np.float64(np.float32(1e-5)))
    off = (cols / 32 + 24) * U / 2 + 4 * U
    assert (np.abs(f64(rstd) - ref) <= off * ref).all()
    s = np.abs(y).max(1) / 127
    assert (np.abs(f64(q.scales) - s) <= (off + 4 * U) * s).all()
    v = q.codes[:, :cols].cpu().numpy() * f64(q.scales)[:, None]
    assert (np.abs(v - y) <= s[:, None] * (0.5 + 127 * (2 * off + 8 * U))).all()
    assert not q.codes[:, cols:].any()


@pytest.mark.parametrize("scale,eps", [(1e-25, 1e-30), (1e-38, 1e-37), (1e15, 1e-6), (1e22, 1e-6), (3e37, 1e-6), (0.0, 1e-30), (1.0, 1e30)])
@pytest.mark.parametrize("cols", [40, 4096, 40000])
def test_norm_at_the_ends(lib, scale, eps, cols):
    """squares past fp32 or below it; a row of zeros; 3e37 times an outlier channel is past fp32 itself, and is reported"""
    if not torch.isfinite(rows_of(3, cols, "f32", 3 + cols, 0, scale)).all():
        with pytest.raises(lib.GptqError) as e:
            _norm(lib, 3, cols, "f32", False, 0, eps, scale)
        assert e.value.status == 7
        return
    x, _, gain, h, (q, _, rstd) = _norm(lib, 3, cols, "f32", False, 0, eps, scale)
    y, ref = I.rms_norm(f64(h), f64(gain), np.float64(np.float32(eps)))
    off = (cols / 32 + 24) * U / 2 + 4 * U
    assert (np.abs(f64(rstd) - ref) <= off * ref + 2.0 ** -149).all()
    v = q.codes[:, :cols].cpu().numpy() * f64(q.scales)[:, None]
    # (rstd below 2^-126 has fewer bits: 2^-150 off at most)
    lost = 2.0 ** -149 / ref.min()
    s = np.abs(y).max(1) / 127
    assert (np.abs(v - y) <= s[:, None] * (0.5 + 127 * (2 * (off + lost) + 8 * U))).all()


def test_norm_in_place(lib):
    for cols in (100, 4096, 40000):
        x, r, gain, h, (q, _, rstd) = _norm(lib, 3, cols, "bf16", True, 0)
        for to in (x, r):
            a, b = x.clone(), r.clone()
            where = a if to is x else b
            q2, h2, _ = lib.gptq_int8_rms_norm(a, gain, 1e-5, b, out=(None, where, None))
            assert h2 is where and torch.equal(h2, h) and torch.equal(q2.codes, q.codes) and torch.equal(q2.scales, q.scales)


def test_norm_reports_what_is_not_finite(lib):
    x = rows_of(3, 50, "bf16", 1)
    gain = torch.ones(50, device=DEV)
    for bad in (float("nan"), float("inf")):
        y = x.clone()
        y[2, 3] = bad
        with pytest.raises(lib.GptqError) as e:
            lib.gptq_int8_rms_norm(y, gain)
        assert e.value.status == 7
    with pytest.raises(lib.GptqError):   # the sum with the residual is past bf16
        lib.gptq_int8_rms_norm(torch.full_like(x, 3e38), gain, 1e-6, torch.full_like(x, 3e38))
    with pytest.raises(lib.GptqError):
        lib.gptq_int8_rms_norm(x, gain, 0.0)


@pytest.mark.parametrize("rows,cols", SHAPES + [(700, 64), (1000, 4096)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("dh", [False, True])
@pytest.mark.parametrize("pad", [0, 1, 8])
def test_norm_gradient(lib, rows, cols, dt, dh, pad):
    x, r, gain, h, (_, _, rstd) = _norm(lib, rows, cols, dt, False, pad)
    dy = rows_of(rows, cols, dt, 77, pad)
    past = rows_of(rows, cols, dt, 78, pad) if dh else None
    dx, dg = lib.gptq_int8_rms_norm_grad(dy, h, gain, rstd, past)
    H, G, R, Y, D = f64(h), f64(gain), f64(rstd)[:, None], f64(dy), f64(past) if dh else 0.0
    ref, refg = I.rms_norm_grad(Y, H, G, R[:, 0], D if dh else None)
    u, v = H * R, Y * G
    mean = np.abs((u * v).mean(1, keepdims=True))
    off = (cols / 32 + 24) * U * R * np.abs(u) * np.abs(u * v).mean(1, keepdims=True)
    off = off + 6 * U * (np.abs(D) + R * (np.abs(v) + np.abs(u) * mean)) + (B * np.abs(ref) if dt == "bf16" else 0)
    assert (np.abs(f64(dx) - ref) <= off).all()
    assert (np.abs(f64(dg) - refg) <= (rows + 4) * U * np.abs(Y * u).sum(0)).all()
    # written over an input, and the same again
    for to in ([dy, h] + ([past] if dh else [])):
        a = [t.clone() if t is not None else None for t in (dy, h, past)]
        where = a[0] if to is dy else a[1] if to is h else a[2]
        dx2, dg2 = lib.gptq_int8_rms_norm_grad(a[0], a[1], gain, rstd, a[2], out=(where, torch.empty_like(dg)))
        if pad == 0:
            assert torch.equal(dx2, dx) and torch.equal(dg2, dg)


def test_norm_gradient_by_differences(lib):
    """L = <dy, y(h)> + <dh, h> in fp64 from the norm's own formula, with the kernel's rstd"""
    x, _, gain, h, (_, _, rstd) = _norm(lib, 4, 30, "f32", False, 0)
    dy, dh = rows_of(4, 30, "f32", 5), rows_of(4, 30, "f32", 6)
    dx, dg = lib.gptq_int8_rms_norm_grad(dy, h, gain, rstd, dh)
    loss = lambda H, G: (I.rms_norm(H, G, np.float64(np.float32(1e-5)))[0] * f64(dy)).sum() + (H * f64(dh)).sum()   # noqa: E731
    H, G = f64(h), f64(gain)
    for i, j in ((0, 0), (1, 13), (3, 29)):
        d = np.zeros_like(H)
        d[i, j] = 1e-4
        assert abs((loss(H + d, G) - loss(H - d, G)) / 2e-4 - dx[i, j].item()) <= 1e-5 * np.abs(f64(dx)).max()
        d = np.zeros_like(G)
        d[j] = 1e-4
        assert abs((loss(H, G + d) - loss(H, G - d)) / 2e-4 - dg[j].item()) <= 1e-5 * np.abs(f64(dg)).max()


def test_norm_of_no_rows(lib):
    x, gain = torch.empty(0, 8, device=DEV), torch.ones(8, device=DEV)
    q, h, rstd = lib.gptq_int8_rms_norm(x, gain)
    assert q.rows == 0 and rstd.shape == (0,)
    dx, dg = lib.gptq_int8_rms_norm_grad(x, x, gain, rstd)
    assert dx.shape == (0, 8) and dg.tolist() == [0] * 8


# ------------------------------------------------------------------------------------- product

def _operands(rng, T, N, K, E=None):
    """codes all over the range (few at the ends, so sums stay below 2^24) and scales over many sizes"""
    def codes(*shape):
        return np.clip(np.rint(rng.normal(size=shape) * 30), -128, 127).astype(np.int8)
    w = codes(*((E, N, K) if E else (N, K)))
    ws = np.exp(rng.normal(size=w.shape[:-1]) - 5).astype(np.float32)
    return codes(T, K), np.exp(rng.normal(size=T) - 3).astype(np.float32), w, ws


def _stored(lib, c, s):
    return lib.Int8(torch.tensor(I.stored(c), device=DEV), torch.tensor(s, device=DEV), c.shape[-1])


def _check(y, ref, dt, extra=0.0):
    got = f64(y)
    assert (np.abs(got - ref) <= (2.1 * U + (B if dt == "bf16" else 0)) * np.abs(ref) + extra).all()


PRODUCTS = [(1, 1, 1), (1, 24, 16), (2, 33, 100), (3, 130, 64), (4, 257, 129), (5, 8, 1000), (8, 300, 515), (9, 40, 128), (16, 256, 256),
            (17, 512, 300), (31, 100, 4096), (33, 777, 1000), (64, 256, 4096), (77, 2310, 1000), (100, 31, 65), (128, 1000, 512),
            (129, 129, 129), (200, 600, 2000), (256, 256, 128), (257, 300, 700), (300, 513, 64), (513, 1025, 1030), (1000, 400, 333)]


@pytest.mark.parametrize("T,N,K", PRODUCTS)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("relu", [False, True])
def test_product(lib, T, N, K, dt, relu):
    xc, xs, wc, ws = _operands(np.random.default_rng(T + N + K), T, N, K)
    y = lib.gptq_int8_matmul(_stored(lib, xc, xs), _stored(lib, wc, ws), relu=relu, out_dtype=DT[dt])
    _check(y, I.matmul(xc, xs, wc, ws, relu=relu), dt)


@pytest.mark.parametrize("T,N,K", [(1, 40, 200), (5, 300, 64), (40, 129, 256), (300, 520, 136)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("pad", [1, 8])
def test_product_into_rows_of_another_stride(lib, T, N, K, dt, pad):
    xc, xs, wc, ws = _operands(np.random.default_rng(T), T, N, K)
    out = torch.full((T + 2, N + pad), 3.0, dtype=DT[dt], device=DEV)
    y = lib.gptq_int8_matmul(_stored(lib, xc, xs), _stored(lib, wc, ws), out_dtype=DT[dt], out=out[1:-1, pad:])
    _check(y, I.matmul(xc, xs, wc, ws), dt)
    assert (out[0] == 3).all() and (out[-1] == 3).all() and (out[:, :pad] == 3).all()


@pytest.mark.parametrize("T", [1, 6, 40, 300])
def test_product_of_the_largest_codes(lib, T):
    """every partial sum past 2^24 is rounded in fp32: off by at most (K / 16 + 4) units of the whole sum"""
    K, N = 5000, 70
    xc, wc = np.full((T, K), -128, np.int8), np.full((N, K), 127, np.int8)
    xc[:, ::2], wc[1::2] = 127, -128
    xs, ws = np.ones(T, np.float32), np.ones(N, np.float32)
    y = lib.gptq_int8_matmul(_stored(lib, xc, xs), _stored(lib, wc, ws))
    size = np.abs(xc.astype(float)) @ np.abs(wc.astype(float)).T
    _check(y, I.matmul(xc, xs, wc, ws), "f32", (K / 16 + 4) * 2 * U * size)


@pytest.mark.parametrize("T", [1, 40, 300])
def test_product_of_far_scales(lib, T):
    """scales whose product is far from fp32's middle while the results are ordinary or just representable"""
    xc, _, wc, _ = _operands(np.random.default_rng(T), T, 50, 100)
    for a, b in ((1e-30, 1e30), (1e30, 1e-30), (1e-44, 1e38), (1e38, 1e-44), (1e-20, 1e-22), (1e20, 1e12), (1e-40, 1.0), (0.0, 1e38)):
        xs, ws = np.full(T, a, np.float32), np.full(50, b, np.float32)
        y = lib.gptq_int8_matmul(_stored(lib, xc, xs), _stored(lib, wc, ws))
        _check(y, I.matmul(xc, xs, wc, ws), "f32", 2.0 ** -149)
    xs = np.ones(T, np.float32)
    xs[-1] = np.nan
    y = lib.gptq_int8_matmul(_stored(lib, xc, xs), _stored(lib, wc, np.ones(50, np.float32)), relu=True)
    assert torch.isnan(y[-1]).all() and torch.isfinite(y[:-1]).all()


@pytest.mark.parametrize("T,N,K", [(40, 256, 8192), (64, 256, 4096), (100, 300, 6000), (200, 512, 4096), (300, 2048, 4096), (2048, 2048, 2048)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_product_is_the_same_every_time(lib, T, N, K, dt):
    """stages in flight, with other work's traffic between the calls"""
    xc, xs, wc, ws = _operands(np.random.default_rng(T), T, N, K)
    X, W = _stored(lib, xc, xs), _stored(lib, wc, ws)
    y = lib.gptq_int8_matmul(X, W, out_dtype=DT[dt])
    if T <= 300:
        _check(y, I.matmul(xc, xs, wc, ws), dt)
    noise = torch.empty(1 << 26, device=DEV)
    with lib.deferred_status():
        for i in range(300):
            if i % 3 == 0:
                noise.add_(1)
            assert torch.equal(lib.gptq_int8_matmul(X, W, out_dtype=DT[dt]), y)
        lib.status_sync()


@pytest.mark.parametrize("T,N", [(1, 3), (3, 50), (40, 300), (300, 300)])
def test_product_over_no_columns_or_of_nothing(lib, T, N):
    none = lambda r: lib.Int8(torch.empty(r, 0, dtype=torch.int8, device=DEV), torch.ones(r, device=DEV), 0)   # noqa: E731
    assert not lib.gptq_int8_matmul(none(T), none(N)).any()
    assert lib.gptq_int8_matmul(none(0), none(N)).shape == (0, N) and lib.gptq_int8_matmul(none(T), none(0)).shape == (T, 0)


@pytest.mark.parametrize("T,N,K", [(3, 60, 100), (33, 129, 200), (300, 300, 120)])
def test_codes_past_the_columns_are_not_read_into_results(lib, T, N, K):
    """whatever the weights hold past their columns meets the zeros of X"""
    xc, xs, wc, ws = _operands(np.random.default_rng(T), T, N, K)
    W = _stored(lib, wc, ws)
    W.codes[:, K:] = 99
    _check(lib.gptq_int8_matmul(_stored(lib, xc, xs), W), I.matmul(xc, xs, wc, ws), "f32")


def _offsets(rng, T, E, kind):
    if kind == "even":
        o = np.linspace(0, T, E + 1).astype(int)
    elif kind == "one":
        o = np.r_[np.zeros(E // 2 + 1), np.full(E - E // 2, T)].astype(int)
    elif kind == "gaps":   # rows before the first range and behind the last one
        o = np.sort(rng.integers(T // 4, T - T // 4 + 1, E + 1))
    elif kind == "none":
        o = np.full(E + 1, T // 2)
    return o


@pytest.mark.parametrize("T,E,N,K", [(1, 1, 30, 40), (5, 8, 70, 100), (32, 16, 200, 513), (32, 3, 256, 256), (100, 7, 129, 100), (257, 2, 300, 64),
                                     (700, 5, 260, 200), (1500, 33, 150, 128)])
@pytest.mark.parametrize("kind", ["even", "one", "gaps", "none"])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_product_by_expert(lib, T, E, N, K, kind, dt):
    rng = np.random.default_rng(T + E)
    xc, xs, wc, ws = _operands(rng, T, N, K, E)
    o = _offsets(rng, T, E, kind)
    out = torch.full((T, N), 5.0, dtype=DT[dt], device=DEV)
    y = lib.gptq_int8_matmul(_stored(lib, xc, xs), _stored(lib, wc, ws), offsets=torch.tensor(o, dtype=torch.int32, device=DEV),
                             out_dtype=DT[dt], out=out, relu=kind == "one")
    _check(y, I.matmul(xc, xs, wc, ws, o, kind == "one"), dt)
    assert not y[:o[0]].any() and not y[o[-1]:].any()


@pytest.mark.parametrize("T", [6, 400])
@pytest.mark.parametrize("o", [[0, 5, 3, 6], [-2, 1, 2, 3], [0, 1, 2, 1000]])
def test_bad_offsets_are_reported(lib, T, o):
    xc, xs, wc, ws = _operands(np.random.default_rng(0), T, 40, 64, 3)
    with pytest.raises(lib.GptqError) as e:
        lib.gptq_int8_matmul(_stored(lib, xc, xs), _stored(lib, wc, ws), offsets=torch.tensor(o, dtype=torch.int32, device=DEV))
    assert e.value.status == 1


# ------------------------------------------------------------------------------------ together

@pytest.mark.parametrize("T", [1, 50, 600])
def test_a_layer_of_experts_in_8_bits(lib, T):
    """norm with the residual, the router on its output, the balance loss, the expert layer: against fp64 up to the codes that the
    hidden rows' rounding to bf16 moves (as for 4 bits, but a step is a 127th of the largest: within 1e-2)"""
    rng = np.random.default_rng(T)
    E, D, H, k = 6, 200, 320, 2
    x, r = rows_of(T, D, "bf16", 1), rows_of(T, D, "bf16", 2)
    gain = torch.ones(D, device=DEV)
    q, h, rstd = lib.gptq_int8_rms_norm(x, gain, 1e-5, r)
    router = lib.gptq_int8_quantize(torch.tensor(rng.normal(size=(E, D)), dtype=torch.float32, device=DEV))
    logits = lib.gptq_int8_matmul(q, router)
    ids = torch.topk(logits, k, 1).indices.to(torch.int32)
    balance = lib.gptq_expert_balance(logits, ids)
    w = torch.softmax(logits, 1).gather(1, ids.long()).contiguous()
    y = lib.gptq_int8_dequantize(q, torch.bfloat16)
    up, down = rng.normal(size=(E, H, D)) / D ** 0.5, rng.normal(size=(E, D, H)) / H ** 0.5
    cu, su = I.quantise(up.reshape(-1, D))
    cd, sd = I.quantise(down.reshape(-1, H))
    W_up = _stored(lib, cu.reshape(E, H, D), su.reshape(E, H))
    W_down = _stored(lib, cd.reshape(E, D, H), sd.reshape(E, D))
    out, route, ys = lib.gptq_expert_mlp(y, ids, w, W_up, W_down)
    assert balance.counts[:E].tolist() == (route.offsets[1:] - route.offsets[:-1]).tolist() and balance.counts[E] == T
    cx, sx = I.quantise(y.float().cpu().numpy())
    ref = np.zeros((T, D))
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            hid = np.maximum((cu.reshape(E, H, D)[e].astype(float) @ cx[t].astype(float)) * su.reshape(E, H)[e] * sx[t], 0)
            hid = torch.tensor(hid, dtype=torch.float32).to(torch.bfloat16).float().numpy()
            ch, sh = I.quantise(hid[None])
            ref[t] += float(w[t, j]) * (cd.reshape(E, D, H)[e].astype(float) @ ch[0].astype(float)) * sd.reshape(E, D)[e] * sh[0]
    assert np.linalg.norm(f64(out) - ref) <= 0.01 * np.linalg.norm(ref)
    dz = lib.gptq_expert_balance_grad(None, logits, balance)
    assert torch.isfinite(dz).all() and abs(float(dz.sum())) <= 1e-5
    dys, dw = lib.gptq_expert_combine_grad(out, ys, route, w)
    dxs = lib.gptq_expert_gather_grad(dys, route)
    dx, dg = lib.gptq_int8_rms_norm_grad(dxs, h, gain, rstd, dxs)
    assert dx.shape == (T, D) and torch.isfinite(dg).all()


def test_on_another_stream_and_captured(lib):
    """the same results from another stream, and from a graph that is replayed on new inputs"""
    xc, xs, wc, ws = _operands(np.random.default_rng(1), 40, 300, 256)
    x, W = rows_of(40, 256, "bf16", 3), _stored(lib, wc, ws)
    gain, z = torch.ones(256, device=DEV), rows_of(40, 8, "f32", 4)
    ids = torch.topk(z, 2, 1).indices.to(torch.int32)

    def step(stream=None):
        q, h, rstd = lib.gptq_int8_rms_norm(x, gain, 1e-5, x, stream=stream)
        y = lib.gptq_int8_matmul(q, W, out_dtype=torch.bfloat16, stream=stream)
        dx, dg = lib.gptq_int8_rms_norm_grad(x, h, gain, rstd, stream=stream)
        b = lib.gptq_expert_balance(z, ids, stream=stream)
        dz = lib.gptq_expert_balance_grad(b.loss, z, b, stream=stream)
        p = lib.gptq_int8_matmul(lib.gptq_int8_quantize(x[:3], stream=stream), W, stream=stream)
        return [h, rstd, y, dx, dg, b.loss, b.counts, dz, p]

    with lib.deferred_status():
        want = step()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        got = step(s)
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = step()
        for k in range(3):
            x.copy_(rows_of(40, 256, "bf16", 10 + k))
            z.copy_(rows_of(40, 8, "f32", 20 + k))
            graph.replay()
            torch.cuda.synchronize()
            got = [t.clone() for t in held]
            assert all(torch.equal(a, b) for a, b in zip(got, step()))
        lib.status_sync()


@pytest.mark.parametrize("rows,cols,dt", [(400, 8200, "bf16"), (400, 8201, "bf16"), (330, 16384, "bf16"), (320, 5001, "f32"), (400, 8192, "f32"),
                                          (310, 16383, "f32"), (700, 3001, "bf16"), (5000, 250, "f32"), (5000, 251, "bf16"), (1500, 1030, "f32"),
                                          (1, 5000, "bf16"), (2, 250, "f32"), (2, 251, "bf16"), (3, 250, "bf16")])
def test_gradient_of_several_rows_per_cta(lib, rows, cols, dt):
    """dX and dgain against the formula, and the same where dX takes the place of any input at its own address."""
    h, dy, dh = (rows_of(rows, cols, dt, s, 1) for s in (1, 2, 3))
    gain, rstd = torch.rand(cols, device=DEV) + 0.5, torch.rand(rows, device=DEV) + 0.5
    dx, dg = lib.gptq_int8_rms_norm_grad(dy, h, gain, rstd, dh)
    H, G, R, Y, D = f64(h), f64(gain), f64(rstd)[:, None], f64(dy), f64(dh)
    ref, refg = I.rms_norm_grad(Y, H, G, R[:, 0], D)
    u, v = H * R, Y * G
    mean = np.abs((u * v).mean(1, keepdims=True))
    off = (cols / 32 + 24) * U * R * np.abs(u) * np.abs(u * v).mean(1, keepdims=True)
    off = off + 6 * U * (np.abs(D) + R * (np.abs(v) + np.abs(u) * mean)) + (B * np.abs(ref) if dt == "bf16" else 0)
    assert (np.abs(f64(dx) - ref) <= off).all()
    assert (np.abs(f64(dg) - refg) <= (rows + 4) * U * np.abs(Y * u).sum(0)).all()
    for i in range(3):
        a = [rows_of(rows, cols, dt, s, 1) for s in (2, 1, 3)]
        dx2, dg2 = lib.gptq_int8_rms_norm_grad(a[0], a[1], gain, rstd, a[2], out=(a[i], torch.empty_like(dg)))
        assert torch.equal(dx2, dx) and torch.equal(dg2, dg), i


@pytest.mark.parametrize("rows,cols,dt", [(700, 4095, "bf16"), (700, 4096, "bf16"), (500, 8201, "bf16"), (600, 2310, "f32"), (400, 9001, "f32"),
                                          (5000, 251, "bf16"), (5000, 100, "f32"), (310, 16384, "f32")])
def test_norm_of_several_rows_per_cta(lib, rows, cols, dt):
    """As row by row, and the same where h takes the place of either input at its own address."""
    x, r = (rows_of(rows, cols, dt, s, 1) for s in (1, 2))
    gain = torch.rand(cols, device=DEV) + 0.5
    q, h, rstd = lib.gptq_int8_rms_norm(x, gain, 1e-5, r)
    assert torch.equal(h, (x.float() + r.float()).to(DT[dt]))
    for at in (0, 1, rows // 3, rows - 1):
        q1, h1, rstd1 = lib.gptq_int8_rms_norm(x[at:at + 1], gain, 1e-5, r[at:at + 1])
        assert torch.equal(q1.codes, q.codes[at:at + 1]) and torch.equal(q1.scales, q.scales[at:at + 1]) and torch.equal(rstd1, rstd[at:at + 1])
    for i in range(2):
        a = [rows_of(rows, cols, dt, s, 1) for s in (1, 2)]
        q2, _, rstd2 = lib.gptq_int8_rms_norm(a[0], gain, 1e-5, a[1], out=(None, a[i], None))
        assert torch.equal(a[i], h) and torch.equal(q2.codes, q.codes) and torch.equal(q2.scales, q.scales) and torch.equal(rstd2, rstd), i


@pytest.mark.parametrize("T,N,K,E", [(64, 4096, 4096, None), (40, 10240, 600, None), (100, 10240, 300, None), (130, 10241, 200, None),
                                     (60, 4000, 2000, None), (96, 4000, 3000, None), (128, 4000, 7000, None), (250, 5000, 9000, None),
                                     (200, 600, 2000, None), (90, 1000, 5000, None), (230, 2600, 6000, None), (250, 3800, 9000, None),
                                     (200, 700, 300, 8), (500, 700, 300, 8), (150, 300, 500, 16), (90, 300, 2000, 3), (300, 300, 3000, 4),
                                     (60, 100, 3000, 3), (250, 300, 4000, 2), (1200, 520, 640, 16), (900, 300, 1000, 40), (24, 2500, 2100, None), (32, 40, 2048, None),
                                     (20, 300, 2032, None), (13, 400, 2100, None)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_product_in_tiles_of_every_width(lib, T, N, K, E, dt):
    """Tiles of 64, 128 and 256 tokens, whole and with the columns in two to four shares; experts with rows at random and all in
    one; the same each time. (Codes small enough for sums below 2^24.)"""
    rng = np.random.default_rng(T + N)
    xc, wc = rng.integers(-40, 41, (T, K)).astype(np.int8), rng.integers(-40, 41, (E, N, K) if E else (N, K)).astype(np.int8)
    xs, ws = (np.exp(rng.normal(size=s) - 4).astype(np.float32) for s in ((T,), wc.shape[:-1]))
    X, W = _stored(lib, xc, xs), _stored(lib, wc, ws)
    for kind in (("gaps", "one") if E else (None,)):
        o = _offsets(rng, T, E, kind) if E else None
        offsets = torch.tensor(o, dtype=torch.int32, device=DEV) if E else None
        y = lib.gptq_int8_matmul(X, W, offsets=offsets, out_dtype=DT[dt])
        ref = torch.zeros(T, N, dtype=torch.float64, device=DEV)   # (whole numbers: exact in 64 bits)
        for e, (a, b) in enumerate(zip(o[:-1], o[1:]) if E else [(0, T)]):
            w, s = (W.codes[e], W.scales[e]) if E else W[:2]
            ref[a:b] = (X.codes[a:b].double() @ w.double().T) * X.scales[a:b, None].double() * s.double()
        _check(y, f64(ref), dt)
        for _ in range(30):
            assert torch.equal(lib.gptq_int8_matmul(X, W, offsets=offsets, out_dtype=DT[dt]), y)
