"""The microscaled 4-bit form on the GPU against its fp64 oracle.

Quantising is a sequence of exactly specified roundings, so codes and scale bytes are compared for
equality, and dequantised values with the one fp32 (or bf16) rounding of code * scale. The product's
bound follows from its arithmetic: products of e2m1 values and block scales are exact in fp32 up to
one rounding per block, sums take at most K additions of relative error 2^-23 (rounded or truncated),
the tensor scales two more roundings, and the result is rounded once:
    |Y - Y_ref| <= ((K + 4) 2^-23) sum_k |x w| (+ 2^-8 |Y_ref| for bf16).
Where scales and codes are chosen so that every partial sum is an integer multiple of one small unit
below 2^24 of it, no rounding happens at all and Y has to be equal: a wrong code, scale, row or tile
shows there.
"""
import numpy as np
import pytest
import torch

from oracle import fp4_oracle as F

pytestmark = pytest.mark.gpu
DEV = "cuda"


def npy(t):
    return t.detach().float().cpu().numpy() if t.dtype == torch.bfloat16 else t.detach().cpu().numpy()


def _matrix(rows, cols, dtype, seed, pad=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols + pad, generator=g) * torch.randn(1, cols + pad, generator=g).exp()
    x[:, ::7] *= 0.01
    x[rows // 2, : min(cols, 40)] = 0.0                 # a block of zeros
    x[rows // 3] = torch.randint(-24, 25, (cols + pad,), generator=g) / 4   # midpoints of the grid
    return x.to(dtype)


SHAPES = [(1, 1), (1, 4096), (3, 31), (5, 33), (128, 128), (129, 65), (300, 1000), (7, 2051)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("fmt,g", [("mx", None), ("nv", 2.0 ** -7), ("nv", 0.0123)])
def test_quantize_is_exact(lib, rows, cols, dtype, fmt, g):
    xh = _matrix(rows, cols, dtype, rows * 31 + cols)
    X = xh.to(DEV)
    gt = None if g is None else torch.tensor([g], device=DEV)
    q = lib.gptq_fp4_quantize(X, fmt, gt)
    gf = None if g is None else float(np.float32(g))
    v, codes, byte = F.quantise(npy(xh), fmt, gf)
    np.testing.assert_array_equal(F.untile_scales(npy(q.scales), rows, byte.shape[1]), byte)
    got = npy(q.codes)
    # every byte of the pitch is written; the sign of a zero is free
    want = F.pack_codes(codes)
    fix = lambda b: np.where((b & 15) == 8, b & 0xF0, b)  # noqa: E731
    zero = lambda b: np.where((b >> 4) == 8, fix(b) & 0x0F, fix(b))  # noqa: E731
    np.testing.assert_array_equal(zero(got), zero(want))
    # blocks past the columns are zero in every row of the matrix
    t = npy(q.scales)
    np.testing.assert_array_equal(F.untile_scales(t, rows, t.shape[1] * 4)[:, byte.shape[1]:], 0)
    d32 = lib.gptq_fp4_dequantize(q)
    np.testing.assert_array_equal(npy(d32), v.astype(np.float32))
    d16 = lib.gptq_fp4_dequantize(q, torch.bfloat16)
    np.testing.assert_array_equal(npy(d16), npy(torch.tensor(v.astype(np.float32)).to(torch.bfloat16)))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_quantize_strides_and_extremes(lib, dtype):
    big = torch.finfo(torch.bfloat16).max
    xh = _matrix(40, 100, torch.float32, 5, pad=29)
    xh[1, :32] = torch.linspace(-1, 1, 32) * big
    xh[2, :32] = 2.0 ** -126
    xh[3, :32] = torch.linspace(0, 2.0 ** -140, 32)
    xh = xh.to(dtype)
    X = xh.to(DEV)
    for view, ref in ((X[:, 3:103], xh[:, 3:103]), (X[::3, :100], xh[::3, :100]), (X[:, 8:108], xh[:, 8:108])):
        q = lib.gptq_fp4_quantize(view, "mx")
        v, codes, byte = F.quantise(npy(ref.contiguous()), "mx")
        np.testing.assert_array_equal(F.untile_scales(npy(q.scales), *byte.shape), byte)
        np.testing.assert_array_equal(npy(lib.gptq_fp4_dequantize(q)), v.astype(np.float32))
    # a tensor scale far below and far above the values: scales saturate, and vanish
    for g in (2.0 ** -20, 2.0 ** 20):
        q = lib.gptq_fp4_quantize(X[4:, 3:103], "nv", torch.tensor([g], device=DEV))
        v, _, byte = F.quantise(npy(xh[4:, 3:103].contiguous()), "nv", g)
        np.testing.assert_array_equal(F.untile_scales(npy(q.scales), *byte.shape), byte)
        np.testing.assert_array_equal(npy(lib.gptq_fp4_dequantize(q)), v.astype(np.float32))


@pytest.mark.parametrize("g", [1e-38, 2.0 ** -126, 3e-30, 1e-20, 1e20, 2.0 ** 110, 1e36, 3e38])
def test_quantize_with_tensor_scales_at_the_ends(lib, g):
    """Scales near the ends of fp32, with values that fit them and values that do not: still the nearest
    codes, saturating with their sign; a scale past fp32 has zeros."""
    rng = np.random.default_rng(3)
    big = np.float32(3.3e38)
    g = np.float32(g)
    with np.errstate(over="ignore", under="ignore"):
        rows = [np.clip(rng.normal(size=64) * np.float64(g) * m, -big, big) for m in (1e-3, 1.0, 100.0, 3000.0, 1e5)]
    rows += [np.linspace(-1, 1, 64) * big, np.full(64, 1e-44), np.zeros(64)]
    x = np.stack(rows).astype(np.float32)
    q = lib.gptq_fp4_quantize(torch.tensor(x, device=DEV), "nv", torch.tensor([g], device=DEV))
    with np.errstate(over="ignore", under="ignore", invalid="ignore", divide="ignore"):
        _, codes, byte = F.quantise(x, "nv", float(g))
        s = np.repeat(np.float32(byte_value(byte)) * g, 16, axis=1)
    codes = np.where(np.isinf(s), 0, codes)
    np.testing.assert_array_equal(F.untile_scales(npy(q.scales), *byte.shape), byte)
    got = npy(q.codes)
    got = np.stack([got & 15, got >> 4], -1).reshape(len(x), -1)[:, :64]
    flat = lambda c: np.where(c == 8, 0, c)  # noqa: E731  (the sign of a zero is free)
    np.testing.assert_array_equal(flat(got), flat(codes))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("g", [1.0, 2.0 ** -9, 2.0 ** -70, 2.0 ** 50])
def test_quantize_midpoints_of_every_scale(lib, dtype, g):
    """All midpoints of the grid under each of e4m3's scales (8 bits hold them), both signs, and the bf16
    numbers next to them."""
    mid = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    rows = []
    for e in (-2, 0, 5):
        for j in range(8):
            s = (1 + j / 8) * 2.0 ** e
            for k in (-1, 0, 1):
                v = np.concatenate((mid, -mid)) * s
                v = np.nextafter(v.astype(np.float32), np.float32(np.inf * k)) if k and dtype == torch.float32 else v * (1 + k * 2.0 ** -7)
                rows.append(np.concatenate(([6 * s], v, [0.0])) * g)
    x = torch.tensor(np.array(rows, dtype=np.float32)).to(dtype)
    q = lib.gptq_fp4_quantize(x.to(DEV), "nv", torch.tensor([g], device=DEV))
    v, _, byte = F.quantise(npy(x), "nv", g)
    np.testing.assert_array_equal(F.untile_scales(npy(q.scales), *byte.shape), byte)
    np.testing.assert_array_equal(npy(lib.gptq_fp4_dequantize(q)), v.astype(np.float32))


def byte_value(byte):
    e, f = byte.astype(int) >> 3, byte.astype(int) & 7
    return np.where(e > 0, np.ldexp(1 + f / 8, e - 7), f / 512)


def test_quantize_gathers_rows(lib):
    X = _matrix(50, 200, torch.bfloat16, 8).to(DEV)
    idx = torch.tensor([0, 99, 41, -1, 40, 7, -1, 98] * 20, dtype=torch.int32, device=DEV)
    q = lib.gptq_fp4_quantize(X, "mx", index=idx, per=2)
    rows = torch.where((idx >= 0).unsqueeze(1), X[(idx.clamp(min=0) // 2).long()], 0)
    ref = lib.gptq_fp4_quantize(rows.contiguous(), "mx")
    assert torch.equal(lib.gptq_fp4_dequantize(q), lib.gptq_fp4_dequantize(ref))
    with pytest.raises(lib.GptqError) as e:
        lib.gptq_fp4_quantize(X, "mx", index=idx, per=1)      # 99 is past the 50 rows
    assert e.value.status == 1


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_nonfinite_is_reported(lib, fmt, bad):
    X = torch.randn(9, 70).to(DEV)
    g = torch.tensor([0.01], device=DEV)
    X[4, 69] = bad
    with pytest.raises(lib.GptqError) as e:
        lib.gptq_fp4_quantize(X, fmt, g)
    assert e.value.status == 7
    with lib.deferred_status():
        q = lib.gptq_fp4_quantize(X, fmt, g)
        with pytest.raises(lib.GptqError) as e:
            lib.status_sync()
        assert e.value.status == 7
        lib.status_sync()
    v = lib.gptq_fp4_dequantize(q)
    assert torch.isnan(v[4, 64:]).all() and torch.isfinite(v[4, :64]).all() and torch.isfinite(v[5:]).all()
    with pytest.raises(lib.GptqError) as e:
        lib.gptq_fp4_tensor_scale(X)
    assert e.value.status == 7


def test_tensor_scale(lib):
    for amax, dtype in ((2688.0, torch.float32), (2689.0, torch.float32), (1e-3, torch.bfloat16), (0.0, torch.float32)):
        X = (torch.rand(33, 77) * 0.5 * amax).to(dtype).to(DEV)
        X[32, 76] = -amax
        a = X.abs().max().item()
        g = lib.gptq_fp4_tensor_scale(X).item()
        assert np.log2(g) == round(np.log2(g))
        assert (a <= 2688 * g and a > 2688 * g / 2) if a else g == 1.0


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_tile_scales(lib, fmt):
    byte = np.random.default_rng(1).integers(0, 120, (261, 7)).astype(np.uint8)
    cols = 7 * F.BLOCK[fmt] - 3
    t = lib.gptq_fp4_tile_scales(torch.tensor(byte, device=DEV), cols, fmt)
    np.testing.assert_array_equal(npy(t), F.tile_scales(byte, cols, fmt))


# ------------------------------------------------------------------------------------- product

def _stored(rng, rows, cols, fmt, exact, g):
    """Random codes and scales; `exact`: few enough bits that sums of products are exact in fp32."""
    codes = rng.integers(0, 16, (rows, cols))
    blocks = -(-cols // F.BLOCK[fmt])
    if fmt == "mx":
        byte = rng.integers(126, 128, (rows, blocks)) if exact else rng.integers(120, 130, (rows, blocks))
    else:
        byte = rng.choice([48, 56], (rows, blocks)) if exact else rng.integers(20, 100, (rows, blocks))   # 0.5, 1
    byte = byte.astype(np.uint8)
    return codes, byte, F.values(codes, byte, fmt, g)


def _fp4(lib, codes, byte, cols, fmt, g):
    return lib.Fp4(torch.tensor(F.pack_codes(codes), device=DEV), torch.tensor(F.tile_scales(byte, cols, fmt), device=DEV), cols,
                   fmt, torch.tensor([g], dtype=torch.float32, device=DEV) if fmt == "nv" else None)


def _check(Y, xv, wv, exact, bf16, K):
    ref = xv @ wv.T
    if exact and not bf16:
        np.testing.assert_array_equal(Y, ref)
        return
    bound = (K + 4) * 2.0 ** -23 * (np.abs(xv) @ np.abs(wv).T) + (2.0 ** -8 * np.abs(ref) if bf16 else 0) + 1e-30
    bad = np.abs(Y - ref) > bound
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:5], float(np.max(np.abs(Y - ref) / bound)))


PRODUCTS = [
    # T, N, K
    (1, 1, 1), (1, 16, 32), (1, 4096, 512), (2, 129, 96), (7, 333, 1000), (16, 128, 1056), (31, 250, 257), (33, 256, 300),
    (64, 512, 768), (77, 2310, 1000), (127, 129, 64), (128, 128, 256), (129, 257, 800), (200, 640, 1500), (300, 1000, 128),
    (513, 300, 1024), (1030, 700, 448), (2100, 1300, 320), (3, 100, 2048), (4, 130, 1500), (2, 2310, 999), (5, 130, 1500),
]


@pytest.mark.parametrize("T,N,K", PRODUCTS)
@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_matmul_exact_sums(lib, T, N, K, fmt):
    rng = np.random.default_rng(T + 3 * N + 7 * K)
    cx, bx, xv = _stored(rng, T, K, fmt, True, 2.0)
    cw, bw, wv = _stored(rng, N, K, fmt, True, 0.25)
    Y = lib.gptq_fp4_matmul(_fp4(lib, cx, bx, K, fmt, 2.0), _fp4(lib, cw, bw, K, fmt, 0.25))
    _check(npy(Y), xv, wv, True, False, K)


@pytest.mark.parametrize("T,N,K", PRODUCTS[::2] + [(5, 300, 5000), (150, 300, 5000)])
@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("bf16,relu", [(False, True), (True, False)])
def test_matmul_bound(lib, T, N, K, fmt, bf16, relu):
    rng = np.random.default_rng(T + 5 * N + 11 * K)
    gx, gw = float(np.float32(0.37)), float(np.float32(1.9))
    cx, bx, xv = _stored(rng, T, K, fmt, False, gx)
    cw, bw, wv = _stored(rng, N, K, fmt, False, gw)
    dt = torch.bfloat16 if bf16 else torch.float32
    wide = torch.full((T, N + 5), -7.0, dtype=dtype_of(bf16), device=DEV)
    Y = lib.gptq_fp4_matmul(_fp4(lib, cx, bx, K, fmt, gx), _fp4(lib, cw, bw, K, fmt, gw), relu=relu, out_dtype=dt, out=wide[:, :N])
    got = npy(Y)
    if relu:
        assert (got >= 0).all()
        plain = npy(lib.gptq_fp4_matmul(_fp4(lib, cx, bx, K, fmt, gx), _fp4(lib, cw, bw, K, fmt, gw)))
        np.testing.assert_array_equal(got, np.maximum(plain, 0))
    else:
        _check(got, xv, wv, False, bf16, K)
    assert (wide[:, N:] == -7).all()              # nothing is written past the columns


def dtype_of(bf16):
    return torch.bfloat16 if bf16 else torch.float32


GROUPED = [
    # rows per expert (0: none), rows past the last one, N, K
    ([1, 0, 2, 0, 0, 1], 0, 200, 96),
    ([0, 0, 0], 5, 64, 64),
    ([5, 130, 0, 127, 1, 300], 9, 300, 320),
    ([33] * 9, 0, 129, 1000),
    ([0, 700, 0, 0, 650], 130, 400, 544),
    ([128, 128, 128], 0, 256, 256),
    ([3, 1, 4, 1, 5, 9, 2, 6, 5, 3, 5, 8, 9, 7, 9, 3], 2, 520, 2048),
]


@pytest.mark.parametrize("sizes,tail,N,K", GROUPED)
@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("per_expert", [False, True])
def test_matmul_grouped(lib, sizes, tail, N, K, fmt, per_expert):
    rng = np.random.default_rng(sum(sizes) + N + K)
    T, E = sum(sizes) + tail, len(sizes)
    cx, bx, xv = _stored(rng, T, K, fmt, True, 2.0)
    gw = [2.0 ** -(e % 3) if per_expert else 0.5 for e in range(E)]
    ws = [_stored(rng, N, K, fmt, True, gw[e]) for e in range(E)]
    W = lib.Fp4(torch.tensor(np.stack([F.pack_codes(w[0]) for w in ws]), device=DEV),
                torch.tensor(np.stack([F.tile_scales(w[1], K, fmt) for w in ws]), device=DEV), K, fmt,
                None if fmt == "mx" else torch.tensor(gw if per_expert else gw[:1], device=DEV))
    off = np.concatenate(([0], np.cumsum(sizes))).astype(np.int32)
    out = torch.full((T, N), 99.0, device=DEV)
    Y = npy(lib.gptq_fp4_matmul(_fp4(lib, cx, bx, K, fmt, 2.0), W, offsets=torch.tensor(off, device=DEV), out=out))
    for e in range(E):
        _check(Y[off[e]:off[e + 1]], xv[off[e]:off[e + 1]], ws[e][2], True, False, K)
    np.testing.assert_array_equal(Y[off[-1]:], 0)


def test_matmul_bounded_waits_time_out_and_unwind(lib):
    """With the library's test hook the waits of the pairs' pipeline give up at once: the product reports
    GPTQ_ERR_TIMEOUT after unwinding, and the next call is as right as the one before."""
    clib = lib.load()
    rng = np.random.default_rng(9)
    T, N, K = 300, 700, 2000
    cx, bx, xv = _stored(rng, T, K, "mx", False, 1)
    cw, bw, wv = _stored(rng, N, K, "mx", False, 1)
    X, W = _fp4(lib, cx, bx, K, "mx", 1.0), _fp4(lib, cw, bw, K, "mx", 1.0)
    ref = lib.gptq_fp4_matmul(X, W)
    try:
        assert clib.gptq_test_set_wait_limit_ns(0) == 0
        with pytest.raises(lib.GptqError) as e:
            lib.gptq_fp4_matmul(X, W)
        assert e.value.status == 5
    finally:
        assert clib.gptq_test_set_wait_limit_ns(2_000_000_000) == 0
    assert torch.equal(lib.gptq_fp4_matmul(X, W), ref)


def test_matmul_reports_bad_offsets(lib):
    rng = np.random.default_rng(2)
    cx, bx, _ = _stored(rng, 40, 64, "mx", True, 1)
    cw, bw, _ = _stored(rng, 60, 64, "mx", True, 1)
    W = _fp4(lib, cw, bw, 64, "mx", 1)
    W3 = lib.Fp4(torch.stack([W.codes] * 3), torch.stack([W.scales] * 3), 64, "mx")
    X = _fp4(lib, cx, bx, 64, "mx", 1)
    for off in ([0, 10, 5, 40], [0, 10, 20, 41], [-1, 10, 20, 40]):
        with pytest.raises(lib.GptqError) as e:
            lib.gptq_fp4_matmul(X, W3, offsets=torch.tensor(off, dtype=torch.int32, device=DEV))
        assert e.value.status == 1


def test_matmul_repeats_bit_for_bit_on_any_stream(lib):
    rng = np.random.default_rng(4)
    for T, N, K in ((1, 900, 4096), (300, 900, 1024)):
        cx, bx, _ = _stored(rng, T, K, "nv", False, 1)
        cw, bw, _ = _stored(rng, N, K, "nv", False, 1)
        X, W = _fp4(lib, cx, bx, K, "nv", 1.0), _fp4(lib, cw, bw, K, "nv", 1.0)
        ref = lib.gptq_fp4_matmul(X, W)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with lib.deferred_status():
            for _ in range(3):
                got = lib.gptq_fp4_matmul(X, W, stream=s, out=torch.empty_like(ref))
                s.synchronize()
                assert torch.equal(got, ref)
            lib.status_sync(s)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("T", [2, 70, 400])
def test_a_nan_scale_stays_in_its_row(lib, fmt, T):
    """A NaN scale (what quantising a NaN leaves) makes its row, or its feature, NaN and nothing else."""
    rng = np.random.default_rng(T)
    N, K = 300, 700
    cx, bx, xv = _stored(rng, T, K, fmt, True, 1)
    cw, bw, wv = _stored(rng, N, K, fmt, True, 1)
    bx[1, 3] = bw[130, 5] = 255 if fmt == "mx" else 127
    Y = npy(lib.gptq_fp4_matmul(_fp4(lib, cx, bx, K, fmt, 1.0), _fp4(lib, cw, bw, K, fmt, 1.0)))
    nan = np.zeros((T, N), bool)
    nan[1] = nan[:, 130] = True
    np.testing.assert_array_equal(np.isnan(Y), nan)
    np.testing.assert_array_equal(Y[~nan], (xv @ wv.T)[~nan])


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("T,N,bf16", [(2, 300, False), (70, 300, False), (70, 304, True), (400, 304, True)])
def test_relu_keeps_a_nan(lib, fmt, T, N, bf16):
    rng = np.random.default_rng(T)
    K = 700
    cx, bx, xv = _stored(rng, T, K, fmt, True, 1)
    cw, bw, wv = _stored(rng, N, K, fmt, True, 1)
    bx[1, 3] = bw[130, 5] = 255 if fmt == "mx" else 127
    Y = npy(lib.gptq_fp4_matmul(_fp4(lib, cx, bx, K, fmt, 1.0), _fp4(lib, cw, bw, K, fmt, 1.0), relu=True,
                                out_dtype=dtype_of(bf16)))
    nan = np.zeros((T, N), bool)
    nan[1] = nan[:, 130] = True
    np.testing.assert_array_equal(np.isnan(Y), nan)
    want = npy(torch.tensor(np.maximum(xv @ wv.T, 0)).to(dtype_of(bf16)))
    np.testing.assert_array_equal(Y[~nan], want[~nan])


@pytest.mark.parametrize("T,first,last", [(3, 1, 2), (4, 4, 4), (70, 9, 61), (400, 130, 399)])
@pytest.mark.parametrize("bf16", [False, True])
def test_rows_in_no_range_are_zero(lib, T, first, last, bf16):
    """Rows before the first range and after the last one, with a Y that held something else."""
    rng = np.random.default_rng(T + first)
    N, K = 136, 320
    cx, bx, xv = _stored(rng, T, K, "mx", True, 1)
    cw, bw, wv = _stored(rng, 2 * N, K, "mx", True, 1)
    one = [_fp4(lib, cw[e * N:(e + 1) * N], bw[e * N:(e + 1) * N], K, "mx", 1.0) for e in range(2)]
    W = one[0]._replace(codes=torch.stack([q.codes for q in one]), scales=torch.stack([q.scales for q in one]))
    mid = (first + last) // 2
    offsets = torch.tensor([first, mid, last], dtype=torch.int32, device=DEV)
    out = torch.full((T, N), 7.0, dtype=dtype_of(bf16), device=DEV)
    lib.gptq_fp4_matmul(_fp4(lib, cx, bx, K, "mx", 1.0), W, offsets=offsets, out_dtype=dtype_of(bf16), out=out)
    want = np.zeros((T, N))
    want[first:mid] = xv[first:mid] @ wv[:N].T
    want[mid:last] = xv[mid:last] @ wv[N:].T
    np.testing.assert_array_equal(npy(out), npy(torch.tensor(want).to(dtype_of(bf16))))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("cols", [64, 65])
def test_zeros_under_a_scale_of_zero(lib, dtype, cols):
    """A tensor scale of max|x| / 2688 is zero for a matrix of zeros, and its blocks are zeros all the same."""
    q = lib.gptq_fp4_quantize(torch.zeros(5, cols, dtype=dtype, device=DEV), "nv", torch.zeros(1, device=DEV))
    assert (lib.gptq_fp4_dequantize(q) == 0).all()
    w = lib.gptq_fp4_quantize(torch.ones(40, cols, device=DEV), "nv")
    assert (lib.gptq_fp4_matmul(q, w) == 0).all()


def test_results_given_and_on_the_current_stream(lib):
    """The forms with `out` and `stream`, and the common form on a stream of the caller's, agree."""
    X = torch.randn(150, 300, device=DEV).to(torch.bfloat16)
    W = lib.gptq_fp4_quantize(torch.randn(200, 300, device=DEV), "nv")
    g = lib.gptq_fp4_tensor_scale(X)
    q = lib.gptq_fp4_quantize(X, "nv", g)
    Y, V = lib.gptq_fp4_matmul(q, W), lib.gptq_fp4_dequantize(q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        q2 = lib.gptq_fp4_quantize(X, "nv", g)
        Y2 = lib.gptq_fp4_matmul(q2, W)
    q3 = lib.Fp4(torch.empty_like(q.codes), torch.zeros_like(q.scales), 300, "nv")
    q3 = lib.gptq_fp4_quantize(X, "nv", g, out=q3, stream=s)
    Y3 = lib.gptq_fp4_matmul(q3, W, out=torch.empty_like(Y), stream=s)
    V3 = lib.gptq_fp4_dequantize(q3, out=torch.empty_like(V), stream=s)
    s.synchronize()
    assert torch.equal(q2.codes, q.codes) and torch.equal(q3.codes, q.codes)
    assert torch.equal(Y2, Y) and torch.equal(Y3, Y) and torch.equal(V3, V)


def test_in_a_cuda_graph(lib):
    """In deferred status mode the calls only enqueue kernels: quantise and product replay as a graph."""
    X = torch.randn(48, 640, device=DEV).to(torch.bfloat16)
    W = lib.gptq_fp4_quantize(torch.randn(300, 640, device=DEV), "mx")
    ref = lib.gptq_fp4_matmul(lib.gptq_fp4_quantize(X, "mx"), W)
    with lib.deferred_status():
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            lib.gptq_fp4_matmul(lib.gptq_fp4_quantize(X, "mx"), W)
        torch.cuda.current_stream().wait_stream(s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            got = lib.gptq_fp4_matmul(lib.gptq_fp4_quantize(X, "mx"), W)
        got.zero_()
        g.replay()
        lib.status_sync()
    torch.cuda.synchronize()
    assert torch.equal(got, ref)


def test_binding_refusals(lib):
    X = torch.randn(8, 64, device=DEV)
    q = lib.gptq_fp4_quantize(X, "mx")
    n = lib.gptq_fp4_quantize(X, "nv")
    for call in (lambda: lib.gptq_fp4_quantize(X.cpu(), "mx"), lambda: lib.gptq_fp4_quantize(X, "fp4"),
                 lambda: lib.gptq_fp4_quantize(X.t(), "mx"), lambda: lib.gptq_fp4_quantize(X.half(), "mx"),
                 lambda: lib.gptq_fp4_quantize(X[0], "mx"), lambda: lib.gptq_fp4_matmul(q, n),
                 lambda: lib.gptq_fp4_matmul(q, q._replace(cols=63)), lambda: lib.gptq_fp4_matmul(q, q, out_dtype=torch.float16),
                 lambda: lib.gptq_fp4_matmul(n, n._replace(tensor_scale=None)),
                 lambda: lib.gptq_fp4_matmul(q, q, offsets=torch.zeros(2, dtype=torch.int32, device=DEV)),
                 lambda: lib.gptq_fp4_dequantize(q, torch.float16), lambda: lib.gptq_fp4_dequantize(q, out=X[:, :63])):
        with pytest.raises(ValueError):
            call()


def test_products_of_two_threads(lib):
    """Two host threads on streams of their own, one with a dense product, one with many experts: what a
    launch needs of the kernel is not what the other thread set for its own."""
    import threading
    rng = np.random.default_rng(6)
    T, N, K, E = 70, 64, 64, 600
    cx, bx, xv = _stored(rng, T, K, "nv", True, 1)
    X = _fp4(lib, cx, bx, K, "nv", 1.0)
    cw, bw, wv = _stored(rng, E * N, K, "nv", True, 1)
    ones = [_fp4(lib, cw[e * N:(e + 1) * N], bw[e * N:(e + 1) * N], K, "nv", 1.0) for e in range(E)]
    W = ones[0]._replace(codes=torch.stack([q.codes for q in ones]), scales=torch.stack([q.scales for q in ones]))
    offsets = torch.tensor([0] * E + [T], dtype=torch.int32, device=DEV)       # all rows to the last one
    torch.cuda.synchronize()
    failed = []

    def work(w, off, want):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(3000):
                    Y = lib.gptq_fp4_matmul(X, w, offsets=off)
                np.testing.assert_array_equal(npy(Y), want)
        except Exception as e:  # noqa: BLE001
            failed.append((off is None, repr(e)))

    with lib.deferred_status():
        threads = [threading.Thread(target=work, args=a)
                   for a in ((ones[0], None, xv @ wv[:N].T), (W, offsets, xv @ wv[-N:].T))]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        lib.status_sync()
    assert not failed, failed


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("T", [0, 3, 200])
def test_product_of_no_columns(lib, fmt, T):
    """A sum over no columns is 0, dense and by expert, into a result that held something else."""
    x, w = torch.empty(T, 0, device=DEV), torch.empty(72, 0, device=DEV, dtype=torch.bfloat16)
    X, W = lib.gptq_fp4_quantize(x, fmt), lib.gptq_fp4_quantize(w, fmt)
    Y = lib.gptq_fp4_matmul(X, W, relu=True)
    assert Y.shape == (T, 72) and (Y == 0).all()
    wide = torch.full((T, 80), 7.0, dtype=torch.bfloat16, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    lib.gptq_fp4_matmul(X, W, out_dtype=torch.bfloat16, out=wide[:, :72], stream=s)
    s.synchronize()
    assert (wide[:, :72] == 0).all() and (wide[:, 72:] == 7).all()
    E = lib.Fp4(torch.stack([W.codes] * 2), torch.stack([W.scales] * 2), 0, fmt, W.tensor_scale)
    offsets = torch.tensor([0, T // 2, T], dtype=torch.int32, device=DEV)
    Y = lib.gptq_fp4_matmul(X, E, offsets=offsets)
    assert Y.shape == (T, 72) and (Y == 0).all()



def _close(Y, xv, wv, bf16, K):
    """The bound of the module for results near the ends of fp32 (plus one unit of its, or bf16's, subnormal numbers)."""
    ref = xv @ wv.T
    bound = (K + 4) * 2.0 ** -23 * (np.abs(xv) @ np.abs(wv).T) + (2.0 ** -8 * np.abs(ref) + 2.0 ** -133 if bf16 else 2.0 ** -148)
    assert np.isfinite(Y).all() and (np.abs(Y - ref) <= bound).all()


@pytest.mark.parametrize("gx,gw", [(1e-22, 1e-22), (3e-30, 7e-12), (1e-8, 2e-37), (1e22, 1e17), (5e37, 20.0)])
@pytest.mark.parametrize("T,N,bf16", [(1, 300, False), (3, 300, True), (70, 300, False), (70, 304, True), (400, 300, True)])
def test_matmul_with_a_product_of_tensor_scales_outside_fp32(lib, gx, gw, T, N, bf16):
    """Both tensor scales and every result are ordinary numbers, their product is subnormal or past fp32.
    The bound of the module, with the product of the tensor scales rounded once as ever."""
    rng = np.random.default_rng(T + N)
    K = 200
    gx, gw = float(np.float32(gx)), float(np.float32(gw))
    cx, cw = rng.integers(0, 16, (T, K)), rng.integers(0, 16, (N, K))
    lo, hi = (100, 126) if gx < 1 else (1, 3)             # large or small block scales: every result fits fp32
    bx, bw = (rng.integers(lo, hi, (r, -(-K // 16))).astype(np.uint8) for r in (T, N))
    cx[0] = 0                                             # a row of zeros
    xv, wv = F.values(cx, bx, "nv", gx), F.values(cw, bw, "nv", gw)
    Y = npy(lib.gptq_fp4_matmul(_fp4(lib, cx, bx, K, "nv", gx), _fp4(lib, cw, bw, K, "nv", gw), out_dtype=dtype_of(bf16)))
    _close(Y, xv, wv, bf16, K)
    assert (Y[0] == 0).all()


def test_grouped_matmul_with_products_of_tensor_scales_outside_fp32(lib):
    rng = np.random.default_rng(12)
    T, N, K, gx, gw = 150, 136, 160, float(np.float32(1e-22)), [1.0, float(np.float32(2e-21)), 0.5]
    cx, bx = rng.integers(0, 16, (T, K)), rng.integers(100, 126, (T, K // 16)).astype(np.uint8)
    cw, bw = rng.integers(0, 16, (3, N, K)), rng.integers(100, 126, (3, N, K // 16)).astype(np.uint8)
    off = [0, 50, 101, 150]
    for t in (T, 3):                                      # (3 rows: the kernel for few rows)
        o = off if t == T else [0, 1, 2, 3]
        W = lib.Fp4(torch.tensor(np.stack([F.pack_codes(c) for c in cw]), device=DEV),
                    torch.tensor(np.stack([F.tile_scales(b, K, "nv") for b in bw]), device=DEV), K, "nv", torch.tensor(gw, device=DEV))
        Y = npy(lib.gptq_fp4_matmul(_fp4(lib, cx[:t], bx[:t], K, "nv", gx), W, offsets=torch.tensor(o, dtype=torch.int32, device=DEV)))
        for e in range(3):
            r = slice(o[e], o[e + 1])
            _close(Y[r], F.values(cx[r], bx[r], "nv", gx), F.values(cw[e], bw[e], "nv", gw[e]), False, K)


@pytest.mark.parametrize("amax", [2.0 ** -149, 1e-42, 2.0 ** -138, 2688 * 2.0 ** -149, 1e-38, 2688 * 2.0 ** -126])
def test_tensor_scale_of_subnormal_numbers(lib, amax):
    """The least power of two that fp32 holds as a normal number, also where max|x| / 2688 vanishes."""
    X = torch.zeros(3, 20, device=DEV)
    X[1, 7] = -amax
    assert lib.gptq_fp4_tensor_scale(X).item() == 2.0 ** -126


@pytest.mark.parametrize("T", [1, 2, 4, 70])
def test_mx_scales_whose_product_is_past_fp32(lib, T):
    """Blocks whose sum is 0, or small enough, count for what they are under any two scales: exactly with a few
    rows, whose blocks are summed one by one, and within the module's bound, which is wide next to products that
    cancel, on the tensor cores. A NaN scale still makes its row NaN."""
    import math
    N, K = 40, 128
    cx, bx = np.zeros((T, K), int), np.full((T, 4), 127, np.uint8)
    cw, bw = np.zeros((N, K), int), np.full((N, 4), 127, np.uint8)

    def check():
        terms = (F.values(cx, bx, "mx") * F.values(cw[:1], bw[:1], "mx"))[0]
        want = math.fsum(terms)                                # (all rows and features are alike)
        Y = npy(lib.gptq_fp4_matmul(_fp4(lib, cx, bx, K, "mx", 1.0), _fp4(lib, cw, bw, K, "mx", 1.0)))
        if T <= 4:
            np.testing.assert_array_equal(Y, np.float32(want))
        else:
            assert np.isfinite(Y).all() and (np.abs(Y - want) <= (K + 4) * 2.0 ** -23 * np.abs(terms).sum()).all()

    cx[:, 0], cw[:, 0] = 2, 4                                  # 1 * 2 in the first block
    cx[:, 32:64], cw[:, 32:64:2], cw[:, 33:64:2] = 2, 2, 10    # 1 and -1 in turn: 0
    for sx, sw in ((227, 157), (157, 227), (252, 252), (10, 252), (252, 10)):
        bx[:, 1], bw[:, 1] = sx, sw
        check()
    cx[:, 32:64], cw[:, 32:64] = 0, 0
    cx[:, 40], cw[:, 40] = 1, 9                                # 0.5 * -0.5
    for sx, sw in ((191, 191), (222, 160), (160, 222), (252, 2), (64, 64)):
        bx[:, 1], bw[:, 1] = sx, sw
        check()
    bx[0, 1], bw[:, 1] = 255, 252
    Y = npy(lib.gptq_fp4_matmul(_fp4(lib, cx, bx, K, "mx", 1.0), _fp4(lib, cw, bw, K, "mx", 1.0)))
    assert np.isnan(Y[0]).all()


def test_a_number_of_columns_past_64_bits_is_refused(lib):
    q = lib.gptq_fp4_quantize(torch.randn(8, 64, device=DEV), "mx")
    wrong = q._replace(cols=2 ** 70)
    for call in (lambda: lib.gptq_fp4_dequantize(wrong), lambda: lib.gptq_fp4_matmul(wrong, q), lambda: lib.gptq_fp4_matmul(q, wrong)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("T,N,K", PRODUCTS[::2] + [(5, 300, 5000), (150, 300, 5000)])
@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_matmul_fp32_bound(lib, T, N, K, fmt):
    """The bound of the module for an fp32 result, general block scales and tensor scales that are no powers of two."""
    rng = np.random.default_rng(T + 5 * N + 13 * K)
    gx, gw = float(np.float32(0.37)), float(np.float32(1.9))
    cx, bx, xv = _stored(rng, T, K, fmt, False, gx)
    cw, bw, wv = _stored(rng, N, K, fmt, False, gw)
    Y = lib.gptq_fp4_matmul(_fp4(lib, cx, bx, K, fmt, gx), _fp4(lib, cw, bw, K, fmt, gw))
    _check(npy(Y), xv, wv, False, False, K)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("sizes", [[1, 0, 2, 1], [70, 3, 0, 200]])
def test_grouped_fp32_bound(lib, fmt, sizes):
    rng = np.random.default_rng(sum(sizes))
    T, E, N, K = sum(sizes) + 1, len(sizes), 200, 600
    gx, gw = float(np.float32(0.37)), [float(np.float32(v)) for v in (1.9, 0.3, 0.011, 70.7)]
    cx, bx, xv = _stored(rng, T, K, fmt, False, gx)
    ws = [_stored(rng, N, K, fmt, False, gw[e]) for e in range(E)]
    W = lib.Fp4(torch.tensor(np.stack([F.pack_codes(w[0]) for w in ws]), device=DEV),
                torch.tensor(np.stack([F.tile_scales(w[1], K, fmt) for w in ws]), device=DEV), K, fmt,
                None if fmt == "mx" else torch.tensor(gw, dtype=torch.float32, device=DEV))
    off = np.concatenate(([0], np.cumsum(sizes))).astype(np.int32)
    Y = npy(lib.gptq_fp4_matmul(_fp4(lib, cx, bx, K, fmt, gx), W, offsets=torch.tensor(off, device=DEV)))
    for e in range(E):
        _check(Y[off[e]:off[e + 1]], xv[off[e]:off[e + 1]], ws[e][2], False, False, K)
    np.testing.assert_array_equal(Y[off[-1]:], 0)


@pytest.mark.slow
@pytest.mark.parametrize("bf16,N", [(True, 14336), (True, 14333), (False, 14336)])
def test_product_past_32_bits(lib, bf16, N):
    """More than 2^31 elements of Y, a third of its rows in no expert's range: rows at both ends and on either side of
    the ranges' ends."""
    rng = np.random.default_rng(N)
    T, K, E = 160001, 64, 3
    off = [1000, 50003, 50003, 108002]
    cx, bx, xv = _stored(rng, T, K, "mx", True, 1)
    ws = [_stored(rng, N, K, "mx", True, 1) for _ in range(E)]
    W = lib.Fp4(torch.tensor(np.stack([F.pack_codes(w[0]) for w in ws]), device=DEV),
                torch.tensor(np.stack([F.tile_scales(w[1], K, "mx") for w in ws]), device=DEV), K, "mx")
    out = torch.full((T, N), 7.0, dtype=dtype_of(bf16), device=DEV)
    assert out.numel() > 1 << 31
    lib.gptq_fp4_matmul(_fp4(lib, cx, bx, K, "mx", 1.0), W, offsets=torch.tensor(off, dtype=torch.int32, device=DEV),
                        out_dtype=dtype_of(bf16), out=out)
    for t in (0, 999, 1000, 50002, 50003, 108001, 108002, T - 1):
        e = 0 if 1000 <= t < 50003 else 2 if 50003 <= t < 108002 else None
        want = np.zeros(N) if e is None else xv[t] @ ws[e][2].T
        np.testing.assert_array_equal(npy(out[t]), npy(torch.tensor(want).to(dtype_of(bf16))))
    rows = torch.cat((out[:1000], out[108002:]))
    assert not rows.any()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("T", [1, 3, 70])
def test_product_right_behind_what_writes_its_operands(lib, fmt, T):
    """Both operands written anew in the same buffers by the call before, many times without a pause: each product is
    that of its own operands."""
    N, K = 256, 512
    rng = np.random.default_rng(T)
    g = 2.0 ** -3 if fmt == "nv" else None
    gt = None if g is None else torch.tensor([g], device=DEV)
    xs = [torch.tensor(rng.normal(size=(T, K)), dtype=torch.bfloat16, device=DEV) for _ in range(8)]
    ws = [torch.tensor(rng.normal(size=(N, K)), dtype=torch.bfloat16, device=DEV) for _ in range(8)]
    want = [[lib.gptq_fp4_matmul(lib.gptq_fp4_quantize(x, fmt, gt), lib.gptq_fp4_quantize(w, fmt, gt)) for w in ws] for x in xs]
    x, w = lib.gptq_fp4_quantize(xs[0], fmt, gt), lib.gptq_fp4_quantize(ws[0], fmt, gt)
    got = []
    with lib.deferred_status():
        for i in range(200):
            if i % 2:
                lib.gptq_fp4_quantize(xs[i // 2 % 8], fmt, gt, out=x)
                lib.gptq_fp4_quantize(ws[i // 3 % 8], fmt, gt, out=w)
            else:
                lib.gptq_fp4_quantize(ws[i // 3 % 8], fmt, gt, out=w)
                lib.gptq_fp4_quantize(xs[i // 2 % 8], fmt, gt, out=x)
            got.append(lib.gptq_fp4_matmul(x, w))
        lib.status_sync()
    assert all(torch.equal(y, want[i // 2 % 8][i // 3 % 8]) for i, y in enumerate(got))
