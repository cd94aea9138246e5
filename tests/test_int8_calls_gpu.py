"""The 8-bit integer operators and the balance loss as calls: given results and streams, several host threads, bounded waits,
matrices past 2^31 elements, rows of other programs' memory around the results."""
import threading

import numpy as np
import pytest
import torch

from oracle import int8_oracle as I
from test_int8_gpu import B, DEV, U, _check, _offsets, _operands, _stored, f64, rows_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,N,K,E", [(300, 700, 2000, None), (300, 700, 300, None), (200, 300, 400, 3)])
def test_bounded_waits_time_out_and_unwind(lib, T, N, K, E):
    """With the library's test hook the waits of the pairs' pipeline give up at once (columns split over a cluster, not split, by
    expert): the product reports GPTQ_ERR_TIMEOUT after unwinding, and the next call is as right as the one before."""
    clib = lib.load()
    rng = np.random.default_rng(9)
    xc, xs, wc, ws = _operands(rng, T, N, K, E)
    o = None if E is None else torch.tensor(_offsets(rng, T, E, "even"), dtype=torch.int32, device=DEV)
    X, W = _stored(lib, xc, xs), _stored(lib, wc, ws)
    ref = lib.gptq_int8_matmul(X, W, offsets=o)
    try:
        assert clib.gptq_test_set_wait_limit_ns(0) == 0
        with pytest.raises(lib.GptqError) as e:
            lib.gptq_int8_matmul(X, W, offsets=o)
        assert e.value.status == 5
    finally:
        assert clib.gptq_test_set_wait_limit_ns(2_000_000_000) == 0
    assert torch.equal(lib.gptq_int8_matmul(X, W, offsets=o), ref)


@pytest.mark.parametrize("T,N,K,E", [(64, 4096, 4096, None), (128, 2000, 3000, None), (40, 10240, 600, None), (100, 10240, 300, None),
                                     (200, 700, 300, 8), (500, 700, 300, 8)])
def test_bounded_waits_in_tiles_of_other_widths(lib, T, N, K, E):
    test_bounded_waits_time_out_and_unwind(lib, T, N, K, E)


def test_several_host_threads(lib):
    """Dense and expert products of several kernels, the norm, its gradient and the balance at once, each thread on a stream of its own"""
    rng = np.random.default_rng(3)
    jobs = []
    for T, N, K, E in ((5, 300, 500, None), (200, 512, 1024, None), (700, 600, 300, None), (64, 200, 256, 600), (900, 300, 256, 4)):
        xc, xs, wc, ws = _operands(rng, T, N, K, E)
        o = None if E is None else torch.tensor(_offsets(rng, T, E, "even"), dtype=torch.int32, device=DEV)
        X, W = _stored(lib, xc, xs), _stored(lib, wc, ws)
        jobs.append(lambda X=X, W=W, o=o: [lib.gptq_int8_matmul(X, W, offsets=o)])
    x, gain = rows_of(300, 4096, "bf16", 1), torch.ones(4096, device=DEV)

    def norm():
        q, h, rstd = lib.gptq_int8_rms_norm(x, gain, 1e-5, x)
        return [q.codes, q.scales, *lib.gptq_int8_rms_norm_grad(x, h, gain, rstd, x)]
    z, ids = rows_of(3000, 64, "f32", 2), torch.zeros(3000, 2, dtype=torch.int32, device=DEV)

    def balance():
        b = lib.gptq_expert_balance(z, ids)
        return [b.loss, b.counts, lib.gptq_expert_balance_grad(None, z, b)]
    jobs += [norm, balance]
    want = [j() for j in jobs]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    got = jobs[i]()
                    torch.cuda.current_stream().synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                        wrong.append(i)
        except Exception as e:   # noqa: BLE001
            wrong.append((i, e))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not wrong


def test_results_given_and_on_a_stream(lib):
    """The forms with `out`, `ws` and `stream` give what the common form gives, and only that memory changes."""
    s = torch.cuda.Stream()
    x, r, dy = rows_of(70, 333, "bf16", 1), rows_of(70, 333, "bf16", 2), rows_of(70, 333, "bf16", 3)
    gain = torch.rand(333, device=DEV) + 0.5
    q, h, rstd = lib.gptq_int8_rms_norm(x, gain, 1e-5, r)
    dx, dg = lib.gptq_int8_rms_norm_grad(dy, h, gain, rstd, r)
    p = lib.gptq_int8_quantize(x)
    v = lib.gptq_int8_dequantize(p, torch.bfloat16)
    z, mask = rows_of(200, 20, "f32", 4), torch.rand(200, device=DEV) < 0.7
    ids = torch.randint(-1, 20, (200, 3), dtype=torch.int32, device=DEV)
    b = lib.gptq_expert_balance(z, ids, mask)
    dz = lib.gptq_expert_balance_grad(b.loss, z, b, mask)

    def wide(like, rows=1, cols=5):
        t = torch.full((like.shape[0] + 2 * rows, like.shape[1] + 2 * cols), 7, dtype=like.dtype, device=DEV)
        return t, t[rows:-rows, cols:-cols]

    def kept(t, view, rows=1, cols=5):
        c = t.clone()
        c[rows:-rows, cols:-cols] = 7
        return bool((c == 7).all())
    th, vh = wide(h)
    tx, vx = wide(dx)
    tv, vv = wide(v)
    tz, vz = wide(dz)
    q2 = lib.Int8(torch.zeros_like(q.codes), torch.zeros_like(q.scales), 333)
    rstd2, dg2 = torch.zeros_like(rstd), torch.zeros_like(dg)
    b2 = lib.Balance(torch.zeros_like(b.loss), torch.zeros_like(b.counts), 0)
    p2 = lib.Int8(torch.zeros_like(p.codes), torch.zeros_like(p.scales), 333)
    work = torch.empty(1 << 22, dtype=torch.uint8, device=DEV)
    s.wait_stream(torch.cuda.current_stream())
    got = lib.gptq_int8_rms_norm(x, gain, 1e-5, r, out=(q2, vh, rstd2), stream=s)
    assert got[1] is vh and got[2] is rstd2
    lib.gptq_int8_rms_norm_grad(dy, vh, gain, rstd2, r, out=(vx, dg2), ws=work, stream=s)
    lib.gptq_int8_quantize(x, out=p2, stream=s)
    lib.gptq_int8_dequantize(p2, torch.bfloat16, out=vv, stream=s)
    b2 = lib.gptq_expert_balance(z, ids, mask, out=b2, ws=work[1 << 21:], stream=s)
    lib.gptq_expert_balance_grad(b2.loss, z, b2, mask, out=vz, stream=s)
    s.synchronize()
    for a, c in ((q.codes, q2.codes), (q.scales, q2.scales), (h, vh), (rstd, rstd2), (dg, dg2), (p.codes, p2.codes), (p.scales, p2.scales),
                 (v, vv), (b.loss, b2.loss), (b.counts, b2.counts), (dz, vz)):
        assert torch.equal(a, c)
    assert torch.equal(dx, vx) and kept(th, vh) and kept(tx, vx) and kept(tv, vv) and kept(tz, vz) and b2.top == 3
    with pytest.raises(lib.GptqError) as e:
        lib.gptq_int8_rms_norm_grad(dy, h, gain, rstd, r, ws=work[:16])
    assert e.value.status == 6
    with pytest.raises(lib.GptqError) as e:
        lib.gptq_expert_balance(z, ids, ws=work[:16])
    assert e.value.status == 6


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(9, 333), (5, 2310), (40, 17), (3, 8195), (6, 1001)])
def test_rows_at_every_address(lib, dt, rows, cols):
    """Inputs and results that start anywhere within 16 bytes, with row strides of every remainder, against whole rows"""
    es = 2 if dt == "bf16" else 4
    x, r, dy = (rows_of(rows, cols, dt, i) for i in (1, 2, 3))
    gain = torch.rand(cols, device=DEV) + 0.5
    q, h, rstd = lib.gptq_int8_rms_norm(x, gain, 1e-5, r)
    dx, dg = lib.gptq_int8_rms_norm_grad(dy, h, gain, rstd, r)
    v = lib.gptq_int8_dequantize(q, x.dtype)

    def moved(t, start, more):
        flat = torch.full((rows * (cols + more) + start + 40,), 3, dtype=t.dtype, device=DEV)
        m = flat[start:start + rows * (cols + more)].view(rows, cols + more)[:, :cols]
        m.copy_(t)
        return flat, m
    for start in range(16 // es):
        for more in (0, 1, 3):
            _, x2 = moved(x, start, more)
            _, r2 = moved(r, (start + 1) % 8, more + 1)
            fh, h2 = moved(torch.zeros_like(h), (start + 3) % 8, more)
            fd, d2 = moved(torch.zeros_like(dx), (start + 2) % 8, more + 2)
            fv, v2 = moved(torch.zeros_like(v), start, more)
            gain2 = torch.cat((gain[:start % 4], gain))[start % 4:]
            q2, _, rstd2 = lib.gptq_int8_rms_norm(x2, gain2, 1e-5, r2, out=(None, h2, None))
            assert torch.equal(h2, h) and (rstd2 - rstd).abs().max() <= 2e-6 * rstd.max()
            lib.gptq_int8_dequantize(q, x.dtype, out=v2)
            assert torch.equal(v2, v)
            dx2, dg2 = lib.gptq_int8_rms_norm_grad(moved(dy, start, 0)[1], h2, gain2, rstd, r2, out=(d2, torch.empty_like(dg)))
            assert (f64(dx2) - f64(dx)).__abs__().max() <= (2 * B if dt == "bf16" else 64 * U) * np.abs(f64(dx)).max()
            for flat, m in ((fh, h2), (fd, d2), (fv, v2)):
                n = flat.numel()
                m.fill_(3)
                assert bool((flat == 3).all()), n


def test_a_product_past_2_31_elements(lib):
    T, N, K = 70001, 32768, 48
    rng = np.random.default_rng(0)
    xc, xs, wc, ws = _operands(rng, 101, 64, K)
    X = lib.Int8(torch.tensor(I.stored(xc), device=DEV).repeat(694, 1)[:T].contiguous(), torch.tensor(xs, device=DEV).repeat(694)[:T].contiguous(), K)
    W = lib.Int8(torch.tensor(I.stored(wc), device=DEV).repeat(N // 64, 1), torch.tensor(ws, device=DEV).repeat(N // 64), K)
    y = lib.gptq_int8_matmul(X, W, out_dtype=torch.bfloat16)
    assert y.numel() > 1 << 31
    ref = I.matmul(xc, xs, wc, ws)
    for t in (0, 1, 65535, 65536, 69999, T - 1):
        for n in (0, 16384, N - 64):
            _check(y[t:t + 1, n:n + 64], ref[t % 101][None], "bf16")
    o = torch.tensor([0, T // 2, T], dtype=torch.int32, device=DEV)
    W2 = lib.Int8(W.codes.view(2, N // 2, -1), W.scales.view(2, N // 2), K)
    z = lib.gptq_int8_matmul(X, W2, offsets=o, out_dtype=torch.bfloat16)
    assert torch.equal(z[-1], y[-1, :N // 2]) and torch.equal(z[0], y[0, :N // 2])


def test_rows_past_2_31_elements(lib):
    rows, cols = 530_000, 4096
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV)
    base = rows_of(1000, cols, "bf16", 1)
    for i in range(0, rows, 1000):
        x[i:i + 1000] = base
    gain = torch.rand(cols, device=DEV) + 0.5
    q0, h0, rstd0 = lib.gptq_int8_rms_norm(base, gain, 1e-5, base)
    q, h, rstd = lib.gptq_int8_rms_norm(x, gain, 1e-5, x)
    v = lib.gptq_int8_dequantize(q, torch.bfloat16)
    v0 = lib.gptq_int8_dequantize(q0, torch.bfloat16)
    dx, dg = lib.gptq_int8_rms_norm_grad(x, h, gain, rstd, x, out=(x, torch.empty(cols, device=DEV)))
    dx0, _ = lib.gptq_int8_rms_norm_grad(base, h0, gain, rstd0, base)
    for i in (0, 524_000, rows - 1000):
        assert torch.equal(q.codes[i:i + 1000], q0.codes) and torch.equal(h[i:i + 1000], h0) and torch.equal(v[i:i + 1000], v0)
        assert torch.equal(dx[i:i + 1000], dx0)


def test_a_balance_past_2_31_logits(lib):
    T, E, n = 2_200_000, 1000, 5000
    base = rows_of(n, E, "bf16", 1)
    z = base.repeat(T // n, 1)
    ids0 = torch.randint(0, E, (n, 2), dtype=torch.int32, device=DEV)
    b0, b = lib.gptq_expert_balance(base, ids0), lib.gptq_expert_balance(z, ids0.repeat(T // n, 1))
    assert z.numel() > 1 << 31 and torch.equal(b.counts, b0.counts * (T // n))
    # the same loss, whose sums have T / 64 + 200 and n / 64 + 200 roundings (see the balance's tests)
    assert abs(float(b.loss) - float(b0.loss)) <= (T / 64 + n / 64 + 400) * U * float(b0.loss)
    dz = lib.gptq_expert_balance_grad(None, z, b)
    dz0 = lib.gptq_expert_balance_grad(torch.full((1,), n / T, device=DEV), base, b0)
    for i in (0, T - n):
        assert (f64(dz[i:i + n]) - f64(dz0)).__abs__().max() <= 2 * B * np.abs(f64(dz0)).max()


@pytest.mark.parametrize("cols", [(1 << 31) - 4096, (1 << 31) - 4099])
def test_a_row_of_almost_2_31_columns(lib, cols):
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("not enough memory")
    x = torch.zeros(1, cols, dtype=torch.bfloat16, device=DEV)
    x[0, 5], x[0, cols // 2], x[0, cols - 1] = 1.0, -2.0, 4.0
    q = lib.gptq_int8_quantize(x)
    scale = np.float32(4.0) / np.float32(127.0)
    assert float(q.scales) == scale
    for at, value in ((5, 1.0), (cols // 2, -2.0), (cols - 1, 4.0)):
        assert int(q.codes[0, at]) == np.rint(np.float32(value) / scale)
    assert int(torch.count_nonzero(q.codes)) == 3
    y = lib.gptq_int8_dequantize(q, torch.bfloat16)
    assert int(torch.count_nonzero(y)) == 3 and float(y[0, cols - 1]) == 4.0
