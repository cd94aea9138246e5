"""Tokens sorted by expert and back, against the fp64 oracle and against differences.

Places and copied rows are compared for equality. A combined row is a sum of `top` products in fp32
(at most 2 `top` roundings) rounded once: |y - ref| <= 2 top 2^-24 sum_j |w ys| (+ 2^-9 |ref| for bf16,
2^-8 with margin for the double rounding). dys is one product, rounded once (twice for bf16); dw a sum
of d products in fp32: |dw - ref| <= (d + 1) 2^-24 sum |dy ys|.
"""
import numpy as np
import pytest
import torch

from oracle import fp4_oracle as F

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def f64(t):
    return t.detach().double().cpu().numpy()


def _ids(T, k, E, seed, drop=0.2):
    rng = np.random.default_rng(seed)
    p = rng.dirichlet(np.full(E, 0.4))
    ids = rng.choice(E, (T, k), p=p)
    ids[rng.random((T, k)) < drop] = -1 - rng.integers(0, 3)
    return ids.astype(np.int32)


CASES = [(1, 1, 1), (1, 2, 8), (5, 2, 8), (33, 6, 64), (100, 1, 1024), (300, 8, 7), (2048, 1, 3), (1500, 3, 300),
         (9000, 2, 5), (40000, 4, 130)]


@pytest.mark.parametrize("T,k,E", CASES)
@pytest.mark.parametrize("drop", [0.0, 0.2, 1.0])
def test_sort(lib, T, k, E, drop):
    ids = _ids(T, k, E, T + k + E, drop)
    r = lib.gptq_expert_sort(torch.tensor(ids, device=DEV), E)
    o, s, p = F.route(ids, E)
    np.testing.assert_array_equal(r.offsets.cpu().numpy(), o)
    np.testing.assert_array_equal(r.pos.cpu().numpy(), p)
    np.testing.assert_array_equal(r.src.cpu().numpy(), s)


def test_sort_reports_ids_past_the_experts(lib):
    ids = torch.tensor([[0, 4], [1, 0]], dtype=torch.int32, device=DEV)
    with pytest.raises(lib.GptqError) as e:
        lib.gptq_expert_sort(ids, 4)
    assert e.value.status == 1
    r = lib.gptq_expert_sort(ids, 5)
    assert r.offsets.tolist() == [0, 2, 3, 3, 3, 4]


def test_sort_of_no_tokens(lib):
    r = lib.gptq_expert_sort(torch.empty(0, 2, dtype=torch.int32, device=DEV), 3)
    assert r.offsets.tolist() == [0, 0, 0, 0]


ROWS = [(1, 1, 1, 1), (1, 2, 8, 4096), (5, 2, 8, 100), (33, 6, 64, 1000), (70, 3, 5, 33), (9, 8, 16, 2056), (130, 2, 4, 9000)]


def _setup(lib, T, k, E, D, dt, drop=0.2, pad=0):
    g = torch.Generator().manual_seed(T + D)
    ids = _ids(T, k, E, T + D, drop)
    r = lib.gptq_expert_sort(torch.tensor(ids, device=DEV), E)
    make = lambda n: torch.randn(n, D + pad, generator=g).to(DT[dt]).to(DEV)[:, pad:]  # noqa: E731
    w = torch.rand(T, k, generator=g).to(DEV)
    return F.route(ids, E), r, make(T), make(T * k), make(T), w


@pytest.mark.parametrize("T,k,E,D", ROWS)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("pad", [0, 3, 8])
def test_rows_there_and_back(lib, T, k, E, D, dt, pad):
    (o, s, p), r, x, ys, dy, w = _setup(lib, T, k, E, D, dt, pad=pad)
    live, b16 = o[-1], dt == "bf16"
    # gather
    xs = lib.gptq_expert_gather(x, r)
    ref = np.where((s >= 0)[:, None], f64(x)[np.maximum(s, 0) // k], 0)
    np.testing.assert_array_equal(f64(xs), ref)
    # its gradient and the combination
    ysd, wd, dyd = f64(ys), f64(w), f64(dy)
    rows = np.where((p >= 0)[..., None], ysd[np.maximum(p, 0)], 0)
    for got, ww in ((lib.gptq_expert_gather_grad(ys, r), np.ones((T, k))), (lib.gptq_expert_combine(ys, r, w), wd)):
        ref = (rows * ww[..., None]).sum(1)
        bound = 2 * k * 2.0 ** -24 * (np.abs(rows) * ww[..., None]).sum(1) + (2.0 ** -8 * np.abs(ref) if b16 else 0)
        assert (np.abs(f64(got) - ref) <= bound).all()
    # the combination's gradient
    dys, dw = lib.gptq_expert_combine_grad(dy, ys, r, w)
    ref = np.where((s >= 0)[:, None], dyd[np.maximum(s, 0) // k] * wd.reshape(-1)[np.maximum(s, 0)][:, None], 0)
    assert (np.abs(f64(dys) - ref) <= (2.0 ** -8 if b16 else 2.0 ** -24) * np.abs(ref)).all()
    assert (f64(dys)[live:] == 0).all()
    ref = (rows * dyd[:, None]).sum(-1)
    assert (np.abs(f64(dw) - ref) <= (D + 1) * 2.0 ** -24 * (np.abs(rows) * np.abs(dyd[:, None])).sum(-1)).all()
    assert (f64(dw)[p < 0] == 0).all()


def test_gradients_against_differences(lib):
    """L = <dy, combine(gather(x) * 2, w)>: changes of x and w in steps of a power of two change L by
    the gradients (L is linear in each, so only rounding is between them)."""
    T, k, E, D = 6, 3, 4, 40
    _, r, x, _, dy, w = _setup(lib, T, k, E, D, "f32")

    def loss(x, w):
        return (f64(lib.gptq_expert_combine(lib.gptq_expert_gather(x, r) * 2, r, w)) * f64(dy)).sum()

    ys = lib.gptq_expert_gather(x, r) * 2
    dys, dw = lib.gptq_expert_combine_grad(dy, ys, r, w)
    dx = lib.gptq_expert_gather_grad(dys * 2, r)
    base, step = loss(x, w), 0.25
    scale = np.abs(f64(dy)).sum() * 8
    for t, j in ((0, 0), (2, 1), (5, 2)):
        w2 = w.clone()
        w2[t, j] += step
        assert abs((loss(x, w2) - base) / step - dw[t, j].item()) <= scale * 2.0 ** -20
        x2 = x.clone()
        x2[t, 7 * j] += step
        assert abs((loss(x2, w) - base) / step - dx[t, 7 * j].item()) <= scale * 2.0 ** -20


def test_nonfinite_rows_that_no_slot_reads_stay_out(lib):
    T, k, E, D = 20, 2, 4, 64
    (o, s, p), r, _, ys, dy, w = _setup(lib, T, k, E, D, "bf16", drop=0.5)
    ys[int(o[-1]):] = float("nan")
    assert torch.isfinite(lib.gptq_expert_combine(ys, r, w)).all()
    dys, dw = lib.gptq_expert_combine_grad(dy, ys, r, w)
    assert torch.isfinite(dys).all() and torch.isfinite(dw).all()


def test_rows_of_no_columns(lib):
    r = lib.gptq_expert_sort(torch.tensor([[0, 1], [1, -1]], dtype=torch.int32, device=DEV), 2)
    x, ys, w = torch.empty(2, 0, device=DEV), torch.empty(4, 0, device=DEV), torch.ones(2, 2, device=DEV)
    assert lib.gptq_expert_gather(x, r).shape == (4, 0) and lib.gptq_expert_combine(ys, r, w).shape == (2, 0)
    dys, dw = lib.gptq_expert_combine_grad(x, ys, r, w)
    assert dys.shape == (4, 0) and (dw == 0).all()


def test_places_past_the_rows_are_reported(lib):
    _, r, x, ys, dy, w = _setup(lib, 8, 2, 4, 64, "f32", drop=0.0)
    r = r._replace(pos=r.pos.clone())
    r.pos[3, 1] = 16
    for call in (lambda: lib.gptq_expert_gather(x, r), lambda: lib.gptq_expert_combine(ys, r, w),
                 lambda: lib.gptq_expert_combine_grad(dy, ys, r, w)):
        with pytest.raises(lib.GptqError) as e:
            call()
        assert e.value.status == 1


@pytest.mark.parametrize("T", [40, 3000])
def test_results_given_and_on_a_stream(lib, T):
    """The forms with `out`, `ws` and `stream` give what the common form gives."""
    _, r, x, ys, dy, w = _setup(lib, T, 3, 6, 96, "bf16")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ids = torch.tensor(_ids(T, 3, 6, T + 96), device=DEV)
    nb = lib.gptq_expert_sort_workspace_bytes(T, 3, 6)
    ws = torch.empty(nb, dtype=torch.uint8, device=DEV) if nb else None
    r2 = lib.gptq_expert_sort(ids, 6, ws=ws, stream=s)
    xs = lib.gptq_expert_gather(x, r2, out=torch.empty_like(ys), stream=s)
    y = lib.gptq_expert_combine(ys, r2, w, out=torch.empty_like(x), stream=s)
    dys, dw = lib.gptq_expert_combine_grad(dy, ys, r2, w, out=(torch.empty_like(ys), torch.empty_like(w)), stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(r, r2))
    ref = lib.gptq_expert_combine_grad(dy, ys, r, w)
    assert torch.equal(xs, lib.gptq_expert_gather(x, r)) and torch.equal(y, lib.gptq_expert_combine(ys, r, w))
    assert torch.equal(dys, ref[0]) and torch.equal(dw, ref[1])


@pytest.mark.slow
def test_offsets_past_32_bits(lib):
    """More than 2^31 elements of gathered rows: the last rows are as right as the first."""
    T, k, E, D = 160000, 2, 4, 7168
    g = torch.Generator(device=DEV).manual_seed(1)
    ids = torch.randint(0, E, (T, k), generator=g, device=DEV, dtype=torch.int32)
    r = lib.gptq_expert_sort(ids, E)
    x = torch.randn(T, D, generator=g, device=DEV, dtype=torch.bfloat16)
    xs = lib.gptq_expert_gather(x, r)
    assert xs.numel() > 1 << 31
    for a in (0, T * k - 3):
        assert torch.equal(xs[a:a + 3], x[(r.src[a:a + 3] // k).long()])
    w = torch.full((T, k), 0.5, device=DEV)
    y = lib.gptq_expert_combine(xs, r, w)
    assert torch.equal(y[-3:], x[-3:]) and torch.equal(y[:3], x[:3])
    q = lib.gptq_fp4_quantize(xs, "mx")
    tail = lib.gptq_fp4_quantize(xs[-3:], "mx")
    assert torch.equal(q.codes[-3:], tail.codes)
    v = lib.gptq_fp4_dequantize(q, torch.bfloat16)
    assert torch.equal(v[-3:], lib.gptq_fp4_dequantize(tail, torch.bfloat16))


def test_binding_refusals(lib):
    _, r, x, ys, dy, w = _setup(lib, 4, 2, 4, 64, "f32")
    for call in (lambda: lib.gptq_expert_sort(r.pos.long(), 4), lambda: lib.gptq_expert_sort(r.pos[0], 4),
                 lambda: lib.gptq_expert_gather(x[:3], r), lambda: lib.gptq_expert_gather(x.half(), r),
                 lambda: lib.gptq_expert_combine(ys[:3], r, w), lambda: lib.gptq_expert_combine(ys, r, w.double()),
                 lambda: lib.gptq_expert_combine_grad(dy.bfloat16(), ys, r, w), lambda: lib.gptq_expert_combine_grad(dy, ys, r, w[:2])):
        with pytest.raises(ValueError):
            call()


# 1025 to 4096 slots are sorted by one CTA of 32 warps, whose counters (128 bytes per expert) need more shared
# memory than a launch has by default from 319 experts on; those run before larger numbers
@pytest.mark.parametrize("T,k", [(1025, 1), (256, 8), (2048, 2)])
@pytest.mark.parametrize("E", [318, 319, 384, 383, 385, 1024])
def test_sort_in_one_block_with_many_experts(lib, T, k, E):
    ids = _ids(T, k, E, T + k + E, 0.1)
    r = lib.gptq_expert_sort(torch.tensor(ids, device=DEV), E)
    o, s, p = F.route(ids, E)
    np.testing.assert_array_equal(r.offsets.cpu().numpy(), o)
    np.testing.assert_array_equal(r.pos.cpu().numpy(), p)
    np.testing.assert_array_equal(r.src.cpu().numpy(), s)


def test_sorts_of_two_threads(lib):
    """Two host threads that sort for other numbers of experts on streams of their own: what a launch needs
    of the kernel is not what the other thread set for its own."""
    import threading
    failed = []

    def work(E):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                ids = _ids(500, 4, E, E)
                want = torch.tensor(F.route(ids, E)[2].astype(np.int32), device=DEV)
                t = torch.tensor(ids, device=DEV)
                for _ in range(3000):
                    r = lib.gptq_expert_sort(t, E)
                assert torch.equal(r.pos, want)
        except Exception as e:  # noqa: BLE001
            failed.append((E, repr(e)))

    with lib.deferred_status():
        threads = [threading.Thread(target=work, args=(E,)) for E in (400, 1024)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        lib.status_sync()
    assert not failed, failed


def test_sort_workspaces(lib):
    """A workspace of the caller's on any word; one that is off a word, on the host, or repeats its memory is refused."""
    ids = torch.tensor(_ids(5000, 2, 9, 1), device=DEV)
    want, nb = lib.gptq_expert_sort(ids, 9), lib.gptq_expert_sort_workspace_bytes(5000, 2, 9)
    ws = torch.empty(nb + 4, dtype=torch.uint8, device=DEV)
    for good in (ws[4:], torch.empty(nb // 4, dtype=torch.int32, device=DEV)):
        got = lib.gptq_expert_sort(ids, 9, ws=good)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    for bad in (ws.cpu(), ws[:1].expand(nb), ws[::2]):
        with pytest.raises(ValueError):
            lib.gptq_expert_sort(ids, 9, ws=bad)
    with pytest.raises(lib.GptqError) as e:
        lib.gptq_expert_sort(ids, 9, ws=ws[1:nb + 1])
    assert e.value.status == 1
    with pytest.raises(lib.GptqError) as e:
        lib.gptq_expert_sort(ids, 9, ws=ws[:nb - 4])
    assert e.value.status == 6
