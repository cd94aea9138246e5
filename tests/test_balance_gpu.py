"""The balance loss of a router and its gradient, against fp64 and against differences.

Bounds, with u = 2^-24: a softmax's p is off by r = (E / 32 + 24 + |z - max|) u of it (the argument's rounding, expf's 2 units, the
sum's chain and the quotient), a sum of p over the tokens by (T / 64 + 200) u more (a lane's chain, then the groups and CTAs in turn),
the loss by both; a gradient by (E / 32 + 12) u more and r of each term (+ 2^-8 of it for bf16).
"""
import numpy as np
import pytest
import torch

from oracle import int8_oracle as I

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
U = 2.0 ** -24


def f64(t):
    return t.detach().double().cpu().numpy()


def _inputs(T, E, k, dt, seed, drop=0.1, pad=0):
    g = torch.Generator().manual_seed(seed)
    z = (torch.randn(T, E + pad, generator=g) * 2).to(DT[dt]).to(DEV)[:, pad:]
    ids = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
    ids[torch.rand(T, k, generator=g) < drop] = -1
    return z, ids.to(DEV), (torch.rand(T, generator=g) < 0.8).to(DEV)


def _check(lib, z, ids, mask, dloss=0.5):
    T, E = z.shape
    b = lib.gptq_expert_balance(z, ids, mask)
    Z, m = f64(z), None if mask is None else mask.cpu().numpy()
    loss, counts, p = I.balance(Z, ids.cpu().numpy(), m)
    np.testing.assert_array_equal(b.counts.cpu().numpy(), counts)
    finite = Z[np.isfinite(Z)]
    r = (E / 32 + 24 + (np.ptp(finite) if finite.size else 0)) * U
    assert abs(float(b.loss) - loss) <= (r + (T / 64 + 200) * U) * loss
    d = torch.full((1,), dloss, device=DEV)
    dz = lib.gptq_expert_balance_grad(d, z, b, mask)
    ref = I.balance_grad(dloss, p, counts, ids.shape[1])
    n, c = max(1, counts[-1]), counts[:-1].astype(float)
    size = dloss * E / (ids.shape[1] * float(n) ** 2) * p * (c + (p * c).sum(1, keepdims=True))
    off = (2 * r + (E / 32 + 12) * U) * size + 2.0 ** -140 + (2.0 ** -8 * np.abs(ref) if z.dtype is torch.bfloat16 else 0)
    assert (np.abs(f64(dz) - ref) <= off).all()
    if m is not None:
        assert not f64(dz)[m == 0].any()
    return b, dz


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (3, 2, 1), (33, 5, 3), (33, 64, 6), (100, 16, 2), (65, 130, 8), (200, 333, 4),
                                   (50, 1024, 8), (5000, 8, 2), (4097, 64, 1), (6000, 200, 2)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("pad", [0, 3])
def test_loss_and_gradient(lib, T, E, k, dt, masked, pad):
    z, ids, mask = _inputs(T, E, k, dt, T + E, pad=pad)
    mask = mask if masked else None
    b, dz = _check(lib, z, ids, mask)
    b2 = lib.gptq_expert_balance(z, ids, mask.to(torch.uint8) * 7 if masked else None)
    assert torch.equal(b.loss, b2.loss) and torch.equal(b.counts, b2.counts)      # the same again
    assert torch.equal(lib.gptq_expert_balance_grad(None, z, b, mask),
                       lib.gptq_expert_balance_grad(torch.ones(1, device=DEV), z, b, mask))
    wide = torch.full((T, E + 2), 3.0, dtype=z.dtype, device=DEV)
    lib.gptq_expert_balance_grad(torch.full((1,), 0.5, device=DEV), z, b, mask, out=wide[:, 1:-1])
    assert torch.equal(wide[:, 1:-1], dz) and (wide[:, 0] == 3).all() and (wide[:, -1] == 3).all()
    z2 = z.clone()
    lib.gptq_expert_balance_grad(torch.full((1,), 0.5, device=DEV), z2, b, mask, out=z2)
    assert torch.equal(z2, dz)


def test_experts_that_are_masked_off(lib):
    """logits of -inf and of the type's lowest value, a row of nothing else, everything dropped, everything masked"""
    for dt in ("f32", "bf16"):
        z, ids, mask = _inputs(70, 40, 2, dt, 3)
        z[:, 5:20] = -float("inf")
        z[7] = -float("inf")
        z[8] = torch.finfo(DT[dt]).min
        z[9, :39] = torch.finfo(DT[dt]).min
        b, dz = _check(lib, z[:7], ids[:7], mask[:7])
        assert not dz[:, 5:20].any()
        b = lib.gptq_expert_balance(z, ids)
        loss, counts, p = I.balance(f64(z), ids.cpu().numpy())
        assert abs(float(b.loss) - loss) <= 1e-5 * loss
        dz = lib.gptq_expert_balance_grad(None, z, b)
        assert torch.isfinite(dz).all() and not dz[7].any()
        b = lib.gptq_expert_balance(z, torch.full_like(ids, -1))
        assert float(b.loss) == 0 and not b.counts[:-1].any() and b.counts[-1] == 70
        b = lib.gptq_expert_balance(z, ids, torch.zeros_like(mask))
        assert float(b.loss) == 0 and not b.counts.any()
        assert not lib.gptq_expert_balance_grad(None, z, b, torch.zeros_like(mask)).any()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_what_is_not_finite_is_reported_where_it_counts(lib, bad):
    z, ids, mask = _inputs(40, 12, 2, "f32", 4)
    mask[:] = True
    b0 = lib.gptq_expert_balance(z, ids, mask)
    mask[11] = False
    z[11, 3] = bad
    b = lib.gptq_expert_balance(z, ids, mask)       # a masked row is not looked at
    assert torch.isfinite(b.loss) and b.counts[-1] == 39
    assert torch.isfinite(lib.gptq_expert_balance_grad(None, z, b, mask)).all()
    for call in (lambda: lib.gptq_expert_balance(z, ids), lambda: lib.gptq_expert_balance_grad(None, z, b0)):
        with pytest.raises(lib.GptqError) as e:
            call()
        assert e.value.status == 7


def test_ids_past_the_experts_are_reported(lib):
    z, ids, _ = _inputs(10, 4, 2, "f32", 5, drop=0)
    ids[3, 1] = 4
    with pytest.raises(lib.GptqError) as e:
        lib.gptq_expert_balance(z, ids)
    assert e.value.status == 1


def test_no_tokens(lib):
    z = torch.empty(0, 6, device=DEV)
    b = lib.gptq_expert_balance(z, torch.empty(0, 2, dtype=torch.int32, device=DEV))
    assert float(b.loss) == 0 and b.counts.tolist() == [0] * 7
    assert lib.gptq_expert_balance_grad(None, z, b).shape == (0, 6)


def test_gradient_by_differences(lib):
    z, ids, mask = _inputs(9, 7, 2, "f32", 6)
    b = lib.gptq_expert_balance(z, ids, mask)
    dz = f64(lib.gptq_expert_balance_grad(None, z, b, mask))
    loss = lambda Z: I.balance(Z, ids.cpu().numpy(), mask.cpu().numpy())[0]   # noqa: E731
    for i, j in ((0, 0), (3, 6), (8, 2)):
        d = np.zeros((9, 7))
        d[i, j] = 1e-4
        assert abs((loss(f64(z) + d) - loss(f64(z) - d)) / 2e-4 - dz[i, j]) <= 1e-6


@pytest.mark.parametrize("T,E,k", [(1024, 3, 2), (1025, 3, 2), (12289, 4, 1), (513, 8, 2), (6144, 7, 3), (6145, 8, 2), (129, 64, 6), (1000, 64, 6),
                                   (1536, 50, 2), (1537, 64, 1), (65, 256, 8), (768, 200, 8), (17, 1024, 8), (192, 1024, 1), (193, 700, 4)])
@pytest.mark.parametrize("masked", [False, True])
def test_loss_by_one_cta_one_cluster_and_two_launches(lib, T, E, k, masked):
    z, ids, mask = _inputs(T, E, k, "f32", T + E)
    b, _ = _check(lib, z, ids, mask if masked else None)
    for _ in range(20):
        b2 = lib.gptq_expert_balance(z, ids, mask if masked else None)
        assert torch.equal(b.loss, b2.loss) and torch.equal(b.counts, b2.counts)
