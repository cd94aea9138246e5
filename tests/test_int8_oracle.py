"""CPU checks of the 8-bit integer operators and the balance loss: the definitions by hand and by differences, and what the
entry points and the binding refuse before anything is launched."""
import ctypes

import numpy as np
import pytest

from oracle import int8_oracle as I
from test_fp4_oracle import ODD, P, Z, _OnDevice


def test_codes_by_hand():
    c, s = I.quantise([[127.0, 0.5, 1.5, -0.5, -127.0], [0, 0, 0, 0, 0], [2.54, 1.26, -0.047, 0.009, 0]])
    assert c.tolist() == [[127, 0, 2, 0, -127], [0, 0, 0, 0, 0], [127, 63, -2, 0, 0]]
    assert s[0] == 1 and s[1] == 0 and abs(s[2] - 0.02) < 1e-8
    c, s = I.quantise(np.full((1, 3), 1e-45, np.float32))      # a / 127 is nothing
    assert s[0] == 0 and not c.any()
    c, s = I.quantise(np.array([[1e-43, -4e-44]], np.float32))   # the scale is the smallest number, rounded up or down by half
    assert np.abs(c).max() <= 127


def test_norm_gradient_by_differences():
    rng = np.random.default_rng(0)
    h, dy, dh, gain = rng.normal(size=(3, 7)), rng.normal(size=(3, 7)), rng.normal(size=(3, 7)), rng.normal(size=7)
    loss = lambda h, g: (I.rms_norm(h, g, 0.1)[0] * dy).sum() + (h * dh).sum()   # noqa: E731
    dx, dg = I.rms_norm_grad(dy, h, gain, I.rms_norm(h, gain, 0.1)[1], dh)
    for i in range(3):
        for j in range(7):
            d = np.zeros((3, 7))
            d[i, j] = 1e-5
            assert abs((loss(h + d, gain) - loss(h - d, gain)) / 2e-5 - dx[i, j]) < 1e-8
    for j in range(7):
        d = 1e-5 * np.eye(7)[j]
        assert abs((loss(h, gain + d) - loss(h, gain - d)) / 2e-5 - dg[j]) < 1e-8


def test_balance_by_hand_and_by_differences():
    z = np.zeros((4, 2))
    assert I.balance(z, np.array([[0], [1], [0], [1]]))[0] == pytest.approx(1)        # even: 1
    assert I.balance(np.array([[50.0, 0], [50, 0]]), np.array([[0], [0]]))[0] == pytest.approx(2)   # all to one of two
    loss, c, p = I.balance(z, np.array([[0], [1], [-1], [1]]), np.array([1, 1, 1, 0]))
    assert c.tolist() == [1, 1, 3] and loss == pytest.approx(2 / 9 * 3)
    loss, c, p = I.balance(np.full((2, 3), -np.inf), np.array([[0], [2]]))
    assert loss == 0 and c.tolist() == [1, 0, 1, 2]
    assert I.balance(z, np.zeros((4, 1), int), np.zeros(4))[0] == 0
    rng = np.random.default_rng(1)
    z, ids = rng.normal(size=(5, 4)), rng.integers(-1, 4, (5, 2))
    mask = np.array([1, 0, 1, 1, 1])
    _, c, p = I.balance(z, ids, mask)
    dz = I.balance_grad(0.7, p, c, 2)
    for i in range(5):
        for j in range(4):
            d = np.zeros((5, 4))
            d[i, j] = 1e-6
            assert abs(0.7 * (I.balance(z + d, ids, mask)[0] - I.balance(z - d, ids, mask)[0]) / 2e-6 - dz[i, j]) < 1e-8


# ------------------------------------------------------------------------------------ refusals

@pytest.fixture(scope="module")
def clib():
    from post_weight_quantization_04_gb300 import build as b
    import post_weight_quantization_04_gb300 as g
    b.build()
    return g.load()


def test_sizes(clib):
    assert [clib.gptq_int8_pitch(c) for c in (0, 1, 16, 17)] == [0, 16, 16, 32]
    assert clib.gptq_int8_rms_norm_grad_workspace_bytes(1, 10) >= 40
    assert clib.gptq_int8_rms_norm_grad_workspace_bytes(-1, 10) == 0
    assert clib.gptq_expert_balance_workspace_bytes(1, 8) >= 4 * 17 and clib.gptq_expert_balance_workspace_bytes(1, 1025) == 0


@pytest.mark.parametrize("change,status", [
    (dict(dtype=2), 1), (dict(rows=-1), 1), (dict(cols=-1), 1), (dict(ldx=63), 1), (dict(codes=ODD), 1), (dict(codes=Z), 1),
    (dict(scales=Z), 1), (dict(X=Z), 1), (dict(src_rows=5), 1), (dict(index=P, per=0), 1), (dict(rows=1 << 31, src_rows=1 << 31), 1),
    (dict(rows=0, src_rows=0), 0)])
def test_quantize_refusals(clib, change, status):
    a = dict(X=P, dtype=1, src_rows=4, cols=64, ldx=64, index=Z, per=1, rows=4, codes=P, scales=P) | change
    assert clib.gptq_int8_quantize(*a.values(), Z) == status


@pytest.mark.parametrize("change,status", [
    (dict(dtype=3), 1), (dict(ldy=63), 1), (dict(Y=Z), 1), (dict(codes=ODD), 1), (dict(scales=Z), 1), (dict(rows=0), 0), (dict(cols=0), 0)])
def test_dequantize_refusals(clib, change, status):
    a = dict(codes=P, scales=P, rows=4, cols=64, Y=P, dtype=0, ldy=64) | change
    assert clib.gptq_int8_dequantize(*a.values(), Z) == status


@pytest.mark.parametrize("change,status", [
    (dict(dtype=2), 1), (dict(cols=0), 1), (dict(rows=-1), 1), (dict(eps=0.0), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
    (dict(eps=float("inf")), 1), (dict(ldx=63), 1), (dict(R=P, ldr=63), 1), (dict(R=P, H=Z), 1), (dict(R=P, ldh=63), 1),
    (dict(gain=Z), 1), (dict(codes=ODD), 1), (dict(rstd=Z), 1), (dict(scales=Z), 1), (dict(rows=0), 0)])
def test_norm_refusals(clib, change, status):
    a = dict(X=P, ldx=64, R=Z, ldr=64, dtype=1, rows=4, cols=64, gain=P, eps=1e-6, codes=P, scales=P, H=P, ldh=64, rstd=P) | change
    assert clib.gptq_int8_rms_norm(*a.values(), Z) == status


@pytest.mark.parametrize("change,status", [
    (dict(dtype=2), 1), (dict(cols=0), 1), (dict(rows=-1), 1), (dict(lddy=63), 1), (dict(ldh=63), 1), (dict(lddh=63), 1),
    (dict(lddx=63), 1), (dict(dgain=Z), 1), (dict(dX=Z), 1), (dict(rstd=Z), 1), (dict(gain=Z), 1), (dict(ws=Z), 6), (dict(n=16), 6),
    (dict(ws=ctypes.c_void_p(66)), 1)])
def test_norm_grad_refusals(clib, change, status):
    a = dict(dY=P, lddy=64, H=P, ldh=64, dH=P, lddh=64, dtype=1, rows=4, cols=64, gain=P, rstd=P, dX=P, lddx=64, dgain=P, ws=P,
             n=1 << 20) | change
    assert clib.gptq_int8_rms_norm_grad(*a.values(), Z) == status


@pytest.mark.parametrize("change,status", [
    (dict(T=-1), 1), (dict(K=-1), 1), (dict(N=0), 0), (dict(T=0), 0), (dict(experts=0), 1), (dict(experts=2), 1),
    (dict(offsets=P, experts=1025), 2), (dict(K=1 << 17), 2), (dict(flags=4), 1), (dict(ldy=31), 1), (dict(Y=Z), 1), (dict(xc=ODD), 1),
    (dict(wc=ODD), 1), (dict(xs=Z), 1), (dict(ws=Z), 1), (dict(wc=Z), 1)])
def test_matmul_refusals(clib, change, status):
    a = dict(xc=P, xs=P, T=4, wc=P, ws=P, N=32, K=64, offsets=Z, experts=1, flags=0, Y=P, ldy=32) | change
    assert clib.gptq_int8_matmul(*a.values(), Z) == status


@pytest.mark.parametrize("change,status", [
    (dict(dtype=2), 1), (dict(T=-1), 1), (dict(E=0), 1), (dict(E=1025, ldz=1025), 2), (dict(top=0), 1), (dict(ldz=7), 1), (dict(ids=Z), 1),
    (dict(Zp=Z), 1), (dict(loss=Z), 1), (dict(counts=Z), 1), (dict(ws=Z), 6), (dict(n=16), 6), (dict(ws=ctypes.c_void_p(66)), 1),
    (dict(T=1 << 31), 1)])
def test_balance_refusals(clib, change, status):
    a = dict(Zp=P, dtype=0, T=4, E=8, ldz=8, ids=P, top=2, mask=Z, loss=P, counts=P, ws=P, n=1 << 20) | change
    assert clib.gptq_expert_balance(*a.values(), Z) == status


@pytest.mark.parametrize("change,status", [
    (dict(dtype=2), 1), (dict(T=-1), 1), (dict(T=0), 0), (dict(E=0), 1), (dict(E=1025, ldz=1025, lddz=1025), 2), (dict(top=0), 1),
    (dict(ldz=7), 1), (dict(lddz=7), 1), (dict(counts=Z), 1), (dict(dZ=Z), 1)])
def test_balance_grad_refusals(clib, change, status):
    a = dict(dl=P, Zp=P, dtype=0, T=4, E=8, ldz=8, counts=P, top=2, mask=Z, dZ=P, lddz=8) | change
    assert clib.gptq_expert_balance_grad(*a.values(), Z) == status


def _tensors():
    import torch
    f32, i32, i8, b = torch.float32, torch.int32, torch.int8, torch.bool
    return dict(x=(f32, 4, 60), r=(f32, 4, 60), gain=(f32, 60), rstd=(f32, 4), dy=(f32, 4, 60), dh=(f32, 4, 60), dgain=(f32, 60),
                xc=(i8, 4, 64), xs=(f32, 4), wc=(i8, 2, 8, 64), ws=(f32, 2, 8), offsets=(i32, 3), index=(i32, 4), y=(f32, 4, 8),
                work=(torch.uint8, 1 << 16), z=(f32, 4, 8), ids=(i32, 4, 2), mask=(b, 4), loss=(f32, 1), counts=(i32, 9), dz=(f32, 4, 8))


def _calls(g):
    X = lambda t: g.Int8(t["xc"], t["xs"], 60)              # noqa: E731
    W = lambda t: g.Int8(t["wc"], t["ws"], 60)              # noqa: E731
    B = lambda t: g.Balance(t["loss"], t["counts"], 2)      # noqa: E731
    return [
        ("x index", lambda t: g.gptq_int8_quantize(t["x"], index=t["index"])),
        ("x xc xs", lambda t: g.gptq_int8_quantize(t["x"], out=X(t))),
        ("xc xs r", lambda t: g.gptq_int8_dequantize(X(t), out=t["r"])),
        ("x gain r", lambda t: g.gptq_int8_rms_norm(t["x"], t["gain"], 1e-6, t["r"])),
        ("x gain r xc xs dh rstd", lambda t: g.gptq_int8_rms_norm(t["x"], t["gain"], 1e-6, t["r"], out=(X(t), t["dh"], t["rstd"]))),
        ("dy x gain rstd dh work", lambda t: g.gptq_int8_rms_norm_grad(t["dy"], t["x"], t["gain"], t["rstd"], t["dh"], ws=t["work"])),
        ("dy x gain rstd dh r dgain", lambda t: g.gptq_int8_rms_norm_grad(t["dy"], t["x"], t["gain"], t["rstd"], t["dh"],
                                                                          out=(t["r"], t["dgain"]), ws=t["work"])),
        ("xc xs wc ws offsets", lambda t: g.gptq_int8_matmul(X(t), W(t), offsets=t["offsets"])),
        ("y", lambda t: g.gptq_int8_matmul(X(t), W(t), offsets=t["offsets"], out=t["y"])),
        ("z ids mask work", lambda t: g.gptq_expert_balance(t["z"], t["ids"], t["mask"], ws=t["work"])),
        ("z ids mask loss counts", lambda t: g.gptq_expert_balance(t["z"], t["ids"], t["mask"], out=B(t), ws=t["work"])),
        ("loss z counts mask", lambda t: g.gptq_expert_balance_grad(t["loss"], t["z"], B(t), t["mask"])),
        ("dz", lambda t: g.gptq_expert_balance_grad(None, t["z"], B(t), out=t["dz"])),
    ]


@pytest.fixture
def fake(clib, monkeypatch):
    import torch
    import post_weight_quantization_04_gb300 as g
    real = torch.empty
    monkeypatch.setattr(g, "_current_device", lambda: 0)
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **k: real(*a, **k))      # (results that are never used)
    g._setup_call(clib)
    yield g
    monkeypatch.undo()
    g._setup_call(clib)


def test_tensors_of_another_device_are_refused(fake):
    for names, call in _calls(fake):
        for n in names.split():
            t = {k: _OnDevice(int(k == n), *v) for k, v in _tensors().items()}
            with pytest.raises(ValueError, match="device"):
                call(t)


def test_tensors_of_another_type_or_shape_are_refused(fake):
    import torch
    for names, call in _calls(fake):
        for n in names.split():
            if n in ("work",):
                continue
            for wrong in ((torch.float64, *_tensors()[n][1:]), (_tensors()[n][0], *(s + 1 for s in _tensors()[n][1:]))):
                if n in ("index", "x", "ids") and wrong[0] is not torch.float64:
                    continue   # (sizes that other arguments follow)
                t = {k: _OnDevice(0, *v) for k, v in _tensors().items()}
                t[n] = _OnDevice(0, *wrong)
                with pytest.raises(ValueError):
                    call(t)


def test_the_expert_layer_takes_one_form(clib):
    import post_weight_quantization_04_gb300 as g
    i8, f4 = g.Int8(None, None, 4), g.Fp4(None, None, 4, "mx")
    with pytest.raises(ValueError, match="both"):
        g.gptq_expert_mlp(None, None, None, i8, f4)


def test_columns_whose_last_unit_passes_31_bits_are_refused(clib):
    """A warp's units reach up to 1024 columns past the row's end, and their numbers have 31 bits."""
    for cols in ((1 << 31) - 513, (1 << 31) - 1024):
        assert clib.gptq_int8_dequantize(P, P, 2, cols, P, 1, cols, Z) == 1


def test_no_rows_of_a_matrix_that_has_some(clib):
    """An empty index has no address."""
    a = dict(X=P, dtype=1, src_rows=4, cols=64, ldx=64, index=Z, per=1, rows=0, codes=Z, scales=Z)
    assert clib.gptq_int8_quantize(*a.values(), Z) == 0
