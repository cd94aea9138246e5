"""Pins of the microscaled 4-bit oracle, by hand, and of the argument checks of its entry points and
the expert routing's (host only)."""
import ctypes

import numpy as np
import pytest

from oracle import fp4_oracle as F


def test_e2m1_by_hand():
    y = np.array([0.25, 0.2500001, 0.75, 1.25, 1.75, 2.5, 2.6, 3.5, 4.9, 5.0, 5.1, 7.0, 100.0, -0.3, -5.5])
    v = F.e2m1_round(y)
    np.testing.assert_array_equal(v, [0, 0.5, 1, 1, 2, 2, 3, 4, 4, 4, 6, 6, 6, -0.5, -6])
    np.testing.assert_array_equal(F.e2m1_code(v), [0, 1, 2, 2, 4, 4, 5, 6, 6, 6, 7, 7, 7, 9, 15])


def test_e4m3_by_hand():
    a = np.array([0.0, 2.0 ** -10, 2.0 ** -9, 1.0, 1.0625, 1.1875, 447.0, 449.0, 1e9, 2.0 ** -6])
    s = F.e4m3_round(a)
    np.testing.assert_array_equal(s, [0, 0, 2.0 ** -9, 1, 1, 1.25, 448, 448, 448, 2.0 ** -6])
    np.testing.assert_array_equal(F.e4m3_byte(s), [0, 0, 1, 56, 56, 58, 126, 126, 126, 8])


def test_mx_block_by_hand():
    x = np.zeros((1, 40), np.float32)
    x[0, :4] = [7.9, -4.0, 0.26, 1.25]     # a = 7.9: s = 1
    x[0, 32] = 3.0                          # the short block: s = 0.5, 3 / 0.5 = 6
    v, c, b = F.quantise(x, "mx")
    np.testing.assert_array_equal(v[0, :4], [6, -4, 0.5, 1])
    np.testing.assert_array_equal(b, [[127, 126]])
    assert v[0, 32] == 3 and c[0, 32] == 7


def test_nv_block_by_hand():
    x = np.zeros((1, 16), np.float32)
    x[0, :3] = [12.0, 1.0, -0.4]            # g = 0.5: 12 / 3 = 4, s = 2
    v, _, b = F.quantise(x, "nv", 0.5)
    assert b[0, 0] == F.e4m3_byte(np.array(4.0))
    np.testing.assert_array_equal(v[0, :3], [12, 1, 0.0])


def test_scale_tiles_round_trip():
    byte = np.random.default_rng(0).integers(0, 255, (300, 9)).astype(np.uint8)
    t = F.tile_scales(byte, 9 * 32, "mx")
    assert t.shape == (3, 3, 512)
    np.testing.assert_array_equal(F.untile_scales(t, 300, 9), byte)
    assert t[1, 2, 5 * 16 + 2 * 4 + 0] == byte[128 + 64 + 5, 8]


def test_route_by_hand():
    ids = np.array([[1, 0], [0, -1], [1, 2]])
    o, s, p = F.route(ids, 4)
    np.testing.assert_array_equal(o, [0, 2, 4, 5, 5])
    np.testing.assert_array_equal(s, [1, 2, 0, 4, 5, -1])
    np.testing.assert_array_equal(p, [[2, 0], [1, -1], [3, 4]])


# --------------------------------------------------------------------------- refusals, on the host
@pytest.fixture(scope="module")
def clib():
    from post_weight_quantization_04_gb300 import build as b
    import post_weight_quantization_04_gb300 as g
    b.build()
    return g.load()


P = ctypes.c_void_p(64)
Z = ctypes.c_void_p(0)
ODD = ctypes.c_void_p(72)


def test_sizes(clib):
    assert clib.gptq_fp4_code_pitch(1) == 16 and clib.gptq_fp4_code_pitch(33) == 32
    assert clib.gptq_fp4_scale_bytes(1, 128, 0) == 512 and clib.gptq_fp4_scale_bytes(129, 129, 0) == 4 * 512
    assert clib.gptq_fp4_scale_bytes(128, 128, 1) == 2 * 512
    assert clib.gptq_fp4_scale_bytes(128, 128, 2) == 0
    assert clib.gptq_expert_sort_workspace_bytes(10, 2, 8) == 0
    assert clib.gptq_expert_sort_workspace_bytes(1 << 20, 2, 8) > 0


@pytest.mark.parametrize("change,status", [
    (dict(dtype=2), 1), (dict(fmt=2), 1), (dict(rows=-1), 1), (dict(cols=-1), 1), (dict(ldx=63), 1), (dict(codes=ODD), 1),
    (dict(scales=ODD), 1), (dict(codes=Z), 1), (dict(fmt=1, g=Z), 1), (dict(src_rows=5), 1), (dict(index=P, per=0), 1),
    (dict(rows=0, src_rows=0), 0), (dict(cols=0), 0)])
def test_quantize_refusals(clib, change, status):
    a = dict(X=P, dtype=1, src_rows=4, cols=64, ldx=64, index=Z, per=1, rows=4, fmt=0, g=P, codes=P, scales=P) | change
    assert clib.gptq_fp4_quantize(*a.values(), Z) == status


@pytest.mark.parametrize("change,status", [
    (dict(dtype=3), 1), (dict(fmt=-1), 1), (dict(ldy=63), 1), (dict(Y=Z), 1), (dict(fmt=1, g=Z), 1), (dict(rows=0), 0)])
def test_dequantize_refusals(clib, change, status):
    a = dict(codes=P, scales=P, g=P, rows=4, cols=64, fmt=0, Y=P, dtype=0, ldy=64) | change
    assert clib.gptq_fp4_dequantize(*a.values(), Z) == status


@pytest.mark.parametrize("change,status", [
    (dict(T=-1), 1), (dict(K=0), 1), (dict(N=0), 0), (dict(T=0), 0), (dict(fmt=2), 1), (dict(experts=0), 1),
    (dict(experts=2), 1), (dict(offsets=P, experts=1025), 2), (dict(flags=8), 1), (dict(ldy=31), 1), (dict(Y=Z), 1),
    (dict(xc=ODD), 1), (dict(ws=ODD), 1), (dict(fmt=1, xg=Z), 1), (dict(fmt=1, wg=Z), 1), (dict(wc=Z), 1)])
def test_matmul_refusals(clib, change, status):
    a = dict(xc=P, xs=P, xg=P, T=4, wc=P, ws=P, wg=P, N=32, K=64, fmt=0, offsets=Z, experts=1, flags=0, Y=P, ldy=32) | change
    assert clib.gptq_fp4_matmul(*a.values(), Z) == status


def test_other_refusals(clib):
    assert clib.gptq_fp4_tile_scales(P, 4, 64, 1, 0, P, Z) == 1        # stride below the blocks
    assert clib.gptq_fp4_tile_scales(Z, 4, 64, 2, 0, P, Z) == 1
    assert clib.gptq_fp4_tensor_scale(P, 1, 4, 64, 63, P, Z) == 1
    assert clib.gptq_fp4_tensor_scale(P, 1, 4, 64, 64, Z, Z) == 1
    sort = lambda **c: clib.gptq_expert_sort(*(dict(ids=P, T=4, k=2, E=8, o=P, s=P, p=P, ws=Z, n=0) | c).values(), Z)  # noqa: E731
    assert sort(k=0) == 1 and sort(E=0) == 1 and sort(E=1025) == 2 and sort(ids=Z) == 1 and sort(o=Z) == 1
    assert sort(T=1 << 20) == 6 and sort(T=1 << 31) == 1
    gather = lambda **c: clib.gptq_expert_gather(*(dict(X=P, dt=1, T=4, d=64, ld=64, p=P, k=2, o=P, E=8, Y=P, ly=64) | c).values(), Z)  # noqa: E731
    assert gather(dt=2) == 1 and gather(ld=63) == 1 and gather(ly=63) == 1 and gather(Y=Z) == 1 and gather(k=0) == 1
    assert gather(T=0) == 0 and gather(d=0) == 0 and gather(o=Z) == 1
    comb = lambda **c: clib.gptq_expert_combine(*(dict(X=P, dt=1, T=4, d=64, ld=64, p=P, k=2, w=Z, Y=P, ly=64) | c).values(), Z)  # noqa: E731
    assert comb(dt=5) == 1 and comb(p=Z) == 1 and comb(ly=1) == 1 and comb(T=0) == 0
    grad = lambda **c: clib.gptq_expert_combine_grad(*(dict(dY=P, l0=64, Y=P, l1=64, dt=1, T=4, d=64, p=P, k=2, o=P, E=8, w=P, dX=P,  # noqa: E731
                                                            l2=64, dw=P) | c).values(), Z)
    assert grad(w=Z) == 1 and grad(dw=Z) == 1 and grad(l0=3) == 1 and grad(T=0) == 0 and grad(E=0) == 1


def test_a_sort_workspace_has_to_be_aligned(clib):
    for at, status in ((66, 1), (65, 1)):
        assert clib.gptq_expert_sort(P, 1 << 20, 2, 8, P, P, P, ctypes.c_void_p(at), 1 << 30, Z) == status


class _OnDevice:
    """What the binding asks a CUDA tensor, which this is not."""
    is_cuda = True

    def __init__(self, device, dtype, *shape):
        import torch
        self.index, self.dtype, self.shape, self.device = device, dtype, torch.Size(shape), torch.device("cuda", device)

    def get_device(self):
        return self.index

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self.dtype.itemsize

    def stride(self):
        return tuple(self.shape[i + 1:].numel() for i in range(len(self.shape)))

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 20


def test_tensors_of_another_device_are_refused(clib, monkeypatch):
    """Each tensor of each call in turn on device 1 while device 0 is the current one."""
    import torch
    import post_weight_quantization_04_gb300 as g
    f32, i32, u8 = torch.float32, torch.int32, torch.uint8
    tensors = dict(x=(f32, 4, 64), w=(f32, 4, 2), ids=(i32, 4, 2), rows=(f32, 8, 64), offsets=(i32, 3), src=(i32, 8), pos=(i32, 4, 2),
                   xc=(u8, 4, 32), xs=(u8, 1, 1, 512), xg=(f32, 1), wc=(u8, 2, 8, 32), ws=(u8, 2, 1, 1, 512), wg=(f32, 2),
                   index=(i32, 4), bytes=(u8, 4, 4), work=(u8, 4096), y=(f32, 4, 8))
    route = lambda t: g.Route(t["offsets"], t["src"], t["pos"])                                     # noqa: E731
    X = lambda t: g.Fp4(t["xc"], t["xs"], 64, "nv", t["xg"])                                        # noqa: E731
    W = lambda t: g.Fp4(t["wc"], t["ws"], 64, "nv", t["wg"])                                        # noqa: E731
    calls = [
        ("x", lambda t: g.gptq_fp4_tensor_scale(t["x"])),
        ("x xg index", lambda t: g.gptq_fp4_quantize(t["x"], "nv", t["xg"], index=t["index"])),
        ("x xc xs", lambda t: g.gptq_fp4_quantize(t["x"], "nv", t["xg"], out=X(t))),
        ("xc xs xg", lambda t: g.gptq_fp4_dequantize(X(t))),
        ("y", lambda t: g.gptq_fp4_dequantize(X(t), out=t["x"] if t["y"].index == 0 else _OnDevice(1, f32, 4, 64))),
        ("bytes", lambda t: g.gptq_fp4_tile_scales(t["bytes"], 64, "nv")),
        ("xc xs xg wc ws wg offsets", lambda t: g.gptq_fp4_matmul(X(t), W(t), offsets=t["offsets"])),
        ("y", lambda t: g.gptq_fp4_matmul(X(t), W(t), offsets=t["offsets"], out=t["y"])),
        ("ids", lambda t: g.gptq_expert_sort(t["ids"], 2)),
        ("work", lambda t: g.gptq_expert_sort(t["ids"], 2, ws=t["work"])),
        ("x offsets src pos", lambda t: g.gptq_expert_gather(t["x"], route(t))),
        ("rows offsets src pos w", lambda t: g.gptq_expert_combine(t["rows"], route(t), t["w"])),
        ("x rows offsets src pos w", lambda t: g.gptq_expert_combine_grad(t["x"], t["rows"], route(t), t["w"])),
    ]
    real = torch.empty
    monkeypatch.setattr(g, "_current_device", lambda: 0)
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **k: real(*a, **k))      # (results that are never used)
    monkeypatch.setattr(torch, "empty_like", lambda t, **k: real(1))
    g._setup_call(clib)
    try:
        for names, call in calls:
            for n in names.split():
                t = {k: _OnDevice(int(k == n), *v) for k, v in tensors.items()}
                with pytest.raises(ValueError, match="device"):
                    call(t)
    finally:
        monkeypatch.undo()
        g._setup_call(clib)
