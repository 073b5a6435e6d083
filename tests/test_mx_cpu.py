"""Argument errors of the MXFP4 and dispatch calls, reported before anything is
launched (no GPU: aligned fake pointers), and the binding's own checks."""
import ctypes

import numpy as np
import pytest

import _mx_ref as R

P = 0x10000      # a fake, aligned device pointer: never read
OK, NULL, SHAPE, ALIGN, WORKSPACE, FORMAT = 0, -1, -2, -4, -5, -8


@pytest.fixture(scope="module")
def L():
    from bit_weight_only_amd import lbq
    return lbq


def _mx(L, rows, cols, codes=P, scales=P):
    return ctypes.byref(L.Mx(rows, cols, codes, scales))


def test_bytes(L):
    lib, a, b = L.lib(), ctypes.c_size_t(), ctypes.c_size_t()
    assert lib.lbq_mx_bytes(10, 256, ctypes.byref(a), ctypes.byref(b)) == OK and (a.value, b.value) == (1280, 80)
    assert lib.lbq_mx_bytes(0, 128, ctypes.byref(a), ctypes.byref(b)) == OK and (a.value, b.value) == (0, 0)
    for rows, cols in ((-1, 128), (1, 0), (1, 64), (1, 130), (2 ** 31 - 1, 128), (2 ** 30 + 1, 128), (2 ** 30, 256), (1, 2 ** 24 + 128)):
        assert lib.lbq_mx_bytes(rows, cols, ctypes.byref(a), ctypes.byref(b)) == SHAPE
    assert lib.lbq_mx_bytes(1, 128, None, ctypes.byref(b)) == NULL


def test_quantize_refusals(L):
    lib = L.lib()
    for f in (lib.lbq_mx_quantize, lib.lbq_mx_quantize_t):
        assert f(P, 3, 128, 128, P, P, None) == FORMAT
        assert f(P, -1, 128, 128, P, P, None) == FORMAT
        assert f(P, 0, -1, 128, P, P, None) == SHAPE
        assert f(P, 0, 128, 0, P, P, None) == SHAPE
        assert f(None, 0, 128, 128, P, P, None) == NULL
        assert f(P, 0, 128, 128, None, P, None) == NULL
        assert f(P, 0, 128, 128, P, None, None) == NULL
        assert f(P + 2, 0, 128, 128, P, P, None) == ALIGN
        assert f(P, 0, 128, 128, P + 8, P, None) == ALIGN
        assert f(P, 0, 0, 128, None, None, None) == OK           # nothing to do
    assert lib.lbq_mx_quantize(P, 0, 4, 100, P, P, None) == SHAPE
    assert lib.lbq_mx_quantize_t(P, 0, 2 ** 31 - 1, 4, P, P, None) == SHAPE
    assert lib.lbq_mx_quantize_t(P, 2, 1, 2 ** 30 - 63, P, P, None) == SHAPE
    assert lib.lbq_mx_dequantize(None, P, 0, None) == NULL
    assert lib.lbq_mx_dequantize(_mx(L, 4, 128), None, 0, None) == NULL
    assert lib.lbq_mx_dequantize(_mx(L, 4, 128), P, 9, None) == FORMAT
    assert lib.lbq_mx_dequantize(_mx(L, 4, 100), P, 0, None) == SHAPE
    assert lib.lbq_mx_dequantize(_mx(L, 0, 128, None, None), None, 0, None) == OK


def test_product_refusals(L):
    lib, n = L.lib(), ctypes.c_size_t()
    a, b = _mx(L, 4, 256), _mx(L, 6, 256)
    assert lib.lbq_mx_matmul_workspace(a, b, ctypes.byref(n)) == OK
    assert lib.lbq_mx_matmul_workspace(a, b, None) == NULL
    assert lib.lbq_mx_matmul_workspace(a, _mx(L, 6, 128), ctypes.byref(n)) == SHAPE
    assert lib.lbq_mx_matmul(a, _mx(L, 6, 128), P, 0, P, 1 << 40, None) == SHAPE
    assert lib.lbq_mx_matmul(a, _mx(L, 6, 256, P, None), P, 0, P, 1 << 40, None) == NULL
    assert lib.lbq_mx_matmul(a, _mx(L, 6, 256, P + 4), P, 0, P, 1 << 40, None) == ALIGN
    assert lib.lbq_mx_matmul(a, b, None, 0, P, 1 << 40, None) == NULL
    assert lib.lbq_mx_matmul(a, b, P + 2, 0, P, 1 << 40, None) == ALIGN
    assert lib.lbq_mx_matmul(a, b, P, 5, P, 1 << 40, None) == FORMAT
    assert lib.lbq_mx_matmul(_mx(L, 0, 256, None, None), b, None, 0, None, 0, None) == OK

    assert lib.lbq_mx_linear_workspace(b, 200, ctypes.byref(n)) == OK and n.value >= 200 * (128 + 8)
    assert lib.lbq_mx_linear_workspace(b, -1, ctypes.byref(n)) == SHAPE
    assert lib.lbq_mx_linear_forward(b, P, 200, P, 0, P, n.value - 1, None) == WORKSPACE
    assert lib.lbq_mx_linear_forward(b, P, 200, P, 2, P, n.value, None) == FORMAT      # fp32 activations
    assert lib.lbq_mx_linear_forward(b, None, 200, P, 0, P, n.value, None) == NULL
    assert lib.lbq_mx_linear_forward(b, P, 200, P, 0, None, n.value, None) == NULL
    assert lib.lbq_mx_linear_forward(b, P, 200, P, 0, P + 8, n.value, None) == ALIGN
    assert lib.lbq_mx_linear_forward(b, None, 0, None, 0, None, 0, None) == OK

    def grouped(w=b, E=3, M=4, T=8, x=P, off=P, perm=P, k=2, y=P, dt=0, ws=P, nb=1 << 40):
        return lib.lbq_mx_grouped_forward(w, E, x, M, off, perm, k, T, y, dt, ws, nb, None)
    assert lib.lbq_mx_grouped_workspace(b, 3, 200, 400, ctypes.byref(n)) == OK and n.value >= 200 * (128 + 8)
    assert grouped(M=200, T=400, nb=n.value - 1) == WORKSPACE and grouped(M=200, T=400, ws=None) == NULL
    assert grouped(E=4) == SHAPE and grouped(E=0) == SHAPE and grouped(k=0) == SHAPE
    assert grouped(w=_mx(L, 2050, 128), E=1025) == SHAPE
    assert grouped(perm=None) == SHAPE                             # without perm x has T rows
    assert grouped(T=2 ** 30 + 1) == SHAPE and grouped(M=-1) == SHAPE
    assert grouped(w=_mx(L, 6, 4096), M=2 ** 21) == SHAPE           # 2^33 values of x
    assert grouped(dt=2) == FORMAT and grouped(off=None) == NULL and grouped(y=P + 2) == ALIGN
    assert grouped(off=P + 2) == ALIGN and grouped(perm=P + 2) == ALIGN
    assert grouped(M=0, x=None, off=None, y=None, ws=None, T=0) == OK


def test_dispatch_refusals(L):
    lib, n = L.lib(), ctypes.c_size_t()
    assert lib.lbq_moe_sort_workspace(16, 8, 2, ctypes.byref(n)) == OK
    for M, E, k in ((-1, 8, 2), (16, 0, 2), (16, 1025, 2), (16, 8, 0), (16, 8, 33), (1 << 20, 8, 2)):
        assert lib.lbq_moe_sort_workspace(M, E, k, ctypes.byref(n)) == SHAPE
        assert lib.lbq_moe_sort(P, M, E, k, P, P, P, P, P, 1 << 40, None) == SHAPE
    assert lib.lbq_moe_sort(None, 16, 8, 2, P, P, P, P, P, 1 << 40, None) == NULL
    assert lib.lbq_moe_sort(P, 16, 8, 2, P, P, P, None, P, 1 << 40, None) == NULL
    assert lib.lbq_moe_sort(P + 2, 16, 8, 2, P, P, P, P, P, 1 << 40, None) == ALIGN
    assert lib.lbq_moe_sort_workspace(1 << 17, 8, 8, ctypes.byref(n)) == OK and n.value > 0
    assert lib.lbq_moe_sort(P, 1 << 17, 8, 8, P, P, P, P, P, n.value - 1, None) == WORKSPACE

    def gather(x=P, dt=0, M=4, H=8, pos=P, k=2, T=8, out=P):
        return lib.lbq_moe_gather(x, dt, M, H, pos, k, T, out, None)

    def gather_b(x=P, dt=0, M=4, H=8, pos=P, k=2, T=8, out=P):
        return lib.lbq_moe_gather_backward(x, dt, T, H, pos, M, k, out, None)

    def combine(x=P, dt=0, M=4, H=8, pos=P, k=2, T=8, out=P, w=P):
        return lib.lbq_moe_combine(x, dt, T, H, pos, w, M, k, out, None)

    def combine_b(x=P, dt=0, M=4, H=8, pos=P, k=2, T=8, out=P, w=P, dw=P):
        return lib.lbq_moe_combine_backward(P, x, dt, T, H, pos, w, M, k, out, dw, None)
    for f in (gather, gather_b, combine, combine_b):
        assert f(dt=3) == FORMAT and f(H=0) == SHAPE and f(H=2 ** 30 + 1) == SHAPE and f(k=33) == SHAPE and f(M=-1) == SHAPE and f(T=-1) == SHAPE
        assert f(x=None) == NULL and f(pos=None) == NULL and f(out=None) == NULL
        assert f(x=P + 4) == ALIGN and f(out=P + 4) == ALIGN and f(pos=P + 2) == ALIGN
        assert f(M=0, x=None, pos=None, out=None) == OK
    assert combine(w=None) == NULL and combine_b(w=None) == NULL and combine_b(dw=None) == NULL


def test_binding_refusals(L):
    """Tensors that are not on a GPU, not contiguous or of another type are refused by the binding."""
    import torch

    x = torch.zeros((4, 128))
    codes, scales = torch.zeros((4, 64), dtype=torch.uint8), torch.zeros((1, 4, 4), dtype=torch.uint8)
    for call in (lambda: L.mx_quantize(x), lambda: L.mx_quantize(x[0]), lambda: L.MxTensor(codes, scales),
                 lambda: L.moe_sort(torch.zeros((4, 2), dtype=torch.int32), 4),
                 lambda: L.moe_gather(x, torch.zeros((4, 2), dtype=torch.int32)),
                 lambda: L.moe_combine(x, torch.zeros((4, 2), dtype=torch.int32), torch.zeros((4, 2)))):
        with pytest.raises(L.LbqError) as e:
            call()
        assert e.value.status in (SHAPE, FORMAT)


def test_who_quantizes(L):
    """The workspace tells which product takes x as it is: few tokens on rows that are not too long. A batch whose
    quantizing every workgroup would repeat at more than a launch's cost has its codes in the workspace."""
    def linear(M, K, N=4096):
        return L._query("lbq_mx_linear_workspace", ((N, K), M))

    def grouped(M, K, E, k, N=256):
        return L._query("lbq_mx_grouped_workspace", ((E * N, K), E, M, M * k))
    for M, K in ((1, 17408), (3, 14336), (4, 14336), (8, 4096), (8, 8192), (16, 4096), (32, 2048)):
        assert linear(M, K) == 0
    for M, K in ((8, 14336), (8, 17408), (5, 17408), (16, 8192), (33, 1024), (32, 4096)):
        assert linear(M, K) >= M * K * 17 // 32
    for M, K, E, k in ((32, 2048, 256, 8), (256, 2048, 256, 8), (20, 4096, 16, 2), (1, 14336, 8, 2)):
        assert grouped(M, K, E, k) == 0
    for M, K, E, k in ((40, 4096, 16, 4), (32, 8192, 16, 4), (8, 14336, 8, 4)):
        assert grouped(M, K, E, k) >= M * K * 17 // 32


def test_sizes_past_32_bits(L, monkeypatch):
    """A size that a C int does not hold is refused, not cut off: 2^32 + n would arrive as n (meta tensors that
    claim to be on a GPU: nothing of them is read)."""
    import torch

    for name, args in (("lbq_mx_linear_workspace", ((256, 128), 2 ** 32)), ("lbq_moe_sort_workspace", (2 ** 32, 8, 2)),
                       ("lbq_moe_sort_workspace", (16, 2 ** 32 + 8, 2)), ("lbq_moe_sort_workspace", (16, 8, 2 ** 32 + 2)),
                       ("lbq_mx_matmul_workspace", ((2 ** 32 + 4, 128), (4, 128))),
                       ("lbq_mx_grouped_workspace", ((256, 128), 2, 4, 2 ** 32 + 4))):
        with pytest.raises(L.LbqError) as e:
            L._query(name, args)
        assert e.value.status == SHAPE

    launched = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: launched.append(name) or 0
    monkeypatch.setattr(L, "_ready", lambda: Lib())
    monkeypatch.setattr(L, "_on", lambda gpu, stream, go, *used: go(0))
    monkeypatch.setattr(L, "_need", lambda *a: None)
    monkeypatch.setattr(L, "_torch", torch)
    monkeypatch.setattr(L, "_dtypes", {torch.float16: 0})
    big, one = 2 ** 32 + 2, 2

    def half(*shape):
        return torch.empty(shape, dtype=torch.float16, device="meta")

    def ints(*shape):
        return torch.empty(shape, dtype=torch.int32, device="meta")

    def floats(*shape):
        return torch.empty(shape, dtype=torch.float32, device="meta")
    # (sizes that fit go through: the stand-ins reach the call)
    assert L.moe_combine(half(one, one), ints(one, one), floats(one, one)).shape == (one, one)
    assert launched == ["lbq_moe_combine"]
    for call in (lambda: L.mx_quantize(half(big, 128)), lambda: L.mx_quantize(half(big, 1), transpose=True),
                 lambda: L.mx_quantize(half(1, big), transpose=True),
                 lambda: L.moe_gather(half(big, 1), ints(big, 1)),
                 lambda: L.moe_gather(half(one, big), ints(one, 1)),
                 lambda: L.moe_gather(half(one, 1), ints(one, 1), out=half(big, 1)),
                 lambda: L.moe_gather_backward(half(big, 1), ints(one, 1)),
                 lambda: L.moe_gather_backward(half(one, 1), ints(big, 1)),
                 lambda: L.moe_combine(half(big, 1), ints(one, 1), floats(one, 1)),
                 lambda: L.moe_combine(half(one, 1), ints(big, 1), floats(big, 1)),
                 lambda: L.moe_combine_backward(half(one, 1), half(big, 1), ints(one, 1), floats(one, 1)),
                 lambda: L.MxTensor(torch.empty((big, 64), dtype=torch.uint8, device="meta"),
                                    torch.empty((1, big, 4), dtype=torch.uint8, device="meta"))):
        with pytest.raises(L.LbqError) as e:
            call()
        assert e.value.status == SHAPE and launched == ["lbq_moe_combine"]
    w = L.MxTensor.__new__(L.MxTensor)
    w.rows, w.cols, w.gpu = 256, 128, 0
    for top_k in (2 ** 32 + 2, -2 ** 32 + 2):
        with pytest.raises(L.LbqError) as e:
            L.mx_grouped_forward(w, 2, half(4, 128), ints(3), ints(8), top_k=top_k)
        assert e.value.status == SHAPE


def test_tensors_of_a_view_stay(L):
    """An MxTensor holds the addresses of its tensors, so another tensor cannot be put in their place (the calls
    would go on reading the old one's memory, which nothing keeps any more)."""
    import torch

    codes, scales = torch.zeros((4, 64), dtype=torch.uint8), torch.zeros((1, 4, 4), dtype=torch.uint8)
    t = L.MxTensor.__new__(L.MxTensor)._set(codes, scales, 4, 128, 0)
    assert t.codes is codes and t.scales is scales and t.device == codes.device
    for name in ("codes", "scales"):
        with pytest.raises(AttributeError):
            setattr(t, name, torch.ones_like(getattr(t, name)))
    assert t.codes is codes and t.scales is scales


def test_reference_quantizer():
    """The tests' quantizer on hand-made blocks: ties to even codes, saturation, the scale of zeros."""
    x = np.zeros((1, 128))
    x[0, :8] = [4.0, 0.25, 0.75, -1.25, 1.75, 2.5, 3.5, -0.0]      # e = 0: middles go to even codes
    x[0, 32:34] = [7.9, 5.0]                                       # e = 0: saturates at 6; 5 is a middle, to 4
    x[0, 64] = 8.0                                                 # e = 1: 4 * 2
    codes, scales = R.quantize(x)
    n = np.stack([codes & 15, codes >> 4], -1).reshape(-1)
    assert n[:8].tolist() == [6, 0, 2, 8 + 2, 4, 4, 6, 8]
    assert n[32:34].tolist() == [7, 6] and n[64] == 6
    assert scales.reshape(-1).tolist() == [127, 127, 128, 0]
    v = R.values(codes, scales)
    assert v[0, :8].tolist() == [4.0, 0.0, 1.0, -1.0, 2.0, 2.0, 4.0, 0.0] and v[0, 64] == 8.0
