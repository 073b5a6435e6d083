"""Low-rank adapters on the GPU: forward and gradients against 64-bit products
within derived bounds, against differences, and next to the library's linears."""
import numpy as np
import pytest

import synth
import _adapters_ref as A
from _helpers import cuda, say

pytestmark = pytest.mark.gpu

DTYPES = ["float16", "bfloat16"]
HALF = {"float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}
TINY = {"float16": 2.0 ** -24, "bfloat16": 2.0 ** -126}


@pytest.fixture(scope="module")
def dev():
    return cuda()


@pytest.fixture(scope="module")
def L():
    from bit_weight_only_amd import lbq
    lbq.lib()
    return lbq


class Case:
    """Inputs on the GPU and as float64; ids with tokens of no adapter, and adapters without tokens."""

    def __init__(self, L, M, K, N, n, r, dtype, item=0, runs=False, none=0.2, scale=1.0):
        import torch

        g = synth.rng(90, item + M + 7 * K + 13 * N + r, synth.ROLE_X)
        dt = getattr(torch, dtype)

        def make(shape, s):
            t = torch.from_numpy((s * g.standard_normal(shape)).astype(np.float32)).to(dt)
            return t.cuda(), t.double().numpy()

        self.M, self.K, self.N, self.n, self.r, self.dtype = M, K, N, n, r, dtype
        self.x, self.x64 = make((M, K), scale)
        self.a, self.a64 = make((n, r, K), K ** -0.5)
        self.b, self.b64 = make((n, N, r), 0.1)
        self.base, self.base64 = make((M, N), 1.0)
        self.dy, self.dy64 = make((M, N), 0.1)
        self.dbase, self.dbase64 = make((M, K), 0.1)
        self.s64 = 2.0 ** g.integers(-2, 2, n)
        ids = g.integers(0, n, M)
        if runs:
            ids = np.sort(ids)[::-1].copy()
        u = g.random(M)
        ids[u < none / 2] = -1
        ids[u > 1 - none / 2] = n + g.integers(0, 100)
        self.ids_h = ids.astype(np.int32)
        self.ids = torch.from_numpy(self.ids_h).cuda()
        self.scales = torch.from_numpy(self.s64.astype(np.float32)).cuda()
        self.ad = L.Adapters(self.a, self.b, self.scales)
        _, off, perm, _ = L.moe_sort(self.ids[:, None].contiguous(), n)
        self.order = (off, perm)


def _near(got, want, bound, dtype=None, what=""):
    got = got.double().cpu().numpy()
    tol = bound * 1.01 + (HALF[dtype] * np.abs(want) + TINY[dtype] if dtype else 2.0 ** -140)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, worst {np.abs(got - want).max()}, at {np.argwhere(bad)[:4].tolist()}"


def _check_forward(L, c, base, order, keep):
    import torch

    h = torch.full((c.M, c.r), 7.0, device="cuda") if keep else None
    y = L.adapters_forward(c.ad, c.x, c.ids, base=c.base if base else None, order=c.order if order else None, h=h)
    wy, wh, by, bh = A.forward(c.x64, c.a64, c.b64, c.s64, c.ids_h, c.base64 if base else None, c.dtype)
    _near(y, wy, by, c.dtype, "y")
    off = (c.ids_h < 0) | (c.ids_h >= c.n)
    if off.any():                                              # copies, to the bit
        want = c.base[torch.from_numpy(off).cuda()] if base else torch.zeros(int(off.sum()), c.N, device="cuda", dtype=y.dtype)
        assert torch.equal(y[torch.from_numpy(off).cuda()], want)
    if keep:
        _near(h, wh, bh + np.abs(wh) * A.U, None, "h")
    return y, h


def _check_backward(L, c, h, base, order):
    dx, da, db = L.adapters_backward(c.ad, c.dy, c.x, h, c.ids, base=c.dbase if base else None,
                                     order=c.order if order else None)
    w, bd = A.backward(c.dy64, c.x64, h.double().cpu().numpy(), c.a64, c.b64, c.s64, c.ids_h, c.dbase64 if base else None,
                       c.dtype)
    _near(dx, w[0], bd[0], c.dtype, "dx")
    _near(da, w[1], bd[1] + np.abs(w[1]) * A.U, None, "d_a")
    _near(db, w[2], bd[2] + np.abs(w[2]) * A.U, None, "d_b")
    return dx, da, db


# (M, K, N, L, r)
SHAPES = [(1, 128, 1, 1, 1), (1, 256, 40, 3, 16), (1, 4096, 4096, 8, 16), (2, 1280, 72, 5, 4), (5, 128, 130, 4, 8),
          (16, 512, 512, 16, 32), (33, 384, 97, 3, 5), (40, 128, 8, 100, 17), (64, 512, 256, 64, 16), (70, 256, 515, 2, 64),
          (100, 896, 333, 1, 7), (131, 128, 64, 5, 128), (257, 2048, 2047, 3, 5), (300, 640, 1000, 7, 33),
          (520, 1024, 768, 2, 100), (1000, 256, 300, 1, 16), (1111, 384, 264, 40, 12)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,K,N,n,r", SHAPES)
def test_forward(L, dev, M, K, N, n, r, dtype):
    say(f"adapters_forward M={M} K={K} N={N} L={n} r={r} {dtype}")
    c = Case(L, M, K, N, n, r, dtype, none=0.0 if M == 1 else 0.2)
    y, h = _check_forward(L, c, True, True, True)
    y2, _ = _check_forward(L, c, True, False, False)
    assert np.array_equal(y.view(-1).cpu().view(dtype=__import__("torch").int16).numpy(),
                          y2.view(-1).cpu().view(dtype=__import__("torch").int16).numpy())
    _check_forward(L, c, False, True, True)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,K,N,n,r", SHAPES)
def test_backward(L, dev, M, K, N, n, r, dtype):
    say(f"adapters_backward M={M} K={K} N={N} L={n} r={r} {dtype}")
    c = Case(L, M, K, N, n, r, dtype, item=1, runs=bool(M % 2), none=0.0 if M == 1 else 0.2)
    _, h = _check_forward(L, c, True, True, True)
    a = _check_backward(L, c, h, True, True)
    b = _check_backward(L, c, h, True, False)
    assert all(bool((p == q).all()) for p, q in zip(a, b))
    _check_backward(L, c, h, False, True)


# several chunks of an adapter, every width of rank with many tokens, rows of fewer than eight values, more adapters
# than lanes, as many as there may be
FORMS = [(3000, 256, 2600, 1, 16), (2500, 512, 1100, 2, 64), (1500, 384, 520, 3, 128), (1300, 256, 777, 2, 30),
         (90, 128, 5, 2, 9), (700, 256, 3, 1, 24), (66, 128, 7, 70, 3), (3, 256, 2, 2, 16), (300, 256, 100, 200, 8),
         (1100, 128, 64, 1024, 4), (70, 14336, 64, 3, 16), (2, 14336, 520, 2, 16), (64, 1024, 4096, 3, 70)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,K,N,n,r", FORMS)
def test_forms(L, dev, M, K, N, n, r, dtype):
    say(f"adapters forms M={M} K={K} N={N} L={n} r={r} {dtype}")
    c = Case(L, M, K, N, n, r, dtype, item=9, runs=bool(n % 2))
    _, h = _check_forward(L, c, True, True, True)
    _check_forward(L, c, True, False, False)
    _check_backward(L, c, h, True, True)


def test_one_adapter_has_nearly_all_tokens(L, dev):
    """Chunks of one adapter next to adapters of one token and of none."""
    import torch

    c = Case(L, 1777, 256, 300, 9, 16, "bfloat16", item=10)
    c.ids_h[:] = 4
    c.ids_h[[3, 700, 1776]] = [0, 8, 5]
    c.ids = torch.from_numpy(c.ids_h).cuda()
    _, off, perm, _ = L.moe_sort(c.ids[:, None].contiguous(), 9)
    c.order = (off, perm)
    _, h = _check_forward(L, c, True, True, True)
    _, da, db = _check_backward(L, c, h, True, False)
    for i in (1, 2, 3, 6, 7):
        assert not da[i].any() and not db[i].any()


@pytest.mark.parametrize("M,K,N,n,r", [(1, 128, 24, 2, 4), (50, 256, 100, 3, 16), (700, 256, 200, 4, 20)])
def test_none_has_an_adapter(L, dev, M, K, N, n, r):
    import torch

    c = Case(L, M, K, N, n, r, "bfloat16", none=2.0)
    assert (c.ids_h < 0).any() or (c.ids_h >= n).any()
    c.ids_h[:] = -1
    c.ids.fill_(-1)
    _, off, perm, _ = L.moe_sort(c.ids[:, None].contiguous(), n)
    c.order = (off, perm)
    for order in (True, False):
        y, h = _check_forward(L, c, True, order, True)
        assert torch.equal(y, c.base) and not h.any()
        dx, da, db = _check_backward(L, c, h, True, order)
        assert torch.equal(dx, c.dbase) and not da.any() and not db.any()


def test_no_tokens(L, dev):
    import torch

    c = Case(L, 3, 128, 40, 2, 4, "float16")
    e = torch.empty(0, 128, device="cuda", dtype=torch.float16)
    ids = torch.empty(0, dtype=torch.int32, device="cuda")
    assert L.adapters_forward(c.ad, e, ids).shape == (0, 40)
    dx, da, db = L.adapters_backward(c.ad, e.new_empty(0, 40), e, torch.empty(0, 4, device="cuda"), ids,
                                     d_a=torch.ones(2, 4, 128, device="cuda"), d_b=torch.ones(2, 40, 4, device="cuda"))
    assert dx.shape == (0, 128) and not da.any() and not db.any()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M", [3, 90, 700])
def test_in_place_and_repeatable(L, dev, M, dtype):
    import torch

    c = Case(L, M, 512, 600, 4, 16, dtype, item=2)
    y, h = _check_forward(L, c, True, True, True)
    for _ in range(3):
        buf = c.base.clone()
        h2 = torch.empty_like(h)
        assert L.adapters_forward(c.ad, c.x, c.ids, base=buf, y=buf, h=h2).data_ptr() == buf.data_ptr()
        assert torch.equal(buf, y) and torch.equal(h, h2)
    g = _check_backward(L, c, h, True, True)
    for _ in range(3):
        buf = c.dbase.clone()
        got = L.adapters_backward(c.ad, c.dy, c.x, h, c.ids, base=buf, dx=buf)
        assert got[0].data_ptr() == buf.data_ptr() and all(torch.equal(a, b) for a, b in zip(got, g))


@pytest.mark.parametrize("M", [6, 70, 300])
def test_values_of_other_tokens_stay_there(L, dev, M):
    """NaN and infinities: in tokens without an adapter they touch nothing else, in a token with one only its own row
    and its adapter's gradients; in an adapter that no token uses, nothing."""
    import torch

    c = Case(L, M, 256, 136, 4, 12, "float16", item=3)
    c.ids_h = (np.arange(M) % 3).astype(np.int32)             # adapter 3 is of no token
    c.ids_h[[0, M - 1]] = -1
    c.ids = torch.from_numpy(c.ids_h).cuda()
    _, off, perm, _ = L.moe_sort(c.ids[:, None].contiguous(), 4)
    c.order = (off, perm)
    _, h0 = _check_forward(L, c, True, True, True)
    want = _check_backward(L, c, h0, True, True)
    for t in (0, M - 1):
        c.x[t], c.dy[t] = float("nan"), float("inf")
    c.a[3], c.b[3] = float("nan"), float("inf")
    y, h = c.base.clone(), torch.empty_like(h0)
    for order in (c.order, None):
        y = L.adapters_forward(c.ad, c.x, c.ids, base=c.base, h=h, order=order)
        assert torch.equal(y[0], c.base[0]) and bool(torch.isfinite(y).all()) and torch.equal(h, h0)
        got = L.adapters_backward(c.ad, c.dy, c.x, h, c.ids, base=c.dbase, order=order)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    # a token of adapter 1
    c.x[4, 5] = float("inf")
    y2 = L.adapters_forward(c.ad, c.x, c.ids, base=c.base, h=h, order=c.order)
    rest = torch.arange(M, device="cuda") != 4
    assert torch.equal(y2[rest], y[rest]) and not bool(torch.isfinite(y2[4]).any())
    c.dy[4, 7] = float("nan")
    dx, da, db = L.adapters_backward(c.ad, c.dy, c.x, h, c.ids, base=c.dbase, order=c.order)
    assert torch.equal(dx[rest], want[0][rest]) and bool(torch.isnan(dx[4]).all())
    for i in (0, 2, 3):
        assert torch.equal(da[i], want[1][i]) and torch.equal(db[i], want[2][i])
    assert bool(torch.isnan(da[1]).any()) and bool(torch.isnan(db[1]).any())


@pytest.mark.parametrize("M", [3, 40, 90])
@pytest.mark.parametrize("r", [9, 64])
def test_values_of_very_different_sizes(L, dev, M, r):
    """fp16: rows of A from 2^-12 to 2^15, columns of B the other way round, so that every value of h counts as much.

    A token's h is brought to at least 2^14 by one power of two for the product with B, and what two pieces leave out
    is below half the smallest fp16 number, 2^-25: 2^-39 of the token's largest h, in each of its r values; the same of u
    for dx. In the sums over tokens a value has its own power of two: 2^-39 of its largest over 32 tokens."""
    import torch

    c = Case(L, M, 1024, 96, 2, r, "float16", item=5)
    size = 2.0 ** np.round(np.linspace(-12, 15, r))
    c.a.copy_((c.a.double().cpu() * torch.from_numpy(size)[None, :, None]).to(c.a.dtype))
    c.b.copy_((c.b.double().cpu() / torch.from_numpy(size)[None, None, :]).to(c.b.dtype))
    c.a64, c.b64 = c.a.double().cpu().numpy(), c.b.double().cpu().numpy()
    h = torch.empty(M, r, device="cuda")
    y = L.adapters_forward(c.ad, c.x, c.ids, base=c.base, order=c.order, h=h)
    wy, wh, by, bh = A.forward(c.x64, c.a64, c.b64, c.s64, c.ids_h, c.base64, c.dtype)
    _near(h, wh, bh + np.abs(wh) * A.U, None, "h")
    h64 = h.double().cpu().numpy()
    on = [t for t in range(M) if 0 <= c.ids_h[t] < c.n]
    for t in on:
        i = c.ids_h[t]
        by[t] += 2.0 ** -39 * np.abs(h64[t]).max() * c.s64[i] * np.abs(c.b64[i]).sum(1)
    _near(y, wy, by, c.dtype, "y")
    dx, da, db = L.adapters_backward(c.ad, c.dy, c.x, h, c.ids, base=c.dbase, order=c.order)
    w, bd = A.backward(c.dy64, c.x64, h64, c.a64, c.b64, c.s64, c.ids_h, c.dbase64, c.dtype)
    for t in on:
        i = c.ids_h[t]
        u = np.abs(c.s64[i] * (c.dy64[t] @ c.b64[i]))
        bd[0][t] += 2.0 ** -38 * u.max() * np.abs(c.a64[i]).sum(0)
    for i in range(c.n):
        t = np.nonzero(c.ids_h == i)[0]
        if len(t) == 0:
            continue
        u = np.abs(c.s64[i] * (c.dy64[t] @ c.b64[i])).max(0)
        bd[1][i] += 2.0 ** -38 * u[:, None] * np.abs(c.x64[t]).sum(0)
        bd[2][i] += 2.0 ** -39 * c.s64[i] * np.abs(h64[t]).max(0) * np.abs(c.dy64[t]).sum(0)[:, None]
    _near(dx, w[0], bd[0], c.dtype, "dx")
    _near(da, w[1], bd[1] + np.abs(w[1]) * A.U, None, "d_a")
    _near(db, w[2], bd[2] + np.abs(w[2]) * A.U, None, "d_b")


@pytest.mark.parametrize("M", [2, 40, 300])
@pytest.mark.parametrize("size", [2.0 ** -9, 2.0 ** 9])
def test_small_and_large_values(L, dev, M, size):
    """fp16: h past its range and u below it are held all the same (y and dx are in range)."""
    import torch

    c = Case(L, M, 1024, 96, 2, 9, "float16", item=4)
    c.x.mul_(size)
    c.a.mul_(8 if size > 1 else 0.125)
    c.b.mul_(2.0 ** -12 if size > 1 else 1.0)
    c.dy.mul_(2.0 ** -8)
    for n in ("x", "a", "b", "dy"):
        setattr(c, n + "64", getattr(c, n).double().cpu().numpy())
    y, h = _check_forward(L, c, True, True, True)
    assert size < 1 or float(h.abs().max()) > 8192
    _check_backward(L, c, h, False, True)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M", [7, 200])
def test_gradients_against_differences(L, dev, M, dtype):
    """y is linear in x, A and B each: <dy, y(v + d) - y(v)> = <gradient, d> up to what y's roundings do."""
    import torch

    c = Case(L, M, 128, 64, 3, 8, dtype, item=5)
    h = torch.empty(M, 8, device="cuda")
    y0 = L.adapters_forward(c.ad, c.x, c.ids, h=h)
    grads = L.adapters_backward(c.ad, c.dy, c.x, h, c.ids)
    room = float((c.dy.double().abs() * (y0.double().abs() + 1)).sum()) * 4 * HALF[dtype]
    for name, g in zip(("x", "a", "b"), grads):
        v = getattr(c, name)
        d = torch.randint(-1, 2, v.shape, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).to(v.dtype)
        d = d * v.abs().amax()                                 # a step as large as the values
        moved = (v + d)
        args = {"x": c.x, "a": c.a, "b": c.b}
        args[name] = moved
        y1 = L.adapters_forward(L.Adapters(args["a"], args["b"], c.scales), args["x"], c.ids)
        lhs = float((c.dy.double() * (y1.double() - y0.double())).sum())
        rhs = float((g.double() * (moved.double() - v.double())).sum())
        more = float((c.dy.double().abs() * y1.double().abs()).sum()) * 2 * HALF[dtype]
        extra = float((g.double().abs() * (moved.double() - v.double()).abs()).sum()) * HALF[dtype]
        assert abs(lhs - rhs) <= room + more + extra, (name, lhs, rhs, room + more + extra)


@pytest.mark.parametrize("order", [True, False])
@pytest.mark.parametrize("M", [4, 333])
def test_streams_and_graphs(L, dev, M, order):
    import torch

    c = Case(L, M, 512, 520, 3, 16, "bfloat16", item=6)
    o = c.order if order else None
    h = torch.empty(M, 16, device="cuda")
    y = L.adapters_forward(c.ad, c.x, c.ids, base=c.base, h=h, order=o)
    g = L.adapters_backward(c.ad, c.dy, c.x, h, c.ids, base=c.dbase, order=o)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    h2 = torch.empty_like(h)
    y2 = L.adapters_forward(c.ad, c.x, c.ids, base=c.base, h=h2, order=o, stream=s)
    g2 = L.adapters_backward(c.ad, c.dy, c.x, h2, c.ids, base=c.dbase, order=o, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, y2) and torch.equal(h, h2) and all(torch.equal(a, b) for a, b in zip(g, g2))
    # two graphs with workspaces of the caller's, shared by both
    ws = torch.empty(max(1, c.ad.workspace_bytes(M, order), c.ad.workspace_bytes(M, order, True)), dtype=torch.uint8,
                     device="cuda")
    x, hg, yg = c.x.clone(), torch.empty_like(h), torch.empty_like(y)
    outs = [torch.empty_like(t) for t in g]
    g1, g2_ = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        L.adapters_forward(c.ad, x, c.ids, base=c.base, y=yg, h=hg, order=o, ws=ws)
    with torch.cuda.graph(g2_):
        L.adapters_backward(c.ad, c.dy, x, hg, c.ids, base=c.dbase, dx=outs[0], d_a=outs[1], d_b=outs[2], order=o, ws=ws)
    for i in range(4):
        x.copy_(c.x * (i + 1))
        g1.replay()
        g2_.replay()
        ws.fill_(255)                                          # nothing is kept in it between calls
        torch.cuda.synchronize()
        hh = torch.empty_like(h)
        assert torch.equal(yg, L.adapters_forward(c.ad, x, c.ids, base=c.base, h=hh, order=o)) and torch.equal(hh, hg)
        for a, b in zip(outs, L.adapters_backward(c.ad, c.dy, x, hh, c.ids, base=c.dbase, order=o)):
            assert torch.equal(a, b)


def test_order_out_of_range(L, dev):
    """An order that is not ids' own gives wrong rows, and nothing outside the buffers."""
    import torch

    for M in (5, 400):
        c = Case(L, M, 256, 200, 3, 8, "float16", item=7)
        h = torch.zeros(M, 8, device="cuda")
        for off, perm in ((torch.tensor([-5, 2 ** 30, 3, 2 ** 31 - 1], dtype=torch.int32, device="cuda"), c.order[1]),
                          (c.order[0], torch.full((M,), 2 ** 31 - 1, dtype=torch.int32, device="cuda")),
                          (c.order[0], torch.full((M,), -7, dtype=torch.int32, device="cuda")),
                          (torch.tensor([0, M, 0, M], dtype=torch.int32, device="cuda"), c.order[1])):
            L.adapters_forward(c.ad, c.x, c.ids, base=c.base, h=h, order=(off, perm))
            L.adapters_backward(c.ad, c.dy, c.x, h, c.ids, base=c.dbase, order=(off, perm))
        torch.cuda.synchronize()


def test_offsets_past_32_bits(L, dev):
    """2^20 tokens with rows of 4104 values: the last rows lie past 2^32 values."""
    import torch

    M, K, N, r, n = 2 ** 20, 128, 4104, 4, 2
    g = torch.Generator("cuda").manual_seed(3)
    x = torch.randn(M, K, device="cuda", generator=g).half()
    a = (torch.randn(n, r, K, device="cuda", generator=g) / 11).half()
    b = torch.randn(n, N, r, device="cuda", generator=g).half()
    sc = torch.ones(n, device="cuda")
    ids = torch.full((M,), -1, dtype=torch.int32, device="cuda")
    ids[:3], ids[-70:] = 0, 1
    ad = L.Adapters(a, b, sc)
    h = torch.empty(M, r, device="cuda")
    y = L.adapters_forward(ad, x, ids, h=h)
    for t, i in ((slice(0, 3), 0), (slice(M - 70, M), 1)):
        want = (x[t].double() @ a[i].double().t()) @ b[i].double().t()
        bound = ((x[t].double().abs() @ a[i].double().abs().t()) @ b[i].double().abs().t()) * (K + 2 * r + 64) * A.U
        assert bool(((y[t].double() - want).abs() <= bound + want.abs() * 2.0 ** -11 + 2.0 ** -24).all())
    assert not bool(y[3:-70].any())
    dx, da, db = L.adapters_backward(ad, y, x, h, ids)
    t = slice(M - 70, M)
    want = y[t].double().t() @ h[t].double()
    bound = (y[t].double().abs().t() @ h[t].double().abs()) * 512 * A.U
    assert bool(((db[1].double() - want).abs() <= bound).all())
    u = y[t].double() @ b[1].double()
    assert bool(((dx[t].double() - u @ a[1].double()).abs()
                 <= (u.abs() @ a[1].double().abs()) * 2.0 ** -10 + (y[t].double().abs() @ b[1].double().abs())
                 @ a[1].double().abs() * (N + 64) * A.U).all())
    assert not bool(dx[3:-70].any())


def test_beside_the_linears(L, dev):
    """A step as it is used: a packed and an MXFP4 projection, adapters of each request beside them in place, one order
    for both layers."""
    import torch
    from _helpers import make_rtn

    M, K, N, n, r = 37, 512, 384, 3, 8
    c = Case(L, M, K, N, n, r, "float16", item=8)
    w, s, planes, meta, pl = make_rtn(N, K, 4, 91, 0)
    y = L.linear_forward(pl, c.x)
    want, _, by, _ = A.forward(c.x64, c.a64, c.b64, c.s64, c.ids_h, y.double().cpu().numpy(), c.dtype)
    L.adapters_forward(c.ad, c.x, c.ids, base=y, y=y, order=c.order)
    _near(y, want, by, "float16", "packed")
    wq = L.mx_quantize(torch.from_numpy(w).cuda())
    y = L.mx_linear_forward(wq, c.x)
    want, _, by, _ = A.forward(c.x64, c.a64, c.b64, c.s64, c.ids_h, y.double().cpu().numpy(), c.dtype)
    h = torch.empty(M, r, device="cuda")
    L.adapters_forward(c.ad, c.x, c.ids, base=y, y=y, h=h, order=c.order)
    _near(y, want, by, "float16", "mx")
    # the projection's own dx, then the adapters' part in place
    dx = L.mx_matmul(L.mx_quantize(c.dy), L.mx_quantize(torch.from_numpy(w).cuda(), transpose=True), torch.float16)
    c.dbase, c.dbase64 = dx, dx.double().cpu().numpy()
    want = _check_backward(L, c, h, True, True)
    got = L.adapters_backward(c.ad, c.dy, c.x, h, c.ids, base=dx, dx=dx, order=c.order)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_routed_block_with_its_router(L, dev):
    """Selection, sort, the experts' products, combine; and back from dy to the logits."""
    import torch

    M, E, k, K, N = 50, 16, 3, 256, 128
    g = synth.rng(92, 0, synth.ROLE_X)
    x = torch.from_numpy(g.standard_normal((M, K)).astype(np.float32)).half().cuda()
    w = L.mx_quantize(torch.from_numpy((0.1 * g.standard_normal((E * N, K))).astype(np.float32)).cuda())
    lg = torch.from_numpy(g.standard_normal((M, E)).astype(np.float32))
    lg[3, 2:] = float("-inf")                                   # two experts left for three picks
    bias = (0.1 * g.standard_normal(E)).astype(np.float32)
    how = dict(score=1, groups=4, top_groups=2, group_picks=2, scale=2.0)
    ids, wts = L.moe_select(lg.cuda(), k, bias=torch.from_numpy(bias).cuda(), **how)
    _, off, perm, pos = L.moe_sort(ids, E)
    o = L.mx_grouped_forward(w, E, x, off, perm, k)
    y = L.moe_combine(o, pos, wts)
    want_ids, ww = A.select(lg.double().numpy(), k, bias.astype(np.float64), **how)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    o64, p = o.double().cpu().numpy(), pos.cpu().numpy()
    rows = np.where((p >= 0)[..., None], o64[p.clip(0)], 0.0)
    want = (ww[..., None] * rows).sum(1)
    room = (np.abs(ww)[..., None] * np.abs(rows)).sum(1)
    _near(y, want, room * 64 * A.U, "float16", "y")
    dy = torch.from_numpy(g.standard_normal((M, N)).astype(np.float32)).half().cuda()
    _, dw = L.moe_combine_backward(dy, o, pos, wts)
    d = L.moe_select_backward(dw, lg.cuda(), ids, score=1, scale=2.0)
    dw64 = (rows * dy.double().cpu().numpy()[:, None]).sum(-1)
    want, bound = A.select_backward(dw64, lg.double().numpy(), want_ids, 1, True, 2.0)
    # d_weights' own error: N roundings of each dot product's absolute sum, through the same derivative
    adw = (np.abs(rows) * np.abs(dy.double().cpu().numpy())[:, None]).sum(-1) * (N + 8) * A.U
    _, p64 = A.scores(lg.double().numpy(), 1)
    S = np.where(want_ids >= 0, np.take_along_axis(p64, want_ids.clip(0), 1), 0).sum(1)
    bound = bound + 4 * (adw.max(1) / np.where(S > 0, S, 1))[:, None]
    assert np.all(np.abs(d.double().cpu().numpy() - want) <= bound + np.abs(want) * A.U)


def test_other_device_index_is_refused(L, dev):
    import torch

    c = Case(L, 4, 256, 100, 2, 8, "float16")
    f, b, h = L.adapters_forward, L.adapters_backward, torch.zeros(4, 8, device="cuda")
    bad = [lambda: f(c.ad, c.x.cpu(), c.ids), lambda: f(c.ad, c.x.bfloat16(), c.ids), lambda: f(c.ad, c.x, c.ids.long()),
           lambda: f(c.ad, c.x, c.ids[:3]), lambda: f(c.ad, c.x[:, :128], c.ids), lambda: f(c.ad, c.x[:, :128].contiguous(), c.ids),
           lambda: f(c.ad, c.x, c.ids, base=c.base[:, :99]), lambda: f(c.ad, c.x, c.ids, h=h.half()),
           lambda: f(c.ad, c.x, c.ids, order=(c.order[0][:2], c.order[1])),
           lambda: f(c.ad, c.x, c.ids, order=(c.order[0], c.order[1].long())),
           lambda: f(c.ad, c.x, c.ids, ws=torch.empty(64, dtype=torch.uint8)),
           lambda: b(c.ad, c.dy, c.x, h[:, :4], c.ids), lambda: b(c.ad, c.dy[:, :8], c.x, h, c.ids),
           lambda: b(c.ad, c.dy, c.x, h, c.ids, dx=c.x.bfloat16()), lambda: b(c.ad, c.dy, c.x, h, c.ids, d_a=torch.zeros(2, 8, 255, device="cuda")),
           lambda: L.Adapters(c.a, c.b[:, :, :4], c.scales), lambda: L.Adapters(c.a, c.b.bfloat16(), c.scales),
           lambda: L.Adapters(c.a.float(), c.b.float(), c.scales) and f(L.Adapters(c.a.float(), c.b.float(), c.scales), c.x.float(), c.ids),
           lambda: L.Adapters(c.a, c.b, c.scales.half())]
    for i, g in enumerate(bad):
        with pytest.raises(L.LbqError):
            g()
            raise AssertionError(i)


def test_no_tokens_with_an_order(L, dev):
    """An empty batch whose program keeps an order: the gradients are zeros, in the workspace that the query names."""
    import torch

    c = Case(L, 3, 128, 40, 2, 4, "float16")
    e = torch.empty(0, 128, device="cuda", dtype=torch.float16)
    ids = torch.empty(0, dtype=torch.int32, device="cuda")
    _, off, perm, _ = L.moe_sort(ids[:, None].contiguous(), 2)
    assert off.tolist() == [0, 0, 0] and perm.numel() == 0
    need = c.ad.workspace_bytes(0, True, True)
    for ws in (None, torch.empty(need, dtype=torch.uint8, device="cuda")):
        for order in ((off, perm), None, (torch.tensor([0, 5, 9], dtype=torch.int32, device="cuda"), perm)):
            if order is None and ws is not None:
                ws = torch.empty(c.ad.workspace_bytes(0, False, True), dtype=torch.uint8, device="cuda")
            h = torch.empty(0, 4, device="cuda")
            assert L.adapters_forward(c.ad, e, ids, h=h, order=order).shape == (0, 40)
            dx, da, db = L.adapters_backward(c.ad, e.new_empty(0, 40), e, h, ids, order=order, ws=ws,
                                             d_a=torch.ones(2, 4, 128, device="cuda"),
                                             d_b=torch.ones(2, 40, 4, device="cuda"))
            assert dx.shape == (0, 128) and not da.any() and not db.any()


def _whole(rows, n, g, r):
    """[rows][r][n] whole numbers 59 .. 121, of which row j + r // 2 is row j but for steps of one at eight places."""
    v = g.integers(60, 121, (rows, r, n))
    half = r // 2
    for i in range(rows):
        for j in range(half):
            at = g.choice(n, 8, replace=False)
            v[i, half + j] = v[i, j]
            v[i, half + j, at] += g.integers(0, 2, 8) * 2 - 1
    v[:, 2 * half:] = 0
    return v


# every form of the forward, every width of rank
WHOLE = [(7, 16384, 40, 3, 16), (9, 8192, 72, 2, 20), (10, 8192, 50, 3, 40), (1, 1024, 40, 2, 2), (2, 1024, 600, 2, 16), (3, 1024, 24, 2, 34), (5, 8192, 100, 3, 9), (40, 1024, 264, 9, 64),
         (30, 1024, 130, 4, 128), (64, 2048, 72, 3, 24), (90, 1024, 5, 2, 6), (300, 1024, 515, 3, 16), (200, 1024, 264, 5, 30),
         (700, 1024, 300, 2, 64), (150, 1024, 97, 3, 128), (1100, 1024, 136, 70, 12)]


@pytest.mark.parametrize("order", [True, False])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,K,N,n,r", WHOLE)
def test_h_and_u_keep_their_bits(L, dev, M, K, N, n, r, dtype, order):
    """Whole numbers of 20 and more bits as h and u, whose differences of a few bits are what y and dx are: all sums are
    below 2^24, exact in 32 bits in any order, and so have to be the results."""
    import torch

    say(f"adapters whole numbers M={M} K={K} N={N} L={n} r={r} {dtype} order={order}")
    g = synth.rng(95, M + K + N + r, synth.ROLE_X)
    dt = getattr(torch, dtype)

    def up(v):
        t = torch.from_numpy(np.ascontiguousarray(v).astype(np.float32)).to(dt)
        assert np.array_equal(t.double().numpy(), v)
        return t.cuda()

    half = r // 2
    ids = g.integers(-1, n, M).astype(np.int32)
    if M == 1:
        ids[:] = 0
    idc = torch.from_numpy(ids).cuda()
    _, off, perm, _ = L.moe_sort(idc[:, None].contiguous(), n)
    o = (off, perm) if order else None
    sc = torch.ones(n, device="cuda")
    on = (ids >= 0)[:, None]
    few = min(K, 1024)                             # so many values at most, and zeros
    for back in (False, True):
        if back and N < 8:
            continue
        long, short = (min(N, 1024), K) if back else (few, N)
        rows = np.zeros((n, r, N if back else K))
        place = np.sort(g.choice(rows.shape[2], long, replace=False))
        rows[:, :, place] = _whole(n, long, g, r)
        x = g.integers(8, 16, (M, rows.shape[2]))
        pick = np.zeros((n, short, r))
        pair = g.integers(0, half, short)
        pick[:, np.arange(short), pair], pick[:, np.arange(short), half + pair] = 1, -1
        base = g.integers(-8, 9, (M, short))
        at = ids.clip(0)
        mid = np.einsum("tk,tjk->tj", x.astype(np.float64), rows[at]) * on
        want = base + np.einsum("tj,tnj->tn", mid, pick[at]) * on
        assert np.abs(mid).max() < 2 ** 24 and np.abs(want).max() <= 256
        if not back:
            h = torch.empty(M, r, device="cuda")
            y = L.adapters_forward(L.Adapters(up(rows), up(pick), sc), up(x), idc, base=up(base), h=h, order=o)
            assert np.array_equal(h.double().cpu().numpy(), mid)
            got = y
        else:
            # B's rows are rows' columns; A's are pick's
            ad = L.Adapters(up(pick.transpose(0, 2, 1)), up(rows.transpose(0, 2, 1)), sc)
            got = L.adapters_backward(ad, up(x), torch.zeros(M, K, device="cuda", dtype=dt), torch.zeros(M, r, device="cuda"),
                                      idc, base=up(base), order=o)[0]
        bad = got.double().cpu().numpy() != want
        assert not bad.any(), f"{'dx' if back else 'y'}: {bad.sum()} of {bad.size}"
