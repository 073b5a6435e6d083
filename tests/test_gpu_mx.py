"""MXFP4 tensors and their products on the GPU against 64-bit NumPy forms:
quantisation bit-exact, products within the error of 32-bit accumulation."""
import numpy as np
import pytest

import synth
import _mx_ref as R
from _helpers import cuda, say

pytestmark = pytest.mark.gpu

DTYPES = ["float16", "bfloat16", "float32"]


@pytest.fixture(scope="module")
def dev():
    return cuda()


@pytest.fixture(scope="module")
def L():
    from bit_weight_only_amd import lbq
    lbq.lib()
    return lbq


def _x(m, k, dtype, item=0, workload=60):
    """Activations with a few large channels, in dtype, and what they are in 64 bits."""
    import torch

    g = synth.rng(workload, item, synth.ROLE_X)
    x = g.standard_normal((m, k)) * np.where(g.random(k) < 0.03, 30.0, 1.0)
    t = torch.from_numpy(x).to(getattr(torch, dtype))
    return t.cuda(), t.double().numpy()


def _tensor(L, r, c, item=0):
    """A random MXFP4 tensor and its values."""
    import torch

    g = synth.rng(61, item, synth.ROLE_W)
    codes = g.integers(0, 256, (r, c // 2), dtype=np.uint8)
    scales = g.integers(118, 126, (c // 128, r, 4), dtype=np.uint8)
    return L.MxTensor(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()), R.values(codes, scales)


def _half_step(dtype):
    """The relative error of one rounding to dtype."""
    return {"float16": 2.0 ** -11, "bfloat16": 2.0 ** -8, "float32": 2.0 ** -24}[dtype]


def _check_product(got, a, b, dtype):
    """got = a b^T: products of e2m1 values and powers of two are exact, so what is left is the order of the
    sums in 32 bits. A product passes at most 64 additions inside an instruction, K / 64 accumulations and 64
    partial sums, each off by at most 2^-23 of the sum of magnitudes (truncation allowed); then one rounding
    to dtype (float16 also 2^-25 below its normal range)."""
    want, mag = a @ b.T, np.abs(a) @ np.abs(b).T
    tol = (a.shape[1] / 64 + 128) * 2.0 ** -23 * mag
    tol += _half_step(dtype) * (np.abs(want) + tol) + (2.0 ** -25 if dtype == "float16" else 0)
    got = got.double().cpu().numpy()
    assert got.shape == want.shape
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], want[bad][:4])


# ------------------------------------------------------------------ quantisation

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,k", [(1, 128), (3, 256), (17, 1152), (130, 384), (5, 17408)])
def test_quantize_bit_exact(L, dev, m, k, dtype):
    say(f"mx quantize {m}x{k} {dtype}")
    x, x64 = _x(m, k, dtype, item=m)
    t = L.mx_quantize(x)
    codes, scales = R.quantize(x64)
    assert np.array_equal(t.scales.cpu().numpy(), scales)
    assert np.array_equal(t.codes.cpu().numpy(), codes)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,k", [(1, 1), (33, 7), (128, 64), (300, 130), (257, 200), (129, 1000)])
def test_quantize_transposed_bit_exact(L, dev, m, k, dtype):
    say(f"mx quantize_t {m}x{k} {dtype}")
    x, x64 = _x(m, k, dtype, item=100 + m)
    t = L.mx_quantize(x, transpose=True)
    codes, scales = R.quantize(R.transposed(x64))
    assert (t.rows, t.cols) == (k, -(-m // 128) * 128)
    assert np.array_equal(t.scales.cpu().numpy(), scales)
    assert np.array_equal(t.codes.cpu().numpy(), codes)


def _special(dtype):
    """Blocks of values where a rule can go wrong, [n][128] in dtype."""
    import torch

    ft = getattr(torch, dtype)
    top, tiny = torch.finfo(ft).max, float(torch.finfo(ft).smallest_normal)
    lowest = {"float16": 2.0 ** -24, "bfloat16": 2.0 ** -133, "float32": 2.0 ** -149}[dtype]
    g = synth.rng(62, DTYPES.index(dtype), synth.ROLE_X)
    rows = []
    # middles between neighbours, and just beside them, under a block maximum of 4..7.5
    mids = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    for top_of_block in (4.0, 6.0, 7.5):
        for scale in (1.0, 2.0 ** -9, 2.0 ** 10):
            v = np.array([s * m * f for m in mids for s in (1, -1) for f in (1, 1 + 2.0 ** -7)] + [top_of_block])
            rows.append(np.resize(v, 128) * scale)
    rows.append(np.zeros(128))
    rows.append(np.full(128, -0.0))
    rows.append(np.where(np.arange(128) % 32 == 0, top, tiny))
    rows.append(np.full(128, -top))
    rows.append(np.where(np.arange(128) % 2 == 0, lowest, -3 * lowest))
    rows.append(g.integers(0, 9, 128) * lowest)
    rows.append(np.where(np.arange(128) % 32 == 5, tiny, lowest))
    rows.append(g.standard_normal(128) * tiny * 8)
    for bad in (np.inf, -np.inf, np.nan):
        v = g.standard_normal(128)
        v[[3, 70]] = bad                 # blocks 0 and 2; 1 and 3 stay as they are
        rows.append(v)
    return torch.from_numpy(np.stack(rows)).to(ft)


@pytest.mark.parametrize("dtype", DTYPES)
def test_quantize_special_values(L, dev, dtype):
    say(f"mx quantize special {dtype}")
    x = _special(dtype)
    codes, scales = R.quantize(x.double().numpy())
    t = L.mx_quantize(x.cuda())
    assert np.array_equal(t.scales.cpu().numpy(), scales)
    assert np.array_equal(t.codes.cpu().numpy(), codes)
    assert (scales == 255).sum() == 6
    # the same blocks along the columns
    t = L.mx_quantize(x.t().contiguous().cuda(), transpose=True)
    assert np.array_equal(t.scales.cpu().numpy(), scales)
    assert np.array_equal(t.codes.cpu().numpy(), codes)


@pytest.mark.parametrize("dtype", DTYPES)
def test_dequantize_every_code_and_scale(L, dev, dtype):
    import torch

    say(f"mx dequantize {dtype}")
    codes = np.tile(np.arange(256, dtype=np.uint8), (256, 1))[:, :64]
    codes = np.concatenate([codes, codes + 64, codes + 128, codes + 192], 1)     # [256][256]: 512 columns
    scales = np.broadcast_to(np.arange(256, dtype=np.uint8)[None, :, None], (4, 256, 4)).copy()
    t = L.MxTensor(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda())
    got = L.mx_dequantize(t, getattr(torch, dtype)).cpu()
    with np.errstate(over="ignore"):
        want = torch.from_numpy(R.values(codes, scales)).float().to(getattr(torch, dtype))
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got[~torch.isnan(want)], want[~torch.isnan(want)])


# ------------------------------------------------------------------ products

SHAPES = [(1, 1, 128), (1, 33, 256), (2, 100, 384), (7, 64, 4096), (16, 130, 1152), (17, 257, 512), (33, 300, 640),
          (64, 96, 2048), (100, 31, 1024), (129, 129, 128), (200, 513, 768), (300, 520, 1280)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_matmul(L, dev, m, n, k, dtype):
    import torch

    say(f"mx matmul {m}x{n}x{k} {dtype}")
    a, av = _tensor(L, m, k, item=m)
    b, bv = _tensor(L, n, k, item=1000 + n)
    y = torch.full((m, n), 7.0, dtype=getattr(torch, dtype), device="cuda")
    _check_product(L.mx_matmul(a, b, y=y), av, bv, dtype)


@pytest.mark.parametrize("m,n,k", [(700, 1100, 2176), (1030, 260, 4096), (5, 9000, 1024), (40, 70, 17408),
                                   (600, 600, 8192), (100, 200, 4096), (130, 500, 14336), (77, 131, 17408),
                                   (64, 640, 4096), (65, 8, 2176), (900, 5000, 128), (2000, 2100, 384),
                                   (1100, 2300, 640), (2100, 1030, 256), (2400, 3600, 384), (4000, 3900, 384)])
def test_matmul_larger(L, dev, m, n, k):
    import torch

    say(f"mx matmul {m}x{n}x{k}")
    a, av = _tensor(L, m, k, item=m)
    b, bv = _tensor(L, n, k, item=1000 + n)
    _check_product(L.mx_matmul(a, b, torch.float32), av, bv, "float32")


@pytest.mark.parametrize("m,n,k", [(3, 70, 512), (200, 300, 1024)])
def test_matmul_nan_blocks_and_wide_scales(L, dev, m, n, k):
    """A NaN block makes its row (A) or column (B) NaN and nothing else; scales far apart stay exact."""
    import torch

    say(f"mx matmul scales {m}x{n}x{k}")
    g = synth.rng(63, m, synth.ROLE_W)
    ca, cb = (g.integers(0, 256, (r, k // 2), dtype=np.uint8) for r in (m, n))
    sa, sb = (g.integers(97, 158, (k // 128, r, 4), dtype=np.uint8) for r in (m, n))
    sa[k // 128 - 1, 1, 3] = 255
    sb[0, n - 1, 0] = 255
    a, b = (L.MxTensor(torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda()) for c, s in ((ca, sa), (cb, sb)))
    y = L.mx_matmul(a, b, torch.float32)
    nan = torch.isnan(y).cpu().numpy()
    want = np.zeros((m, n), bool)
    want[1], want[:, n - 1] = True, True
    assert np.array_equal(nan, want)
    rows, cols = [i for i in range(m) if i != 1], list(range(n - 1))
    _check_product(y[rows][:, cols], R.values(ca, sa)[rows], R.values(cb, sb)[cols], "float32")


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("m,n,k", [(1, 40, 128), (1, 4096, 4096), (3, 100, 1152), (4, 1000, 512), (5, 333, 2048),
                                   (16, 512, 1024), (31, 200, 640), (65, 130, 384), (150, 700, 1536), (2, 9000, 256),
                                   (16, 77, 17408), (9, 1100, 14336), (32, 2500, 8192), (20, 30, 4224),
                                   (1, 17000, 2048)])
def test_linear(L, dev, m, n, k, dtype):
    say(f"mx linear {m}x{n}x{k} {dtype}")
    x, x64 = _x(m, k, dtype, item=200 + m)
    w, wv = _tensor(L, n, k, item=2000 + n)
    _check_product(L.mx_linear_forward(w, x), R.values(*R.quantize(x64)), wv, dtype)


def _routing(m, E, k, item):
    g = synth.rng(64, item, synth.ROLE_LOGITS)
    ids = np.stack([g.permutation(E)[:k] for _ in range(m)]).astype(np.int32)
    return ids


# experts without rows, with one row, with several row tiles; odd sizes
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("m,E,top_k,n,k", [(1, 4, 1, 40, 128), (3, 256, 8, 64, 256), (32, 16, 4, 130, 512),
                                           (150, 3, 2, 100, 384), (400, 2, 1, 300, 640), (9, 1, 1, 33, 1024),
                                           (70, 1024, 6, 16, 128), (900, 5, 3, 140, 256), (700, 6, 3, 500, 384),
                                           (3000, 4, 2, 1100, 128), (2100, 4, 2, 3500, 384)])
def test_grouped(L, dev, m, E, top_k, n, k, dtype):
    import torch

    say(f"mx grouped m={m} E={E} k={top_k} {n}x{k} {dtype}")
    x, x64 = _x(m, k, dtype, item=300 + m)
    w, wv = _tensor(L, E * n, k, item=3000 + E)
    ids = _routing(m, E, top_k, m)
    counts, offsets, perm, pos = R.sort(ids, E)
    y = L.mx_grouped_forward(w, E, x, torch.from_numpy(offsets).cuda(), torch.from_numpy(perm).cuda(), top_k)
    q = R.values(*R.quantize(x64))
    for e in range(E):
        if counts[e]:
            rows = slice(offsets[e], offsets[e + 1])
            _check_product(y[rows], q[perm[rows] // top_k], wv[e * n:(e + 1) * n], dtype)


def test_grouped_rows_behind_the_last_and_no_perm(L, dev):
    """Dropped picks: rows from offsets[E] on stay as they were. Without perm x is already in list order."""
    import torch

    E, n, k, top_k, m = 6, 96, 256, 2, 90
    x, x64 = _x(m, k, "bfloat16", item=7)
    w, wv = _tensor(L, E * n, k, item=7)
    ids = _routing(m, E, top_k, 7)
    ids[::3] = -1
    ids[5] = E
    ids[ids == 2] = 4                      # expert 2 gets none, expert 4 a token's two picks at times
    counts, offsets, perm, pos = R.sort(ids, E)
    od, pd = torch.from_numpy(offsets).cuda(), torch.from_numpy(perm).cuda()
    y = torch.full((m * top_k, n), 3.5, dtype=torch.bfloat16, device="cuda")
    L.mx_grouped_forward(w, E, x, od, pd, top_k, y=y)
    end = offsets[-1]
    assert end < m * top_k and (y[end:] == 3.5).all()
    xs = x[torch.from_numpy(perm[:end] // top_k).long().cuda()].contiguous()
    z = torch.full((end, n), 3.5, dtype=torch.bfloat16, device="cuda")
    L.mx_grouped_forward(w, E, xs, od, y=z)
    assert torch.equal(y[:end], z)
    # an empty list
    y.fill_(3.5)
    L.mx_grouped_forward(w, E, x, torch.zeros_like(od), pd, top_k, y=y)
    assert (y == 3.5).all()


def test_empty_and_repeat(L, dev):
    import torch

    w, _ = _tensor(L, 300, 1024, item=9)
    for m in (0, 1, 20, 200):
        x, _ = _x(m, 1024, "float16", item=400 + m)
        a, b = L.mx_linear_forward(w, x), L.mx_linear_forward(w, x)
        assert a.shape == (m, 300) and torch.equal(a, b)
    e = L.mx_quantize(torch.empty((0, 256), dtype=torch.float32, device="cuda"))
    assert L.mx_matmul(e, _tensor(L, 5, 256)[0], torch.float32).shape == (0, 5)
    assert L.mx_dequantize(e, torch.float16).shape == (0, 256)


# ------------------------------------------------------------------ streams and graphs

def test_captured_and_replayed(L, dev):
    """The calls in a graph, with two graphs' workspaces of their own, replayed with new inputs and eager work
    between: every replay equals the eager result."""
    import torch

    w, _ = _tensor(L, 600, 2048, item=11)
    E = 4
    ids = torch.from_numpy(_routing(24, E, 2, 11)).cuda()
    xs = [_x(m, 2048, "bfloat16", item=500 + m)[0] for m in (3, 24)]

    def work(x):
        y = L.mx_linear_forward(w, x)
        t = L.mx_quantize(x.float(), transpose=True)
        if x.shape[0] != 24:
            return [y, t.codes, t.scales]
        counts, offsets, perm, pos = L.moe_sort(ids, E)
        h = L.mx_grouped_forward(w, E, x, offsets, perm, 2)
        return [y, t.codes, t.scales, h, L.moe_combine(h, pos, torch.ones(24, 2, device="cuda"))]

    for x in xs:
        work(x)
    graphs, outs, keep = [], [], [x.clone() for x in xs]
    torch.cuda.synchronize()
    for x in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(work(x))
        graphs.append(g)
    for step in range(3):
        for i, x in enumerate(xs):
            x.copy_(keep[i] * (step + 1) + step)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for i, x in enumerate(xs):
            for a, b in zip(outs[i], work(x)):
                assert torch.equal(a, b), (step, i)


def test_on_another_stream(L, dev):
    """Calls on two streams at once, workspaces allocated by the calls: the results are those of one stream."""
    import torch

    w, _ = _tensor(L, 2000, 4096, item=12)
    x = [_x(m, 4096, "float16", item=600 + m)[0] for m in (2, 90)]
    want = [L.mx_linear_forward(w, v) for v in x]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(6):
        for i, s in enumerate(streams):
            got[i].append(L.mx_linear_forward(w, x[i], stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        for y in got[i]:
            assert torch.equal(y, want[i])


def _stream_calls(L):
    """name -> (makes the tensors, the call on them); every tensor 2 MB or more, so a block of its own."""
    import torch

    def codes(r, c):
        return [torch.randint(0, 256, (r, c // 2), dtype=torch.uint8, device="cuda"),
                torch.randint(118, 126, (c // 128, r, 4), dtype=torch.uint8, device="cuda")]

    def rows(r, c, dtype=torch.float16):
        return torch.randn(r, c, device="cuda").to(dtype)
    m, k, n, E = 1 << 17, 4, 8192, 8        # tokens, picks, rows of the products, experts
    H = 64

    def ids():
        return torch.randint(0, E, (m, k), dtype=torch.int32, device="cuda")

    def pos():
        return torch.randperm(m * k, device="cuda").to(torch.int32).reshape(m, k)

    def grouped():
        off = torch.arange(E + 1, device="cuda", dtype=torch.int32) * (m * k // E)
        return codes(E * 1024, 8192) + [rows(n, 8192), off, torch.arange(m * k, device="cuda", dtype=torch.int32) % n]
    return {
        "quantize": (lambda: [rows(n, 4096)], lambda x, s: L.mx_quantize(x, stream=s)),
        "quantize_t": (lambda: [rows(n, 4096)], lambda x, s: L.mx_quantize(x, transpose=True, stream=s)),
        "dequantize": (lambda: codes(n, 8192),
                       lambda c, e, s: L.mx_dequantize(L.MxTensor(c, e), torch.float16, stream=s)),
        "matmul": (lambda: codes(n, 8192) + codes(n, 8192),
                   lambda a, b, c, d, s: L.mx_matmul(L.MxTensor(a, b), L.MxTensor(c, d), torch.bfloat16, stream=s)),
        "linear": (lambda: codes(n, 8192) + [rows(256, 8192)],
                   lambda c, e, x, s: L.mx_linear_forward(L.MxTensor(c, e), x, stream=s)),
        "grouped": (grouped, lambda c, e, x, o, p, s: L.mx_grouped_forward(L.MxTensor(c, e), E, x, o, p, 1, stream=s)),
        "sort": (lambda: [ids()], lambda i, s: L.moe_sort(i, E, stream=s)),
        "gather": (lambda: [rows(m, H), pos()], lambda x, p, s: L.moe_gather(x, p, stream=s)),
        "gather_backward": (lambda: [rows(m * k, H), pos()], lambda d, p, s: L.moe_gather_backward(d, p, stream=s)),
        "combine": (lambda: [rows(m * k, H), pos(), torch.rand(m, k, device="cuda")],
                    lambda o, p, w, s: L.moe_combine(o, p, w, stream=s)),
        "combine_backward": (lambda: [rows(m, H), rows(m * k, H), pos(), torch.rand(m, k, device="cuda")],
                             lambda d, o, p, w, s: L.moe_combine_backward(d, o, p, w, stream=s)),
    }


STREAM_CALLS = ["quantize", "quantize_t", "dequantize", "matmul", "linear", "grouped", "sort", "gather",
                "gather_backward", "combine", "combine_backward"]


@pytest.mark.parametrize("name", STREAM_CALLS)
def test_tensors_let_go_while_another_stream_reads_them(L, dev, name):
    """The caller drops a call's tensors while the stream has not come to it yet: their memory is not given out
    again until it has (tensors of the same sizes, made meanwhile, lie elsewhere)."""
    import torch

    say(f"mx let go {name}")
    make, call = _stream_calls(L)[name]
    busy = torch.randn(8192, 8192, device="cuda")
    s = torch.cuda.Stream()
    tensors = make()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(24):
            busy @ busy                              # some 170 ms of work before the call's
    out = call(*tensors, s)
    at = {t.data_ptr() for t in tensors if t.numel() * t.element_size() >= 2 << 20}
    sizes = [(t.shape, t.dtype) for t in tensors]
    assert at
    del tensors
    new = [torch.zeros(shape, dtype=dtype, device="cuda") for shape, dtype in sizes * 2]
    assert not s.query()
    assert not at & {t.data_ptr() for t in new}
    torch.cuda.synchronize()
    del out, new, busy


def test_captured_with_the_stream_given(L, dev):
    """A capture whose calls name its stream, with tensors dropped inside it and after it."""
    import torch

    w, _ = _tensor(L, 600, 4096, item=13)
    x = _x(90, 4096, "bfloat16", item=650)[0]
    first = x.clone()
    ids = torch.from_numpy(_routing(90, 5, 2, 13)).cuda()

    def work(x, stream):
        t = x * 2
        y = L.mx_linear_forward(w, t, stream=stream)
        del t
        pos = L.moe_sort(ids, 5, stream=stream)[3]
        xs = L.moe_gather(x, pos, stream=stream)
        return [y, L.moe_combine(xs, pos, torch.ones(90, 2, device="cuda"), stream=stream)]
    work(x, None)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = work(x, torch.cuda.current_stream())
    for step in range(3):
        x.copy_(first * (step + 1))
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, work(x, None)):
            assert torch.equal(a, b), step
    del w, x, ids
    assert torch.isfinite(torch.zeros(1 << 20, device="cuda")).all()


# ------------------------------------------------------------------ the operators together

def test_training_step_of_one_linear(L, dev):
    """y, dx and dW of a linear in MXFP4: each product's operands quantized along what it sums over."""
    import torch

    m, k, n = 200, 256, 384
    x, x64 = _x(m, k, "bfloat16", item=21)
    w, w64 = _x(n, k, "bfloat16", item=22)
    dy, dy64 = _x(m, n, "bfloat16", item=23)

    def q(v):
        return R.values(*R.quantize(v))
    y = L.mx_matmul(L.mx_quantize(x), L.mx_quantize(w), torch.bfloat16)
    _check_product(y, q(x64), q(w64), "bfloat16")
    dx = L.mx_matmul(L.mx_quantize(dy), L.mx_quantize(w, transpose=True), torch.bfloat16)
    _check_product(dx, q(dy64), q(R.transposed(w64)), "bfloat16")
    dw = L.mx_matmul(L.mx_quantize(dy, transpose=True), L.mx_quantize(x, transpose=True), torch.float32)
    _check_product(dw, q(R.transposed(dy64)), q(R.transposed(x64)), "float32")


def test_gradients_against_differences(L, dev):
    """Values on the e2m1 grid with a 6 in every block of 32 along both axes: quantizing keeps them, and every
    sum is a multiple of 1/4 below 2^22, exact in fp32. L = <dy, x W^T> is linear in each value, so its
    difference over one value's step equals the gradient's value times the step, exactly."""
    import torch

    m, k, n = 128, 256, 128
    g = synth.rng(64, 41, synth.ROLE_LOGITS)
    grid = np.array([-6, -4, -3, -2, -1.5, -1, -0.5, 0, 0.5, 1, 1.5, 2, 3, 4, 6])

    def tensor(rows, cols):
        v = g.choice(grid, (rows, cols))
        for i in range(32):
            v[i::32, i::32] = 6.0
        return v

    def dev32(v):
        return torch.from_numpy(v.astype(np.float32)).cuda()

    x, w, dy = tensor(m, k), tensor(n, k), tensor(m, n)
    dx = L.mx_matmul(L.mx_quantize(dev32(dy)), L.mx_quantize(dev32(w), transpose=True)).double().cpu().numpy()
    dw = L.mx_matmul(L.mx_quantize(dev32(dy), transpose=True),
                     L.mx_quantize(dev32(x), transpose=True)).double().cpu().numpy()
    assert np.array_equal(dx, dy @ w) and np.array_equal(dw, dy.T @ x)

    def loss(a, b):
        y = L.mx_matmul(L.mx_quantize(dev32(a)), L.mx_quantize(dev32(b)))
        return float((y.double().cpu().numpy() * dy).sum())
    at = loss(x, w)
    for which, v, grad in (("x", x, dx), ("w", w, dw)):
        for _ in range(8):
            i, j = int(g.integers(0, v.shape[0])), int(g.integers(0, v.shape[1]))
            if i % 32 == j % 32:
                j = (j + 1) % v.shape[1]               # the 6 that holds the block's scale stays
            step = v.copy()
            step[i, j] = 1.0 if v[i, j] != 1.0 else -2.0
            moved = loss(step, w) if which == "x" else loss(x, step)
            assert moved - at == grad[i, j] * (step[i, j] - v[i, j]), (which, i, j)


def test_moe_block_end_to_end(L, dev):
    """A routed block in MXFP4: route, sort, gate|up, SwiGLU, down, combine. Each step is compared on the inputs
    that the GPU's own earlier steps gave, so a rounding that falls the other way does not spread."""
    import torch

    m, E, k, hidden, ffn = 70, 8, 3, 512, 256
    x, x64 = _x(m, hidden, "bfloat16", item=31)
    gu, guv = _tensor(L, E * 2 * ffn, hidden, item=31)
    dn, dnv = _tensor(L, E * hidden, ffn, item=32)
    logits = torch.from_numpy(synth.logits(m, E, workload=60, item=31)).cuda()
    ids, weights, counts, offsets, perm = L.moe_route(logits, k)
    c2, o2, p2, pos = L.moe_sort(ids, E)
    assert torch.equal(counts, c2) and torch.equal(offsets, o2) and torch.equal(perm, p2)
    h = L.mx_grouped_forward(gu, E, x, offsets, perm, k)
    a = torch.nn.functional.silu(h[:, :ffn].float()).mul(h[:, ffn:].float()).to(torch.bfloat16)
    o = L.mx_grouped_forward(dn, E, a, offsets)
    y = L.moe_combine(o, pos, weights)
    off, pn = offsets.cpu().numpy(), perm.cpu().numpy()
    qx, qa = R.values(*R.quantize(x64)), R.values(*R.quantize(a.double().cpu().numpy()))
    for e in range(E):
        r = slice(off[e], off[e + 1])
        _check_product(h[r], qx[pn[r] // k], guv[e * 2 * ffn:(e + 1) * 2 * ffn], "bfloat16")
        _check_product(o[r], qa[r], dnv[e * hidden:(e + 1) * hidden], "bfloat16")
    wn, on = weights.double().cpu().numpy(), o.double().cpu().numpy()
    terms = wn[..., None] * on[pos.cpu().numpy()]
    want, mag = terms.sum(1), np.abs(terms).sum(1)
    tol = k * 2.0 ** -24 * mag + _half_step("bfloat16") * (np.abs(want) + k * 2.0 ** -24 * mag)
    assert (np.abs(y.double().cpu().numpy() - want) <= tol).all()
