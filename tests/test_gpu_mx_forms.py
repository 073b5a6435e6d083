"""The forms of the MXFP4 product kernels that large, long and decode-sized calls
run: each tile with its two ways out, the streaming kernel by K, tokens and row
tiles at a time, x quantized on the way or before. Against 64-bit products."""
import numpy as np
import pytest

import synth
import _mx_ref as R
from _helpers import cuda, say
from test_gpu_mx import _check_product, _routing, _tensor, _x

pytestmark = pytest.mark.gpu

HALVES = ["float16", "bfloat16"]


@pytest.fixture(scope="module")
def dev():
    return cuda()


@pytest.fixture(scope="module")
def L():
    from bit_weight_only_amd import lbq
    lbq.lib()
    return lbq


# 256 x 256 and 128 x 128 tiles with ragged last ones; N a multiple of 8 (results through LDS) and not; two,
# four and eight slices of K (their sum in every type), even and odd numbers of 128-groups
@pytest.mark.parametrize("dtype", HALVES + ["float32"])
@pytest.mark.parametrize("m,n,k", [(4000, 3912, 384), (4000, 3901, 128), (2400, 3608, 384), (2400, 3601, 256),
                                   (700, 1104, 2176), (100, 200, 4096), (77, 131, 17408)])
def test_matmul_tiles(L, dev, m, n, k, dtype):
    import torch

    say(f"mx tiles {m}x{n}x{k} {dtype}")
    a, av = _tensor(L, m, k, item=m)
    b, bv = _tensor(L, n, k, item=1000 + n)
    y = torch.full((m + 1, n), 7.0, dtype=getattr(torch, dtype), device="cuda")
    _check_product(L.mx_matmul(a, b, y=y[:m]), av, bv, dtype)
    assert (y[m] == 7.0).all()


# up to 16 tokens at every length of K (to 2048, 4096, 8192, 17536 and past it), 17 to 32, 33 to 64; row tiles
# walked in more than one batch (N past 4096); x quantized on the way and in a launch before
@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("m,n,k", [(1, 333, 5120), (8, 200, 8192), (16, 200, 8192), (3, 4500, 5120), (1, 4096, 14336),
                                   (3, 130, 14336), (7, 40, 9216), (9, 70, 17408), (12, 4200, 14336),
                                   (24, 500, 2560), (24, 500, 4096), (32, 100, 2048), (20, 4200, 6400),
                                   (64, 300, 2048), (50, 300, 4096), (40, 4200, 3200), (1, 200, 18944),
                                   (3, 72, 28672), (1777, 3904, 384)])
def test_linear_forms(L, dev, m, n, k, dtype):
    say(f"mx linear forms {m}x{n}x{k} {dtype}")
    x, x64 = _x(m, k, dtype, item=700 + m)
    w, wv = _tensor(L, n, k, item=4000 + n)
    _check_product(L.mx_linear_forward(w, x), R.values(*R.quantize(x64)), wv, dtype)


def _check_grouped(L, x, x64, w, wv, ids, E, n, top_k, dtype):
    import torch

    counts, offsets, perm, pos = R.sort(ids, E)
    y = torch.full((ids.size, n), 7.0, dtype=getattr(torch, dtype), device="cuda")
    L.mx_grouped_forward(w, E, x, torch.from_numpy(offsets).cuda(), torch.from_numpy(perm).cuda(), top_k, y=y)
    q = R.values(*R.quantize(x64))
    for e in range(E):
        if counts[e]:
            rows = slice(offsets[e], offsets[e + 1])
            _check_product(y[rows], q[perm[rows] // top_k], wv[e * n:(e + 1) * n], dtype)
    assert (y[offsets[E]:] == 7.0).all()


# the streaming kernel with one, two and four row tiles at a time, with walkers that take one batch and several;
# K to 2048, 4096, 8192 and past it, x quantized on the way and before; the 64, 128 and 256-row tiles
@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("m,E,top_k,n,k", [(32, 64, 4, 300, 2048), (70, 1024, 6, 250, 256), (50, 64, 1, 300, 512),
                                           (20, 16, 2, 1000, 4096), (200, 256, 2, 130, 2304), (64, 8, 1, 200, 4096),
                                           (8, 8, 2, 270, 8192), (40, 16, 4, 100, 8192), (2, 4, 2, 90, 14336),
                                           (5, 4, 2, 90, 14336), (700, 6, 3, 504, 384), (3000, 4, 2, 1104, 128),
                                           (2000, 4, 2, 1800, 384), (2100, 4, 2, 3528, 384)])
def test_grouped_forms(L, dev, m, E, top_k, n, k, dtype):
    say(f"mx grouped forms m={m} E={E} k={top_k} {n}x{k} {dtype}")
    x, x64 = _x(m, k, dtype, item=800 + m)
    w, wv = _tensor(L, E * n, k, item=5000 + E)
    ids = _routing(m, E, top_k, 50 + m)
    ids[::7] = -1                                        # a dropped token in seven
    _check_grouped(L, x, x64, w, wv, ids, E, n, top_k, dtype)


@pytest.mark.parametrize("m,E,n,k", [(50, 64, 300, 512), (70, 64, 130, 4096), (40, 32, 40, 9216)])
def test_grouped_crowded_expert(L, dev, m, E, n, k):
    """Every row goes to one expert: several of the streaming kernel's row tiles for it, none for the others."""
    say(f"mx grouped crowded m={m} E={E} {n}x{k}")
    x, x64 = _x(m, k, "bfloat16", item=900 + m)
    w, wv = _tensor(L, E * n, k, item=6000 + E)
    for e in (0, 3, E - 1):
        _check_grouped(L, x, x64, w, wv, np.full((m, 1), e, np.int32), E, n, 1, "bfloat16")


# ------------------------------------------------------------------ values out of the ordinary

@pytest.mark.parametrize("m,n,k", [(1, 40, 1152), (3, 100, 1152), (7, 40, 9216), (9, 70, 17408), (24, 60, 2560),
                                   (24, 60, 4096), (60, 60, 1024), (200, 130, 512), (4000, 3912, 128)])
def test_linear_rows_with_nan_and_infinity(L, dev, m, n, k):
    """A NaN or an infinity in x makes the results of its own row NaN and leaves the others' bits alone."""
    import torch

    say(f"mx linear nan {m}x{n}x{k}")
    x, _ = _x(m, k, "bfloat16", item=750 + m)
    w, _ = _tensor(L, n, k, item=4500 + n)
    clean = L.mx_linear_forward(w, x)
    assert torch.isfinite(clean).all()
    bad = x.clone()
    bad[m // 2, k - 1] = torch.inf
    bad[0, k // 2] = torch.nan
    got = L.mx_linear_forward(w, bad)
    hit = torch.zeros(m, dtype=torch.bool, device="cuda")
    hit[[0, m // 2]] = True
    assert torch.isnan(got[hit]).all() and torch.equal(got[~hit], clean[~hit])


@pytest.mark.parametrize("m,n,k", [(1, 64, 512), (16, 70, 9216), (40, 64, 512), (200, 72, 1024), (100, 200, 4096)])
def test_scales_at_the_ends(L, dev, m, n, k):
    """Scales from 2^-126 to 2^126 whose products are 1, and a subnormal scale against the largest: the products
    are exact. Results below 2^-126 keep fp32's subnormal steps: every addition and the partial products may each
    be off by 2^-149."""
    import torch

    say(f"mx scales {m}x{n}x{k}")
    g = synth.rng(65, m, synth.ROLE_W)
    ca, cb = (g.integers(0, 256, (r, k // 2), dtype=np.uint8) for r in (m, n))

    def product(sa, sb):
        sa, sb = (np.ascontiguousarray(np.broadcast_to(s, (k // 128, r, 4)), np.uint8) for s, r in ((sa, m), (sb, n)))
        a, b = (L.MxTensor(torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda()) for c, s in ((ca, sa), (cb, sb)))
        return L.mx_matmul(a, b, torch.float32), R.values(ca, sa), R.values(cb, sb)
    per_block = g.integers(1, 254, (k // 128, 1, 4))
    _check_product(*product(per_block, 254 - per_block), "float32")
    for sa, sb in ((0, 254), (254, 0), (0, 200), (1, 253)):
        _check_product(*product(sa, sb), "float32")
    for together in (-126, -140, -149):
        y, av, bv = product(127 + together // 2, 127 + together - together // 2)
        want, mag = av @ bv.T, np.abs(av) @ np.abs(bv).T
        tol = (k / 64 + 128) * (2.0 ** -23 * mag + 2.0 ** -149)
        assert (np.abs(y.double().cpu().numpy() - want) <= tol).all()
