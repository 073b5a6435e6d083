"""Expert dispatch on the GPU: the sort exact against a Python sort, the row
moves and their gradients against 64-bit sums and against differences."""
import numpy as np
import pytest

import synth
import _mx_ref as R
from _helpers import cuda, say

pytestmark = pytest.mark.gpu

DTYPES = ["float16", "bfloat16", "float32"]
HALF = {"float16": 2.0 ** -11, "bfloat16": 2.0 ** -8, "float32": 2.0 ** -24}


@pytest.fixture(scope="module")
def dev():
    return cuda()


@pytest.fixture(scope="module")
def L():
    from bit_weight_only_amd import lbq
    lbq.lib()
    return lbq


def _ids(m, k, E, item=0, drop=0.2):
    g = synth.rng(70, item, synth.ROLE_LOGITS)
    ids = g.integers(0, E, (m, k)).astype(np.int32)          # a token may name an expert twice
    u = g.random((m, k))
    ids[u < drop / 2] = -1
    ids[u > 1 - drop / 2] = E + g.integers(0, 1000)
    return ids


def _check_sort(L, ids, E):
    import torch

    got = [t.cpu().numpy() for t in L.moe_sort(torch.from_numpy(ids).cuda(), E)]
    for name, a, b in zip(("counts", "offsets", "perm", "pos"), got, R.sort(ids, E)):
        assert a.dtype == np.int32 and np.array_equal(a, b), name


# one and several workgroups, ragged chunks, one expert, the limits
@pytest.mark.parametrize("m,k,E", [(1, 1, 1), (1, 32, 4), (5, 3, 1024), (32, 8, 256), (100, 7, 3), (2048, 8, 256),
                                   (5000, 8, 1000), (16385, 1, 64), (131072, 8, 256)])
def test_sort(L, dev, m, k, E):
    say(f"moe_sort m={m} k={k} E={E}")
    _check_sort(L, _ids(m, k, E, item=m), E)


def test_sort_crowded_and_empty(L, dev):
    import torch

    _check_sort(L, np.full((3000, 8), 5, np.int32), 7)                     # all to one expert
    _check_sort(L, np.full((3000, 8), -1, np.int32), 7)                    # none at all
    _check_sort(L, np.full((1, 1), 2 ** 31 - 1, np.int32), 7)
    counts, offsets, perm, pos = L.moe_sort(torch.empty((0, 4), dtype=torch.int32, device="cuda"), 9)
    assert counts.tolist() == [0] * 9 and offsets.tolist() == [0] * 10 and perm.numel() == 0


def test_sort_agrees_with_the_router(L, dev):
    import torch

    lg = torch.from_numpy(synth.logits(333, 64, workload=70)).cuda()
    ids, _, counts, offsets, perm = L.moe_route(lg, 6)
    c, o, p, pos = L.moe_sort(ids, 64)
    assert torch.equal(c, counts) and torch.equal(o, offsets) and torch.equal(p, perm)
    assert torch.equal(perm[pos.reshape(-1).long()], torch.arange(333 * 6, device="cuda", dtype=torch.int32))


def _setup(m, k, E, H, dtype, item=0, drop=0.2):
    """ids, pos (device, host), x, o, dy, d_out in dtype (device) and in 64 bits."""
    import torch

    g = synth.rng(71, item, synth.ROLE_X)
    ids = _ids(m, k, E, item, drop)
    if m > 2:
        ids[1] = -1                                            # a token without any expert
    pos = R.sort(ids, E)[3]
    out = {"pos": pos, "pd": torch.from_numpy(pos).cuda()}
    w = g.random((m, k), dtype=np.float32)
    out["w"], out["wd"] = w.astype(np.float64), torch.from_numpy(w).cuda()
    for name, rows in (("x", m), ("dy", m), ("o", m * k), ("dxs", m * k)):
        t = torch.from_numpy(g.standard_normal((rows, H))).to(getattr(torch, dtype))
        out[name], out[name + "d"] = t.double().numpy(), t.cuda()
    return out


SIZES = [(1, 1, 1, 1), (3, 2, 4, 8), (17, 8, 64, 2048), (40, 3, 5, 333), (9, 32, 256, 40), (300, 4, 16, 1024),
         (6, 5, 12, 5000)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,k,E,H", SIZES)
def test_rows_and_gradients(L, dev, m, k, E, H, dtype):
    import torch

    say(f"dispatch m={m} k={k} E={E} H={H} {dtype}")
    s = _setup(m, k, E, H, dtype, item=m * 100 + H)
    ft, hs = getattr(torch, dtype), HALF[dtype]
    small = 2.0 ** -25 if dtype == "float16" else 2.0 ** -133
    there = (s["pos"] >= 0)[..., None]
    rows = s["pos"].clip(0)
    named = np.zeros(m * k, bool)
    named[s["pos"][s["pos"] >= 0]] = True

    # gather: copies; rows that no place names stay
    xs = torch.full((m * k, H), 2.5, dtype=ft, device="cuda")
    L.moe_gather(s["xd"], s["pd"], out=xs)
    want = np.full((m * k, H), 2.5)
    for t in range(m):
        want[s["pos"][t][s["pos"][t] >= 0]] = s["x"][t]
    assert np.array_equal(xs.double().cpu().numpy(), want)

    # its gradient and the combine: k products and sums in 32 bits, then one rounding
    for got, terms in ((L.moe_gather_backward(s["dxsd"], s["pd"]), np.where(there, s["dxs"][rows], 0)),
                       (L.moe_combine(s["od"], s["pd"], s["wd"]),
                        np.where(there, s["w"][..., None] * s["o"][rows], 0))):
        want, mag = terms.sum(1), np.abs(terms).sum(1)
        tol = k * 2.0 ** -24 * mag + small
        tol += hs * (np.abs(want) + tol)
        assert (np.abs(got.double().cpu().numpy() - want) <= tol).all()

    # the combine's gradients: one product in 32 bits rounded to dtype; a sum of H products in 32 bits
    d_o = torch.full((m * k, H), 2.5, dtype=ft, device="cuda")
    _, d_w = L.moe_combine_backward(s["dyd"], s["od"], s["pd"], s["wd"], d_o=d_o)
    got = d_o.double().cpu().numpy()
    assert (got[~named] == 2.5).all()
    want = np.zeros((m * k, H))
    for t in range(m):
        for j in range(k):
            if s["pos"][t, j] >= 0:
                want[s["pos"][t, j]] = s["w"][t, j] * s["dy"][t]
    assert (np.abs(got - want)[named] <= ((hs + 2.0 ** -23) * np.abs(want) + small)[named]).all()
    terms = np.where(there, s["o"][rows] * s["dy"][:, None], 0)
    tol = (H + 8) * 2.0 ** -24 * np.abs(terms).sum(-1)
    got = d_w.double().cpu().numpy()
    assert (np.abs(got - terms.sum(-1)) <= tol).all() and (got[s["pos"] < 0] == 0).all()

    # in place of o: the same
    o2 = s["od"].clone()
    _, d_w2 = L.moe_combine_backward(s["dyd"], o2, s["pd"], s["wd"], d_o=o2)
    assert torch.equal(d_w, d_w2)
    assert torch.equal(o2[torch.from_numpy(named).cuda()], d_o[torch.from_numpy(named).cuda()])


def test_gradients_against_differences(L, dev):
    """The scalar <dy, combine(gather(x), w)> moved along random directions, central differences: it is linear
    in x and in w, so the difference has no truncation error, only that of 32-bit sums (2 H k terms of size one
    around a sum of size sqrt(H k m): 1e-4 relative to the sum of magnitudes is 2^-24 times over 1000)."""
    import torch

    m, k, E, H = 24, 3, 8, 64
    s = _setup(m, k, E, H, "float32", item=5)
    pos, w, x, dy = s["pd"], s["wd"], s["xd"], s["dyd"]

    def f(x, w):
        xs = torch.zeros((m * k, H), device="cuda")
        return (L.moe_combine(L.moe_gather(x, pos, out=xs), pos, w).double() * dy.double()).sum().item()
    xs = torch.zeros((m * k, H), device="cuda")
    L.moe_gather(x, pos, out=xs)
    d_o, d_w = L.moe_combine_backward(dy, xs, pos, w, d_o=torch.zeros_like(xs))
    dx = L.moe_gather_backward(d_o, pos)
    g = torch.Generator(device="cuda").manual_seed(3)
    scale = (dy.abs().sum() * w.max()).item()
    vx = torch.randn(x.shape, device="cuda", generator=g)
    vw = torch.randn(w.shape, device="cuda", generator=g)
    num = (f(x + vx, w) - f(x - vx, w)) / 2
    assert abs(num - (dx.double() * vx.double()).sum().item()) <= 1e-4 * scale
    num = (f(x, w + vw) - f(x, w - vw)) / 2
    assert abs(num - (d_w.double() * vw.double()).sum().item()) <= 1e-4 * scale


def test_dropped_values_do_not_count(L, dev):
    """NaN in rows that no place names, and NaN weights of dropped picks, reach nothing."""
    import torch

    s = _setup(50, 4, 8, 96, "bfloat16", item=9, drop=0.5)
    named = torch.zeros(200, dtype=torch.bool, device="cuda")
    named[s["pd"][s["pd"] >= 0].long()] = True
    o, w = s["od"].clone(), s["wd"].clone()
    o[~named] = torch.nan
    w[s["pd"] < 0] = torch.nan
    assert torch.equal(L.moe_combine(o, s["pd"], w), L.moe_combine(s["od"], s["pd"], s["wd"]))
    assert torch.isfinite(L.moe_gather_backward(o, s["pd"])).all()
    d_o, d_w = L.moe_combine_backward(s["dyd"], o, s["pd"], w)
    assert torch.isfinite(d_w).all() and torch.isfinite(d_o[named]).all()
    # a list shorter than the places: those behind its end count nothing
    T = 60
    cut = torch.where(s["pd"] < T, s["pd"], -1)
    assert torch.equal(L.moe_combine(s["od"][:T], s["pd"], s["wd"]), L.moe_combine(s["od"], cut, s["wd"]))
    short = torch.zeros((T, 96), dtype=torch.bfloat16, device="cuda")
    full = torch.zeros((200, 96), dtype=torch.bfloat16, device="cuda")
    L.moe_gather(s["xd"], s["pd"], out=short)
    L.moe_gather(s["xd"], s["pd"], out=full)
    assert torch.equal(short, full[:T])


def test_gather_larger_than_the_memory_side_cache(L, dev):
    """A list of over 256 MB is stored past the caches; smaller ones are not: the same rows."""
    import torch

    m, k, H = 17000, 4, 2048
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(m, H, device="cuda", generator=g).to(torch.bfloat16)
    ids = torch.randint(-1, 40, (m, k), device="cuda", generator=g, dtype=torch.int32)
    counts, offsets, perm, pos = L.moe_sort(ids, 40)
    n = int(offsets[-1])
    out = torch.full((m * k, H), 2.5, dtype=torch.bfloat16, device="cuda")
    assert out.numel() * 2 > 256 << 20
    L.moe_gather(x, pos, out=out)
    assert torch.equal(out[:n], x[(perm[:n] // k).long()]) and (out[n:] == 2.5).all()
