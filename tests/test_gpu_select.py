"""Expert selection on the GPU: ids exact against Python sorts of 64-bit values,
weights and gradients within derived bounds, and against differences."""
import numpy as np
import pytest

import synth
import _adapters_ref as A
from _helpers import cuda, say

pytestmark = pytest.mark.gpu

DTYPES = ["float32", "float16", "bfloat16"]
HALF = {"float16": 2.0 ** -11, "bfloat16": 2.0 ** -8, "float32": 2.0 ** -24}
TINY = {"float16": 2.0 ** -25, "bfloat16": 2.0 ** -133, "float32": 2.0 ** -126}


@pytest.fixture(scope="module")
def dev():
    return cuda()


@pytest.fixture(scope="module")
def L():
    from bit_weight_only_amd import lbq
    lbq.lib()
    return lbq


def _logits(m, E, dtype, item, spread=2.0):
    import torch

    g = synth.rng(80, item, synth.ROLE_LOGITS)
    return torch.from_numpy((spread * g.standard_normal((m, E))).astype(np.float32)).to(getattr(torch, dtype))


def _check(L, lg, top_k, bias=None, **how):
    import torch

    ids, w = L.moe_select(lg.cuda(), top_k, bias=None if bias is None else torch.from_numpy(bias).cuda(), **how)
    want_ids, want = A.select(lg.double().numpy(), top_k, None if bias is None else bias.astype(np.float64), **how)
    assert ids.dtype == torch.int32 and w.dtype == torch.float32
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    w = w.cpu().numpy().astype(np.float64)
    # exp is off by its argument's rounding, the score, the sum over picks and the quotient by a few roundings each;
    # an argument below -128 gives zero in 32 bits
    fin = lg.double().numpy()
    span = min(128, np.abs(np.where(np.isfinite(fin), fin, 0)).max()) * (how.get("score", 0) == 0)
    tol = (40 + top_k + 4 * span) * A.U
    # (scores below fp32's normal range keep an absolute step only)
    assert np.all(np.abs(w - want) <= tol * np.abs(want) + 2.0 ** -120), np.abs(w - want).max()
    return ids, w


# (tokens, experts, picks, groups, top groups, group picks)
SHAPES = [(1, 1, 1, 1, 1, 1), (1, 256, 8, 1, 1, 1), (33, 256, 8, 8, 4, 2), (7, 60, 4, 1, 1, 1), (64, 64, 6, 8, 3, 1),
          (5, 1024, 32, 1, 1, 1), (19, 1000, 13, 10, 4, 2), (9, 30, 10, 10, 10, 2), (11, 16, 16, 2, 2, 1),
          (3, 1024, 32, 512, 100, 2), (6, 65, 3, 1, 1, 1), (4, 257, 9, 1, 1, 1), (130, 17, 2, 17, 5, 2),
          (8, 1022, 4, 73, 2, 2), (1030, 128, 8, 4, 2, 2)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,E,k,G,tg,gp", SHAPES)
def test_select(L, dev, m, E, k, G, tg, gp, dtype):
    say(f"moe_select m={m} E={E} k={k} groups={G}/{tg}/{gp} {dtype}")
    lg = _logits(m, E, dtype, m * 7 + E)
    g = synth.rng(81, E, synth.ROLE_X)
    bias = (0.1 * g.standard_normal(E)).astype(np.float32)
    for score in (L.SCORE_SOFTMAX, L.SCORE_SIGMOID):
        for b in (None, bias):
            for renorm, scale in ((True, 1.0), (False, 2.5)):
                _check(L, lg, k, b, score=score, groups=G, top_groups=tg, group_picks=gp, renormalise=renorm, scale=scale)


@pytest.mark.parametrize("score", [0, 1])
def test_ties_and_near_ties(L, dev, score):
    """Equal logits go to the lower id; choice values that differ by less than 32 bits can tell are told apart."""
    import torch

    E = 256
    g = synth.rng(82, score, synth.ROLE_X)
    lg = torch.from_numpy(g.integers(-2, 3, (200, E)).astype(np.float32))             # five values only
    _check(L, lg, 8, None, score=score)
    _check(L, lg, 8, np.zeros(E, np.float32), score=score)
    _check(L, lg, 8, None, score=score, groups=8, top_groups=3, group_picks=2)
    _check(L, lg, 32, (g.integers(0, 2, E) * 0.25).astype(np.float32), score=score, groups=32, top_groups=4, group_picks=2)
    # logits one fp32 step apart, in falling and rising order, with a bias that swallows the step in 32 bits
    v = np.full((2, E), 1.0, np.float32)
    for e in range(1, E):
        v[0, e] = np.nextafter(v[0, e - 1], np.float32(0))
        v[1, e] = np.nextafter(v[1, e - 1], np.float32(2))
    for b in (None, np.full(E, 1.0, np.float32), np.full(E, 64.0, np.float32)):
        _check(L, torch.from_numpy(v), 8, b, score=score)
        _check(L, torch.from_numpy(v), 8, b, score=score, groups=16, top_groups=2, group_picks=2)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("score", [0, 1])
def test_masked(L, dev, score, dtype):
    """Experts that are switched off, rows that leave fewer than top_k or none, the type's lowest value, NaN."""
    import torch

    m, E = 12, 40
    lg = _logits(m, E, dtype, 3)
    lg[0, :] = float("-inf")                       # none
    lg[1, 3:] = float("-inf")                      # three
    lg[2, :] = torch.finfo(lg.dtype).min           # the lowest value everywhere: equal, not off
    lg[3, 1:] = torch.finfo(lg.dtype).min
    lg[4, 5] = float("nan")
    lg[5, :] = float("nan")
    lg[6, 7] = float("inf")
    lg[7, [7, 9]] = float("inf")
    lg[8, 10:] = float("-inf")
    lg[9, :] = torch.finfo(lg.dtype).max
    bias = (0.05 * synth.rng(83, 0, synth.ROLE_X).standard_normal(E)).astype(np.float32)
    off = bias.copy()
    off[[0, 1, 11, 30]] = [-np.inf, np.nan, -np.inf, -np.inf]
    for b in (None, bias, off):
        for how in (dict(), dict(groups=5, top_groups=2, group_picks=2), dict(groups=10, top_groups=6, group_picks=1)):
            for renorm in (True, False):
                ids, w = _check(L, lg, 6, b, score=score, renormalise=renorm, **how)
                assert np.all(w[ids.cpu().numpy() < 0] == 0) and np.all(np.isfinite(w))
    ids, _ = L.moe_select(lg.cuda(), 6, score=score)
    assert ids[0].tolist() == [-1] * 6 and ids[1].tolist()[3:] == [-1] * 3
    # what it calls no pick is none to the sort
    counts = L.moe_sort(ids, E)[0]
    assert int(counts.sum()) == int((ids >= 0).sum())


def test_agrees_with_the_router(L, dev):
    lg = _logits(300, 256, "float32", 9).cuda()
    ids, w = L.moe_select(lg, 8)
    i2, w2 = L.moe_route(lg, 8)[:2]
    assert np.array_equal(ids.cpu().numpy(), i2.cpu().numpy())
    np.testing.assert_allclose(w.cpu().numpy(), w2.cpu().numpy(), rtol=80 * A.U)


def test_no_tokens(L, dev):
    import torch

    lg = torch.empty(0, 16, device="cuda")
    ids, w = L.moe_select(lg, 4)
    assert ids.shape == (0, 4) and w.shape == (0, 4)
    assert L.moe_select_backward(w, lg, ids).shape == (0, 16)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,E,k,G,tg,gp", SHAPES)
def test_gradient(L, dev, m, E, k, G, tg, gp, dtype):
    import torch

    say(f"moe_select_backward m={m} E={E} k={k} {dtype}")
    lg = _logits(m, E, dtype, m * 3 + E)
    if E > 2 and m > 2:
        lg[1, ::2] = float("-inf")
        lg[2, :] = float("-inf")
    g = synth.rng(84, E, synth.ROLE_X).standard_normal((m, k)).astype(np.float32)
    for score in (0, 1):
        for renorm, scale in ((True, 1.0), (False, 2.5)):
            ids, _ = L.moe_select(lg.cuda(), k, score=score, groups=G, top_groups=tg, group_picks=gp)
            gd = torch.from_numpy(g).cuda()
            gd[ids < 0] = float("nan")             # not read where there is no pick
            d = L.moe_select_backward(gd, lg.cuda(), ids, score=score, renormalise=renorm, scale=scale)
            assert d.dtype == lg.dtype
            want, bound = A.select_backward(g.astype(np.float64), lg.double().numpy(), ids.cpu().numpy(), score, renorm,
                                            scale)
            err = np.abs(d.double().cpu().numpy() - want)
            assert np.all(err <= bound * 1.01 + HALF[dtype] * np.abs(want) + TINY[dtype] + 2.0 ** -120), err.max()


def test_gradient_of_given_picks(L, dev):
    """Picks of the caller's own: an expert named twice gets both slots' gradients, numbers out of range none; in place."""
    import torch

    lg = _logits(6, 20, "float32", 5)
    ids = np.array([[3, 3, 7], [-1, 5, 20], [2 ** 31 - 1, -2 ** 31, 0], [1, 2, 3], [-1, -1, -1], [19, 0, 19]], np.int32)
    g = synth.rng(85, 0, synth.ROLE_X).standard_normal((6, 3)).astype(np.float32)
    for score in (0, 1):
        for renorm in (True, False):
            x = lg.cuda()
            d = L.moe_select_backward(torch.from_numpy(g).cuda(), x, torch.from_numpy(ids).cuda(), score=score,
                                      renormalise=renorm, d_logits=x)
            assert d.data_ptr() == x.data_ptr()
            want, bound = A.select_backward(g.astype(np.float64), lg.double().numpy(), ids, score, renorm)
            assert np.all(np.abs(d.double().cpu().numpy() - want) <= bound * 1.01 + HALF["float32"] * np.abs(want))


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_against_differences(L, dev, score, renorm):
    """Central differences of the weights themselves: with a step e their own error is e^2 / 6 times a third
    derivative (below 2 here) and the weights' roundings over 2 e."""
    import torch

    lg = _logits(1, 24, "float32", 11, spread=1.0)
    k, e = 4, 2.0 ** -6
    g = synth.rng(86, 0, synth.ROLE_X).standard_normal((1, k)).astype(np.float32)
    ids, _ = L.moe_select(lg.cuda(), k, score=score, renormalise=renorm)
    d = L.moe_select_backward(torch.from_numpy(g).cuda(), lg.cuda(), ids, score=score, renormalise=renorm).cpu().numpy()[0]
    step = torch.zeros(48, 24)
    for i in range(24):
        step[2 * i, i], step[2 * i + 1, i] = e, -e
    i2, w = L.moe_select((lg + step).cuda(), 24, score=score, renormalise=False)
    # the picks of lg, whatever their order after the step
    p = torch.zeros(48, 24, dtype=torch.double, device="cuda").scatter_(1, i2.long(), w.double())[:, ids[0].long()]
    if renorm:
        p = p / p.sum(1, keepdim=True)
    f = (p.cpu().numpy() * g).sum(1)
    diff = (f[0::2] - f[1::2]) / (2 * e)
    tol = np.abs(g).sum() * (e * e / 3 + 64 * A.U / e)
    assert np.all(np.abs(diff - d) <= tol), np.abs(diff - d).max()


def test_repeatable_other_stream_and_graph(L, dev):
    import torch

    lg = _logits(500, 256, "bfloat16", 21).cuda()
    bias = torch.from_numpy((0.05 * synth.rng(87, 0, synth.ROLE_X).standard_normal(256)).astype(np.float32)).cuda()
    how = dict(score=1, groups=8, top_groups=4, group_picks=2, scale=2.5)
    want = L.moe_select(lg, 8, bias=bias, **how)
    gw = torch.randn(500, 8, device="cuda")
    want_d = L.moe_select_backward(gw, lg, want[0], score=1, scale=2.5)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = L.moe_select(lg, 8, bias=bias, stream=s, **how)
    d = L.moe_select_backward(gw, lg, got[0], score=1, scale=2.5, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(d, want_d)
    ids, w = torch.empty_like(want[0]), torch.empty_like(want[1])
    src = lg.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L.moe_select(src, 8, bias=bias, ids=ids, weights=w, **how)
        dl = L.moe_select_backward(gw, src, ids, score=1, scale=2.5)
    for i in range(3):
        new = _logits(500, 256, "bfloat16", 30 + i).cuda()
        src.copy_(new)
        g.replay()
        torch.cuda.synchronize()
        a, b = L.moe_select(new, 8, bias=bias, **how)
        assert torch.equal(ids, a) and torch.equal(w, b)
        assert torch.equal(dl, L.moe_select_backward(gw, new, a, score=1, scale=2.5))


def test_many_tokens(L, dev):
    """A long batch against 64-bit torch on the GPU."""
    import torch

    lg = (torch.randn(70001, 160, device="cuda", generator=torch.Generator("cuda").manual_seed(5))).to(torch.bfloat16)
    bias = 0.05 * torch.randn(160, device="cuda", generator=torch.Generator("cuda").manual_seed(6))
    ids, w = L.moe_select(lg, 6, bias=bias, score=1, scale=2.0)
    p = torch.sigmoid(lg.double())
    want = torch.sort(p + bias.double(), dim=1, descending=True, stable=True).indices[:, :6]
    assert torch.equal(ids.long(), want)
    s = p.gather(1, want)
    s = 2.0 * s / s.sum(1, keepdim=True)
    assert float(((w.double() - s).abs() / s).max()) <= 46 * A.U


# more tokens than go to a wavefront each
@pytest.mark.parametrize("m,E,k,G,tg,gp", [(2100, 256, 8, 8, 4, 2), (2049, 200, 17, 10, 5, 2), (2060, 72, 32, 1, 1, 1)])
def test_more_tokens_than_wavefronts(L, dev, m, E, k, G, tg, gp):
    bias = (0.1 * synth.rng(88, E, synth.ROLE_X).standard_normal(E)).astype(np.float32)
    lg = _logits(m, E, "bfloat16", m)
    lg[5, 2:] = float("-inf")
    for score in (0, 1):
        for b in (None, bias, np.zeros(E, np.float32)):
            _check(L, lg, k, b, score=score, groups=G, top_groups=tg, group_picks=gp)


def test_far_below_zero(L, dev):
    """Sigmoids that 32 bits cannot hold still have a ratio, and a gradient."""
    import torch

    for shift in (-50.0, -95.0, -300.0):
        lg = _logits(40, 96, "float32", 3) + shift
        ids, _ = _check(L, lg, 6, score=1)
        g = synth.rng(89, 0, synth.ROLE_X).standard_normal((40, 6)).astype(np.float32)
        d = L.moe_select_backward(torch.from_numpy(g).cuda(), lg.cuda(), ids, score=1)
        want, bound = A.select_backward(g.astype(np.float64), lg.double().numpy(), ids.cpu().numpy(), 1)
        # (the argument of exp is off by its own rounding)
        assert np.all(np.abs(d.double().cpu().numpy() - want) <= bound * (1.01 + abs(shift) / 4) + 1e-30)


def test_refusals(L, dev):
    import torch

    lg = torch.zeros(4, 16, device="cuda")
    ids, w = L.moe_select(lg, 2)
    bad = [lambda: L.moe_select(lg[:, ::2], 2), lambda: L.moe_select(lg.double(), 2), lambda: L.moe_select(lg, 17),
           lambda: L.moe_select(lg, 2, bias=torch.zeros(15, device="cuda")),
           lambda: L.moe_select(lg, 2, bias=torch.zeros(16)), lambda: L.moe_select(lg[0], 2),
           lambda: L.moe_select(lg, 2, groups=3), lambda: L.moe_select(lg, 2, score=2),
           lambda: L.moe_select(lg, 2, ids=ids.long()), lambda: L.moe_select_backward(w, lg, ids.long()),
           lambda: L.moe_select_backward(w[:2], lg, ids), lambda: L.moe_select_backward(w, lg[:3], ids),
           lambda: L.moe_select_backward(w, lg, ids, d_logits=lg.half())]
    for f in bad:
        with pytest.raises(L.LbqError):
            f()


# (tokens, experts, picks, groups, top groups, group picks): every form of the kernel
FAR_SHAPES = [(9, 40, 3, 1, 1, 1), (9, 48, 4, 6, 3, 2), (12, 256, 8, 1, 1, 1), (2052, 200, 5, 1, 1, 1), (2049, 256, 8, 8, 4, 2),
              (10, 300, 32, 1, 1, 1), (7, 1000, 13, 1, 1, 1), (5, 960, 6, 80, 30, 2)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,E,k,G,tg,gp", FAR_SHAPES)
def test_picks_far_below_the_rows_largest(L, dev, m, E, k, G, tg, gp, dtype):
    """Softmax: where the bias keeps the row's largest from being picked, the picks' weights still have their ratio, and
    the gradient is that ratio's. More than 745 below it 64 bits hold their p as 0: weights and gradient are 0."""
    import torch

    g = synth.rng(93, E, synth.ROLE_X)
    bias = (0.1 * g.standard_normal(E)).astype(np.float32)
    dw = g.standard_normal((m, k)).astype(np.float32)
    first = E // 3
    for gap in (60, 80, 90, 100, 110, 300, 690, 800):
        say(f"moe_select far below m={m} E={E} groups={G} {dtype} gap={gap}")
        lg = _logits(m, E, dtype, 17, spread=1.0)
        lg[:, first] = lg.amax(1) + gap
        for b0 in (-np.inf, -3.0):
            b = bias.copy()
            b[first] = b0
            how = dict(score=0, groups=G, top_groups=tg, group_picks=gp)
            ids, w = _check(L, lg, k, b, **how)
            assert not bool((ids == first).any())
            assert bool((w.sum(1) == 0).all()) if gap == 800 else np.all(np.abs(w.sum(1) - 1) <= 16 * A.U)
            d = L.moe_select_backward(torch.from_numpy(dw).cuda(), lg.cuda(), ids, score=0)
            want, bound = A.select_backward(dw.astype(np.float64), lg.double().numpy(), ids.cpu().numpy(), 0)
            err = np.abs(d.double().cpu().numpy() - want)
            assert np.all(err <= bound * 1.01 + HALF[dtype] * np.abs(want) + TINY[dtype] + 2.0 ** -120), err.max()
            _check(L, lg, k, b, renormalise=False, **how)


def test_one_pick_past_the_border(L, dev):
    """One pick just inside what 64 bits hold, the other outside."""
    import torch

    lg = torch.tensor([[0.0, -740.0, -750.0, -751.0], [0.0, -80.0, -120.0, -800.0]])
    b = np.array([-np.inf, 0.3, 0.2, 0.1], np.float32)
    g = np.array([[1.0, 0.5], [-0.5, 1.0]], np.float32)
    ids, w = _check(L, lg, 2, b)
    assert ids.tolist() == [[1, 2], [1, 2]] and w[0].tolist() == [1.0, 0.0]
    d = L.moe_select_backward(torch.from_numpy(g).cuda(), lg.cuda(), ids).double().cpu().numpy()
    # w (g - sum w g): with S = 4e-322 the oracle's g / S overflows
    _, w = A.select(lg.double().numpy(), 2, b.astype(np.float64))
    want, bound = np.zeros((2, 4)), np.zeros((2, 4))
    want[:, 1:3] = w * (g - (w * g).sum(1, keepdims=True))
    bound[:, 1:3] = w * (np.abs(g) + (w * np.abs(g)).sum(1, keepdims=True)) * (42 + 4 * 80) * A.U
    assert np.all(np.abs(d - want) <= bound * 1.01 + A.U * np.abs(want) + 2.0 ** -120)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("shift", [-690.0, -720.0, -800.0])
def test_sigmoids_that_64_bits_cannot_hold(L, dev, shift, dtype):
    """1 / (1 + exp(-l)) is 0 in 64 bits from l = -709.78 down: weights and gradient end at the same place."""
    import torch

    for bias in (None, (0.1 * synth.rng(94, 0, synth.ROLE_X).standard_normal(96)).astype(np.float32)):
        lg = (_logits(40, 96, "float32", 3) + shift).to(getattr(torch, dtype))
        ids, w = _check(L, lg, 6, bias, score=1)
        assert np.all(w == 0) if shift < -710 else np.all(np.abs(w.sum(1) - 1) <= 16 * A.U)
        g = synth.rng(89, 0, synth.ROLE_X).standard_normal((40, 6)).astype(np.float32)
        d = L.moe_select_backward(torch.from_numpy(g).cuda(), lg.cuda(), ids, score=1).double().cpu().numpy()
        want, bound = A.select_backward(g.astype(np.float64), lg.double().numpy(), ids.cpu().numpy(), 1)
        # (the argument of exp is off by its own rounding)
        assert np.all(np.abs(d - want) <= bound * (1.01 + abs(shift) / 4) + HALF[dtype] * np.abs(want) + 1e-30)


def test_sigmoids_around_the_border(L, dev):
    """Some picks on this side of it, some on the other."""
    import torch

    edge = np.float32(-709.7827)                               # the last that 64 bits hold is one step above
    lg = torch.tensor([[-709.0, -710.0, -711.0], [float(np.nextafter(edge, np.float32(0))), float(edge), -800.0],
                       [float(edge), -710.0, -720.0], [-100.0, -705.0, -715.0]])
    g = np.array([[1.0, 0.5], [-0.5, 1.0], [1.0, 2.0], [3.0, -1.0]], np.float32)
    ids, w = _check(L, lg, 2, score=1)
    assert w.tolist()[:3] == [[1.0, 0.0], [1.0, 0.0], [0.0, 0.0]]
    d = L.moe_select_backward(torch.from_numpy(g).cuda(), lg.cuda(), ids, score=1).double().cpu().numpy()
    # w (1 - p) (g - sum w g), 1 - p = 1 here: with S = 6e-309 the oracle's g / S overflows
    _, w = A.select(lg.double().numpy(), 2, score=1)
    want, bound = np.zeros((4, 3)), np.zeros((4, 3))
    want[:, :2] = w * (g - (w * g).sum(1, keepdims=True))
    bound[:, :2] = w * (np.abs(g) + (w * np.abs(g)).sum(1, keepdims=True)) * 42 * A.U
    # (the argument of exp is off by its own rounding)
    assert np.all(np.abs(d - want) <= bound * (1.01 + 720 / 4) + A.U * np.abs(want) + 1e-30)


@pytest.mark.parametrize("m,E,k", [(40, 24, 6), (60, 256, 32), (2070, 200, 8), (30, 700, 12)])
def test_sigmoids_of_very_different_sizes(L, dev, m, E, k):
    """Picks whose own sigmoid fp32 cannot hold, beside others: their ratio may be one that it can. Logits are multiples of
    1/8, whose differences are exact."""
    import torch

    g = synth.rng(96, E, synth.ROLE_X)
    v = np.round(g.standard_normal((m, E)) * 8 * g.choice([8.0, 30.0, 60.0], (m, 1)) + 8 * g.choice([0.0, -41.0, -90.0], (m, 1))) / 8
    keep = np.argsort(g.random((m, E)), 1) < np.minimum(E, g.integers(1, 2 * k, (m, 1)))
    keep[:, 0] = True
    v[0, :3], keep[0] = (-41.0, -95.0, -120.0), np.arange(E) < 3
    lg = torch.from_numpy(np.where(keep, v, -np.inf).astype(np.float32))
    ids, w = _check(L, lg, k, score=1)
    dw = g.standard_normal((m, k)).astype(np.float32)
    d = L.moe_select_backward(torch.from_numpy(dw).cuda(), lg.cuda(), ids, score=1).double().cpu().numpy()
    want, bound = A.select_backward(dw.astype(np.float64), lg.double().numpy(), ids.cpu().numpy(), 1)
    assert np.all(np.abs(d - want) <= bound * 1.01 + HALF["float32"] * np.abs(want) + 2.0 ** -120)
    _check(L, lg, k, (0.1 * g.standard_normal(E)).astype(np.float32), score=1)
    _check(L, lg, k, score=1, renormalise=False)
