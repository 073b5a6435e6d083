"""The expert dispatch in captured graphs and on streams of its own: sorts by one
workgroup and by several, gather, combine and both gradients."""
import pytest

from _helpers import cuda, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return cuda()


@pytest.fixture(scope="module")
def L():
    from bit_weight_only_amd import lbq
    lbq.lib()
    return lbq


class Pass:
    """One routed pass there and back on m tokens of k picks; refill() gives it other ids, rows and gradients."""

    def __init__(self, L, m, k, E, H, dtype):
        import torch

        self.L, self.m, self.k, self.E, self.H = L, m, k, E, H
        ft = getattr(torch, dtype)
        self.ids = torch.zeros((m, k), dtype=torch.int32, device="cuda")
        self.w = torch.zeros((m, k), device="cuda")
        self.x, self.dy = (torch.zeros((m, H), dtype=ft, device="cuda") for _ in range(2))

    def refill(self, seed):
        import torch

        g = torch.Generator(device="cuda").manual_seed(seed)
        self.ids.copy_(torch.randint(-1, self.E + 1, (self.m, self.k), device="cuda", generator=g, dtype=torch.int32))
        self.w.copy_(torch.rand((self.m, self.k), device="cuda", generator=g))
        self.x.copy_(torch.randn((self.m, self.H), device="cuda", generator=g))
        self.dy.copy_(torch.randn((self.m, self.H), device="cuda", generator=g))

    def run(self, stream=None):
        """Every result; rows that no place names are zeros."""
        L, T = self.L, self.m * self.k
        counts, offsets, perm, pos = L.moe_sort(self.ids, self.E, stream=stream)
        xs, d_o = self.x.new_empty((T, self.H)), self.x.new_empty((T, self.H))
        xs.zero_(), d_o.zero_()
        L.moe_gather(self.x, pos, out=xs, stream=stream)
        y = L.moe_combine(xs, pos, self.w, stream=stream)
        _, d_w = L.moe_combine_backward(self.dy, xs, pos, self.w, d_o=d_o, stream=stream)
        dx = L.moe_gather_backward(d_o, pos, stream=stream)
        return [counts, offsets, perm, pos, xs, y, d_o, d_w, dx]


# 64 picks (one workgroup) and 12000 (several, with a workspace of their own); rows of whole vectors and not
SIZES = [(32, 2, 8, 256, "float16"), (4000, 3, 40, 100, "bfloat16"), (1500, 8, 256, 129, "float32")]


def test_captured_and_replayed(L, dev):
    """Each size in a graph of its own, replayed in turn with new ids and rows and eager work between: every replay
    equals the eager result."""
    import torch

    say("dispatch graphs")
    passes = [Pass(L, *size) for size in SIZES]
    for i, p in enumerate(passes):
        p.refill(i)
        p.run()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for p in passes:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(p.run())
        graphs.append(g)
    for step in range(4):
        for i, p in enumerate(passes):
            p.refill(100 * step + i)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for i, p in enumerate(passes):
            for j, (a, b) in enumerate(zip(outs[i], p.run())):
                assert torch.equal(a, b), (step, i, j)


def test_on_two_streams(L, dev):
    """Passes on two streams at once, each call's workspace its own: the results are those of the current stream."""
    import torch

    say("dispatch streams")
    passes = [Pass(L, *size) for size in SIZES[1:]]
    for i, p in enumerate(passes):
        p.refill(40 + i)
    want = [p.run() for p in passes]
    streams = [torch.cuda.Stream() for _ in passes]
    torch.cuda.synchronize()
    got = [[] for _ in passes]
    for _ in range(6):
        for i, (p, s) in enumerate(zip(passes, streams)):
            with torch.cuda.stream(s):
                got[i].append(p.run(stream=s if len(got[i]) % 2 else None))
    torch.cuda.synchronize()
    for i in range(len(passes)):
        for r in got[i]:
            for j, (a, b) in enumerate(zip(r, want[i])):
                assert torch.equal(a, b), (i, j)
