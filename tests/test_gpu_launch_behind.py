"""Kernels that are set up while the one before them in the stream ends: they read nothing
before it has ended, and nothing behind them begins before they have, whatever comes before and
behind: copies, kernels, themselves, another stream's work, in a graph or not."""
import numpy as np
import pytest
import torch

from broadcast_gemm_attention_gb300 import binding as B

pytestmark = pytest.mark.gpu

H, D, LQ = 4, 128, 8
LENS = {"steps": [3, 1, 0, 2], "registers": [60, 100, 0, 33], "tiles": [500, 130, 0, 700], "cut": [3000, 10, 0, 900]}
BOUND = {"steps": 3, "registers": 100, "tiles": 700, "cut": 0}


class Step:
    """A user's program: positions, the states of the users' rows, candidates' reads, and all gradients."""

    def __init__(self, kind, seed):
        g = torch.Generator().manual_seed(seed)
        rows, n_users, n = sum(LENS[kind]), len(LENS[kind]), 200
        draw = lambda *s: torch.randn(s, generator=g)  # noqa: E731
        self.kind = kind
        self.m = torch.sort(torch.randint(0, n_users, (n,), generator=g)).values.int().cuda()
        self.off = torch.tensor(np.concatenate([[0], np.cumsum(LENS[kind])]), dtype=torch.int32).cuda()
        self.decay = torch.linspace(0.9, 0.999, H).cuda()
        self.rope = B.Rope(D, B.ikbo_rope_frequencies(D), axes=[j % 2 for j in range(D // 2)], n_axes=2)
        self.fresh = [[draw(rows, H, D).bfloat16().cuda() for _ in range(4)] + [draw(n_users, H, D, D).cuda() for _ in range(2)] +
                      [draw(n, H, LQ, D).bfloat16().cuda() for _ in range(2)] +
                      [torch.randint(0, 5000, (n, LQ, 2), generator=g, dtype=torch.int32).cuda()] for _ in range(2)]
        self.ins = [torch.zeros_like(t) for t in self.fresh[0]]
        Q, _, _, _, S, _, X, _, _ = self.ins
        self.outs = [torch.zeros_like(t) for t in (X, X, Q, S, Q, Q, Q, S, X, S, X)]

    def fill(self, which):
        for to, x in zip(self.ins, self.fresh[which]):
            to.copy_(x)

    def run(self, p):
        Q, K, V, dO, S, dS, X, dX, place = self.ins
        X2, Y, O, S2, dQ, dK, dV, dS2, dX2, dS3, dX3 = self.outs
        kw = dict(offsets=self.off, max_len=BOUND[self.kind])
        p.rope_axes_forward(self.rope, X, X2, positions=place)
        p.linattn_forward(Q, K, V, self.decay, O, state_in=S, state_out=S2, **kw)
        p.linattn_read_forward(X2, S2, Y)
        p.linattn_read_backward(X2, S2, dX, dX2, dS3)
        p.linattn_backward(Q, K, V, dO, self.decay, dQ, dK, dV, state_in=S, d_state_out=dS3, d_state_in=dS2, **kw)
        p.rope_axes_backward(self.rope, dX2, dX3, positions=place)

    def spoil(self):
        for t in self.ins + self.outs:
            t.fill_(3)


@pytest.mark.parametrize("kind", list(LENS))
def test_every_order_gives_the_same(kind):
    s = Step(kind, 40 + len(kind))
    with B.Plan(256, 4, H) as p:
        p.plan(s.m, 4, H, LQ)
        want = []
        for i in range(2):  # each call by itself
            s.spoil()
            s.fill(i)
            torch.cuda.synchronize()
            s.run(_Alone(p))
            torch.cuda.synchronize()
            want.append([t.clone() for t in s.outs])
        ref = states(s)
        assert torch.allclose(want[1][3].double().cpu(), ref, rtol=0, atol=2.0 ** -10 * float(ref.abs().max()))
        wrong = torch.zeros((), dtype=torch.int64, device="cuda")

        def once(i):
            s.fill(i)
            s.run(p)
            for t, w in zip(s.outs, want[i]):
                wrong.add_((t != w).sum())
            s.spoil()

        for i in range(30):
            once(i % 2)
        assert int(wrong) == 0

        side = torch.cuda.Stream()

        def across(i):  # inputs from one stream, results to another
            main = torch.cuda.current_stream()
            side.wait_stream(main)
            with torch.cuda.stream(side):
                s.fill(i)
            main.wait_stream(side)
            s.run(p)
            side.wait_stream(main)
            with torch.cuda.stream(side):
                for t, w in zip(s.outs, want[i]):
                    wrong.add_((t != w).sum())
                s.spoil()
            main.wait_stream(side)

        torch.cuda.synchronize()
        for i in range(30):
            across(i % 2)
        torch.cuda.synchronize()
        assert int(wrong) == 0
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            once(0)
            across(1)
            across(0)
            once(1)
        for _ in range(10):
            graph.replay()
        torch.cuda.synchronize()
        assert int(wrong) == 0 and p.status() == B.IKBO_OK


class _Alone:
    """A plan whose calls wait for each other on the host."""

    def __init__(self, p):
        self.p = p

    def __getattr__(self, name):
        call = getattr(self.p, name)

        def wait(*a, **k):
            call(*a, **k)
            torch.cuda.synchronize()

        return wait


def states(s):
    """The states after the rows, in 64 bits."""
    _, K, V, _, S = (t.double().cpu() for t in s.fresh[1][:5])
    off, decay = s.off.cpu().tolist(), s.decay.double().cpu()
    out = S.clone()
    for u in range(len(off) - 1):
        n = off[u + 1] - off[u]
        if n == 0:
            continue
        w = decay[None, :] ** torch.arange(n - 1, -1, -1, dtype=torch.float64)[:, None]  # [n, H]
        out[u] = out[u] * (decay ** n)[:, None, None] + torch.einsum("th,thi,thj->hij", w, K[off[u]:off[u + 1]], V[off[u]:off[u + 1]])
    return out
