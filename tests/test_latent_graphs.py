"""Captured and overlapping calls of the latent cache, bit for bit against eager
calls."""
import pytest
import torch

from bwd_tcgen05_tma_gb300 import attn as A
from latent_util import Latent

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bwd_tcgen05_tma_gb300 import build

    build.build()


def bits(t):
    return t.contiguous().view(torch.uint8)


BATCHES = {
    "decode": dict(new=[1] * 4, ctx=[30, 400, 1000, 2500], one=True),
    "decode_128": dict(new=[1] * 3, ctx=[400, 1000, 2500], one=True, H=128),
    "verify": dict(new=[4, 1, 3], ctx=[900, 30, 2000], H=8),
    "chunk": dict(new=[70, 1, 0, 33], ctx=[1900, 300, 40, 700], d_c=256, dtype="fp16"),
}


class Step:
    def __init__(self, seed, name):
        self.c = Latent(seed=seed, **BATCHES[name])
        self.p = self.c.params()
        self.o, self.lse = self.c.fresh_outputs()
        self.ws = torch.empty(A.attn_latent_workspace_size(self.p), dtype=torch.uint8,
                              device="cuda")
        self.saved = {n: self.c.t[n].clone() for n in ("cache", "lens")}

    def run(self):
        A.attn_latent_append(self.p)
        A.attn_latent_fwd(self.p, self.o, self.lse, self.ws)

    def restore(self, delta):
        for n, x in self.saved.items():
            self.c.t[n].copy_(x)
        self.c.t["lens"].sub_(delta)
        self.o.fill_(float("nan"))
        self.lse.fill_(float("nan"))
        self.ws.fill_(255)

    def results(self):
        return [bits(x).clone() for x in (self.o, self.lse, self.c.t["cache"], self.c.t["q_rot"])]


@pytest.mark.parametrize("name", list(BATCHES))
def test_two_graphs_on_two_streams(name):
    """Two captured steps with a workspace each, replayed together on two
    streams at lengths other than the captured ones."""
    steps = [Step(81 + i, name) for i in range(2)]
    graphs, streams = [], [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()
    for st, stream in zip(steps, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            st.run()
        graphs.append(g)
    for delta in (0, 1, 17):
        want = []
        for st in steps:
            st.restore(delta)
            st.run()
            torch.cuda.synchronize()
            want.append(st.results())
            st.restore(delta)
        torch.cuda.synchronize()
        for _ in range(3):  # the same step again appends the same tokens
            for g, stream in zip(graphs, streams):
                with torch.cuda.stream(stream):
                    g.replay()
        torch.cuda.synchronize()
        for st, w in zip(steps, want):
            assert all(torch.equal(x, y) for x, y in zip(st.results(), w)), delta
            assert st.c.status() == 0


@pytest.mark.parametrize("name", list(BATCHES))
def test_captured_step_that_forks_and_joins(name):
    st = Step(85, name)
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    st.restore(0)
    st.run()
    torch.cuda.synchronize()
    want = st.results()

    def forked():
        side.wait_stream(main)
        with torch.cuda.stream(side):
            A.attn_latent_append(st.p)
        main.wait_stream(side)
        A.attn_latent_fwd(st.p, st.o, st.lse, st.ws)

    st.restore(0)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=main):
        forked()
    for _ in range(2):
        st.restore(0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(st.results(), want))


@pytest.mark.parametrize("name", list(BATCHES))
def test_overlapping_calls_and_repeats(name):
    """Many calls of two batches on two streams: every call gives the bits of
    the first."""
    steps = [Step(87 + i, name) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in steps]
    want = []
    for st in steps:
        st.run()
        torch.cuda.synchronize()
        want.append(st.results())
    outs = [[(torch.empty_like(st.o), torch.empty_like(st.lse)) for _ in range(10)] for st in steps]
    for o in outs:
        for x, lse in o:  # padding rows and rows of no sequence stay as they are
            x.fill_(float("nan"))
            lse.fill_(float("nan"))
    torch.cuda.synchronize()
    for i in range(10):
        for st, stream, o in zip(steps, streams, outs):
            A.attn_latent_fwd(st.p, *o[i], st.ws, stream)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        for x, lse in o:
            assert torch.equal(bits(x), w[0]) and torch.equal(bits(lse), w[1])


@pytest.mark.parametrize("names", [("decode", "decode_128"), ("verify", "chunk"),
                                   ("decode_128", "verify")])
def test_graphs_that_share_a_workspace(names):
    """Two captured steps of other sizes on one workspace, replayed in turn on one
    stream without a pause, with an eager call of the first between them."""
    steps = [Step(91 + i, n) for i, n in enumerate(names)]
    ws = max((st.ws for st in steps), key=lambda w: w.numel())
    want = []
    for st in steps:
        st.restore(0)
        st.run()
        torch.cuda.synchronize()
        want.append(st.results())
        st.ws = ws
    stream, graphs = torch.cuda.Stream(), []
    for st in steps:
        st.restore(0)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            st.run()
        graphs.append(g)
    with torch.cuda.stream(stream):
        for _ in range(4):
            graphs[0].replay()
            graphs[1].replay()
            steps[0].run()
            graphs[1].replay()
    torch.cuda.synchronize()
    for st, w in zip(steps, want):
        assert all(torch.equal(x, y) for x, y in zip(st.results(), w))
        assert st.c.status() == 0
