"""Captured and overlapping calls of the paged cache, of single tokens and of
chunks (each kernel with the one that joins its pieces), bit for bit against
eager calls."""
import pytest
import torch

from paged_util import Paged

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
    "verify": dict(new=[4, 1, 3], ctx=[900, 30, 2000], Hq=8, Hkv=2),
    "chunk": dict(new=[70, 1, 0, 33], ctx=[1900, 300, 40, 700]),
}
CACHES = ["fp8_e4m3", "bf16"]
SAVED = ("k_cache", "v_cache", "k_scale", "v_scale", "lens")


class Step:
    """One sequence batch with the outputs and the workspace of its step."""

    def __init__(self, seed, name, cache):
        from bwd_tcgen05_tma_gb300 import attn as A

        self.A, self.c = A, Paged(seed=seed, cache=cache, **BATCHES[name])
        self.p = self.c.params()
        self.o, self.lse = self.c.fresh_outputs()
        self.ws = torch.empty(A.attn_paged_workspace_size(self.p), dtype=torch.uint8,
                              device="cuda")
        self.saved = {n: self.c.t[n].clone() for n in SAVED if self.c.t[n] is not None}

    def run(self):
        self.A.attn_paged_append(self.p)
        self.A.attn_paged_fwd(self.p, self.o, self.lse, self.ws)

    def restore(self, delta):
        for n, x in self.saved.items():
            self.c.t[n].copy_(x)
        self.c.t["lens"].sub_(delta)
        self.o.fill_(float("nan"))
        self.lse.fill_(float("nan"))
        self.ws.fill_(255)

    def results(self):
        out = [self.o, self.lse, self.c.t["k_cache"], self.c.t["v_cache"]]
        return [bits(x).clone() for x in out]


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("name", list(BATCHES))
def test_two_graphs_on_two_streams(name, cache):
    """Two captured steps with a workspace each, replayed together on two
    streams at lengths other than the captured ones."""
    steps = [Step(81 + i, name, cache) for i in range(2)]
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
    """Append on one stream, attention on another behind an event, in a graph
    and eagerly."""
    st = Step(85, name, "fp8_e4m3")
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    st.restore(0)
    st.run()
    torch.cuda.synchronize()
    want = st.results()

    def forked():
        side.wait_stream(main)
        with torch.cuda.stream(side):
            st.A.attn_paged_append(st.p)
        main.wait_stream(side)
        st.A.attn_paged_fwd(st.p, st.o, st.lse, st.ws)

    st.restore(0)
    torch.cuda.synchronize()
    with torch.cuda.stream(main):
        forked()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(st.results(), want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=main):
        forked()
    for _ in range(2):
        st.restore(0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(st.results(), want))


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("name", list(BATCHES))
def test_overlapping_calls_and_repeats(name, cache):
    """Many calls of two batches on two streams: every call gives the bits of
    the first."""
    steps = [Step(87 + i, name, cache) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in steps]
    want = []
    for st in steps:
        st.run()
        torch.cuda.synchronize()
        want.append(st.results())
    outs = [[(torch.empty_like(st.o), torch.empty_like(st.lse)) for _ in range(10)] for st in steps]
    torch.cuda.synchronize()
    for i in range(10):
        for st, stream, o in zip(steps, streams, outs):
            st.A.attn_paged_fwd(st.p, *o[i], st.ws, stream)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        for x, lse in o:
            assert torch.equal(bits(x), w[0]) and torch.equal(bits(lse), w[1])
