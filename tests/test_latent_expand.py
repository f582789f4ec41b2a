"""The expanded form of latent attention on the GPU: keys, values and gradients
against the float64 oracle, and a training step from the projections' outputs
through the attention and back."""
import numpy as np
import pytest
import torch

from bwd_tcgen05_tma_gb300 import attn as A
from latent_util import dev16, turn_tolerance
from oracle import attn_ref as R
from oracle import latent_ref as L
from paged_util import UNIT
from test_rope import angles, bits, draw, tables

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bwd_tcgen05_tma_gb300 import build

    build.build()


SHAPES = {
    "wide": dict(T=70, H=16, d_n=128, d_r=64, d_v=128),
    "one_token": dict(T=1, H=1, d_n=128, d_r=64, d_v=128),
    "seven": dict(T=33, H=7, d_n=64, d_r=64, d_v=64),
    "narrow": dict(T=33, H=3, d_n=96, d_r=32, d_v=64),
    "shared128": dict(T=20, H=5, d_n=64, d_r=128, d_v=128),
    "small": dict(T=300, H=2, d_n=8, d_r=32, d_v=8),
    "widest": dict(T=9, H=3, d_n=256, d_r=64, d_v=256),
    "many_heads": dict(T=5, H=130, d_n=24, d_r=32, d_v=40),
}


class Case:
    """Tensors of one shape; `apart`: rows further apart than their width."""

    def __init__(self, T, H, d_n, d_r, d_v, dtype, apart=False, seed=71, rows=64):
        rng = np.random.default_rng(seed)
        self.shape, self.dtype = (T, H, d_n, d_r, d_v), dtype
        widths = dict(kv=(H, d_n + d_v), k_rope=(1, d_r), k=(H, d_n + d_r), v=(H, d_v))
        self.host = {n: draw(rng, (T, h, d), dtype) for n, (h, d) in widths.items()}
        self.host["k_rope"] = self.host["k_rope"][:, 0]
        self.cos, self.sin = tables(rows, d_r, 1.2)
        self.pos = rng.integers(0, rows, T)
        self.apart = apart

    def dev(self, name, fill=None):
        x = dev16(self.host[name], self.dtype)
        if self.apart:
            wide = torch.full((x.shape[0], x[0].numel() + 24), 5.0, dtype=x.dtype, device="cuda")
            part = wide[:, 8:8 + x[0].numel()].view_as(x) if x.dim() == 2 else wide[
                :, 8:8 + x[0].numel()].unflatten(1, x.shape[1:])
            part.copy_(x)
            x = part
        if fill is not None:
            x.fill_(fill)
        return x

    def run(self, back, interleaved, fill=float("nan"), **kw):
        ins, outs = (("k", "v"), ("kv", "k_rope")) if back else (("kv", "k_rope"), ("k", "v"))
        t = {n: self.dev(n) for n in ins}
        t.update({n: self.dev(n, fill) for n in outs})
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        if not {"cu_seqlens", "seq_len"} & set(kw):
            kw["positions"] = torch.tensor(self.pos, dtype=torch.int32, device="cuda")
        p = A.make_latent_expand_params(dtype=self.dtype, rope_cos=self.cos, rope_sin=self.sin,
                                        interleaved=interleaved, status=status, **t, **kw)
        (A.attn_latent_expand_bwd if back else A.attn_latent_expand)(p)
        return t, status.item()


def check_forward(c, t, interleaved, rows=slice(None), pos=None):
    T, H, d_n, d_r, d_v = c.shape
    cc, ss = angles(c.cos, c.sin, c.pos if pos is None else pos)
    k, v = L.expand(c.host["kv"][rows], c.host["k_rope"][rows], cc, ss, d_n, interleaved)
    got_k, got_v = (t[n].double().cpu().numpy()[rows] for n in ("k", "v"))
    assert np.array_equal(got_v, v)
    assert np.array_equal(got_k[..., :d_n], k[..., :d_n])
    big = np.abs(c.host["k_rope"][rows]).max(-1)[:, None, None]
    tol = turn_tolerance(k[..., d_n:], big, c.dtype, 1.2)
    assert (np.abs(got_k - k)[..., d_n:] <= tol).all()


def check_backward(c, t, interleaved, rows=slice(None), pos=None):
    """The sum over H heads is off by at most (H - 1) 2^-24 of the sum of
    magnitudes, then turned as a value of that size."""
    T, H, d_n, d_r, d_v = c.shape
    cc, ss = angles(c.cos, c.sin, c.pos if pos is None else pos)
    dk, dv = c.host["k"][rows], c.host["v"][rows]
    kv, pe = L.expand_bwd(dk, dv, cc, ss, d_n, interleaved)
    assert np.array_equal(t["kv"].double().cpu().numpy()[rows], kv)
    big = np.abs(dk[..., d_n:]).sum(1).max(-1, keepdims=True)
    tol = turn_tolerance(pe, big, c.dtype, 1.2) + 2 * (H - 1) * 2.0 ** -24 * big * 1.2
    err = np.abs(t["k_rope"].double().cpu().numpy()[rows] - pe)
    assert (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("apart", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("name", list(SHAPES))
def test_expand(name, back, interleaved, apart):
    c = Case(dtype="fp16" if apart else "bf16", apart=apart, **SHAPES[name])
    t, status = c.run(back, interleaved)
    assert status == 0
    (check_backward if back else check_forward)(c, t, interleaved)
    for n in ("kv", "k_rope", "k", "v") if apart else ():  # what lies between rows
        base = t[n]._base
        w = c.host[n][0].size
        assert (base[:, :8] == 5).all() and (base[:, 8 + w:] == 5).all()


@pytest.mark.parametrize("back", [False, True])
def test_segments_padding_and_rows(back):
    c = Case(40, 3, 64, 64, 64, "bf16", seed=72)
    cu = [2, 2, 20, 21, 33]
    t, status = c.run(back, False, fill=9.0,
                      cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"))
    assert status == 0
    pos = np.concatenate([np.arange(b - a) for a, b in zip(cu, cu[1:])])
    (check_backward if back else check_forward)(c, t, False, slice(2, 33), pos)
    for n in ("kv", "k_rope") if back else ("k", "v"):
        assert (t[n][:2] == 9).all() and (t[n][33:] == 9).all()
    t, status = c.run(back, False, seq_len=10)
    assert status == 0
    (check_backward if back else check_forward)(c, t, False, slice(None), np.arange(40) % 10)


@pytest.mark.parametrize("back", [False, True])
def test_bad_positions_are_reported(back):
    c = Case(6, 2, 64, 32, 64, "bf16", seed=73, rows=4)
    c.pos = np.array([0, -1, 3, 4, 2 ** 31 - 1, 1])
    t, status = c.run(back, True, fill=9.0)
    assert status == 7
    for n in ("kv", "k_rope") if back else ("k", "v"):
        left = (t[n] == 9).flatten(1).all(1).tolist()
        assert left == [False, True, False, True, True, False]


def test_no_tokens():
    c = Case(0, 2, 64, 32, 64, "bf16")
    for back in (False, True):
        assert c.run(back, False)[1] == 0


@pytest.mark.parametrize("interleaved", [False, True])
def test_backward_against_differences(interleaved):
    """Of sum(wk K) + sum(wv V) in float64; the map is linear."""
    c = Case(3, 2, 8, 32, 8, "bf16", seed=74)
    T, H, d_n, d_r, d_v = c.shape
    cc, ss = angles(c.cos, c.sin, c.pos)
    wk, wv = c.host["k"], c.host["v"]

    def loss(kv, pe):
        k, v = L.expand(kv, pe, cc, ss, d_n, interleaved)
        return (wk * k).sum() + (wv * v).sum()

    kv, pe = c.host["kv"], c.host["k_rope"]
    t, _ = c.run(True, interleaved)
    for x, name in ((kv, "kv"), (pe, "k_rope")):
        got = t[name].double().cpu().numpy()
        for idx in np.ndindex(x.shape):
            e = np.zeros_like(x)
            e[idx] = 0.5
            a = (kv + e, kv - e, pe, pe) if name == "kv" else (kv, kv, pe + e, pe - e)
            g = loss(a[0], a[2]) - loss(a[1], a[3])
            big = np.abs(wk[idx[0], :, d_n:]).sum(0).max()
            assert abs(got[idx] - g) <= turn_tolerance(g, big, "bf16", 1.2) + 2.0 ** -30


def test_training_step():
    """Two packed sequences: queries turned, keys and values expanded, attention
    forward and backward, gradients folded and turned back, against the whole in
    float64, within the tolerances of the attention (1.5e-2 on gradients)."""
    rng = np.random.default_rng(75)
    H, d_n, d_r, d_v, lens = 4, 128, 64, 128, [150, 106]
    T, scale = sum(lens), 192 ** -0.5
    cu = torch.tensor([0, 150, 256], dtype=torch.int32, device="cuda")
    pos = np.concatenate([np.arange(n) for n in lens])
    cos, sin = (torch.empty(160, 32, device="cuda") for _ in "cs")
    A.attn_rope_table(A.make_rope_table_params(cos=cos, sin=sin, scaling="TURNS", factor=4.0,
                                               trained_len=40))
    host = {n: draw(rng, s, "bf16") for n, s in
            (("q", (T, H, 192)), ("kv", (T, H, 256)), ("k_rope", (T, 64)), ("do", (T, H, 128)))}
    dev = {n: dev16(x, "bf16") for n, x in host.items()}
    rope = dict(dtype="bf16", rope_cos=cos, rope_sin=sin, cu_seqlens=cu, interleaved=True)
    q = torch.empty_like(dev["q"])
    k = torch.empty(T, H, 192, dtype=torch.bfloat16, device="cuda")
    v = torch.empty(T, H, 128, dtype=torch.bfloat16, device="cuda")
    A.attn_rope(A.make_rope_params(q=dev["q"], q_out=q, rot_start=128, **rope))
    A.attn_latent_expand(A.make_latent_expand_params(kv=dev["kv"], k_rope=dev["k_rope"], k=k, v=v,
                                                     **rope))
    p = A.make_params(layout="HD_HD_HD", fmt="THD_CU_SEQLENS", mask="PADDING_CAUSAL", B=1, Sq=T,
                      Skv=T, Hq=H, Hkv=H, d_qk=192, d_v=128, scale=scale, q=q, k=k, v=v,
                      cu_seqlens_q=cu, cu_seqlens_kv=cu)
    ws = torch.zeros(A.attn_bwd_workspace_size(p), dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(v), torch.empty(1, H, T, device="cuda")
    A.attn_fwd(p, o, lse, ws)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    A.attn_bwd(p, o, dev["do"], lse, dq, dk, dv, None, ws)
    assert A.attn_read_status(ws)[0] == 0
    dkv, dpe = torch.empty_like(dev["kv"]), torch.empty_like(dev["k_rope"])
    A.attn_rope(A.make_rope_params(q=dq, rot_start=128, inverse=True, **rope))
    A.attn_latent_expand_bwd(A.make_latent_expand_params(kv=dkv, k_rope=dpe, k=dk, v=dv, **rope))

    cc, ss = angles(cos, sin, pos)
    rq = L.turn(host["q"], cc, ss, 128, True)
    rk, rv = L.expand(host["kv"], host["k_rope"], cc, ss, 128, True)
    ids, ps = R.metadata_from_cu_seqlens(np.array([0, 150, 256]), T)
    ro, _ = R.attention_forward(rq[None], rk[None], rv[None], ids, ps, ids, ps, True, scale)
    gq, gk, gv, _ = R.attention_backward(rq[None], rk[None], rv[None], host["do"][None], ids, ps,
                                         ids, ps, True, scale)
    gq = L.turn(gq[0], cc, ss, 128, True, True)
    gkv, gpe = L.expand_bwd(gk[0], gv[0], cc, ss, 128, True)
    # the rotated parts enter the attention rounded to bf16, which adds about one
    # half step (2^-8 relative) to errors of two in the tolerances' measure
    assert R.rel_frobenius(o.double().cpu().numpy(), ro[0]) <= 5e-3 + UNIT["bf16"]
    for got, ref in ((dq, gq), (dkv, gkv), (dpe, gpe)):
        assert R.rel_frobenius(got.double().cpu().numpy(), ref) <= 1.5e-2 + UNIT["bf16"]


def test_captured_step_and_repeats():
    """The pair captured into a graph beside an eager pair on another stream:
    the bits of the first call, every time."""
    c = Case(200, 8, 128, 64, 128, "bf16", seed=76)
    eager, _ = c.run(True, True)
    first = {n: eager[n].clone() for n in ("kv", "k_rope")}
    pos = torch.tensor(c.pos, dtype=torch.int32, device="cuda")
    t = {n: c.dev(n) for n in ("kv", "k_rope", "k", "v")}
    p = A.make_latent_expand_params(dtype="bf16", rope_cos=c.cos, rope_sin=c.sin, positions=pos,
                                    interleaved=True, **t)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        A.attn_latent_expand_bwd(p)
    for _ in range(3):
        t["kv"].fill_(float("nan"))
        t["k_rope"].fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        with torch.cuda.stream(side):
            again, _ = c.run(True, True)
        torch.cuda.synchronize()
        for n, x in first.items():
            assert torch.equal(bits(t[n]), bits(x)) and torch.equal(bits(again[n]), bits(x))
