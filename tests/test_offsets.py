"""Offsets that are not in order or lie outside the tokens, in the calls that look
a token's place up: every such pair is reported, wherever it stands, a token is
written only by a sequence whose own offsets are sound and hold it, and the last
offset ends the tokens only where it is sound itself."""
import numpy as np
import pytest
import torch

from bwd_tcgen05_tma_gb300 import attn as A
from latent_util import Latent, turn_tolerance
from oracle import latent_ref as L
from paged_util import Paged
from test_latent_expand import Case
from test_rope import angles, bits, draw, tables

pytestmark = pytest.mark.gpu

BOUNDS = 7
T = 10
I32 = dict(dtype=torch.int32, device="cuda")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bwd_tcgen05_tma_gb300 import build

    build.build()


def sound(cu, tokens=T):
    return [(a, b) for a, b in zip(cu, cu[1:]) if 0 <= a <= b <= tokens]


def places(cu, t):
    """Positions that sound segments give token t."""
    return [t - a for a, b in sound(cu) if a <= t < b]


# offsets, rows that have to be written
BAD = {
    "last_decreases": ([0, 10, 5], range(10)),
    "last_below_zero": ([0, 2, -5], range(2)),
    "inner_decreases": ([0, 8, 4, 10], range(4)),
    "only_one_below_zero": ([0, -1], ()),
    "behind_all_tokens": ([20, 30], ()),
    "first_below_zero": ([-3, 10], ()),
    "end_behind_the_tokens": ([0, 4, 11], range(4)),
    "inner_behind_the_tokens": ([0, 3, 50, 6], range(3)),
    "far_behind": ([0] + [10] * 700 + [3] + [10] * 500, range(10)),
    "no_segment": ([50], ()),
    "in_order": ([2, 2, 5, 9], range(2, 9)),
}


def expected_status(name):
    return 0 if name == "in_order" else BOUNDS


def check_rows(name, written, right):
    """written(t): has row t changed; right(t, pos): is it what position pos makes."""
    cu, must = BAD[name]
    for t in range(T):
        at = places(cu, t)
        if t in must:
            assert written(t), t
        if not at:
            assert not written(t), t
        elif written(t):
            assert any(right(t, p) for p in at), t


@pytest.mark.parametrize("name", list(BAD))
def test_rope(name):
    x = draw(np.random.default_rng(90), (T, 2, 64), "bf16")
    q = torch.from_numpy(x).cuda().bfloat16()
    cos, sin = tables(T, 64)
    out, status = torch.full_like(q, 77.0), torch.zeros(1, **I32)
    A.attn_rope(A.make_rope_params(dtype="bf16", q=q, q_out=out, rope_cos=cos, rope_sin=sin,
                                   cu_seqlens=torch.tensor(BAD[name][0], **I32), status=status))
    assert status.item() == expected_status(name)
    got = out.double().cpu().numpy()

    def right(t, pos):
        ref = L.turn(x[t:t + 1], *angles(cos, sin, [pos]))
        return (np.abs(got[t:t + 1] - ref) <=
                turn_tolerance(ref, np.abs(x[t]).max(), "bf16")).all()

    check_rows(name, lambda t: (got[t] != 77).any(), right)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("name", list(BAD))
def test_expand(name, back):
    c = Case(T, 2, 64, 64, 64, "bf16", seed=91)
    t, status = c.run(back, False, fill=77.0, cu_seqlens=torch.tensor(BAD[name][0], **I32))
    assert status == expected_status(name)
    got = {n: t[n].double().cpu().numpy() for n in (("kv", "k_rope") if back else ("k", "v"))}

    def right(r, pos):
        cc, ss = angles(c.cos, c.sin, [pos])
        row = slice(r, r + 1)
        if back:
            kv, pe = L.expand_bwd(c.host["k"][row], c.host["v"][row], cc, ss, 64)
            big = np.abs(c.host["k"][r, :, 64:]).sum(0).max()
            tol = turn_tolerance(pe, big, "bf16", 1.2) + 2 * 2.0 ** -24 * big * 1.2
            return (np.array_equal(got["kv"][row], kv) and
                    (np.abs(got["k_rope"][row] - pe) <= tol).all())
        k, v = L.expand(c.host["kv"][row], c.host["k_rope"][row], cc, ss, 64)
        tol = turn_tolerance(k, np.abs(c.host["k_rope"][r]).max(), "bf16", 1.2)
        return np.array_equal(got["v"][row], v) and (np.abs(got["k"][row] - k) <= tol).all()

    check_rows(name, lambda r: any((x[r] != 77).any() for x in got.values()), right)


# ---------------------------------------------------------------- appends

CACHES = {
    "latent": (Latent, A.attn_latent_append, ["cache"]),
    "paged": (Paged, A.attn_paged_append, ["k_cache", "v_cache"]),
}


def appended(kind, new, ctx, change):
    """A batch appended whole, and again with its offsets or lengths changed."""
    make, call, caches = CACHES[kind]
    kw = dict(page=16) if kind == "latent" else dict(cache="bf16")
    good, bad = (make(new, ctx, seed=92, **kw) for _ in range(2))
    call(good.params())
    assert good.status() == 0
    before = {n: bad.t[n].clone() for n in caches}
    change(bad.t)
    call(bad.params())
    return good, bad, before, caches


def same_pages(x, y, pages):
    return all(torch.equal(bits(x[p]), bits(y[p])) for p in pages)


@pytest.mark.parametrize("kind", list(CACHES))
@pytest.mark.parametrize("last", [-5, 1])
def test_append_with_a_bad_last_offset(kind, last):
    """The sequences before the last are appended; the last is left out and
    reported."""
    def change(t):
        t["cu"][2] = last

    good, bad, before, caches = appended(kind, [2, 3], [3, 4], change)
    assert bad.status() == BOUNDS
    for n in caches:
        own = [int(good.table[0, 0])]
        assert same_pages(bad.t[n], good.t[n], own)
        assert same_pages(bad.t[n], before[n], [i for i in range(len(before[n])) if i not in own])
    assert torch.equal(bits(bad.t["q_rot"][:2]), bits(good.t["q_rot"][:2]))
    assert torch.isnan(bad.t["q_rot"][2:]).all()


@pytest.mark.parametrize("kind", list(CACHES))
@pytest.mark.parametrize("what", ["offset", "length"])
def test_append_reports_what_no_token_meets(kind, what):
    """Among empty sequences, hundreds of them away from the tokens: an offset or a
    length that is negative.  The tokens are appended all the same."""
    new = [1, 1] + [0] * 900 + [1] + [0] * 300

    def change(t):
        if what == "length":
            t["lens"][1100] = -4
        else:
            t["cu"][700] = -1

    good, bad, before, caches = appended(kind, new, [3] * len(new), change)
    assert bad.status() == BOUNDS
    for n in caches:
        assert same_pages(bad.t[n], good.t[n], range(len(before[n])))
    assert torch.equal(bits(bad.t["q_rot"]), bits(good.t["q_rot"]))


@pytest.mark.parametrize("kind", list(CACHES))
def test_append_with_an_inner_decrease(kind):
    """Offsets 0, 8, 4, 10: reported; nothing is written but to the pages of the two
    sequences whose own offsets are in order."""
    def change(t):
        t["cu"][1], t["cu"][2] = 8, 4

    good, bad, before, caches = appended(kind, [4, 4, 2], [8, 8, 8], change)
    assert bad.status() == BOUNDS
    left = int(good.table[1, 0])
    for n in caches:
        assert same_pages(bad.t[n], before[n], [left])
    assert torch.isfinite(bad.t["q_rot"]).all()


@pytest.mark.parametrize("kind", list(CACHES))
def test_append_with_padding_reports_nothing(kind):
    """Sound offsets that end before the last row: no report, and padding stays."""
    make, call, _ = CACHES[kind]
    c = make([3, 0, 2], [5, 7, 1], seed=93, pad=70)
    call(c.params())
    assert c.status() == 0
    assert torch.isfinite(c.t["q_rot"][:5]).all() and torch.isnan(c.t["q_rot"][5:]).all()


def test_more_segments_than_half_of_32_bits():
    """2^30 + 1000 segments, all but the last two empty (4.3 GB of offsets)."""
    n = (1 << 30) + 1000
    cu = torch.zeros(n + 1, **I32)
    cu[-2], cu[-1] = 4, T
    x = draw(np.random.default_rng(94), (T, 2, 64), "bf16")
    q = torch.from_numpy(x).cuda().bfloat16()
    cos, sin = tables(T, 64)
    status = torch.zeros(1, **I32)
    A.attn_rope(A.make_rope_params(dtype="bf16", q=q, rope_cos=cos, rope_sin=sin, cu_seqlens=cu,
                                   status=status))
    assert status.item() == 0
    ref = L.turn(x, *angles(cos, sin, [0, 1, 2, 3, 0, 1, 2, 3, 4, 5]))
    tol = turn_tolerance(ref, np.abs(x).max(), "bf16")
    assert (np.abs(q.double().cpu().numpy() - ref) <= tol).all()
    cu[1 << 29] = 3  # in order with nothing behind it
    A.attn_rope(A.make_rope_params(dtype="bf16", q=q, rope_cos=cos, rope_sin=sin, cu_seqlens=cu,
                                   status=status))
    assert status.item() == BOUNDS
