"""Offsets that are not in order or lie outside the tokens, in the calls that look
a token's place up: every such pair is reported, wherever it stands, a token is
written only by a sequence whose own offsets are sound and hold it, and the last
offset ends the tokens only where it is sound itself."""
import numpy as np
import pytest
import torch

from bwd_tcgen05_tma_gb300 import attn as A
from latent_util import turn_tolerance
from oracle import latent_ref as L
from test_latent_expand import Case
from test_rope import angles, draw, tables

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
