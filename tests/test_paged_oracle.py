"""Pins of the paged cache's float64 oracle against independent statements of
the same definitions (no GPU)."""
import numpy as np
import pytest
import torch

from oracle import attn_ref as R
from oracle import paged_ref as P


def test_e4m3_values_and_rounding_match_the_type():
    v = P.e4m3_values()
    t = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double()
    assert np.array_equal(np.isnan(v), torch.isnan(t).numpy())
    ok = ~np.isnan(v)
    assert np.array_equal(v[ok], t.numpy()[ok])
    rng = np.random.default_rng(1)
    x = rng.standard_normal(20000) * np.exp(rng.uniform(-12, 5, 20000))
    x = np.clip(x, -448, 448).astype(np.float32)
    mid = (v[:126] + v[1:127]) / 2  # ties of neighbouring codes
    x = np.concatenate([x, mid.astype(np.float32), v[:127].astype(np.float32)])
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(P.e4m3_round(x), want)
    assert np.isnan(P.e4m3_round([np.inf, -np.inf, np.nan])).all()


@pytest.mark.parametrize("amax", [0.0, 1e-30, 447.9, 448.0, 448.1, 1.0, 3e38, 2.0 ** -70])
def test_page_scale_is_the_smallest(amax):
    s = P.page_scale(np.array([amax, -amax / 3, np.inf, np.nan]))
    assert amax <= 448 * s
    assert s == 2.0 ** P.MIN_EXP or amax > 448 * (s / 2)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_norms_and_depends_on_distance(interleaved):
    rng = np.random.default_rng(2)
    q, k = rng.standard_normal((2, 1, 32))
    inv = 10000.0 ** (-np.arange(8) / 8)

    def turn(x, pos):
        return P.rotate(x, np.cos(pos * inv), np.sin(pos * inv), interleaved)

    assert np.allclose(np.linalg.norm(turn(q, 77)), np.linalg.norm(q))
    assert np.array_equal(turn(q, 77)[:, 16:], q[:, 16:])
    assert np.allclose((turn(q, 9) * turn(k, 4)).sum(), (turn(q, 105) * turn(k, 100)).sum())


def test_append_in_one_call_or_token_by_token():
    """Where the page's scale never grows the codes do not depend on how the
    tokens were cut into calls; where it does, a value is off by at most one
    more rounding under the final scale."""
    rng = np.random.default_rng(3)
    page, n = 16, 37
    x = rng.standard_normal((n, 2, 64)) * np.exp(rng.standard_normal((n, 1, 1)))
    table = np.array([[2, 0, 1]])
    once, s1 = np.zeros((3, 2, page, 64)), np.zeros((3, 2))
    P.append(once, s1, table, page, [n], [0, n], x)
    step, s2 = np.zeros((3, 2, page, 64)), np.zeros((3, 2))
    for j in range(n):
        P.append(step, s2, table, page, [j + 1], [0, 1], x[j:j + 1])
    assert np.array_equal(s1, s2)
    a, b = (P.gather(c, s, table[0], page, n) for c, s in ((once, s1), (step, s2)))
    ref = x.transpose(1, 0, 2)
    tiny = s1.max() * 2.0 ** -10
    assert (np.abs(a - ref) <= np.abs(ref) * 2.0 ** -4 + tiny).all()
    assert (np.abs(b - ref) <= np.abs(ref) * 2.0 ** -4 + 2 * tiny).all()


@pytest.mark.parametrize("causal", [False, True])
def test_attend_matches_the_attention_oracle(causal):
    rng = np.random.default_rng(4)
    n, length, hq, hkv, d = 5, 23, 4, 2, 16
    q, k, v = (rng.standard_normal(s) for s in ((n, hq, d), (hkv, length, d), (hkv, length, d)))
    o, lse, _, _ = P.attend(q, lambda s: k, lambda s: v, [length], [0, n], 0.3, causal)
    qi, qp = R.dense_metadata(1, n)
    ki, kp = R.dense_metadata(1, length)
    mask = R.Window(None, 0, length - n) if causal else False
    ro, rl = R.attention_forward(q[None], k.transpose(1, 0, 2)[None], v.transpose(1, 0, 2)[None],
                                 qi, qp, ki, kp, mask, 0.3)
    assert np.allclose(o, ro[0]) and np.allclose(lse, rl[0])


def test_attend_window_sink_and_empty_rows():
    rng = np.random.default_rng(5)
    q, k, v = rng.standard_normal((3, 1, 8)), rng.standard_normal((1, 9, 8)), np.ones((1, 9, 8))
    o, lse, _, _ = P.attend(q, lambda s: k, lambda s: v, [9], [0, 3], 0.5, True, 0)
    assert np.allclose(o, 1.0)  # a window of 0 keeps the row's own key
    assert np.allclose(lse[0], [k[0, 6 + i] @ q[i, 0] * 0.5 for i in range(3)])
    o, lse, _, _ = P.attend(q[:1], lambda s: k[:, :0], lambda s: v[:, :0], [0], [0, 1], 0.5,
                            sink=np.array([0.25]))
    assert np.array_equal(o, np.zeros_like(o)) and lse[0, 0] == 0.25
