"""Pins of the float64 oracle of rotary positions and latent attention against
independent statements of the same definitions (no GPU)."""
import numpy as np
import pytest

from oracle import attn_ref as R
from oracle import latent_ref as L


def test_frequencies():
    f = L.frequencies(64)
    assert f[0] == 1.0 and np.allclose(f[1:] / f[:-1], 10000.0 ** (-2 / 64))
    assert np.allclose(L.frequencies(64, scaling="LINEAR", factor=4.0), f / 4)
    b = L.frequencies(64, scaling="BASE", factor=4.0)
    assert b[0] == f[0] and np.isclose(b[-1], f[-1] / 4)
    t = L.frequencies(64, scaling="TURNS", factor=4.0, trained_len=1000, turns=(1.0, 8.0))
    turns = 1000 * f / (2 * np.pi)
    assert np.array_equal(t[turns >= 8], f[turns >= 8])
    assert np.allclose(t[turns <= 1], f[turns <= 1] / 4)
    mid = (turns > 1) & (turns < 8)
    assert mid.any() and (t[mid] > f[mid] / 4).all() and (t[mid] < f[mid]).all()


def test_linear_scaling_reads_positions_between():
    """Positions 4 times as far with a factor of 4 are the unscaled ones."""
    a = L.rope_table(40, L.frequencies(32, scaling="LINEAR", factor=4.0))
    b = L.rope_table(10, L.frequencies(32))
    assert np.allclose(a[0][::4], b[0]) and np.allclose(a[1][::4], b[1])


@pytest.mark.parametrize("interleaved", [False, True])
def test_turn_keeps_norms_and_depends_on_distance(interleaved):
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((2, 1, 1, 48))
    cos, sin = L.rope_table(200, L.frequencies(32))

    def at(x, p, inverse=False):
        return L.turn(x, cos[[p]], sin[[p]], 8, interleaved, inverse)

    assert np.allclose(np.linalg.norm(at(q, 77)), np.linalg.norm(q))
    assert np.array_equal(at(q, 77)[..., :8], q[..., :8])
    assert np.array_equal(at(q, 77)[..., 40:], q[..., 40:])
    assert np.allclose((at(q, 9) * at(k, 4)).sum(), (at(q, 105) * at(k, 100)).sum())
    assert np.allclose(at(at(q, 77), 77, True), q)


def test_gradients_against_differences():
    rng = np.random.default_rng(2)
    T, H, d_n, d_r, d_v = 3, 2, 4, 8, 4
    cos, sin = L.rope_table(T, L.frequencies(d_r))
    kv, pe = rng.standard_normal((T, H, d_n + d_v)), rng.standard_normal((T, d_r))
    wk, wv = rng.standard_normal((T, H, d_n + d_r)), rng.standard_normal((T, H, d_v))

    def loss(kv, pe):
        k, v = L.expand(kv, pe, cos, sin, d_n)
        return (wk * k).sum() + (wv * v).sum()

    gkv, gpe = L.expand_bwd(wk, wv, cos, sin, d_n)
    for x, g, f in ((kv, gkv, lambda y: loss(y, pe)), (pe, gpe, lambda y: loss(kv, y))):
        for idx in np.ndindex(x.shape):
            e = np.zeros_like(x)
            e[idx] = 1e-3
            assert abs((f(x + e) - f(x - e)) / 2e-3 - g[idx]) < 1e-9


def test_absorbed_equals_expanded():
    """The same attention with the up-projections taken into queries and outputs,
    through the oracle of the dense attention."""
    rng = np.random.default_rng(3)
    T, n, H, d_c, d_n, d_r, d_v = 20, 6, 3, 16, 8, 4, 8
    W_k, W_v = rng.standard_normal((H, d_c, d_n)), rng.standard_normal((H, d_c, d_v))
    c, pe = rng.standard_normal((T, d_c)), rng.standard_normal((T, d_r))
    q_n, q_r = rng.standard_normal((n, H, d_n)), rng.standard_normal((n, H, d_r))
    cos, sin = L.rope_table(T, L.frequencies(d_r))
    kv = np.concatenate([np.einsum("tc,hcn->thn", c, W_k), np.einsum("tc,hcv->thv", c, W_v)], -1)
    k, v = L.expand(kv, pe, cos, sin, d_n)
    q_rot = L.turn(q_r, cos[-n:], sin[-n:])
    qi, qp = R.dense_metadata(1, n)
    ki, kp = R.dense_metadata(1, T)
    ro, rl = R.attention_forward(np.concatenate([q_n, q_rot], -1)[None], k[None], v[None], qi, qp,
                                 ki, kp, R.Window(None, 0, T - n), 0.3)
    rows = np.concatenate([c, L.turn(pe[:, None], cos, sin)[:, 0]], 1)
    q = np.concatenate([np.einsum("thn,hcn->thc", q_n, W_k), q_rot], -1)
    o, lse, _, _ = L.attend(q, lambda s: rows, d_c, [T], [0, n], 0.3)
    assert np.allclose(np.einsum("thc,hcv->thv", o, W_v), ro[0]) and np.allclose(lse, rl[0])
