"""Page scales at the ends of their range: pages of zeros (whose scale is the
smallest an append writes) under queries of zeros and near it, V scales down to
zero and far apart."""
import numpy as np
import pytest
import torch

from bwd_tcgen05_tma_gb300 import inputs as I
from paged_util import Paged, check_attend

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bwd_tcgen05_tma_gb300 import build

    build.build()


@pytest.mark.parametrize("window", [None, 20])
@pytest.mark.parametrize("q_size", [0.0, 2.0 ** -120, 2.0 ** -90, 2.0 ** -20])
@pytest.mark.parametrize("new", [[3, 1], [20, 70], [300, 129]])
def test_zero_keys_give_the_mean_of_the_values(new, q_size, window):
    """Scores are exactly 0, whatever the queries are: O is the mean of the
    values that the mask keeps and LSE the logarithm of their number."""
    from bwd_tcgen05_tma_gb300 import attn as A

    c = Paged(new, [0] * len(new), seed=61)
    c.k_new[:] = 0
    c.q = I.round_to(c.q * q_size, "bf16").astype(np.float64)
    c.t["k_new"].zero_()
    c.t["q"].copy_(torch.from_numpy(c.q))
    A.attn_paged_append(c.params())
    o, lse = c.attend(c.params(q_rot=None, window_left=window))
    assert c.status() == 0
    check_attend(c, o, lse, c.oracle_attend(c.q, window=-1 if window is None else window))


@pytest.mark.parametrize("new,one", [([1], True), ([40], False)])
def test_smallest_value_scales(new, one):
    """V scales below 2^-80 are read as 2^-80: weights and LSE stay right over a
    long context, and no value exceeds 448 times its scale."""
    from bwd_tcgen05_tma_gb300 import attn as A

    c = Paged(new, [20000], seed=62, one=one, Hq=8, Hkv=1, d_qk=64, d_v=64, page=64)
    A.attn_paged_append(c.params())
    c.t["k_scale"].fill_(2.0 ** -30)  # weights within 2^-10 of one another
    for scale in (0.0, 2.0 ** -140, 2.0 ** -101, 2.0 ** -80, 2.0 ** -64):
        c.t["v_scale"].fill_(scale)
        o, lse = c.attend(c.params(q_rot=None))
        assert c.status() == 0
        _, rl, _, rD = c.oracle_attend(c.q)
        assert o.abs().max().item() <= 448 * max(scale, 2.0 ** -80)
        # as in check_attend
        tol = (c.d_qk + 16) * 2.0 ** -24 * rD.T + 2.0 ** -20 * (1 + np.abs(rl))
        assert (np.abs(lse.double().cpu().numpy() - rl) <= tol).all()


@pytest.mark.parametrize("new", [[1, 1], [1, 4], [4, 60], [200, 17]])
def test_value_scales_far_apart(new):
    """V scales that are no powers of two, spread over 2^85, and one page of
    each sequence at zero.  Beyond check_attend's terms: a score and its scale's
    logarithm are added, and the maximum taken off, at magnitudes below 128 (two
    roundings of 2^-18), and the logarithm itself is good to 2^-18 there; the
    three move P and the normaliser by at most 2^-16 relatively (LSE: twice,
    once for itself and once for what P loses against it)."""
    from bwd_tcgen05_tma_gb300 import attn as A

    c = Paged(new, [200, 300], seed=63)
    A.attn_paged_append(c.params())
    rng = np.random.default_rng(8)
    for name, lo, hi in (("k_scale", -9, -5), ("v_scale", -60, 25)):
        s = np.exp2(rng.uniform(lo, hi, tuple(c.t[name].shape))).astype(np.float32)
        c.t[name].copy_(torch.from_numpy(s))
    for s in range(2):
        c.t["v_scale"][int(c.table[s, 3])] = 0.0
    o, lse = c.attend(c.params(q_rot=None))
    assert c.status() == 0
    ro, rl, rA, rD = c.oracle_attend(c.q)
    got, gl = o.double().cpu().numpy(), lse.double().cpu().numpy()
    delta = (c.d_qk + 16) * 2.0 ** -24 * rD
    more = 2.0 ** -16
    tol = 2.0 ** -8 * np.abs(ro) + (2.0 ** -11 + 2.0 ** -17 + 2 * delta[..., None] + 2 * more) * (
        rA * (1 + 2.0 ** -8)) + 1e-7
    assert (np.abs(got - ro) <= tol).all()
    assert (np.abs(gl - rl) <= delta.T + 2.0 ** -20 * (1 + np.abs(rl)) + 2 * more).all()
