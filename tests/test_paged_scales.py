"""Page scales at the ends of their range: pages of zeros (whose scale is the
smallest there is) under queries of zeros and near it."""
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
