"""The absorbed attention where the work is cut otherwise than usual: scores of
-inf in pieces of their own."""
import numpy as np
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


# ------------------------------------------------- scores of -inf

@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("H", [16, 32, 64, 128])
@pytest.mark.parametrize("ctx", [256, 64, 0])
def test_infinite_key_in_a_piece_of_its_own(ctx, H, dtype):
    """The last key's latent part holds +inf: rows whose score it makes -inf keep
    the other keys' weights, and NaN (0 * inf) in that coordinate, whether the key
    shares its tile, its piece or nothing with the others."""
    c = Latent([1], [max(ctx, 1)], seed=95, H=H, dtype=dtype)
    A.attn_latent_append(c.params())
    last = c.lens[0] - 1
    ref, ref_lse = c.attend(c.params())
    c.t["cache"][int(c.table[0, last // 64]), last % 64, 9] = float("inf")
    o, lse = c.attend(c.params())
    down = c.t["q_lat"][..., 9].float() < 0
    assert down.any() and (~down).any()
    assert torch.isnan(o[~down]).all() and torch.isnan(lse.t()[~down]).all()
    got = o[down]
    assert torch.isfinite(lse.t()[down]).all()
    assert torch.isnan(got[:, 9]).all()
    assert torch.isfinite(torch.cat([got[:, :9], got[:, 10:]], 1)).all()
    assert c.status() == 0


@pytest.mark.parametrize("sink", [False, True])
@pytest.mark.parametrize("H", [16, 64, 128])
@pytest.mark.parametrize("new,ctx", [(2, 0), (3, 0), (2, 257)])
def test_rows_whose_scores_are_all_minus_infinity(new, ctx, H, sink):
    """Every key holds +inf in its latent part and every query a negative number
    there: no score is above -inf, so O = 0 and LSE = -inf (the sink), also for
    rows that keep a key that others mask."""
    c = Latent([new], [ctx], seed=96, H=H)
    A.attn_latent_append(c.params())
    for j in range(c.lens[0]):
        c.t["cache"][int(c.table[0, j // 64]), j % 64, 9] = float("inf")
    c.t["q_lat"][..., 9] = -1.0
    s = torch.linspace(-1, 2, H, device="cuda") if sink else None
    o, lse = c.attend(c.params(sink=s))
    assert (o == 0).all()
    want = s[:, None].expand(-1, new) if sink else torch.full_like(lse, -np.inf)
    assert torch.equal(lse, want)
    assert c.status() == 0
