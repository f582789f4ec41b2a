"""What a call reports in its status word and what it refuses."""
import numpy as np
import pytest
import torch

from bwd_tcgen05_tma_gb300 import attn as A
from paged_util import Paged


def bits(t):
    return t.contiguous().view(torch.uint8)


@pytest.mark.gpu
@pytest.mark.parametrize("mask", ["CAUSAL", "NONE"])
@pytest.mark.parametrize("new", [4, 80])
def test_attention_reports_positions_below_zero(new, mask):
    """Fewer tokens than new ones: the first rows stand below position 0.  The
    call says so; they keep no key under a causal mask, and the other rows are
    right.  A sequence of length 0 is padding and no such case."""
    from bwd_tcgen05_tma_gb300 import build

    build.build()
    c = Paged([new, 3], [0, 20], seed=71)
    A.attn_paged_append(c.params())
    assert c.status() == 0
    short = new - new // 4
    p = c.params(q_rot=None, mask=mask)
    c.t["lens"][0] = 0
    c.attend(p)
    assert c.status() == 0
    ref, ref_lse = c.attend(p)
    c.t["lens"][0] = short
    o, lse = c.attend(p)
    assert c.status() == 7
    assert torch.equal(bits(o[new:]), bits(ref[new:]))
    assert torch.equal(bits(lse[:, new:]), bits(ref_lse[:, new:]))
    below = new - short
    if mask == "CAUSAL":
        assert (o[:below] == 0).all() and (lse[:, :below] == -np.inf).all()
    assert torch.isfinite(o[below:]).all() and torch.isfinite(lse[:, below:]).all()


def test_rotation_in_place_needs_one_layout():
    """q_rot == q with rows at other distances would overwrite queries that are
    still to be read: refused (on the host, nothing is launched)."""
    from bwd_tcgen05_tma_gb300 import build
    from test_paged_abi import INVALID, append, params, size

    build.build()
    lib = A.load_library()
    assert append(lib, params(q_rot_stride=8 * 128 + 8)) == INVALID
    assert append(lib, params(q_stride=8 * 128 + 64)) == INVALID
    assert size(lib, params(q_rot_stride=8 * 128 + 8)) > 0  # the attention reads q_rot only
