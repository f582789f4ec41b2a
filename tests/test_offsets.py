"""Offsets in the calls that look a token's place up."""
import numpy as np
import pytest
import torch

from bwd_tcgen05_tma_gb300 import attn as A
from latent_util import turn_tolerance
from oracle import latent_ref as L
from test_rope import angles, draw, tables

pytestmark = pytest.mark.gpu

T = 10
I32 = dict(dtype=torch.int32, device="cuda")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bwd_tcgen05_tma_gb300 import build

    build.build()


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
