"""Bounds of the paged calls' sizes that are checked on the host (nothing is
launched)."""
import pytest

from bwd_tcgen05_tma_gb300 import attn as A
from test_paged_abi import FAKE, UNSUPPORTED, append, fwd, params, size


@pytest.fixture(scope="module")
def lib():
    from bwd_tcgen05_tma_gb300 import build

    build.build()
    return A.load_library()


def test_sequences_beyond_32_bits_of_work(lib):
    """Offsets allow more sequences than tokens: their number is bounded by itself."""
    for n in ((1 << 30) + 1, (1 << 31) - 1):
        p = params(num_seqs=n, cu_seqlens_q=FAKE)
        assert size(lib, p) == 0
        assert append(lib, p) == UNSUPPORTED
        assert fwd(lib, p) == UNSUPPORTED
    assert size(lib, params(num_seqs=1 << 30, cu_seqlens_q=FAKE)) > 0
