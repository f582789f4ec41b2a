"""Scores that are NaN (a NaN in a query or in a kept key) make O and LSE of
their rows NaN in both kernels, however the keys are shared out, and change no
bit of any other row."""
import numpy as np
import pytest
import torch

from paged_util import Paged

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bwd_tcgen05_tma_gb300 import build

    build.build()


def bits(t):
    return t.contiguous().view(torch.uint8)


def only_hit_rows_are_nan(c, p, hit, before):
    """hit: bool [tokens, Hq].  before: O and LSE of the same call without the
    NaN."""
    o, lse = c.attend(p)
    assert c.status() == 0
    hit = torch.from_numpy(hit).cuda()
    assert hit.any() and torch.isnan(o[hit]).all() and torch.isnan(lse.t()[hit]).all()
    assert torch.equal(bits(o[~hit]), bits(before[0][~hit]))
    assert torch.equal(bits(lse.t()[~hit]), bits(before[1].t()[~hit]))


# new, ctx: one block's whole item, items cut into pieces, warps that take items
# alone; the same of the many-row kernel
BATCHES = {
    "shared": dict(new=[1] * 4, ctx=[0, 15, 40, 127], one=True),
    "split": dict(new=[1, 1], ctx=[3000, 700], one=True),
    "solo": dict(new=[1] * 700, ctx=[33 + i % 16 for i in range(700)], one=True, Hq=16, Hkv=4,
                 d_qk=64, d_v=64),
    "rows24": dict(new=[5, 4], ctx=[90, 300], Hq=8, Hkv=2),
    "chunk": dict(new=[40, 70], ctx=[3, 100]),
    "chunk_split": dict(new=[140, 33], ctx=[2500, 700], Hq=4, Hkv=1, page=64),
}
TYPES = {"e4m3": {}, "bf16": dict(cache="bf16"), "fp16": dict(cache="fp16", dtype="fp16")}


@pytest.mark.parametrize("sink", [False, True])
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("name", list(BATCHES))
def test_nan_in_queries(name, kind, sink):
    from bwd_tcgen05_tma_gb300 import attn as A

    c = Paged(seed=51, **BATCHES[name], **TYPES[kind])
    A.attn_paged_append(c.params())
    s = torch.linspace(-1, 2, c.Hq, device="cuda") if sink else None
    p = c.params(q_rot=None, sink=s)
    before = c.attend(p)
    hit = np.zeros((c.T, c.Hq), bool)
    for row, head, dim in ((0, 1, 0), (c.T - 1, c.Hq - 1, c.d_qk - 1), (c.T // 2, 0, 17)):
        c.t["q"][row, head, dim] = float("nan")
        hit[row, head] = True
    only_hit_rows_are_nan(c, p, hit, before)


@pytest.mark.parametrize("sink", [False, True])
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("name", list(BATCHES))
def test_nan_in_the_newest_key(name, kind, sink):
    """The rows that keep the key are those of its KV head's last token."""
    from bwd_tcgen05_tma_gb300 import attn as A

    c = Paged(seed=52, **BATCHES[name], **TYPES[kind])
    A.attn_paged_append(c.params())
    s = torch.linspace(-1, 2, c.Hq, device="cuda") if sink else None
    p = c.params(q_rot=None, sink=s)
    before = c.attend(p)
    hit = np.zeros((c.T, c.Hq), bool)
    group = c.Hq // c.Hkv
    k = c.t["k_cache"].view(torch.uint8 if kind == "e4m3" else torch.int16)
    for i in range(0, len(c.lens), max(1, len(c.lens) // 4)):
        j, head = c.lens[i] - 1, i % c.Hkv
        k[int(c.table[i, j // c.page]), head, j % c.page, 3] = 0x7F if kind == "e4m3" else 0x7FFF
        hit[c.cu[i + 1] - 1, head * group:(head + 1) * group] = True
    only_hit_rows_are_nan(c, p, hit, before)


@pytest.mark.parametrize("cache", ["fp8_e4m3", "bf16"])
@pytest.mark.parametrize("length", [1, 16, 17, 33, 64, 97, 113, 129, 257])
def test_nan_key_alone_in_a_share(length, cache):
    """One sequence: the newest key stands alone in a warp's, a block's or a
    piece's share at some of these lengths."""
    from bwd_tcgen05_tma_gb300 import attn as A

    c = Paged([1], [length - 1], seed=53, cache=cache, one=True)
    A.attn_paged_append(c.params())
    p = c.params(q_rot=None)
    before = c.attend(p)
    k = c.t["k_cache"].view(torch.uint8 if cache == "fp8_e4m3" else torch.int16)
    j = length - 1
    k[int(c.table[0, j // 16]), 1, j % 16, 100] = 0x7F if cache == "fp8_e4m3" else 0x7FFF
    hit = np.zeros((1, 4), bool)
    hit[0, 2:] = True
    only_hit_rows_are_nan(c, p, hit, before)


@pytest.mark.parametrize("cache", ["fp8_e4m3", "bf16"])
@pytest.mark.parametrize("new", [4, 100])
def test_nan_in_the_only_key(new, cache):
    """A window of 0: every row keeps its own key and no other."""
    from bwd_tcgen05_tma_gb300 import attn as A

    c = Paged([new, new], [0, 200], seed=54, cache=cache)
    A.attn_paged_append(c.params())
    p = c.params(q_rot=None, window_left=0)
    before = c.attend(p)
    k = c.t["k_cache"].view(torch.uint8 if cache == "fp8_e4m3" else torch.int16)
    hit = np.zeros((2 * new, 4), bool)
    for s, first in ((0, 0), (1, 200)):
        for i in (0, new // 2, new - 1):
            j = first + i
            k[int(c.table[s, j // 16]), 0, j % 16, 64] = 0x7F if cache == "fp8_e4m3" else 0x7FFF
            hit[s * new + i, :2] = True
    only_hit_rows_are_nan(c, p, hit, before)


@pytest.mark.parametrize("cache", ["fp8_e4m3", "bf16"])
@pytest.mark.parametrize("new", [1, 4, 80])
def test_nan_value_beside_a_page_that_is_none(new, cache):
    """A value that is NaN reaches the rows that keep it also where another page
    of its 128 tokens is masked for its id."""
    from bwd_tcgen05_tma_gb300 import attn as A

    c = Paged([new], [300], seed=55, cache=cache)
    A.attn_paged_append(c.params())
    c.t["table"][0, 2] = -1
    p = c.params(q_rot=None)
    ref, ref_lse = c.attend(p)
    assert c.status() == 7
    v = c.t["v_cache"].view(torch.uint8 if cache == "fp8_e4m3" else torch.int16)
    v[int(c.table[0, 0]), 1, 5, 9] = 0x7F if cache == "fp8_e4m3" else 0x7FC0
    o, lse = c.attend(p)
    assert torch.equal(bits(lse), bits(ref_lse))
    got, want = o.float().cpu(), ref.float().cpu()
    assert torch.isnan(got[:, 2:, 9]).all()
    want[:, 2:, 9] = got[:, 2:, 9]
    assert torch.equal(bits(got), bits(want))
