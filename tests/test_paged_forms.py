"""Forms of the paged calls that the header allows beside the usual ones: head
widths in every pair, padded batches of chunks, offsets that start behind row
0, outputs aligned to 16 bytes only, calls without LSE, many sequences, empty
pools and tables."""
import numpy as np
import pytest
import torch

from bwd_tcgen05_tma_gb300 import attn as A
from paged_util import Paged, check_attend

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bwd_tcgen05_tma_gb300 import build

    build.build()


def bits(t):
    return t.contiguous().view(torch.uint8)


def attend_and_check(c, sink=None, **kw):
    A.attn_paged_append(c.params())
    s = None if sink is None else torch.from_numpy(sink).float().cuda()
    o, lse = c.attend(c.params(q_rot=None, sink=s, **kw))
    assert c.status() == 0
    check_attend(c, o, lse, c.oracle_attend(c.q, sink=sink))
    return o, lse


@pytest.mark.parametrize("kind", ["e4m3", "bf16", "fp16"])
@pytest.mark.parametrize("d_qk,d_v", [(64, 64), (64, 128), (128, 64), (128, 128), (192, 64),
                                      (192, 128)])
@pytest.mark.parametrize("new", [1, 3, 5, 70])
def test_head_widths(new, d_qk, d_v, kind):
    """8, 16, 24 (of two heads' groups of 4 and 5 tokens: 20) and many rows."""
    types = {"e4m3": {}, "bf16": dict(cache="bf16"), "fp16": dict(cache="fp16", dtype="fp16")}
    c = Paged([new, 1], [150, 33], seed=91, Hq=8, Hkv=2, d_qk=d_qk, d_v=d_v, **types[kind])
    attend_and_check(c)


@pytest.mark.parametrize("cache", ["fp8_e4m3", "bf16"])
@pytest.mark.parametrize("name,kw", [
    ("decode", dict(new=[1, 1], ctx=[600, 20], one=True)),
    ("chunk", dict(new=[70, 33], ctx=[900, 300])),
    ("padded_chunk", dict(new=[70, 0, 33], ctx=[900, 30, 300], pad=40)),
])
def test_outputs_aligned_to_16_bytes_and_no_lse(name, kw, cache):
    c = Paged(seed=92, Hq=4, Hkv=1, cache=cache, **kw)
    o, _ = attend_and_check(c, sink=np.array([0.5, -3.0, 8.0, 0.0]))
    p = c.params(q_rot=None, sink=torch.tensor([0.5, -3.0, 8.0, 0.0], device="cuda"))
    ws = torch.empty(A.attn_paged_workspace_size(p), dtype=torch.uint8, device="cuda")
    room = torch.full((o.numel() + 16,), float("nan"), dtype=o.dtype, device="cuda")
    shifted = room[8:8 + o.numel()].view(o.shape)
    assert shifted.data_ptr() % 32 == 16
    A.attn_paged_fwd(p, shifted, None, ws)
    assert torch.equal(bits(shifted), bits(o))
    assert torch.isnan(room[:8]).all() and torch.isnan(room[-8:]).all()


@pytest.mark.parametrize("cache", ["fp8_e4m3", "bf16"])
def test_many_sequences_in_the_many_row_kernel(cache):
    c = Paged([i % 4 for i in range(1100)], [(i * 7) % 50 for i in range(1100)], seed=93, Hq=2,
              Hkv=1, d_qk=64, d_v=64, cache=cache)
    attend_and_check(c, max_q_len=5000)


@pytest.mark.parametrize("cache", ["fp8_e4m3", "bf16"])
@pytest.mark.parametrize("new", [2, 60])
def test_offsets_that_start_behind_row_0(new, cache):
    """The calls of a batch without its first sequence leave that one's rows and
    pages alone and give the others' bits."""
    whole, part = (Paged([3, new, 1], [40, 200, 7], seed=94, cache=cache) for _ in range(2))
    A.attn_paged_append(whole.params())
    o, lse = whole.attend(whole.params(q_rot=None))
    keep = {n: part.t[n].clone() for n in ("k_cache", "v_cache")}
    t = part.t
    kw = dict(page_table=t["table"][1:], seq_lens=t["lens"][1:], cu_seqlens_q=t["cu"][1:])
    A.attn_paged_append(part.params(**kw))
    o2, lse2 = part.attend(part.params(q_rot=None, **kw))
    assert whole.status() == 0 and part.status() == 0
    assert torch.isnan(o2[:3]).all() and torch.isnan(lse2[:, :3]).all()
    assert torch.isnan(t["q_rot"][:3]).all()
    assert torch.equal(bits(t["q_rot"][3:]), bits(whole.t["q_rot"][3:]))
    first = part.table[0, :3].tolist()
    for n, x in keep.items():
        others = [i for i in range(x.shape[0]) if i not in first]
        assert torch.equal(bits(t[n])[first], bits(x)[first])
        assert torch.equal(bits(t[n])[others], bits(whole.t[n])[others])
    # shares are cut elsewhere, so sums may be in another order
    ref = whole.oracle_attend(whole.q)
    got, gl = o2[3:].double().cpu().numpy(), lse2[:, 3:].double().cpu().numpy()
    u_p = 2.0 ** -8 if cache == "bf16" else 2.0 ** -11
    delta = (128 + 16) * 2.0 ** -24 * ref[3][3:]
    tol = 2.0 ** -8 * np.abs(ref[0][3:]) + (u_p + 2.0 ** -17 + 2 * delta[..., None]) * (
        ref[2][3:] * (1 + 2.0 ** -8)) + 1e-7
    assert (np.abs(got - ref[0][3:]) <= tol).all()
    assert (np.abs(gl - ref[1][:, 3:]) <= delta.T + 2.0 ** -20 * (1 + np.abs(ref[1][:, 3:]))).all()


@pytest.mark.parametrize("cache", ["fp8_e4m3", "bf16"])
@pytest.mark.parametrize("new", [1, 80])
@pytest.mark.parametrize("what", ["pool", "table"])
def test_empty_pool_or_table(what, new, cache):
    """Nothing can be kept: O = 0, LSE = -inf, reported; nothing is appended."""
    c = Paged([new, new], [30, 0], seed=95, cache=cache)
    t = c.t
    if what == "pool":
        for n in ("k_cache", "v_cache", "k_scale", "v_scale"):
            t[n] = None if t[n] is None else t[n][:0]
    else:
        keep = {n: t[n].clone() for n in ("k_cache", "v_cache")}
        t["table"] = t["table"][:, :0]
    A.attn_paged_append(c.params())
    assert c.status() == 7
    t["status"].zero_()
    o, lse = c.attend(c.params(q_rot=None))
    assert c.status() == 7
    assert (o == 0).all() and (lse == -np.inf).all()
    if what == "table":
        assert all(torch.equal(bits(t[n]), bits(x)) for n, x in keep.items())
    t["status"].zero_()
    t["lens"].zero_()
    o, lse = c.attend(c.params(q_rot=None))
    assert c.status() == 0
    assert (o == 0).all() and (lse == -np.inf).all()


@pytest.mark.parametrize("cache", ["fp8_e4m3", "bf16"])
@pytest.mark.parametrize("new", [1, 20, 100])
def test_pool_of_one_page(new, cache):
    c = Paged([new], [0], seed=96, page=128, spare=0, cache=cache)
    assert c.t["k_cache"].shape[0] == 1
    attend_and_check(c)
