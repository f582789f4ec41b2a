"""The absorbed attention where the work is cut otherwise than usual: scores of
-inf in pieces of their own, values that are not finite behind long contexts, many
sequences with long runs of empty ones, and pieces that take seconds."""
import numpy as np
import pytest
import torch

from bwd_tcgen05_tma_gb300 import attn as A
from latent_util import SCALE, Latent
from paged_util import check_attend

pytestmark = pytest.mark.gpu

I32 = dict(dtype=torch.int32, device="cuda")


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


# ------------------------------------------------- long contexts

class Aliased:
    """Contexts of any length over few pages: the table of every sequence lists the
    same pages over and over, its last page apart (its own)."""

    def __init__(self, seqs, new, ctx, *, seed, H=16, d_c=512, page=256, pages=8):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def randn(*shape):
            return torch.randn(*shape, generator=g, device="cuda").bfloat16()

        assert ctx % page == 0
        own = -(-new // page)
        cols = ctx // page + own
        self.cache = randn(pages + seqs * own, page, d_c + 64)
        self.table = (torch.arange(cols, **I32) % pages).repeat(seqs, 1)
        self.table[:, cols - own:] = pages + torch.arange(seqs * own, **I32).view(seqs, own)
        self.T, self.H, self.new = seqs * new, H, new
        q_lat, q_rot = randn(self.T, H, d_c), randn(self.T, H, 64)
        self.status = torch.zeros(1, **I32)
        self.p = A.make_latent_params(
            dtype="bf16", cache=self.cache, d_c=d_c, page_table=self.table,
            seq_lens=torch.full((seqs,), ctx + new, **I32), q_lat=q_lat, q_rot=q_rot,
            cu_seqlens_q=torch.arange(0, self.T + 1, new, **I32), max_q_len=new, scale=SCALE,
            status=self.status)
        self.ws = torch.empty(A.attn_latent_workspace_size(self.p), dtype=torch.uint8,
                              device="cuda")
        self.d_c = d_c

    def attend(self):
        o = torch.full((self.T, self.H, self.d_c), float("nan"), dtype=torch.bfloat16,
                       device="cuda")
        lse = torch.full((self.H, self.T), float("nan"), device="cuda")
        A.attn_latent_fwd(self.p, o, lse, self.ws)
        torch.cuda.synchronize()
        return o, lse


def test_nan_behind_a_long_context():
    """A chunk of 700 tokens behind 4 M keys.  The 303rd, the third of the four in its
    block of rows, is NaN: the rows that keep it are NaN, those before it have the
    bits that they have without it, and their block's epilogue does not go through
    all its keys for it (which took seconds, past the limit of the waits)."""
    c = Aliased(1, 700, 1 << 22, seed=97)
    ref, ref_lse = c.attend()
    assert c.status.item() == 0
    c.cache[c.table[0, -2], 302 - 256, 3] = float("nan")
    o, lse = c.attend()
    assert c.status.item() == 0
    assert torch.isnan(o[302:]).all() and torch.isnan(lse[:, 302:]).all()
    assert torch.equal(bits(o[:302]), bits(ref[:302]))
    assert torch.equal(bits(lse[:, :302]), bits(ref_lse[:, :302]))


def test_pieces_that_take_longer_than_a_wait():
    """160 contexts of 140 M keys: a block works on one of them for some 3 s, which
    is no failure."""
    c = Aliased(160, 1, 550000 * 256, seed=98, H=64, pages=64)
    o, lse = c.attend()
    assert c.status.item() == 0
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()


# ------------------------------------------------- many sequences

@pytest.mark.parametrize("H", [2, 40])
@pytest.mark.parametrize("kind", ["spread", "runs"])
def test_thousands_of_sequences(kind, H):
    """Several sequences for every thread that sums their work, empty ones among them
    one by one or in long runs, and a prompt of many row blocks."""
    n = 5000
    if kind == "spread":
        new = [1 if i % 7 == 3 else 2 if i % 41 == 0 else 0 for i in range(n)]
    else:
        new = [1 if i // 600 % 2 else 0 for i in range(n)]
    new[2345] = 150
    ctx = [(i * 7) % 90 if new[i] else 0 for i in range(n)]
    c = Latent(new, ctx, seed=99, H=H, d_c=256, page=16)
    o, lse = c.append_and_attend()
    assert c.status() == 0
    check_attend(c, o, lse, c.oracle_attend())


def test_a_long_run_of_empty_sequences():
    """Two prompts with 2^25 empty sequences between them: the block that goes from
    one to the other finds it without a look at each (which took it past the limit
    of the waits)."""
    gap = 1 << 25
    c = Latent([400, 250], [0, 30], seed=100, H=16, d_c=256, page=256)
    ref = c.append_and_attend()
    check_attend(c, *ref, c.oracle_attend())
    cols = c.table.shape[1]
    table = torch.full((gap + 2, cols), 2 ** 31 - 1, **I32)
    lens = torch.full((gap + 2,), 5, **I32)
    cu = torch.full((gap + 3,), 400, **I32)
    cu[0], cu[-1] = 0, 650
    for at, s in ((0, 0), (-1, 1)):
        table[at] = c.t["table"][s]
        lens[at] = c.lens[s]
    o, lse = c.attend(c.params(page_table=table, seq_lens=lens, cu_seqlens_q=cu))
    assert c.status() == 0
    check_attend(c, o, lse, c.oracle_attend())
