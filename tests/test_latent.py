"""The paged latent cache on the GPU against the float64 oracle: appending with
rotation, the absorbed attention over the pages, and both in turn as a decoder
runs them."""
import numpy as np
import pytest
import torch

from bwd_tcgen05_tma_gb300 import attn as A
from latent_util import SCALE, Latent, dev16, turn_tolerance, written_slots
from oracle import latent_ref as L
from oracle import paged_ref as P
from paged_util import UNIT, check_attend

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bwd_tcgen05_tma_gb300 import build

    build.build()


def bits(t):
    return t.contiguous().view(torch.uint8)


# ---------------------------------------------------------------- append

APPEND = {
    "decode": dict(new=[1] * 5, ctx=[0, 15, 16, 17, 63], one=True, page=16),
    "decode_offsets": dict(new=[1, 0, 1, 1], ctx=[31, 40, 0, 5], pad=3, H=7),
    "ragged": dict(new=[40, 0, 1, 17, 33], ctx=[0, 9, 16, 15, 3], pad=2, H=20, page=32),
    "one_head": dict(new=[1], ctx=[0], one=True, page=256, H=1),
    "d256_fp16": dict(new=[70, 3], ctx=[5, 64], d_c=256, dtype="fp16", interleaved=True),
    "interleaved": dict(new=[20, 3], ctx=[5, 16], interleaved=True, page=128),
    "fused_shifted": dict(new=[18, 2], ctx=[15, 16], fused=True, pos_shift=100, H=17),
    "wide_by_head": dict(new=[18, 2], ctx=[15, 16], layout="wide", by_head=True, H=33),
    "slots": dict(new=[18, 2], ctx=[15, 16], layout="slots", dtype="fp16"),
    "many_seqs": dict(new=[i % 3 for i in range(600)], ctx=[i % 7 for i in range(600)], H=2,
                      d_c=256, page=16),
}


def check_append(c):
    new = written_slots(c)
    got = c.cache_host()
    assert np.array_equal(got[~new], c.host[~new], equal_nan=True)
    pe, rq = c.rotated(c.k_rope[:, None])[:, 0], c.rotated(c.q_rope)
    for s, row, pos in P.new_rows(c.lens, c.cu):
        at = got[c.table[s, pos // c.page], pos % c.page]
        assert np.array_equal(at[:c.d_c], c.c_new[row])
        tol = turn_tolerance(pe[row], np.abs(c.k_rope[row]).max(), c.dtype)
        assert (np.abs(at[c.d_c:] - pe[row]) <= tol).all()
    q, n = c.t["q_rot"].double().cpu().numpy(), c.cu[-1]
    tol = turn_tolerance(rq, np.abs(c.q_rope).max(-1, keepdims=True), c.dtype)
    assert (np.abs(q - rq)[:n] <= tol[:n]).all()
    assert np.isnan(q[n:]).all()


@pytest.mark.parametrize("name", list(APPEND))
def test_append(name):
    c = Latent(seed=11, **APPEND[name])
    A.attn_latent_append(c.params())
    assert c.status() == 0
    check_append(c)


def test_append_in_place_and_without_queries():
    c, d = (Latent([5, 1], [3, 16], seed=12) for _ in range(2))
    c.t["q_rot"] = c.t["q_rope"]
    A.attn_latent_append(c.params())
    check_append(c)
    A.attn_latent_append(d.params(q_rope=None))
    torch.cuda.synchronize()
    assert torch.equal(bits(c.t["cache"]), bits(d.t["cache"]))
    assert torch.isnan(d.t["q_rot"]).all()


def test_append_copies_every_pattern():
    """The latent vector is copied, whatever its bits."""
    c = Latent([130], [0], seed=13)
    c.t["c_new"].view(torch.int16).copy_(
        (torch.arange(130 * 512, device="cuda") - 32768).to(torch.int16).view(130, 512))
    A.attn_latent_append(c.params())
    j = np.arange(130)
    got = c.t["cache"].view(torch.int16)[c.table[0, j // 64], j % 64]
    assert torch.equal(got[:, :512], c.t["c_new"].view(torch.int16))


def test_append_reports_and_skips():
    """Bad pages, rotation positions, lengths and offsets: reported, and nothing
    of the tokens concerned is written."""
    c = Latent([3, 1, 1, 2], [63, 0, 4, 1], seed=14)
    before = c.t["cache"].clone()
    c.t["table"][0, 1] = 99999
    c.t["table"][1, 0] = -1
    c.t["lens"][2] = -4
    A.attn_latent_append(c.params())
    assert c.status() == 7
    got = c.t["cache"]
    page0, page3 = int(c.table[0, 0]), int(c.table[3, 0])
    same = [i for i in range(got.shape[0]) if i not in (page0, page3)]
    assert torch.equal(bits(got)[same], bits(before)[same])
    assert torch.equal(got[page0, 63, :512], c.t["c_new"][0])
    # a query is left out for its sequence's length, not for its key's page
    q = c.t["q_rot"]
    assert torch.isfinite(q[:4]).all() and torch.isnan(q[4]).all() and torch.isfinite(q[5:]).all()

    d = Latent([2, 1], [3, 4], seed=15, pos_shift=0)
    d.t["pos"][0], d.t["pos"][2] = -1, 1 << 20
    before = d.t["cache"].clone()
    A.attn_latent_append(d.params())
    assert d.status() == 7
    assert torch.isnan(d.t["q_rot"][[0, 2]]).all() and torch.isfinite(d.t["q_rot"][1]).all()
    page = int(d.table[1, 0])
    assert torch.equal(bits(d.t["cache"])[page], bits(before)[page])

    e = Latent([2, 1], [3, 4], seed=16)
    e.t["cu"][1] = 50
    A.attn_latent_append(e.params())
    assert e.status() == 7
    assert torch.equal(bits(e.t["cache"]), bits(torch.from_numpy(e.host).cuda().bfloat16()))


# ---------------------------------------------------------------- attention

ATTEND = {
    "decode": dict(new=[1] * 4, ctx=[0, 15, 64, 700], one=True),
    "decode_one_head": dict(new=[1, 1], ctx=[200, 63], H=1, one=True),
    "decode_7": dict(new=[1, 1, 1], ctx=[64, 65, 127], H=7, page=16),
    "decode_20": dict(new=[1, 1, 1], ctx=[64, 65, 127], H=20, page=32, dtype="fp16"),
    "decode_33": dict(new=[1, 1], ctx=[190, 191], H=33, page=128),
    "decode_64": dict(new=[1, 1], ctx=[1000, 3], H=64, one=True),
    "decode_100": dict(new=[1, 1], ctx=[100, 600], H=100, page=256),
    "decode_128": dict(new=[1] * 6, ctx=[0, 63, 64, 500, 1300, 127], H=128, one=True),
    "decode_128_fp16": dict(new=[1, 1], ctx=[900, 10], H=128, d_c=256, dtype="fp16", page=16),
    "pairs_ragged": dict(new=[2, 1, 0, 5, 1], ctx=[700, 64, 9, 200, 1], H=50),
    "decode_256": dict(new=[1], ctx=[300], H=256, d_c=256, one=True),
    "one_token_total": dict(new=[1], ctx=[0], one=True),
    "verify": dict(new=[4, 1, 3, 2], ctx=[63, 0, 129, 62]),
    "verify_fp16": dict(new=[2, 2], ctx=[500, 61], dtype="fp16", interleaved=True),
    "d256": dict(new=[1, 1, 1], ctx=[5, 300, 1500], d_c=256, one=True),
    "d256_verify": dict(new=[3, 2], ctx=[64, 300], d_c=256, H=8, dtype="fp16"),
    "d256_chunk": dict(new=[70, 9], ctx=[64, 300], d_c=256, H=5),
    "chunk": dict(new=[70, 0, 33], ctx=[130, 7, 0], H=5, pad=3),
    "chunk_fp16": dict(new=[65], ctx=[100], H=4, dtype="fp16", page=16),
    "prompt": dict(new=[130], ctx=[0], H=2, page=32),
    "batch": dict(new=[1] * 64, ctx=[(i * i * 37) % 900 for i in range(64)], one=True),
    "batch_verify": dict(new=[2] * 40, ctx=[(i * i * 37) % 500 for i in range(40)]),
    "chunks": dict(new=[90, 100, 40], ctx=[500, 100, 900]),
    "wide": dict(new=[1, 5], ctx=[100, 200], layout="wide", H=12),
    "slots_by_head": dict(new=[1, 5], ctx=[100, 200], layout="slots", by_head=True, H=12),
    "fused": dict(new=[2, 5], ctx=[100, 200], fused=True, H=12),
    "many": dict(new=[i % 3 for i in range(500)], ctx=[(i * 7) % 90 for i in range(500)], H=2,
                 d_c=256, page=16),
    "small_values": dict(new=[1, 2], ctx=[100, 90], std=1e-3),
    "peaked": dict(new=[1, 2], ctx=[400, 90], std=4.0),
}


def attend_and_check(c, sink=None, **kw):
    s = None if sink is None else torch.from_numpy(sink).float().cuda()
    o, lse = c.append_and_attend(sink=s, **kw)
    assert c.status() == 0
    ok = {k: v for k, v in kw.items() if k != "max_q_len"}
    causal = ok.get("mask", "CAUSAL") == "CAUSAL"
    w = ok.get("window_left")
    check_attend(c, o, lse, c.oracle_attend(sink=sink, causal=causal, window=-1 if w is None else w))
    return o, lse


@pytest.mark.parametrize("name", list(ATTEND))
def test_attend(name):
    attend_and_check(Latent(seed=21, **ATTEND[name]))


@pytest.mark.parametrize("kw", [dict(mask="NONE"), dict(window_left=0), dict(window_left=20),
                                dict(mask="NONE", window_left=70), dict(window_left=1 << 30)])
@pytest.mark.parametrize("name", ["decode", "verify", "chunk", "d256_chunk", "decode_128"])
def test_attend_masks(name, kw):
    attend_and_check(Latent(seed=22, **ATTEND[name]), **kw)


@pytest.mark.parametrize("name", ["decode_7", "verify", "chunk", "decode_100", "decode_128"])
def test_attend_sink(name):
    c = Latent(seed=23, **ATTEND[name])
    attend_and_check(c, sink=np.random.default_rng(1).uniform(-3, 9, c.H).astype(np.float32))


@pytest.mark.parametrize("kw", [dict(), dict(window_left=100), dict(mask="NONE")])
@pytest.mark.parametrize("name", ["chunk", "chunks", "decode_256", "d256_chunk", "pairs_ragged"])
def test_attend_in_a_long_table(name, kw):
    """A table that could hold more than the L2 cache: blocks work in pairs on more
    than two row blocks of a sequence too, of which the last may be alone."""
    c = Latent(seed=42, **ATTEND[name])
    wide = torch.full((len(c.new), 4000), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    wide[:, :c.table.shape[1]] = c.t["table"]
    c.t["table"] = wide
    attend_and_check(c, **kw)


@pytest.mark.parametrize("hint", [1, 2, 3, 4, 5, 5000])
@pytest.mark.parametrize("name", ["decode_7", "chunk"])
def test_attend_any_length_hint(name, hint):
    attend_and_check(Latent(seed=24, **ATTEND[name]), max_q_len=hint)


@pytest.mark.parametrize("H", [16, 32, 64])
@pytest.mark.parametrize("length", [1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 191, 193, 450])
def test_attend_lengths(length, H):
    attend_and_check(Latent([1], [length - 1], seed=25, H=H, d_c=256 if length % 2 else 512,
                            one=True, page=16))


def test_attend_grows_its_maximum_late():
    """Keys whose scores rise from tile to tile, by more than the maximum may lag:
    O is rescaled many times."""
    c = Latent([1, 3], [900, 500], seed=26, H=32)
    for s in range(2):
        for j in range(c.ctx[s]):
            pid, slot = c.table[s, j // 64], j % 64
            c.t["cache"][int(pid), slot] *= 0.02 * (j // 64) ** 2
    attend_and_check(c)


def test_attend_without_lse_and_outputs_aligned_to_16_bytes():
    c = Latent([3, 1], [100, 700], seed=27)
    o, _ = attend_and_check(c)
    p = c.params()
    ws = torch.empty(A.attn_latent_workspace_size(p), dtype=torch.uint8, device="cuda")
    room = torch.full((o.numel() + 16,), float("nan"), dtype=o.dtype, device="cuda")
    shifted = room[8:8 + o.numel()].view(o.shape)
    assert shifted.data_ptr() % 32 == 16
    A.attn_latent_fwd(p, shifted, None, ws)
    assert torch.equal(bits(shifted), bits(o))
    assert torch.isnan(room[:8]).all() and torch.isnan(room[-8:]).all()


def test_shared_prefix_and_strided_table():
    """Two sequences whose first pages are the same, in a table with wider rows."""
    c = Latent([1, 1], [300, 300], seed=28, one=True)
    c.table[1, :4] = c.table[0, :4]
    wide = torch.full((2, 40), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    wide[:, :c.table.shape[1]] = torch.tensor(c.table, dtype=torch.int32)
    c.t["table"] = wide[:, :c.table.shape[1]]
    attend_and_check(c)


@pytest.mark.parametrize("new", [1, 3, 20])
def test_empty_sequences_and_windows(new):
    """Length 0 (padding rows) and rows before every key of their window."""
    c = Latent([new, new, new], [30, 0, 200], seed=29)
    A.attn_latent_append(c.params())
    c.t["lens"][1] = 0
    o, lse = c.attend(c.params())
    assert c.status() == 0
    assert (o[new:2 * new] == 0).all() and (lse[:, new:2 * new] == -np.inf).all()
    rest = [*range(new), *range(2 * new, 3 * new)]
    assert torch.isfinite(o[rest]).all() and torch.isfinite(lse[:, rest]).all()
    sink = torch.linspace(-2, 2, c.H, device="cuda")
    o2, lse2 = c.attend(c.params(sink=sink))
    assert (o2[new:2 * new] == 0).all()
    assert torch.equal(lse2[:, new:2 * new], sink[:, None].expand(-1, new))


@pytest.mark.parametrize("what", ["pool", "table"])
@pytest.mark.parametrize("new", [1, 80])
def test_empty_pool_or_table(what, new):
    """Nothing can be kept: O = 0, LSE = -inf, reported; nothing is appended."""
    c = Latent([new, new], [30, 0], seed=30, H=4)
    keep = c.t["cache"].clone()
    if what == "pool":
        c.t["cache"] = c.t["cache"][:0]
    else:
        c.t["table"] = c.t["table"][:, :0]
    A.attn_latent_append(c.params())
    assert c.status() == 7
    c.t["status"].zero_()
    c.t["q_rot"].zero_()
    o, lse = c.attend(c.params())
    assert c.status() == 7
    assert (o == 0).all() and (lse == -np.inf).all()
    if what == "table":
        assert torch.equal(bits(c.t["cache"]), bits(keep))


def test_lengths_behind_the_table_are_reported():
    c = Latent([1, 2], [70, 100], seed=31, page=16)
    attend_and_check(c)
    ref = c.attend(c.params())
    c.t["lens"][0] = c.table.shape[1] * 16 + 5
    o, lse = c.attend(c.params())
    assert c.status() == 7
    assert torch.equal(bits(o[1:]), bits(ref[0][1:]))
    assert torch.equal(bits(lse[:, 1:]), bits(ref[1][:, 1:]))


@pytest.mark.parametrize("H,new", [(16, 1), (16, 2), (16, 4), (3, 40), (128, 1)])
def test_attend_reports_bad_pages(H, new):
    """A page that is none counts as masked; the rest of its sequence, and the
    other sequences, are right."""
    c = Latent([new, new], [300, 200], seed=32, H=H, page=16)
    A.attn_latent_append(c.params())
    whole = c.table.copy()
    for bad in (-1, c.host.shape[0], 2 ** 31 - 1):
        c.t["status"].zero_()
        c.table = whole.copy()
        c.t["table"].copy_(torch.tensor(np.minimum(whole, 2 ** 31 - 1), dtype=torch.int32))
        for col in (0, 5, 6):
            c.t["table"][0, col] = bad
        o, lse = c.attend(c.params())
        assert c.status() == 7
        host = c.cache_host()

        def rows_of(s):
            j = np.arange(c.lens[s])
            if s == 0:
                j = j[~np.isin(j // 16, (0, 5, 6))]
            return host[whole[s, j // 16], j % 16]

        lens = [c.lens[0] - 48, c.lens[1]]
        check_attend(c, o, lse, L.attend(c.queries(), rows_of, c.d_c, lens, c.cu, SCALE))


def test_offsets_that_start_behind_row_0():
    """The calls of a batch without its first sequence leave that one's rows and
    pages alone."""
    c = Latent([3, 9, 1], [40, 200, 7], seed=44)
    t = c.t
    kw = dict(page_table=t["table"][1:], seq_lens=t["lens"][1:], cu_seqlens_q=t["cu"][1:])
    before = t["cache"].clone()
    A.attn_latent_append(c.params(**kw))
    o, lse = c.attend(c.params(**kw))
    assert c.status() == 0
    assert torch.isnan(o[:3]).all() and torch.isnan(lse[:, :3]).all()
    assert torch.isnan(t["q_rot"][:3]).all() and torch.isfinite(t["q_rot"][3:]).all()
    page = int(c.table[0, 0])
    assert torch.equal(bits(t["cache"])[page], bits(before)[page])
    ref = c.oracle_attend()
    rows = slice(3, 13)
    u = UNIT["bf16"]
    delta = (576 + 16) * 2.0 ** -24 * ref[3][rows]
    tol = u * np.abs(ref[0][rows]) + (u + 2.0 ** -17 + 2 * delta[..., None]) * (
        ref[2][rows] * (1 + u)) + 1e-7
    assert (np.abs(o.double().cpu().numpy()[rows] - ref[0][rows]) <= tol).all()


def test_offsets_out_of_range_are_reported():
    for bad in (-3, 1000):
        c = Latent([2, 1, 1], [30, 40, 50], seed=33)
        attend_and_check(c)
        ref = c.attend(c.params())
        c.t["cu"][1] = bad
        o, lse = c.attend(c.params())
        assert c.status() == 7
        assert torch.equal(bits(o[3:]), bits(ref[0][3:]))


def test_attention_reports_positions_below_zero():
    c = Latent([8, 3], [0, 20], seed=34)
    A.attn_latent_append(c.params())
    ref, _ = c.attend(c.params())
    assert c.status() == 0
    c.t["lens"][0] = 6
    o, lse = c.attend(c.params())
    assert c.status() == 7
    assert torch.equal(bits(o[8:]), bits(ref[8:]))
    assert (o[:2] == 0).all() and (lse[:, :2] == -np.inf).all()
    assert torch.isfinite(o[2:]).all()


# ------------------------------------------------- values that are not finite

@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("H,new", [(16, 1), (16, 2), (16, 4), (3, 40), (64, 1), (128, 1), (50, 4)])
def test_masked_values_have_no_influence(H, new, dtype):
    """NaN and infinities in slots behind a sequence's end, in front of every
    row's window, and in tokens that only later rows see."""
    c = Latent([new, new], [300, 100], seed=35, H=H, dtype=dtype)
    A.attn_latent_append(c.params())
    p = c.params(window_left=130)
    ref = c.attend(p)
    cache = c.t["cache"]
    for s in range(2):
        for j in range(0, max(0, c.ctx[s] - 130)):
            cache[int(c.table[s, j // 64]), j % 64] = float("nan") if j % 2 else float("inf")
        for j in range(c.lens[s], -(-c.lens[s] // 64) * 64):
            cache[int(c.table[s, j // 64]), j % 64] = float("-inf") if j % 2 else float("nan")
    got = c.attend(p)
    for a, b in zip(ref, got):
        assert torch.equal(bits(a), bits(b))
    if new > 1:  # the newest token: its own row keeps it, the others do not
        last = c.cu[1] - 1
        j = c.lens[0] - 1
        cache[int(c.table[0, j // 64]), j % 64, 3] = float("nan")
        cache[int(c.table[0, j // 64]), j % 64, c.d_c - 1] = float("inf")
        o, lse = c.attend(p)
        assert torch.isnan(o[last]).all() and torch.isnan(lse[:, last]).all()
        rest = [i for i in range(c.T) if i != last]
        assert torch.equal(bits(o[rest]), bits(ref[0][rest]))
        assert torch.equal(bits(lse.t()[rest]), bits(ref[1].t()[rest]))
    assert c.status() == 0


@pytest.mark.parametrize("sink", [False, True])
@pytest.mark.parametrize("name", ["decode", "verify", "chunk", "decode_64", "decode_128"])
def test_nan_in_queries(name, sink):
    c = Latent(seed=36, **ATTEND[name])
    A.attn_latent_append(c.params())
    p = c.params(sink=torch.linspace(-1, 2, c.H, device="cuda") if sink else None)
    before = c.attend(p)
    n = c.cu[-1]
    hit = torch.zeros(c.T, c.H, dtype=torch.bool, device="cuda")
    for row, head, part, dim in ((0, 1, "q_lat", 0), (n - 1, c.H - 1, "q_rot", 63),
                                 (n // 2, 0, "q_lat", c.d_c - 1)):
        c.t[part][row, head, dim] = float("nan")
        hit[row, head] = True
    o, lse = c.attend(p)
    assert c.status() == 0
    assert torch.isnan(o[hit]).all() and torch.isnan(lse.t()[hit]).all()
    assert torch.equal(bits(o[~hit]), bits(before[0][~hit]))
    assert torch.equal(bits(lse.t()[~hit]), bits(before[1].t()[~hit]))


@pytest.mark.parametrize("where", [0, 70, 299])
@pytest.mark.parametrize("new", [1, 4])
def test_kept_infinities(where, new):
    """An infinity in a kept key's shared part: scores of +inf and NaN make their
    rows NaN; scores of -inf take the key out.  In the latent part also its
    coordinate of O becomes NaN for rows that do keep it."""
    c = Latent([new], [300], seed=37)
    A.attn_latent_append(c.params())
    ref, ref_lse = c.attend(c.params())
    at = c.t["cache"][int(c.table[0, where // 64]), where % 64]
    for dim in (512 + 5, 9):
        old = at[dim].clone()
        at[dim] = float("inf")
        q = c.t["q_rot"][..., 5] if dim > 512 else c.t["q_lat"][..., 9]
        o, lse = c.attend(c.params())
        up = (q.float() >= 0)  # 0 * inf is NaN
        assert up.any() and (~up).any()
        assert torch.isnan(o[up]).all() and torch.isnan(lse.t()[up]).all()
        down = o[~up]
        assert torch.isfinite(lse.t()[~up]).all()
        if dim > 512:
            assert torch.isfinite(down).all()
        else:
            assert torch.isnan(down[:, 9]).all()
            assert torch.isfinite(torch.cat([down[:, :9], down[:, 10:]], 1)).all()
        at[dim] = old
    o, lse = c.attend(c.params())
    assert torch.equal(bits(o), bits(ref)) and torch.equal(bits(lse), bits(ref_lse))


def test_all_scores_minus_infinity():
    """No key whose score is above -inf: O = 0 in the coordinates that are finite,
    LSE = -inf."""
    c = Latent([1], [100], seed=38, one=True)
    A.attn_latent_append(c.params())
    c.t["q_rot"][0, :, 7] = -1.0
    for j in range(c.lens[0]):
        c.t["cache"][int(c.table[0, j // 64]), j % 64, 512 + 7] = float("inf")
    o, lse = c.attend(c.params())
    assert (o == 0).all() and (lse == -np.inf).all()
    sink = torch.linspace(-1, 1, 16, device="cuda")
    o, lse = c.attend(c.params(sink=sink))
    assert (o == 0).all() and torch.equal(lse[:, 0], sink)


# ---------------------------------------------------------------- addresses

def test_offsets_beyond_32_bits():
    """Pages and queries that lie more than 2^32 bytes apart."""
    far = (5 << 30) // 2
    c = Latent([1, 1], [60, 60], seed=39, H=16, spare=0)
    assert c.host.shape[0] == 2
    span = far + 64 * 576
    pool = torch.empty(span + (1 << 20), dtype=torch.bfloat16, device="cuda")
    cache = torch.as_strided(pool, (2, 64, 576), (far, 576, 1))
    cache.copy_(c.t["cache"])
    c.t["cache"] = cache
    qs = torch.empty(far + 16 * 512, dtype=torch.bfloat16, device="cuda")
    q = torch.as_strided(qs, (2, 16, 512), (far, 512, 1))
    q.copy_(c.t["q_lat"])
    c.t["q_lat"] = q
    attend_and_check(c)
    check_append(c)


@pytest.mark.parametrize("H", [16, 100])
def test_long_context(H):
    """100000 keys of one sequence, cut over all blocks, against the oracle."""
    c = Latent([1], [99999], seed=40, H=H, one=True)
    attend_and_check(c)


# ---------------------------------------------------------------- as used

def test_decoder_loop():
    """A prompt in two chunks, then token by token: every step's rows against the
    oracle over everything appended so far."""
    rng = np.random.default_rng(41)
    H, page, steps = 8, 16, [37, 20, 1, 1, 2, 1, 1]
    total = sum(steps)
    i32 = dict(dtype=torch.int32, device="cuda")
    cache = torch.full((8, page, 576), float("nan"), dtype=torch.bfloat16, device="cuda")
    table = torch.tensor([[3, 1, 7, 0, 5, 2]], **i32)
    cos, sin = (torch.empty(96, 32, device="cuda") for _ in "cs")
    A.attn_rope_table(A.make_rope_table_params(cos=cos, sin=sin, scaling="LINEAR", factor=2.0))
    data = {n: dev16(rng.standard_normal(s), "bf16") for n, s in
            (("c_new", (total, 512)), ("k_rope", (total, 64)), ("q_rope", (total, H, 64)),
             ("q_lat", (total, H, 512)))}
    lens, at = torch.zeros(1, **i32), 0
    cc, ss = cos.double().cpu().numpy(), sin.double().cpu().numpy()
    host = {n: x.double().cpu().numpy() for n, x in data.items()}
    for n in steps:
        lens += n
        new = {k: x[at:at + n] for k, x in data.items()}
        q_rot = torch.empty(n, H, 64, dtype=torch.bfloat16, device="cuda")
        p = A.make_latent_params(dtype="bf16", cache=cache, d_c=512, page_table=table,
                                 seq_lens=lens, cu_seqlens_q=torch.tensor([0, n], **i32),
                                 max_q_len=n, rope_cos=cos, rope_sin=sin, q_rot=q_rot, scale=SCALE,
                                 **new)
        o = torch.empty(n, H, 512, dtype=torch.bfloat16, device="cuda")
        lse = torch.empty(H, n, device="cuda")
        ws = torch.empty(A.attn_latent_workspace_size(p), dtype=torch.uint8, device="cuda")
        A.attn_latent_append(p)
        A.attn_latent_fwd(p, o, lse, ws)
        at += n
        pos = np.arange(at)
        pe = L.turn(host["k_rope"][:at, None], cc[pos], ss[pos])[:, 0]
        rows = np.concatenate([host["c_new"][:at], pe], 1)
        q = np.concatenate([host["q_lat"][at - n:at],
                            L.turn(host["q_rope"][at - n:at], cc[pos[-n:]], ss[pos[-n:]])], -1)
        ro, rl, rA, rD = L.attend(q, lambda s: rows, 512, [at], [0, n], SCALE)
        # against exact keys and queries: their rotated parts are rounded once
        # (u each), which moves a score by at most 2 u D and a weight by twice that
        u = UNIT["bf16"]
        tol = u * np.abs(ro) + (2 * u + 8 * u * rD[..., None]) * rA + 1e-6
        assert (np.abs(o.double().cpu().numpy() - ro) <= tol).all()
        assert (np.abs(lse.double().cpu().numpy() - rl) <= 2 * u * rD.T + 1e-5).all()


def test_absorbed_is_expanded():
    """The absorbed form over the cache gives what the expanded form gives, with
    the up-projections taken into queries and outputs."""
    rng = np.random.default_rng(42)
    H, T, d_n, d_v = 4, 100, 128, 128
    W_k = rng.standard_normal((H, d_n, 512)) / 512 ** 0.5
    W_v = rng.standard_normal((H, 512, d_v)) / 512 ** 0.5
    c = Latent([T], [0], seed=43, H=H)
    q_n = rng.standard_normal((T, H, d_n))
    q_lat = dev16(np.einsum("thn,hnc->thc", q_n, W_k), "bf16")
    c.t["q_lat"], c.q_lat = q_lat, q_lat.double().cpu().numpy()
    o, lse = c.append_and_attend()
    out = np.einsum("thc,hcv->thv", o.double().cpu().numpy(), W_v)
    # expanded, in float64
    kv = np.concatenate([np.einsum("tc,hnc->thn", c.c_new, W_k),
                         np.einsum("tc,hcv->thv", c.c_new, W_v)], -1)
    cos, sin = c.angles(np.arange(T))
    k, v = L.expand(kv, c.k_rope, cos, sin, d_n)
    q = np.concatenate([q_n, L.turn(c.q_rope, cos, sin)], -1)
    ro, rl, _, rD = P.attend(q, lambda s: k.transpose(1, 0, 2), lambda s: v.transpose(1, 0, 2),
                             [T], [0, T], SCALE)
    # roundings of q_lat, of the rotated parts, of P and of O, all of half a step of
    # bf16: relative Frobenius errors well below 8 of them
    rel = np.linalg.norm(out - ro) / np.linalg.norm(ro)
    assert rel <= 8 * UNIT["bf16"], rel
    assert np.abs(lse.double().cpu().numpy() - rl).max() <= 4 * UNIT["bf16"] * rD.max()
