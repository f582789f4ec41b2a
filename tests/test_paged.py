"""The paged KV cache on the GPU against the float64 oracle: appending with
rotation, attention over the pages, and both in turn as a decoder runs them."""
import numpy as np
import pytest
import torch

from oracle import paged_ref as P
from paged_util import TORCH, UNIT, Paged, check_attend, written_slots

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
    "decode": dict(new=[1] * 5, ctx=[0, 15, 16, 17, 63], one=True, grow=20.0),
    "decode_offsets": dict(new=[1, 0, 1, 1], ctx=[31, 40, 0, 5], pad=3, grow=20.0),
    "ragged": dict(new=[40, 0, 1, 17, 33], ctx=[0, 9, 16, 15, 3], pad=2, grow=8.0),
    "one_token_total": dict(new=[1], ctx=[0], one=True, page=256),
    "page64": dict(new=[130, 64, 65], ctx=[0, 64, 7], page=64, grow=30.0),
    "page256": dict(new=[300, 5], ctx=[200, 255], page=256, d_qk=192, grow=8.0),
    "bf16": dict(new=[20, 3], ctx=[5, 16], cache="bf16"),
    "fp16": dict(new=[20, 3], ctx=[5, 16], cache="fp16", dtype="fp16"),
    "fp16_e4m3": dict(new=[20, 3], ctx=[5, 16], dtype="fp16", page=32, grow=5.0),
    "wide_partial": dict(new=[20, 3], ctx=[5, 16], d_qk=192, rot=64, interleaved=True,
                         cache="bf16", Hq=3, Hkv=3),
    "d64": dict(new=[70], ctx=[20], d_qk=64, d_v=64, Hq=7, Hkv=1, interleaved=True, page=32),
    "no_rotation": dict(new=[10, 1], ctx=[3, 4], rot=0),
    "rot16": dict(new=[10, 1], ctx=[3, 4], rot=16),
    "nhd": dict(new=[18, 2], ctx=[15, 16], layout="nhd", grow=20.0),
    "nhd_fused_bf16": dict(new=[18, 2], ctx=[15, 16], layout="nhd", fused=True, cache="bf16"),
    "fused_shifted": dict(new=[18, 2], ctx=[15, 16], fused=True, pos_shift=100),
    "packed": dict(new=[18, 2], ctx=[15, 16], layout="packed", d_qk=192, grow=20.0),
    "many_seqs": dict(new=[i % 3 for i in range(600)], ctx=[i % 7 for i in range(600)], Hq=2,
                      Hkv=1, d_qk=64, d_v=64),
}


def check_append(c):
    """Codes and scales of earlier tokens are exact; a new 16-bit value is off
    by half a step plus the rotation's fp32 roundings (each product and the
    sum: 3 * 2^-24 of |a| + |b|), a new code by half an E4M3 step of its
    page's scale plus the same."""
    c.oracle_append()
    new = written_slots(c)
    for name, x in (("k", c.k_new), ("v", c.v_new)):
        vals, scale = c.host[name]
        got, got_scale = c.cache_host(name)
        old = ~np.broadcast_to(new[:, None, :, None], vals.shape)
        assert np.array_equal(got[old], vals[old], equal_nan=True), name
        if scale is not None:
            assert np.array_equal(got_scale, scale, equal_nan=True), name
        exact = c.rotated(x) if name == "k" else x
        big = np.abs(x).max(-1)  # bounds |a| and |b| of every pair
        for s, row, pos in P.new_rows(c.lens, c.cu):
            pid, slot = c.table[s, pos // c.page], pos % c.page
            f32 = 6 * 2.0 ** -24 * big[row][:, None]
            if scale is None:
                tol = UNIT[c.cache] * np.abs(exact[row]) + f32 + 2.0 ** -25
                err = np.abs(got[pid, :, slot] - exact[row])
            else:
                sc = scale[pid][:, None]
                tol = np.maximum(2.0 ** -4 * np.abs(exact[row]), 2.0 ** -10 * sc) + 2 * f32
                err = np.abs(got[pid, :, slot] * sc - exact[row])
            assert (err <= tol).all(), (name, row, float((err / tol).max()))
    rq = c.rotated(c.q)
    got = c.t["q_rot"].double().cpu().numpy()
    n = c.cu[-1]
    tol = UNIT[c.dtype] * np.abs(rq) + 6 * 2.0 ** -24 * np.abs(c.q).max(-1, keepdims=True) + 2.0 ** -25
    assert (np.abs(got - rq)[:n] <= tol[:n]).all()
    assert np.isnan(got[n:]).all()


@pytest.mark.parametrize("name", list(APPEND))
def test_append(name):
    from bwd_tcgen05_tma_gb300 import attn as A

    c = Paged(seed=11, **APPEND[name])
    p = c.params()
    A.attn_paged_append(p)
    assert c.status() == 0
    first = {n: c.t[n].clone() for n in ("q_rot", "k_cache", "v_cache")}
    check_append(c)
    # the same call again: the scales are there already and nothing changes
    A.attn_paged_append(p)
    torch.cuda.synchronize()
    for n, x in first.items():
        assert torch.equal(bits(x), bits(c.t[n])), n


def test_scale_growth_rounds_earlier_codes_again():
    """A page filled token by token, each larger than the last: the scale grows
    many times and every earlier code follows."""
    from bwd_tcgen05_tma_gb300 import attn as A

    for j in range(16):
        c = Paged([1], [j], seed=30 + j, one=True, Hq=2, Hkv=2, std=2.0 ** j)
        pid = c.table[0, 0]
        before = c.host["k"][1][pid].copy()
        A.attn_paged_append(c.params())
        check_append(c)
        assert j < 3 or (c.host["k"][1][pid] > before).all()


def test_append_in_place_and_without_queries():
    from bwd_tcgen05_tma_gb300 import attn as A

    c = Paged([5, 1], [3, 16], seed=12)
    c.t["q_rot"] = c.t["q"]
    A.attn_paged_append(c.params())
    check_append(c)
    d = Paged([5, 1], [3, 16], seed=12)
    A.attn_paged_append(d.params(q=None, q_rot=None))
    torch.cuda.synchronize()
    for n in ("k_cache", "v_cache"):
        assert torch.equal(bits(c.t[n]), bits(d.t[n]))


def test_append_nonfinite_values():
    """Infinities and NaN become NaN codes and leave the scale to the others."""
    from bwd_tcgen05_tma_gb300 import attn as A

    c = Paged([3], [2], seed=13, rot=0)
    for x, name in ((c.k_new, "k_new"), (c.v_new, "v_new")):
        x[0, 0, 3], x[1, 1, 5], x[2, 0, 0] = np.inf, -np.inf, np.nan
        c.t[name].copy_(torch.from_numpy(x))
    A.attn_paged_append(c.params())
    torch.cuda.synchronize()
    c.oracle_append()
    for name in ("k", "v"):
        got, scale = c.cache_host(name)
        assert np.array_equal(got, c.host[name][0], equal_nan=True)
        assert np.array_equal(scale, c.host[name][1], equal_nan=True)


def test_append_reports_and_skips_bad_pages_and_positions():
    from bwd_tcgen05_tma_gb300 import attn as A

    good = Paged([20, 4, 4], [0, 0, 3], seed=14)
    A.attn_paged_append(good.params())
    torch.cuda.synchronize()
    for what in ("page", "negative_page", "rope", "length"):
        c = Paged([20, 4, 4], [0, 0, 3], seed=14, pos_shift=0)
        hit = int(c.table[1, 0])
        keep = c.t["k_cache"].clone()
        if what == "page":
            c.t["table"][1, 0] = c.t["k_cache"].shape[0]
        elif what == "negative_page":
            c.t["table"][1, 0] = -1
        elif what == "rope":
            c.t["pos"][20:24] = c.cos.shape[0]
        else:
            c.t["lens"][1] = 2  # four new tokens of a sequence of two
        A.attn_paged_append(c.params())
        assert c.status() == 7, what
        for n in ("k_cache", "v_cache"):
            got, want = bits(c.t[n]), bits(good.t[n]).clone()
            others = torch.ones(got.shape[0], dtype=torch.bool)
            others[hit] = False
            assert torch.equal(got[others.cuda()], want[others.cuda()]), what
        if what != "length":
            assert torch.equal(bits(c.t["k_cache"])[hit], bits(keep)[hit])


# ---------------------------------------------------------------- attention

ATTEND = {
    "one_key": dict(new=[1], ctx=[0], one=True),
    "decode": dict(new=[1] * 6, ctx=[0, 1, 15, 16, 200, 700], one=True),
    "decode_group8": dict(new=[1] * 3, ctx=[5, 130, 257], one=True, Hq=16, Hkv=2, page=64),
    "decode_group7": dict(new=[1] * 3, ctx=[5, 130, 257], one=True, Hq=14, Hkv=2, page=32),
    "decode_group12": dict(new=[1] * 2, ctx=[33, 400], one=True, Hq=12, Hkv=1),
    "decode_group1": dict(new=[1] * 3, ctx=[33, 400, 64], one=True, Hq=3, Hkv=3),
    "decode_bf16": dict(new=[1] * 3, ctx=[33, 300, 64], one=True, cache="bf16"),
    "decode_fp16": dict(new=[1] * 3, ctx=[33, 300, 64], one=True, cache="fp16", dtype="fp16"),
    "decode_fp16_e4m3": dict(new=[1] * 3, ctx=[33, 300, 64], one=True, dtype="fp16"),
    "decode_192": dict(new=[1] * 3, ctx=[33, 300, 64], one=True, d_qk=192),
    "decode_192_bf16": dict(new=[1] * 3, ctx=[33, 300, 64], one=True, d_qk=192, cache="bf16"),
    "decode_64": dict(new=[1] * 3, ctx=[33, 300, 64], one=True, d_qk=64, d_v=64),
    "decode_192_64": dict(new=[1] * 2, ctx=[33, 300], one=True, d_qk=192, d_v=64, cache="fp16",
                          dtype="fp16"),
    "decode_64_128_bf16": dict(new=[1] * 2, ctx=[33, 300], one=True, d_qk=64, cache="bf16"),
    "decode_nhd": dict(new=[1] * 3, ctx=[33, 300, 64], one=True, layout="nhd"),
    "decode_many": dict(new=[1] * 300, ctx=[i % 40 for i in range(300)], one=True, Hq=2, Hkv=1),
    "decode_group64": dict(new=[1] * 3, ctx=[33, 300, 0], one=True, Hq=64, Hkv=1),
    "decode_group256": dict(new=[1] * 2, ctx=[200, 0], one=True, Hq=256, Hkv=1, d_qk=64, d_v=64),
    "decode_page256": dict(new=[1] * 3, ctx=[255, 700, 256], one=True, page=256),
    "decode_packed_192": dict(new=[1] * 2, ctx=[33, 300], one=True, d_qk=192, layout="packed"),
    "decode_nhd_bf16": dict(new=[1] * 2, ctx=[33, 300], one=True, layout="nhd", cache="bf16",
                            page=128),
    "verify_many": dict(new=[1 + i % 5 for i in range(200)], ctx=[i % 60 for i in range(200)],
                        Hq=8, Hkv=1, d_qk=64, d_v=64),
    "padded": dict(new=[1, 0, 1], ctx=[20, 30, 0], pad=5),
    "verify": dict(new=[4, 1, 0, 5, 2], ctx=[100, 0, 50, 16, 31]),
    "verify_fp16_64": dict(new=[3, 2], ctx=[150, 40], d_qk=64, d_v=64, dtype="fp16", page=32),
    "verify_bf16": dict(new=[8, 7], ctx=[150, 40], cache="bf16", Hq=8, Hkv=1),
    "chunk": dict(new=[40, 130], ctx=[100, 0], page=64),
    "chunk_group8": dict(new=[33, 20], ctx=[300, 7], Hq=8, Hkv=1),
    "chunk_bf16": dict(new=[70, 129], ctx=[3, 140], cache="bf16", page=32),
    "chunk_fp16": dict(new=[70], ctx=[300], cache="fp16", dtype="fp16", Hq=2, Hkv=2),
    "chunk_192": dict(new=[65, 20], ctx=[100, 0], d_qk=192, Hq=2, Hkv=1),
    "chunk_64": dict(new=[65, 128], ctx=[130, 0], d_qk=64, d_v=64),
    "chunk_192_64_bf16": dict(new=[65], ctx=[130], d_qk=192, d_v=64, cache="bf16"),
    "chunk_64_128": dict(new=[65], ctx=[130], d_qk=64, d_v=128, dtype="fp16"),
    "chunk_uneven_group": dict(new=[50, 61], ctx=[30, 0], Hq=6, Hkv=2, layout="nhd", fused=True),
    "chunk_page256": dict(new=[100, 33], ctx=[500, 200], page=256),
    "chunk_page256_bf16": dict(new=[100, 33], ctx=[500, 200], page=256, cache="bf16"),
    "chunk_packed": dict(new=[100], ctx=[130], layout="packed", d_qk=192, page=32),
    "chunk_packed_fp16": dict(new=[100], ctx=[130], layout="packed", cache="fp16", dtype="fp16"),
    "chunk_many_tiles": dict(new=[300, 150], ctx=[1500, 700], Hq=8, Hkv=1, page=64),
    "chunk_many_tiles_bf16": dict(new=[129, 64], ctx=[1500, 700], Hq=8, Hkv=2, cache="bf16"),
    "chunk_many_tiles_192": dict(new=[129, 64], ctx=[1500, 700], Hq=4, Hkv=1, d_qk=192, page=128),
    "chunk_many_seqs": dict(new=[(i * 37) % 90 for i in range(70)],
                            ctx=[(i * 53) % 200 for i in range(70)], Hq=2, Hkv=1),
    "chunk_mixed_with_decode": dict(new=[1, 200, 1, 0, 3], ctx=[500, 20, 0, 3, 100]),
}
MASKS = {"causal": {}, "window": dict(window_left=20), "window0": dict(window_left=0),
         "full": dict(mask="NONE"), "full_window": dict(mask="NONE", window_left=33)}


def _attend(c, sink=None, **kw):
    """Queries unrotated; the new tokens' keys and values come from the cache,
    which holds NaN behind every sequence's end."""
    from bwd_tcgen05_tma_gb300 import attn as A

    A.attn_paged_append(c.params())
    s = None if sink is None else torch.from_numpy(sink).float().cuda()
    p = c.params(q_rot=None, sink=s, **kw)
    o, lse = c.attend(p)
    assert c.status() == 0
    ref = c.oracle_attend(c.q, causal=kw.get("mask", "CAUSAL") == "CAUSAL",
                          window=-1 if kw.get("window_left") is None else kw["window_left"],
                          sink=sink)
    check_attend(c, o, lse, ref)
    o2, lse2 = c.attend(p)
    assert torch.equal(bits(o), bits(o2)) and torch.equal(bits(lse), bits(lse2))


@pytest.mark.parametrize("name", list(ATTEND))
def test_attend(name):
    _attend(Paged(seed=21, **ATTEND[name]))


@pytest.mark.parametrize("mask", list(MASKS))
@pytest.mark.parametrize("name", ["decode", "verify", "verify_many", "chunk", "chunk_bf16",
                                  "chunk_page256", "chunk_mixed_with_decode"])
def test_attend_masks(name, mask):
    _attend(Paged(seed=22, **ATTEND[name]), **MASKS[mask])


@pytest.mark.parametrize("name", ["decode_group7", "padded", "verify", "chunk_group8"])
def test_attend_sink(name):
    c = Paged(seed=23, **ATTEND[name])
    _attend(c, sink=np.random.default_rng(1).standard_normal(c.Hq).astype(np.float32).astype(float),
            window_left=50)


@pytest.mark.parametrize("hint", [1, 2, 40, 5000])
def test_attend_any_length_hint(hint):
    c = Paged(seed=24, **ATTEND["chunk_mixed_with_decode"])
    _attend(c, max_q_len=hint)


@pytest.mark.parametrize("window", [None, 20])
@pytest.mark.parametrize("cache", ["fp8_e4m3", "bf16"])
@pytest.mark.parametrize("new", [8, 9, 16, 17])
def test_attend_on_both_sides_of_the_choice(new, cache, window):
    """32, 36, 64 and 68 rows a KV head over a long table and inside a narrow
    window: the last sizes of one kernel and the first of the other."""
    _attend(Paged([new, 1, new - 3], [900, 300, 40], seed=25, Hq=8, Hkv=2, cache=cache),
            window_left=window)


def test_shared_prefix_and_strided_table():
    """Two sequences that list the same pages for their first 48 tokens, tables
    with rows further apart than their columns, windows of any size."""
    from bwd_tcgen05_tma_gb300 import attn as A

    c = Paged([3, 20], [60, 90], seed=41)
    c.table[1, :3] = c.table[0, :3]
    wide = torch.full((2, c.table.shape[1] + 5), -7, dtype=torch.int32, device="cuda")
    wide[:, :c.table.shape[1]] = torch.tensor(c.table, dtype=torch.int32)
    c.t["table"] = wide[:, :c.table.shape[1]]
    A.attn_paged_append(c.params())
    for window in (None, 2 ** 31 - 1, 70):
        p = c.params(q_rot=None, window_left=window)
        o, lse = c.attend(p)
        assert c.status() == 0
        check_attend(c, o, lse, c.oracle_attend(c.q, window=-1 if window is None else window))


def test_lengths_behind_the_table_are_reported():
    """A length beyond the table's row: what the table has counts, the rest is
    masked, and the status says so (few rows and many)."""
    from bwd_tcgen05_tma_gb300 import attn as A

    for new in (1, 80):
        c = Paged([new], [100], seed=42, spare=0)
        A.attn_paged_append(c.params())
        assert c.status() == 0
        full = c.t["table"]
        c.t["table"] = full[:, :5].contiguous()  # 80 of the tokens
        o, lse = c.attend(c.params(q_rot=None, mask="NONE"))
        assert c.status() == 7
        lens, c.lens = c.lens, [80]
        src = {n: c.cache_host(n) for n in ("k", "v")}
        ref = P.attend(c.q, lambda s: P.gather(*src["k"], c.table[s], 16, 80),
                       lambda s: P.gather(*src["v"], c.table[s], 16, 80), [80], c.cu,
                       c.d_qk ** -0.5, causal=False)
        check_attend(c, o, lse, ref)
        c.lens = lens


def test_attend_without_lse():
    from bwd_tcgen05_tma_gb300 import attn as A

    c = Paged(seed=25, **ATTEND["verify"])
    A.attn_paged_append(c.params())
    p = c.params(q_rot=None)
    o, _ = c.attend(p)
    o2, _ = c.fresh_outputs()
    ws = torch.empty(A.attn_paged_workspace_size(p), dtype=torch.uint8, device="cuda")
    A.attn_paged_fwd(p, o2, None, ws)
    assert torch.equal(bits(o), bits(o2))


@pytest.mark.parametrize("cache", ["fp8_e4m3", "bf16"])
@pytest.mark.parametrize("new", [1, 3, 40])
def test_empty_sequences_and_windows(cache, new):
    """Sequences without tokens, lengths below the new tokens' number, and a
    batch of none: rows without a key give 0 and -inf (or the sink)."""
    from bwd_tcgen05_tma_gb300 import attn as A

    c = Paged([new, new], [10, 0], seed=26, cache=cache)
    A.attn_paged_append(c.params())
    c.t["lens"][1] = 0
    c.lens[1] = 0
    for sink in (None, np.array([0.5, -1.0, 2.0, 0.0])):
        s = None if sink is None else torch.from_numpy(sink).float().cuda()
        o, lse = c.attend(c.params(q_rot=None, sink=s))
        torch.cuda.synchronize()
        assert (o[new:] == 0).all()
        want = -np.inf if sink is None else sink[:, None]
        assert np.array_equal(lse[:, new:].cpu().numpy(), np.broadcast_to(want, (4, new)))
        assert torch.isfinite(o[:new]).all()
        assert c.status() == 0
    # a sequence of length 0 takes no tokens, without a report
    keep = bits(c.t["k_cache"]).clone()
    c.t["q_rot"].fill_(7.0)
    A.attn_paged_append(c.params())
    assert c.status() == 0 and (c.t["q_rot"][new:] == 7.0).all()
    assert torch.equal(bits(c.t["k_cache"]), keep)
    c.t["cu"].zero_()
    o, lse = c.attend(c.params(q_rot=None))
    assert torch.isnan(o).all() and torch.isnan(lse).all()


@pytest.mark.parametrize("cache", ["fp8_e4m3", "bf16", "fp16"])
@pytest.mark.parametrize("new", [1, 4, 50, 140])
def test_masked_values_have_no_influence(cache, new):
    """NaN and infinities in keys and values that a row does not keep: behind
    its position, before its window, and behind the sequence's end."""
    dtype = "fp16" if cache == "fp16" else "bf16"
    from bwd_tcgen05_tma_gb300 import attn as A

    window = 30
    c = Paged([new, 2], [70, 9], seed=27, cache=cache, dtype=dtype)
    A.attn_paged_append(c.params())
    p = c.params(q_rot=None, window_left=window)
    ref, ref_lse = (x.clone() for x in c.attend(p))
    torch.cuda.synchronize()
    view = {n: c.t[n].view(torch.uint8 if cache == "fp8_e4m3" else torch.int16)
            for n in ("k_cache", "v_cache")}
    bad = {"fp8_e4m3": 0x7F, "bf16": 0x7F80, "fp16": 0x7E00}[cache]
    last = 70 + new - 1  # poisoned: only the last row keeps it
    first = 70 - window  # only the first row keeps it
    for j in range(0, first):
        for v in view.values():
            v[c.table[0, j // 16], :, j % 16] = bad
    for j in (last, first):
        for i, v in enumerate(view.values()):
            v[c.table[0, j // 16], :, j % 16, i::7] = bad
    o, lse = c.attend(p)
    torch.cuda.synchronize()
    clean = [r for r in range(new + 2) if r >= new or (r != new - 1 and r != 0)]
    assert torch.equal(bits(o[clean]), bits(ref[clean]))
    assert torch.equal(lse[:, clean], ref_lse[:, clean])
    # the rows that keep one: NaN scores and NaN or infinite values
    for r in {0, new - 1}:
        assert not torch.isfinite(lse[:, r]).any() or not torch.isfinite(o[r]).all()


@pytest.mark.parametrize("cache", ["fp8_e4m3", "bf16"])
@pytest.mark.parametrize("Hq", [2, 16])
def test_masked_values_in_a_wide_batch(cache, Hq):
    """As above where a warp takes whole sequences: a NaN in the last token's
    value reaches the last row of its sequence only."""
    from bwd_tcgen05_tma_gb300 import attn as A

    n = 300
    c = Paged([3] * n, [20 + i % 17 for i in range(n)], seed=43, cache=cache, Hq=Hq, Hkv=1)
    A.attn_paged_append(c.params())
    p = c.params(q_rot=None)
    ref, ref_lse = (x.clone() for x in c.attend(p))
    v = c.t["v_cache"].view(torch.uint8 if cache == "fp8_e4m3" else torch.int16)
    hit = list(range(0, n, 7))
    for s in hit:
        j = c.lens[s] - 1
        v[c.table[s, j // 16], 0, j % 16, 5] = 0x7F if cache == "fp8_e4m3" else 0x7FC0
    o, lse = c.attend(p)
    assert torch.equal(bits(lse), bits(ref_lse))
    got, want = o.float().cpu(), ref.float().cpu()
    rows = [3 * s + 2 for s in hit]
    assert torch.isnan(got[rows, :, 5]).all()
    want[rows, :, 5] = got[rows, :, 5]
    assert torch.equal(bits(got), bits(want))


@pytest.mark.parametrize("new", [1, 4, 60, 140])
def test_nonfinite_values_stay_in_their_dims(new):
    """A NaN in one dim of a value reaches that dim of the rows that keep it
    and nothing else."""
    from bwd_tcgen05_tma_gb300 import attn as A

    c = Paged([new], [70], seed=28, cache="bf16")
    A.attn_paged_append(c.params())
    p = c.params(q_rot=None)
    ref, ref_lse = (x.clone() for x in c.attend(p))
    j = 70 + new // 2
    c.t["v_cache"][c.table[0, j // 16], 0, j % 16, 5] = float("nan")
    c.t["v_cache"][c.table[0, 1], 1, 3, 9] = float("inf")
    o, lse = c.attend(p)
    assert torch.equal(bits(lse), bits(ref_lse))
    got, want = o.float().cpu(), ref.float().cpu()
    assert torch.isnan(got[new // 2:, :2, 5]).all()
    assert torch.isinf(got[:, 2:, 9]).all()
    want[new // 2:, :2, 5] = got[new // 2:, :2, 5]
    want[:, 2:, 9] = got[:, 2:, 9]
    assert torch.equal(bits(got), bits(want))


@pytest.mark.parametrize("new", [1, 3, 40])
def test_attend_reports_bad_pages(new):
    """A page id that is none: its tokens count as masked, the rest is right."""
    from bwd_tcgen05_tma_gb300 import attn as A

    c = Paged([new, new], [100, 40], seed=29)
    A.attn_paged_append(c.params())
    torch.cuda.synchronize()
    for bad in (-1, c.t["k_cache"].shape[0], 2 ** 31 - 1):
        c.t["status"].zero_()
        c.t["table"][0, 2] = bad
        o, lse = c.attend(c.params(q_rot=None))
        assert c.status() == 7
        src = {n: c.cache_host(n) for n in ("k", "v")}
        keep = [j for j in range(100 + new) if j // 16 != 2]

        def of(name):
            def f(s):
                if s:
                    return P.gather(*src[name], c.table[s], 16, c.lens[s])
                return P.gather(*src[name], c.table[s], 16, c.lens[s])[:, keep]
            return f

        lens = [len(keep), c.lens[1]]
        ref = P.attend(c.q, of("k"), of("v"), lens, c.cu, c.d_qk ** -0.5)
        check_attend(c, o, lse, ref)


def test_offsets_out_of_range_are_reported():
    from bwd_tcgen05_tma_gb300 import attn as A

    c = Paged([3, 2], [20, 5], seed=31)
    A.attn_paged_append(c.params())
    ref, _ = c.attend(c.params(q_rot=None))
    assert c.status() == 0
    c.t["cu"][2] = 1000
    o, _ = c.attend(c.params(q_rot=None))
    assert c.status() == 7
    assert torch.equal(bits(o[:3]), bits(ref[:3])) and torch.isnan(o[3:]).all()
    c.t["status"].zero_()
    A.attn_paged_append(c.params())
    assert c.status() == 7


def test_caller_scales_of_any_size():
    """Scales that are no powers of two, far apart, and zero."""
    c = Paged([1, 4], [200, 100], seed=32)
    from bwd_tcgen05_tma_gb300 import attn as A

    A.attn_paged_append(c.params())
    rng = np.random.default_rng(5)
    for name, lo, hi in (("k_scale", -9, -5), ("v_scale", -40, 20)):
        s = np.exp2(rng.uniform(lo, hi, tuple(c.t[name].shape))).astype(np.float32)
        c.t[name].copy_(torch.from_numpy(s))
    c.t["v_scale"][int(c.table[0, 3])] = 0.0
    o, lse = c.attend(c.params(q_rot=None))
    assert c.status() == 0
    # a 16-bit type of O with enough range for these values
    check_attend(c, o, lse, c.oracle_attend(c.q))


# ------------------------------------------------------------- as it is used


def test_decoder_loop():
    """Prefill in two chunks, then decode steps, appending and attending in
    turn on the same buffers; every step's attention against the oracle, and
    the cache against the oracle's at the end."""
    from bwd_tcgen05_tma_gb300 import attn as A

    rng = np.random.default_rng(6)
    total, page, Hq, Hkv, d = 75, 16, 4, 2, 128
    steps = [40, 23] + [1] * 12
    c = Paged([total, 8], [0, 0], seed=33, Hq=Hq, Hkv=Hkv, page=page, grow=6.0)
    host = {n: [np.zeros_like(v), np.zeros_like(s)] for n, (v, s) in c.host.items()}
    done = 0
    for n in steps:
        c.t["lens"].copy_(torch.tensor([done + n, 1 if n == 1 else 8], dtype=torch.int32))
        new = [n, 0]
        c.new, c.lens, c.cu = new, [done + n, 0], [0, n, n]
        c.T = n
        rows = slice(done, done + n)
        d_ = Paged.__new__(Paged)
        d_.__dict__.update(c.__dict__)
        d_.t = dict(c.t, q=c.t["q"][rows], k_new=c.t["k_new"][rows], v_new=c.t["v_new"][rows],
                    q_rot=torch.empty(n, Hq, d, dtype=torch.bfloat16, device="cuda"),
                    cu=torch.tensor([0, n, n], dtype=torch.int32, device="cuda"))
        d_.q, d_.k_new, d_.v_new = c.q[rows], c.k_new[rows], c.v_new[rows]
        p = d_.params(max_q_len=n)
        A.attn_paged_append(p)
        o, lse = d_.attend(p)
        assert c.status() == 0
        done += n
        qr = d_.t["q_rot"].double().cpu().numpy()
        check_attend(d_, o, lse, d_.oracle_attend(qr))
        for name, x in (("k", d_.rotated(d_.k_new)), ("v", d_.v_new)):
            P.append(*host[name], d_.table, page, d_.lens, d_.cu, x)
    for name, x in (("k", c.k_new), ("v", c.v_new)):
        vals, scale = c.cache_host(name)
        used = c.table[0, :-(-total // page)]
        assert np.array_equal(scale[used], host[name][1][used])
        got = P.gather(vals, scale, c.table[0], page, total)
        want = P.gather(*host[name], c.table[0], page, total)
        # a value near a tie may fall to either side
        step = np.maximum(np.abs(want) * 2.0 ** -3, 2.0 ** -9 * scale[used].max())
        assert (np.abs(got - want) <= step * 1.01).all()
        assert (got != want).mean() < 1e-3


def test_graph_serves_later_steps():
    """One captured step replayed with other lengths, tables and values equals
    the eager calls; two graphs with a workspace each on two streams."""
    from bwd_tcgen05_tma_gb300 import attn as A

    c = Paged([1] * 4, [3, 40, 100, 250], seed=34, one=True)
    p = c.params()
    o, lse = c.fresh_outputs()
    ws = torch.empty(A.attn_paged_workspace_size(p), dtype=torch.uint8, device="cuda")

    def step():
        A.attn_paged_append(p)
        A.attn_paged_fwd(p, o, lse, ws)

    saved = {n: c.t[n].clone() for n in ("k_cache", "v_cache", "k_scale", "v_scale", "lens")}
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph):
            step()
    torch.cuda.current_stream().wait_stream(side)

    def restore(delta):
        for n, x in saved.items():
            c.t[n].copy_(x)
        c.t["lens"].sub_(delta).clamp_(min=0)
        o.fill_(float("nan"))
        lse.fill_(float("nan"))
        c.t["status"].zero_()

    for delta in (0, 1, 17):
        restore(delta)
        step()
        torch.cuda.synchronize()
        want = [x.clone() for x in (o, lse, c.t["k_cache"], c.t["v_scale"])]
        restore(delta)
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(want, (o, lse, c.t["k_cache"], c.t["v_scale"])):
            assert torch.equal(bits(x), bits(y)), delta


def test_two_streams_with_two_workspaces():
    from bwd_tcgen05_tma_gb300 import attn as A

    cs = [Paged([1] * 3, [700, 300, 5 + i], seed=35 + i, one=True) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in cs]
    ref, got = [], []
    for c in cs:
        A.attn_paged_append(c.params())
        ref.append(c.attend(c.params(q_rot=None))[0])
    torch.cuda.synchronize()
    ws = [torch.empty(A.attn_paged_workspace_size(c.params()), dtype=torch.uint8, device="cuda")
          for c in cs]
    outs = [c.fresh_outputs() for c in cs]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s, w, (o, lse) in zip(cs, streams, ws, outs):
            A.attn_paged_fwd(c.params(q_rot=None), o, lse, w, s)
    torch.cuda.synchronize()
    for (o, _), r in zip(outs, ref):
        assert torch.equal(bits(o), bits(r))


@pytest.mark.slow
def test_offsets_beyond_32_bits():
    """Pages whose element offset in the pool passes 2^31."""
    from bwd_tcgen05_tma_gb300 import attn as A

    c = Paged([1, 6, 100], [50, 150, 0], seed=37, page=128)
    pages = 70000
    for name in ("k", "v"):
        small = c.t[name + "_cache"]
        big = torch.empty(pages, *small.shape[1:], dtype=torch.uint8, device="cuda")
        assert big.numel() > 2 ** 31
        big[-small.shape[0]:] = small.view(torch.uint8)
        c.t[name + "_cache"] = big.view(torch.float8_e4m3fn)
        sc = torch.zeros(pages, c.Hkv, device="cuda")
        sc[-small.shape[0]:] = c.t[name + "_scale"]
        c.t[name + "_scale"] = sc
        shift = pages - small.shape[0]
    c.t["table"] = torch.where(c.t["table"] < 1000, c.t["table"] + shift, c.t["table"])
    A.attn_paged_append(c.params())
    o, lse = c.attend(c.params(q_rot=None))
    assert c.status() == 0
    for name in ("k", "v"):
        n = c.host[name][0].shape[0]
        c.t[name + "_cache"] = c.t[name + "_cache"][-n:]
        c.t[name + "_scale"] = c.t[name + "_scale"][-n:]
    check_attend(c, o, lse, c.oracle_attend(c.q))
    check_append(c)


def test_long_context_on_sampled_heads():
    """A context of 20000 tokens beside short ones; E4M3 and bf16 caches."""
    for cache in ("fp8_e4m3", "bf16"):
        c = Paged([1, 1, 1], [20000, 3, 900], seed=38, one=True, Hq=8, Hkv=1, page=64, cache=cache)
        _attend(c)
        assert c.t["k_cache"].dtype == TORCH[cache]
