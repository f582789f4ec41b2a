"""Host-side checks of the rotary and latent calls (no GPU needed): every
refusal the header names, workspace sizes, and the binding's own checks of
tensors.  Pointers are fake addresses that no refused call dereferences."""
import ctypes

import pytest
import torch

from bwd_tcgen05_tma_gb300 import attn as A

FAKE = 0x10000000
OK, INVALID, UNSUPPORTED, SHAPE, SMALL = 0, 1, 2, 3, 4
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    from bwd_tcgen05_tma_gb300 import build

    build.build()
    return A.load_library()


def fill(block, values, kw):
    p = block()
    for k, v in {**values, **kw}.items():
        if isinstance(v, tuple):
            field = getattr(p, k)
            for i, x in enumerate(v):
                field[i] = x
        else:
            setattr(p, k, v)
    return p


def call(lib, name, p):
    return getattr(lib, name)(ctypes.byref(p), None)


# ---------------------------------------------------------------- tables

def table(**kw):
    return fill(A.attn_rope_table_params_t,
                dict(struct_version=1, scaling=3, rope_len=64, rot_dim=64, base=1e4, factor=2.0,
                     turns_low=1.0, turns_high=4.0, trained_len=32, magnitude=1.0, rope_cos=FAKE,
                     rope_sin=FAKE), kw)


@pytest.mark.parametrize("kw,code", [
    (dict(struct_version=0), INVALID), (dict(struct_version=2), INVALID),
    (dict(scaling=-1), INVALID), (dict(scaling=4), INVALID), (dict(rope_len=-1), INVALID),
    (dict(rope_len=(1 << 30) + 1), UNSUPPORTED), (dict(rot_dim=0), INVALID),
    (dict(rot_dim=-16), INVALID), (dict(rot_dim=24), UNSUPPORTED), (dict(rot_dim=272), UNSUPPORTED),
    (dict(base=0.5), INVALID), (dict(base=NAN), INVALID), (dict(base=INF), INVALID),
    (dict(factor=0.99), INVALID), (dict(factor=NAN), INVALID), (dict(factor=INF), INVALID),
    (dict(magnitude=NAN), INVALID), (dict(magnitude=INF), INVALID),
    (dict(turns_low=4.0), INVALID), (dict(turns_low=NAN), INVALID), (dict(turns_high=INF), INVALID),
    (dict(trained_len=0), INVALID), (dict(rope_cos=None), INVALID), (dict(rope_sin=None), INVALID),
    (dict(rope_cos=FAKE + 8), INVALID), (dict(rope_sin=FAKE + 4), INVALID),
    (dict(scaling=2, base=1e300, factor=1e300), INVALID),  # the stretched base overflows
])
def test_table_refuses(lib, kw, code):
    assert call(lib, "attn_rope_table", table(**kw)) == code


def test_table_without_rows(lib):
    assert call(lib, "attn_rope_table", table(rope_len=0, rope_cos=None, rope_sin=None)) == OK
    # what a scaling does not read is not looked at
    assert call(lib, "attn_rope_table", table(rope_len=0, scaling=0, factor=NAN, turns_low=NAN,
                                              trained_len=0)) == OK


# ---------------------------------------------------------------- rope

def rope(**kw):
    return fill(A.attn_rope_params_t,
                dict(struct_version=1, dtype=0, num_tokens=10, Hq=4, Hkv=2, d=128, rot_start=0,
                     rot_dim=128, rope_len=64, seq_len=10, positions=FAKE, rope_cos=FAKE,
                     rope_sin=FAKE, q=FAKE, k=FAKE + 65536, q_out=2 * FAKE, k_out=3 * FAKE,
                     q_stride=512, k_stride=256, q_out_stride=512, k_out_stride=256), kw)


PLACES = [
    (dict(num_tokens=-1), INVALID), (dict(num_tokens=(1 << 30) + 1), UNSUPPORTED),
    (dict(rope_len=-1), INVALID), (dict(cu_seqlens=FAKE), INVALID),  # and positions
    (dict(positions=None, cu_seqlens=FAKE, num_segments=-1), INVALID),
    (dict(positions=None, seq_len=0), INVALID), (dict(positions=FAKE + 2), INVALID),
    (dict(positions=None, cu_seqlens=FAKE + 2), INVALID), (dict(status=FAKE + 1), INVALID),
    (dict(rope_cos=FAKE + 8), INVALID), (dict(rope_sin=FAKE + 4), INVALID),
    (dict(rope_cos=None), INVALID), (dict(rope_sin=None), INVALID),
    (dict(struct_version=0), INVALID), (dict(dtype=2), INVALID), (dict(dtype=-1), INVALID),
]


@pytest.mark.parametrize("kw,code", PLACES + [
    (dict(Hq=-1), INVALID), (dict(Hkv=-1), INVALID), (dict(Hq=0, Hkv=0), INVALID),
    (dict(Hq=1025, q_stride=1 << 20, q_out_stride=1 << 20), UNSUPPORTED), (dict(d=0), INVALID),
    (dict(d=120, rot_dim=64), UNSUPPORTED), (dict(d=272, rot_dim=64), UNSUPPORTED),
    (dict(rot_start=-8), INVALID), (dict(rot_start=4, rot_dim=64), UNSUPPORTED),
    (dict(rot_start=8), INVALID), (dict(rot_dim=0), INVALID), (dict(rot_dim=40), UNSUPPORTED),
    (dict(rot_dim=(1 << 31) - 16, rot_start=(1 << 31) - 8), INVALID),
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(q_out=None), INVALID),
    (dict(k_out=None), INVALID), (dict(q=FAKE + 8), INVALID), (dict(k_out=FAKE + 2), INVALID),
    (dict(q_stride=504), INVALID), (dict(q_stride=516), INVALID), (dict(k_out_stride=0), INVALID),
    (dict(q_out=FAKE, q_out_stride=520), INVALID),  # in place needs one layout
])
def test_rope_refuses(lib, kw, code):
    assert call(lib, "attn_rope", rope(**kw)) == code


def test_rope_without_tokens(lib):
    assert call(lib, "attn_rope", rope(num_tokens=0, q=None, k=None, q_out=None, k_out=None,
                                       rope_cos=None, rope_sin=None)) == OK


# ---------------------------------------------------------------- expand

def expand(**kw):
    return fill(A.attn_latent_expand_params_t,
                dict(struct_version=1, dtype=0, num_tokens=10, H=4, d_n=128, d_v=128, d_r=64,
                     rope_len=64, seq_len=10, positions=FAKE, rope_cos=FAKE, rope_sin=FAKE,
                     kv=FAKE, k_rope=2 * FAKE, k=3 * FAKE, v=4 * FAKE, kv_stride=1024,
                     k_rope_stride=64, k_stride=768, v_stride=512), kw)


@pytest.mark.parametrize("call_name", ["attn_latent_expand", "attn_latent_expand_bwd"])
@pytest.mark.parametrize("kw,code", PLACES + [
    (dict(H=0), INVALID), (dict(d_n=0), INVALID), (dict(d_v=-8), INVALID), (dict(d_r=0), INVALID),
    (dict(H=1025), UNSUPPORTED), (dict(d_n=124), UNSUPPORTED), (dict(d_n=264), UNSUPPORTED),
    (dict(d_v=12), UNSUPPORTED), (dict(d_v=264), UNSUPPORTED), (dict(d_r=48), UNSUPPORTED),
    (dict(kv=None), INVALID), (dict(k_rope=None), INVALID), (dict(k=None), INVALID),
    (dict(v=None), INVALID), (dict(kv=FAKE + 8), INVALID), (dict(k=FAKE + 2), INVALID),
    (dict(kv_stride=1016), INVALID), (dict(k_rope_stride=60), INVALID),
    (dict(k_stride=772), INVALID), (dict(v_stride=0), INVALID),
])
def test_expand_refuses(lib, call_name, kw, code):
    assert call(lib, call_name, expand(**kw)) == code


def test_expand_without_tokens(lib):
    p = expand(num_tokens=0, kv=None, k_rope=None, k=None, v=None, rope_cos=None, rope_sin=None)
    assert call(lib, "attn_latent_expand", p) == OK
    assert call(lib, "attn_latent_expand_bwd", p) == OK


# ---------------------------------------------------------------- paged

def params(**kw):
    return fill(A.attn_latent_params_t,
                dict(struct_version=1, dtype=0, mask=1, num_seqs=4, num_tokens=4, max_q_len=1, H=16,
                     d_c=512, d_r=64, page_size=64, num_pages=100, max_pages=10, page_table=FAKE,
                     table_stride=10, seq_lens=FAKE, cache=FAKE, cache_stride=(64 * 576, 576),
                     c_new=FAKE, k_rope=FAKE, q_rope=FAKE, q_lat=FAKE, q_rot=2 * FAKE,
                     c_new_stride=512, k_rope_stride=64, q_rope_stride=(1024, 64),
                     q_lat_stride=(8192, 512), q_rot_stride=(1024, 64), rope_len=640,
                     rope_cos=FAKE, rope_sin=FAKE, scale=0.1, window_left=-1), kw)


def size(lib, p):
    return lib.attn_latent_workspace_size(ctypes.byref(p))


def fwd(lib, p, o=FAKE, lse=FAKE, ws=FAKE, ws_bytes=1 << 30):
    v = ctypes.c_void_p
    return lib.attn_latent_fwd(ctypes.byref(p), v(o), v(lse), v(ws), ctypes.c_size_t(ws_bytes),
                               None)


@pytest.mark.parametrize("kw,code", [
    (dict(struct_version=0), INVALID), (dict(struct_version=2), INVALID), (dict(dtype=2), INVALID),
    (dict(dtype=-1), INVALID), (dict(mask=2), INVALID), (dict(mask=-1), INVALID),
    (dict(num_seqs=-1), INVALID), (dict(num_tokens=-1), INVALID), (dict(max_q_len=0), INVALID),
    (dict(num_pages=-1), INVALID), (dict(max_pages=-1), INVALID), (dict(H=0), INVALID),
    (dict(H=257), UNSUPPORTED), (dict(d_c=128), UNSUPPORTED), (dict(d_c=576), UNSUPPORTED),
    (dict(d_r=32), UNSUPPORTED), (dict(page_size=8), UNSUPPORTED), (dict(page_size=48), UNSUPPORTED),
    (dict(page_size=512), UNSUPPORTED),
    (dict(max_pages=(1 << 24) + 1, table_stride=1 << 25), UNSUPPORTED),  # over 2^30 positions
    (dict(num_seqs=(1 << 26) + 1, num_tokens=(1 << 26) + 1), UNSUPPORTED),  # over 2^30 rows
    (dict(num_tokens=5), SHAPE),  # one token per sequence without offsets
    (dict(seq_lens=None), INVALID), (dict(page_table=None), INVALID), (dict(cache=None), INVALID),
    (dict(seq_lens=FAKE + 2), INVALID), (dict(page_table=FAKE + 1), INVALID),
    (dict(cu_seqlens_q=FAKE + 2), INVALID), (dict(status=FAKE + 2), INVALID),
    (dict(cache=FAKE + 8), INVALID), (dict(table_stride=9), INVALID),
    (dict(cache_stride=(0, 576)), INVALID), (dict(cache_stride=(64 * 576, 568)), INVALID),
    (dict(cache_stride=(64 * 576, 580)), INVALID), (dict(cache_stride=(-64 * 576, 576)), INVALID),
    (dict(q_rot=FAKE + 8), INVALID), (dict(q_rot_stride=(1024, 56)), INVALID),
    (dict(q_rot_stride=(1020, 64)), INVALID),
])
def test_both_calls_refuse(lib, kw, code):
    p = params(**kw)
    assert size(lib, p) == 0
    assert call(lib, "attn_latent_append", p) == code
    assert fwd(lib, p) == code


@pytest.mark.parametrize("kw", [
    dict(c_new=None), dict(k_rope=None), dict(q_rot=None), dict(c_new=FAKE + 8),
    dict(k_rope=FAKE + 2), dict(q_rope=FAKE + 4), dict(c_new_stride=504), dict(k_rope_stride=68),
    dict(q_rope_stride=(1024, 60)), dict(q_rope_stride=(0, 64)),
    dict(q_rope=2 * FAKE, q_rope_stride=(2048, 64)), dict(q_rope=2 * FAKE, q_rope_stride=(1024, 72)),
    dict(rope_len=-1), dict(rope_cos=None), dict(rope_sin=None), dict(rope_cos=FAKE + 4),
    dict(rope_sin=FAKE + 8), dict(rope_pos=FAKE + 2),
])
def test_append_refuses(lib, kw):
    assert call(lib, "attn_latent_append", params(**kw)) == INVALID
    if "q_rot" not in kw:
        assert size(lib, params(**kw)) > 0  # the attention does not read these fields


def test_fwd_refuses(lib):
    for kw in (dict(q_lat=None), dict(q_rot=None), dict(q_lat=FAKE + 8), dict(sink=FAKE + 2),
               dict(q_lat_stride=(8192, 504)), dict(q_lat_stride=(8196, 512)),
               *(dict(scale=s) for s in (0.0, -1.0, NAN, INF))):
        assert fwd(lib, params(**kw)) == INVALID and size(lib, params(**kw)) == 0
    p = params()
    need = size(lib, p)
    assert need > 0
    assert fwd(lib, p, o=0) == INVALID and fwd(lib, p, o=FAKE + 8) == INVALID
    assert fwd(lib, p, lse=FAKE + 2) == INVALID
    assert fwd(lib, p, ws=0) == INVALID and fwd(lib, p, ws=FAKE + 128) == INVALID
    assert fwd(lib, p, ws_bytes=need - 1) == SMALL


def test_nothing_to_do(lib):
    """No sequences or no tokens: nothing is launched, whatever is missing."""
    for kw in (dict(num_seqs=0, num_tokens=0), dict(num_tokens=0, cu_seqlens_q=FAKE)):
        p = params(cache=None, num_pages=0, c_new=None, k_rope=None, q_rope=None, q_lat=None,
                   q_rot=None, seq_lens=None, page_table=None, rope_cos=None, rope_sin=None, **kw)
        assert call(lib, "attn_latent_append", p) == OK
        assert fwd(lib, p, o=0, ws=0, ws_bytes=0) == OK


def test_sequences_beyond_32_bits_of_work(lib):
    """Offsets allow more sequences than tokens: their number is bounded by itself."""
    for n in ((1 << 30) + 1, (1 << 31) - 1):
        p = params(num_seqs=n, cu_seqlens_q=FAKE)
        assert size(lib, p) == 0
        assert call(lib, "attn_latent_append", p) == UNSUPPORTED
        assert fwd(lib, p) == UNSUPPORTED
    assert size(lib, params(num_seqs=1 << 30, cu_seqlens_q=FAKE)) > 0


def test_workspace_grows_with_the_rows_expected(lib):
    sizes = [size(lib, params(max_q_len=n)) for n in (1, 2, 3, 100)]
    assert sizes == sorted(sizes) and sizes[0] < sizes[1] < sizes[2] == sizes[3]
    assert size(lib, params(max_q_len=(1 << 31) - 1)) == sizes[3]


# ---------------------------------------------------------------- the binding

def tensors():
    bf = dict(dtype=torch.bfloat16)
    return dict(dtype="bf16", cache=torch.zeros(10, 16, 576, **bf), d_c=512,
                page_table=torch.zeros(3, 4, dtype=torch.int32),
                seq_lens=torch.ones(3, dtype=torch.int32), c_new=torch.zeros(3, 512, **bf),
                k_rope=torch.zeros(3, 64, **bf), q_rope=torch.zeros(3, 8, 64, **bf),
                q_lat=torch.zeros(3, 8, 512, **bf), q_rot=torch.zeros(3, 8, 64, **bf),
                rope_cos=torch.zeros(64, 32), rope_sin=torch.zeros(64, 32), scale=0.1)


def test_binding_fills_the_block():
    t = tensors()
    wide = torch.zeros(10, 16, 600, dtype=torch.bfloat16)
    both = torch.zeros(3, 576, dtype=torch.bfloat16)
    t.update(cache=wide[..., :576], c_new=both[:, :512], k_rope=both[:, 512:],
             q_lat=torch.zeros(8, 3, 512, dtype=torch.bfloat16).transpose(0, 1))
    p = A.make_latent_params(window_left=7, rope_interleaved=True, **t)
    assert (p.num_seqs, p.num_tokens, p.H, p.d_c, p.d_r) == (3, 3, 8, 512, 64)
    assert (p.page_size, p.num_pages, p.max_pages, p.table_stride) == (16, 10, 4, 4)
    assert list(p.cache_stride) == [16 * 600, 600]
    assert (p.c_new_stride, p.k_rope_stride) == (576, 576)
    assert list(p.q_lat_stride) == [512, 3 * 512] and list(p.q_rot_stride) == [512, 64]
    assert (p.rope_len, p.rot_interleaved, p.window_left, p.mask) == (64, 1, 7, 1)


BF = dict(dtype=torch.bfloat16)


@pytest.mark.parametrize("kw", [
    dict(cache=torch.zeros(10, 16, 576)), dict(cache=torch.zeros(10, 576, 16, **BF).transpose(1, 2)),
    dict(cache=torch.zeros(10, 576, **BF)), dict(c_new=torch.zeros(4, 512, **BF)),
    dict(c_new=torch.zeros(3, 256, **BF)), dict(k_rope=torch.zeros(3, 32, **BF)),
    dict(q_rope=torch.zeros(3, 4, 64, **BF)), dict(q_rot=torch.zeros(3, 8, 64)),
    dict(q_lat=torch.zeros(3, 8, 256, **BF)), dict(q_lat=torch.zeros(3, 512, 8, **BF).transpose(1, 2)),
    dict(seq_lens=torch.ones(3, dtype=torch.int64)), dict(seq_lens=torch.ones(6, dtype=torch.int32)[::2]),
    dict(page_table=torch.zeros(2, 4, dtype=torch.int32)),
    dict(page_table=torch.zeros(4, 3, dtype=torch.int32).t()),
    dict(cu_seqlens_q=torch.zeros(3, dtype=torch.int32)), dict(rope_sin=None),
    dict(rope_sin=torch.zeros(64, 16)), dict(rope_cos=torch.zeros(64, 16), rope_sin=torch.zeros(64, 16)),
    dict(rope_pos=torch.zeros(4, dtype=torch.int32)), dict(sink=torch.zeros(2)),
    dict(sink=torch.zeros(8, device="meta")), dict(dtype="fp8_e4m3"),
    dict(c_new=None, q_rope=None, q_lat=None, q_rot=None),
])
def test_binding_refuses(kw):
    t = tensors()
    t.update(kw)
    with pytest.raises(ValueError):
        A.make_latent_params(**t)


def rope_tensors():
    return dict(dtype="bf16", q=torch.zeros(5, 4, 128, **BF), k=torch.zeros(5, 2, 128, **BF),
                rope_cos=torch.zeros(8, 64), rope_sin=torch.zeros(8, 64))


@pytest.mark.parametrize("kw", [
    dict(q=None, k=None), dict(q=torch.zeros(5, 4, 128)), dict(q=torch.zeros(4, 4, 128, **BF)),
    dict(q=torch.zeros(5, 128, 4, **BF).transpose(1, 2)), dict(q_out=torch.zeros(5, 3, 128, **BF)),
    dict(k_out=torch.zeros(4, 2, 128, **BF)), dict(q=None, q_out=torch.zeros(5, 4, 128, **BF)),
    dict(rope_sin=torch.zeros(8, 32)), dict(rope_cos=torch.zeros(64, 8).t()),
    dict(positions=torch.zeros(4, dtype=torch.int32)), dict(positions=torch.zeros(5)),
    dict(positions=torch.zeros(5, dtype=torch.int32), cu_seqlens=torch.zeros(2, dtype=torch.int32)),
    dict(cu_seqlens=torch.zeros(0, dtype=torch.int32)),
    dict(positions=torch.zeros(5, dtype=torch.int32, device="meta")), dict(dtype="fp16"),
])
def test_rope_binding_refuses(kw):
    t = rope_tensors()
    t.update(kw)
    with pytest.raises(ValueError):
        A.make_rope_params(**t)


def test_rope_binding_fills_the_block():
    t = rope_tensors()
    qkv = torch.zeros(5, 8 * 128, **BF)
    t.update(q=qkv[:, :512].unflatten(1, (4, 128)), k=qkv[:, 512:768].unflatten(1, (2, 128)))
    p = A.make_rope_params(cu_seqlens=torch.zeros(4, dtype=torch.int32), inverse=True, **t)
    assert (p.Hq, p.Hkv, p.d, p.rot_dim, p.num_tokens, p.num_segments) == (4, 2, 128, 128, 5, 3)
    assert p.q == p.q_out and p.k == p.k_out and p.k - p.q == 1024
    assert (p.q_stride, p.k_stride, p.q_out_stride, p.inverse) == (1024, 1024, 1024, 1)
    assert A.make_rope_params(**t).seq_len == 5


def expand_tensors():
    return dict(dtype="bf16", kv=torch.zeros(5, 4, 192, **BF), k_rope=torch.zeros(5, 64, **BF),
                k=torch.zeros(5, 4, 192, **BF), v=torch.zeros(5, 4, 64, **BF),
                rope_cos=torch.zeros(8, 32), rope_sin=torch.zeros(8, 32))


@pytest.mark.parametrize("kw", [
    dict(kv=torch.zeros(5, 4, 200, **BF)), dict(kv=torch.zeros(5, 4, 192)),
    dict(k_rope=torch.zeros(4, 64, **BF)), dict(k=torch.zeros(5, 3, 192, **BF)),
    dict(v=torch.zeros(6, 4, 64, **BF)), dict(k_rope=torch.zeros(64, 5, **BF).t()),
    dict(rope_cos=torch.zeros(8, 16), rope_sin=torch.zeros(8, 16)),
])
def test_expand_binding_refuses(kw):
    t = expand_tensors()
    t.update(kw)
    with pytest.raises(ValueError):
        A.make_latent_expand_params(**t)


@pytest.mark.parametrize("kw", [
    dict(cos=torch.zeros(8, 8), sin=torch.zeros(8, 4)), dict(cos=torch.zeros(8, 8).half(),
                                                             sin=torch.zeros(8, 8)),
    dict(cos=torch.zeros(8, 8).t(), sin=torch.zeros(16, 8)[::2]),
])
def test_table_binding_refuses(kw):
    with pytest.raises(ValueError):
        A.make_rope_table_params(**kw)


def test_fwd_refuses_outputs_of_another_type_or_device(monkeypatch):
    """Raised before the library is called: nothing is launched."""
    p = A.attn_latent_params_t()
    p.device, p.num_tokens, p.H, p.d_c, p.dtype = 0, 2, 4, 256, A.DTYPES["bf16"]
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(A, "load_library", lambda: pytest.fail("the library was called"))
    o, lse = torch.empty(2, 4, 256, **BF), torch.empty(4, 2)
    ws = torch.empty(1 << 20, dtype=torch.uint8)
    with pytest.raises(ValueError):
        A.attn_latent_fwd(p, o, lse, ws)
    # as if on the device: the types alone are wrong, or the workspace lies in parts
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    for bad in ((o.half(), lse, ws), (o, lse.int(), ws), (o, lse, ws[::2]), (o[:1], lse, ws)):
        with pytest.raises(ValueError):
            A.attn_latent_fwd(p, *bad)
    p.device = 1  # the block's tensors are elsewhere
    for f in (A.attn_latent_append, A.attn_rope, A.attn_rope_table, A.attn_latent_expand):
        with pytest.raises(ValueError):
            f(p)
