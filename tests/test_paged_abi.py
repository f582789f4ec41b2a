"""Host-side checks of the paged-cache calls (no GPU needed): every refusal
the header names, workspace sizes, and the binding's own checks of tensors.
Pointers are fake addresses that no refused call dereferences."""
import ctypes

import pytest
import torch

from bwd_tcgen05_tma_gb300 import attn as A

FAKE = 0x10000000
OK, INVALID, UNSUPPORTED, SHAPE, SMALL = 0, 1, 2, 3, 4


@pytest.fixture(scope="module")
def lib():
    from bwd_tcgen05_tma_gb300 import build

    build.build()
    return A.load_library()


def params(**kw):
    p = A.attn_paged_params_t()
    p.struct_version = A.ATTN_PAGED_PARAMS_VERSION
    p.dtype, p.cache_dtype, p.mask = 0, 2, 1
    p.num_seqs, p.num_tokens, p.max_q_len = 4, 4, 1
    p.Hq, p.Hkv, p.d_qk, p.d_v = 8, 2, 128, 128
    p.page_size, p.num_pages, p.max_pages = 64, 100, 10
    p.page_table, p.table_stride, p.seq_lens = FAKE, 10, FAKE
    p.k_cache, p.v_cache = FAKE, FAKE
    for s in (p.k_cache_stride, p.v_cache_stride):
        s[0], s[1], s[2] = 2 * 64 * 128, 64 * 128, 128
    p.k_scale, p.v_scale = FAKE, FAKE
    p.q, p.k_new, p.v_new, p.q_rot = FAKE, FAKE, FAKE, FAKE
    p.q_stride = p.q_rot_stride = 8 * 128
    p.k_new_stride = p.v_new_stride = 2 * 128
    p.rot_dim, p.rope_len, p.rope_cos, p.rope_sin = 128, 640, FAKE, FAKE
    p.scale, p.window_left = 0.1, -1
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def size(lib, p):
    return lib.attn_paged_workspace_size(ctypes.byref(p))


def append(lib, p):
    return lib.attn_paged_append(ctypes.byref(p), None)


def fwd(lib, p, o=FAKE, lse=FAKE, ws=FAKE, ws_bytes=1 << 30):
    v = ctypes.c_void_p
    return lib.attn_paged_fwd(ctypes.byref(p), v(o), v(lse), v(ws), ctypes.c_size_t(ws_bytes), None)


BOTH = [
    (dict(struct_version=0), INVALID), (dict(struct_version=2), INVALID),
    (dict(dtype=2), INVALID), (dict(dtype=-1), INVALID),
    (dict(cache_dtype=1), INVALID),  # a 16-bit cache has the tensors' type
    (dict(cache_dtype=3), INVALID), (dict(mask=2), INVALID), (dict(mask=-1), INVALID),
    (dict(num_seqs=-1), INVALID), (dict(num_tokens=-1), INVALID), (dict(max_q_len=0), INVALID),
    (dict(num_pages=-1), INVALID), (dict(max_pages=-1), INVALID),
    (dict(Hq=0), INVALID), (dict(Hkv=0), INVALID), (dict(Hq=7), INVALID),
    (dict(Hq=512, q_stride=1 << 20, q_rot_stride=1 << 20), UNSUPPORTED),
    (dict(d_qk=96), UNSUPPORTED), (dict(d_v=192), UNSUPPORTED),
    (dict(page_size=8), UNSUPPORTED), (dict(page_size=48), UNSUPPORTED),
    (dict(page_size=512), UNSUPPORTED),
    (dict(max_pages=(1 << 24) + 1, table_stride=1 << 25), UNSUPPORTED),  # over 2^30 positions
    (dict(num_seqs=(1 << 28) + 1, num_tokens=(1 << 28) + 1), UNSUPPORTED),  # over 2^30 rows
    (dict(num_tokens=5), SHAPE),  # one token per sequence without offsets
    (dict(seq_lens=None), INVALID), (dict(page_table=None), INVALID),
    (dict(k_cache=None), INVALID), (dict(v_cache=None), INVALID),
    (dict(k_scale=None), INVALID), (dict(v_scale=None), INVALID),
    (dict(seq_lens=FAKE + 2), INVALID), (dict(page_table=FAKE + 1), INVALID),
    (dict(cu_seqlens_q=FAKE + 2), INVALID), (dict(status=FAKE + 2), INVALID),
    (dict(k_scale=FAKE + 2), INVALID), (dict(k_cache=FAKE + 8), INVALID),
    (dict(v_cache=FAKE + 1), INVALID), (dict(table_stride=9), INVALID),
    (dict(q=FAKE + 8), INVALID), (dict(q_rot=FAKE + 2), INVALID),
    (dict(q_stride=8 * 128 - 8), INVALID), (dict(q_stride=8 * 128 + 4), INVALID),
    (dict(q_rot_stride=0), INVALID),
]


@pytest.mark.parametrize("kw,code", BOTH)
def test_both_calls_refuse(lib, kw, code):
    p = params(**kw)
    assert size(lib, p) == 0
    assert append(lib, p) == code
    assert fwd(lib, p) == code


@pytest.mark.parametrize("field", ["k_cache_stride", "v_cache_stride"])
@pytest.mark.parametrize("axis", [0, 1, 2])
@pytest.mark.parametrize("value", [0, -128, 8, 130])
def test_cache_strides(lib, field, axis, value):
    p = params()
    getattr(p, field)[axis] = value
    assert append(lib, p) == INVALID and fwd(lib, p) == INVALID


def test_scales_only_with_e4m3(lib):
    p = params(cache_dtype=0)
    assert size(lib, p) == 0 and append(lib, p) == INVALID
    p = params(cache_dtype=0, k_scale=None, v_scale=None)
    assert size(lib, p) > 0


@pytest.mark.parametrize("kw,code", [
    (dict(k_new=None), INVALID), (dict(v_new=None), INVALID), (dict(q_rot=None), INVALID),
    (dict(k_new=FAKE + 8), INVALID), (dict(v_new_stride=2 * 128 - 8), INVALID),
    (dict(k_new_stride=2 * 128 + 1), INVALID), (dict(rot_dim=-16), INVALID),
    (dict(rot_dim=144), INVALID), (dict(rot_dim=24), UNSUPPORTED), (dict(rope_cos=None), INVALID),
    (dict(rope_sin=FAKE + 4), INVALID), (dict(rope_len=0), INVALID), (dict(rope_pos=FAKE + 2), INVALID),
])
def test_append_refuses(lib, kw, code):
    assert append(lib, params(**kw)) == code
    if code == INVALID and "q_rot" not in kw:
        assert size(lib, params(**kw)) > 0  # the attention does not read these fields


def test_fwd_refuses(lib):
    assert fwd(lib, params(q=None, q_rot=None)) == INVALID
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert fwd(lib, params(scale=scale)) == INVALID
    assert fwd(lib, params(sink=FAKE + 2)) == INVALID
    p = params()
    need = size(lib, p)
    assert need > 0 and need % 256 == 0
    assert fwd(lib, p, o=0) == INVALID and fwd(lib, p, o=FAKE + 8) == INVALID
    assert fwd(lib, p, lse=FAKE + 2) == INVALID
    assert fwd(lib, p, ws=0) == INVALID and fwd(lib, p, ws=FAKE + 128) == INVALID
    assert fwd(lib, p, ws_bytes=need - 1) == SMALL


def test_nothing_to_do(lib):
    """No sequences or no tokens: nothing is launched, whatever is missing."""
    for kw in (dict(num_seqs=0, num_tokens=0), dict(num_tokens=0, cu_seqlens_q=FAKE)):
        p = params(k_cache=None, v_cache=None, k_scale=None, v_scale=None, num_pages=0, k_new=None,
                   v_new=None, q=None, q_rot=None, seq_lens=None, page_table=None, **kw)
        assert append(lib, p) == OK
        assert fwd(lib, p, o=0, ws=0, ws_bytes=0) == OK


def test_workspace_grows_with_the_rows_expected(lib):
    sizes = [size(lib, params(max_q_len=n)) for n in (1, 3, 5, 100)]
    assert sizes == sorted(sizes) and sizes[0] < sizes[-1]
    assert size(lib, params(max_q_len=1 << 30)) == sizes[-1]


def tensors():
    c = torch.zeros(10, 2, 16, 128, dtype=torch.float8_e4m3fn)
    s = torch.ones(10, 2)
    return dict(dtype="bf16", cache_dtype="fp8_e4m3", k_cache=c, v_cache=c.clone(), k_scale=s,
                v_scale=s.clone(), page_table=torch.zeros(3, 4, dtype=torch.int32),
                seq_lens=torch.ones(3, dtype=torch.int32),
                q=torch.zeros(3, 8, 128, dtype=torch.bfloat16),
                k_new=torch.zeros(3, 2, 128, dtype=torch.bfloat16),
                v_new=torch.zeros(3, 2, 128, dtype=torch.bfloat16),
                q_rot=torch.zeros(3, 8, 128, dtype=torch.bfloat16),
                rope_cos=torch.zeros(64, 32), rope_sin=torch.zeros(64, 32))


def test_binding_fills_the_block():
    t = tensors()
    nhd = torch.zeros(10, 16, 2, 128, dtype=torch.uint8)
    qkv = torch.zeros(3, 12 * 128, dtype=torch.bfloat16)
    t.update(k_cache=nhd.transpose(1, 2), q=qkv[:, :1024].unflatten(1, (8, 128)))
    p = A.make_paged_params(window_left=7, rope_interleaved=True, **t)
    assert (p.num_seqs, p.num_tokens, p.Hq, p.Hkv, p.d_qk, p.d_v) == (3, 3, 8, 2, 128, 128)
    assert (p.page_size, p.num_pages, p.max_pages, p.table_stride) == (16, 10, 4, 4)
    assert list(p.k_cache_stride) == [16 * 2 * 128, 128, 2 * 128]
    assert list(p.v_cache_stride) == [16 * 2 * 128, 16 * 128, 128]
    assert (p.q_stride, p.k_new_stride) == (12 * 128, 2 * 128)
    assert (p.rot_dim, p.rope_len, p.rot_interleaved, p.window_left) == (64, 64, 1, 7)
    assert abs(p.scale - 128 ** -0.5) < 1e-7


@pytest.mark.parametrize("kw", [
    dict(k_cache=torch.zeros(10, 2, 16, 128)),
    dict(v_cache=torch.zeros(10, 2, 32, 128, dtype=torch.float8_e4m3fn)),
    dict(k_cache=torch.zeros(10, 2, 128, 16, dtype=torch.float8_e4m3fn).transpose(2, 3)),
    dict(q=torch.zeros(3, 8, 128)), dict(q=torch.zeros(3, 128, 8, dtype=torch.bfloat16).transpose(1, 2)),
    dict(q=torch.zeros(4, 8, 128, dtype=torch.bfloat16)),
    dict(k_new=torch.zeros(3, 4, 128, dtype=torch.bfloat16)),
    dict(seq_lens=torch.ones(3, dtype=torch.int64)), dict(seq_lens=torch.ones(6, dtype=torch.int32)[::2]),
    dict(page_table=torch.zeros(2, 4, dtype=torch.int32)),
    dict(page_table=torch.zeros(4, 3, dtype=torch.int32).t()),
    dict(cu_seqlens_q=torch.zeros(3, dtype=torch.int32)), dict(k_scale=torch.ones(10, 3)),
    dict(k_scale=torch.ones(2, 10).t()), dict(rope_sin=None), dict(rope_sin=torch.zeros(64, 16)),
    dict(rope_pos=torch.zeros(4, dtype=torch.int32)), dict(sink=torch.zeros(2)),
    dict(sink=torch.zeros(8, device="meta")),
])
def test_binding_refuses(kw):
    t = tensors()
    t.update(kw)
    with pytest.raises(ValueError):
        A.make_paged_params(**t)


def test_fwd_refuses_outputs_of_another_type_or_device(monkeypatch):
    """Raised before the library is called: nothing is launched."""
    p = A.attn_paged_params_t()
    p.device, p.num_tokens, p.Hq, p.d_v, p.dtype = 0, 2, 4, 64, A.DTYPES["bf16"]
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(A, "load_library", lambda: pytest.fail("the library was called"))
    meta = dict(device="meta")
    o, lse = torch.empty(2, 4, 64, dtype=torch.bfloat16), torch.empty(4, 2)
    ws = torch.empty(1 << 20, dtype=torch.uint8)
    for bad in ((o, lse, ws), (o.half(), lse, ws), (o, lse.int(), ws),
                (o.to(**meta), lse.to(**meta), ws.to(**meta))):
        with pytest.raises(ValueError):
            A.attn_paged_fwd(p, *bad)
    # as if on the device: the types alone are wrong, or the workspace lies in parts
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    for bad in ((o.half(), lse, ws), (o, lse.int(), ws), (o, lse, ws[::2])):
        with pytest.raises(ValueError):
            A.attn_paged_fwd(p, *bad)
