"""Rotary positions on the GPU against the float64 oracle: tables, turning in
every layout, the inverse as gradient, and positions given in each way."""
import numpy as np
import pytest
import torch

from bwd_tcgen05_tma_gb300 import attn as A
from bwd_tcgen05_tma_gb300 import inputs as I
from latent_util import dev16, turn_tolerance
from oracle import latent_ref as L

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bwd_tcgen05_tma_gb300 import build

    build.build()


def bits(t):
    return t.contiguous().view(torch.uint8)


# ---------------------------------------------------------------- tables

TABLES = {
    "plain": dict(rope_len=1000, rot=128),
    "one_row": dict(rope_len=1, rot=16),
    "odd": dict(rope_len=333, rot=48, base=500000.0),
    "widest": dict(rope_len=77, rot=256),
    "linear": dict(rope_len=500, rot=64, scaling="LINEAR", factor=4.0),
    "base": dict(rope_len=500, rot=64, scaling="BASE", factor=8.0),
    "base_16": dict(rope_len=500, rot=16, scaling="BASE", factor=2.5),
    "turns": dict(rope_len=2000, rot=64, scaling="TURNS", factor=16.0, trained_len=4096,
                  turns=(1.0, 32.0), magnitude=1.277),
    "turns_all_kept": dict(rope_len=300, rot=32, scaling="TURNS", factor=16.0, trained_len=1 << 30,
                           turns=(0.25, 0.5)),
    "base_1": dict(rope_len=300, rot=32, base=1.0, magnitude=-0.5),
    "far": dict(rope_len=1 << 20, rot=16),
}


@pytest.mark.parametrize("name", list(TABLES))
def test_table(name):
    """Off by at most 2^-22 of the magnitude.  (A frequency is off by a unit or
    two of fp64, 2^-52 relative, which over 2^20 positions of at most one radian
    each is 2^-32; the oracle's angles the same.)"""
    c = dict(TABLES[name])
    n, rot, mag = c.pop("rope_len"), c.pop("rot"), c.pop("magnitude", 1.0)
    cos, sin = (torch.full((n, rot // 2), float("nan"), device="cuda") for _ in "cs")
    A.attn_rope_table(A.make_rope_table_params(cos=cos, sin=sin, magnitude=mag, **c))
    freq = L.frequencies(rot, **c)
    for got, ref in zip((cos, sin), L.rope_table(n, freq, np.float32(mag))):
        err = np.abs(got.double().cpu().numpy() - ref).max()
        assert err <= 2.0 ** -22 * abs(mag), err / (2.0 ** -22 * abs(mag))


def test_table_at_far_positions():
    """The last of 2^24 positions against angles reduced exactly."""
    from fractions import Fraction
    import math

    n = 1 << 24
    cos, sin = (torch.empty(n, 8, device="cuda") for _ in "cs")
    A.attn_rope_table(A.make_rope_table_params(cos=cos, sin=sin, base=10000.0))
    freq = L.frequencies(16)
    turn = Fraction(2 * math.pi)
    for j in (n - 1, n - 2, n // 2 + 1):
        for p in range(8):
            # the angle modulo the fp64 value of 2 pi, whose own error of 2^-52
            # relative adds j f 2^-53 < 2^-29
            a = float((j * Fraction(float(freq[p]))) % turn)
            assert abs(float(cos[j, p]) - math.cos(a)) <= 2.0 ** -22
            assert abs(float(sin[j, p]) - math.sin(a)) <= 2.0 ** -22


def test_empty_table():
    cos, sin = (torch.empty(0, 8, device="cuda") for _ in "cs")
    A.attn_rope_table(A.make_rope_table_params(cos=cos, sin=sin))


# ---------------------------------------------------------------- turning

def tables(n, rot, mag=1.0):
    cos, sin = (torch.empty(n, rot // 2, device="cuda") for _ in "cs")
    A.attn_rope_table(A.make_rope_table_params(cos=cos, sin=sin, base=100.0, magnitude=mag))
    return cos, sin


def angles(cos, sin, pos):
    return cos.double().cpu().numpy()[pos], sin.double().cpu().numpy()[pos]


def draw(rng, shape, dtype):
    return I.round_to(rng.standard_normal(shape), dtype).astype(np.float64)


ROPE = {
    "d128": dict(T=37, Hq=4, Hkv=2, d=128, rot=128),
    "one_token": dict(T=1, Hq=1, Hkv=1, d=64, rot=64),
    "wide_gqa": dict(T=20, Hq=33, Hkv=3, d=128, rot=128),
    "partial": dict(T=50, Hq=7, Hkv=1, d=128, rot=64),
    "partial_16": dict(T=50, Hq=3, Hkv=2, d=64, rot=16),
    "behind": dict(T=50, Hq=5, Hkv=5, d=192, start=128, rot=64),
    "middle": dict(T=9, Hq=5, Hkv=2, d=192, start=40, rot=96),
    "d192": dict(T=9, Hq=5, Hkv=2, d=192, rot=192),
    "rot48": dict(T=33, Hq=6, Hkv=1, d=64, rot=48, start=8),
    "d256": dict(T=9, Hq=3, Hkv=2, d=256, rot=256),
    "d16": dict(T=300, Hq=3, Hkv=2, d=16, rot=16),
    "queries": dict(T=20, Hq=4, Hkv=0, d=128, rot=128),
    "keys": dict(T=20, Hq=0, Hkv=4, d=128, rot=64),
}


def check(got, x, cos, sin, c, dtype, mag, inverse):
    start, rot = c.get("start", 0), c["rot"]
    ref = L.turn(x, cos, sin, start, c["interleaved"], inverse)
    out = got.double().cpu().numpy()
    turned = np.zeros(x.shape[-1], bool)
    turned[start:start + rot] = True
    assert np.array_equal(out[..., ~turned], x[..., ~turned])
    tol = turn_tolerance(ref, np.abs(x).max(-1, keepdims=True), dtype, mag)
    err = np.abs(out - ref)
    assert (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("name", list(ROPE))
def test_rope(name, interleaved, inverse):
    """Out of place and in place give the same bits, which are right."""
    c = dict(ROPE[name], interleaved=interleaved)
    dtype = "fp16" if len(name) % 2 else "bf16"
    rng = np.random.default_rng(61)
    T, mag = c["T"], 1.25
    cos, sin = tables(64, c["rot"], mag)
    pos = rng.integers(0, 64, T)
    cc, ss = angles(cos, sin, pos)
    kw = dict(dtype=dtype, rope_cos=cos, rope_sin=sin, rot_start=c.get("start", 0),
              positions=torch.tensor(pos, dtype=torch.int32, device="cuda"),
              interleaved=interleaved, inverse=inverse,
              status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    host = {n: draw(rng, (T, h, c["d"]), dtype) for n, h in (("q", c["Hq"]), ("k", c["Hkv"])) if h}
    dev = {n: dev16(x, dtype) for n, x in host.items()}
    outs = {n + "_out": torch.full_like(x, float("nan")) for n, x in dev.items()}
    keep = {n: x.clone() for n, x in dev.items()}
    A.attn_rope(A.make_rope_params(**dev, **outs, **kw))
    for n, x in dev.items():
        assert torch.equal(bits(x), bits(keep[n]))
        check(outs[n + "_out"], host[n], cc, ss, c, dtype, mag, inverse)
    A.attn_rope(A.make_rope_params(**dev, **kw))
    for n, x in dev.items():
        assert torch.equal(bits(x), bits(outs[n + "_out"]))
    assert kw["status"].item() == 0


@pytest.mark.parametrize("layout", ["3HD", "HD_2HD"])
def test_rope_in_place_of_packed_layouts(layout):
    """Slices of the fused projections; the rest of their rows stays."""
    rng = np.random.default_rng(62)
    T, Hq, Hkv, d = 75, 6, 2, 128
    cos, sin = tables(T, d)
    if layout == "3HD":
        buf = dev16(draw(rng, (T, (Hq + 2 * Hkv) * d), "bf16"), "bf16")
        q = buf[:, :Hq * d].unflatten(1, (Hq, d))
        k = buf[:, Hq * d:(Hq + Hkv) * d].unflatten(1, (Hkv, d))
        v = buf[:, (Hq + Hkv) * d:]
    else:
        q = dev16(draw(rng, (T, Hq, d), "bf16"), "bf16")
        buf = dev16(draw(rng, (T, 2, Hkv, d), "bf16"), "bf16")
        k, v = buf[:, 0], buf[:, 1]
    host = {n: x.double().cpu().numpy() for n, x in (("q", q), ("k", k))}
    keep = v.clone()
    A.attn_rope(A.make_rope_params(dtype="bf16", q=q, k=k, rope_cos=cos, rope_sin=sin))
    cc, ss = angles(cos, sin, np.arange(T))
    c = dict(rot=d, interleaved=False)
    for n, x in (("q", q), ("k", k)):
        check(x, host[n], cc, ss, c, "bf16", 1.0, False)
    assert torch.equal(bits(v), bits(keep))


def test_positions_of_rows_and_segments():
    """Dense rows restart at every row; offsets restart at every segment, leave
    empty ones out and do not touch padding."""
    rng = np.random.default_rng(63)
    cos, sin = tables(40, 64)
    x = draw(rng, (3 * 37, 2, 64), "bf16")
    c = dict(rot=64, interleaved=True)
    kw = dict(dtype="bf16", rope_cos=cos, rope_sin=sin, interleaved=True)
    q = dev16(x, "bf16")
    A.attn_rope(A.make_rope_params(q=q, seq_len=37, **kw))
    check(q, x, *angles(cos, sin, np.arange(111) % 37), c, "bf16", 1.0, False)

    cu = [5, 5, 35, 36, 36, 70, 109]
    q = dev16(x, "bf16")
    q[:5], q[109:] = float("nan"), float("nan")
    out = torch.full_like(q, 7.0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    A.attn_rope(A.make_rope_params(q=q, q_out=out, status=status, cu_seqlens=torch.tensor(
        cu, dtype=torch.int32, device="cuda"), **kw))
    assert status.item() == 0
    assert (out[:5] == 7).all() and (out[109:] == 7).all()
    pos = np.concatenate([np.arange(b - a) for a, b in zip(cu, cu[1:])])
    check(out[5:109], x[5:109], *angles(cos, sin, pos), c, "bf16", 1.0, False)


def test_bad_positions_and_offsets_are_reported():
    x = torch.randn(6, 2, 64, device="cuda").bfloat16()
    cos, sin = tables(4, 64)
    i32 = dict(dtype=torch.int32, device="cuda")

    def run(**kw):
        out, status = torch.full_like(x, 7.0), torch.zeros(1, **i32)
        A.attn_rope(A.make_rope_params(dtype="bf16", q=x, q_out=out, rope_cos=cos, rope_sin=sin,
                                       status=status, **kw))
        return out, status.item()

    out, s = run(positions=torch.tensor([0, -1, 3, 4, 2 ** 31 - 1, 1], **i32))
    assert s == 7
    left = (out == 7).flatten(1).all(1)
    assert left.tolist() == [False, True, False, True, True, False]
    out, s = run(positions=torch.tensor([0, 3, 2, 1, 1, 1], **i32))
    assert s == 0 and not (out == 7).flatten(1).all(1).any()
    out, s = run()  # one row of six tokens, a table of four
    assert s == 7 and (out == 7).flatten(1).all(1).tolist() == [False] * 4 + [True] * 2
    # the second offset lies behind the last token
    out, s = run(cu_seqlens=torch.tensor([0, 9, 3, 6], **i32))
    assert s == 7
    out, s = run(cu_seqlens=torch.tensor([0], **i32))  # no segment: all padding
    assert s == 0 and (out == 7).all()


def test_no_tokens():
    x = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    cos, sin = tables(4, 64)
    A.attn_rope(A.make_rope_params(dtype="bf16", q=x, k=x, rope_cos=cos, rope_sin=sin))


def test_rows_beyond_32_bits():
    """Rows more than 2^32 bytes apart."""
    far = (5 << 30) // 2
    pool = torch.empty(far + 256, dtype=torch.bfloat16, device="cuda")
    q = torch.as_strided(pool, (2, 2, 64), (far, 64, 1))
    x = draw(np.random.default_rng(64), (2, 2, 64), "bf16")
    q.copy_(dev16(x, "bf16"))
    cos, sin = tables(4, 64)
    A.attn_rope(A.make_rope_params(dtype="bf16", q=q, rope_cos=cos, rope_sin=sin))
    check(q, x, *angles(cos, sin, np.arange(2)), dict(rot=64, interleaved=False), "bf16", 1.0,
          False)


@pytest.mark.parametrize("interleaved", [False, True])
def test_inverse_is_the_gradient(interleaved):
    """Against central differences of sum(w * turn(x)) in float64: the map is
    linear, so they are exact but for fp64 rounding (2^-40 here)."""
    rng = np.random.default_rng(65)
    cos, sin = tables(16, 32, 1.1)
    pos = np.arange(4)
    cc, ss = angles(cos, sin, pos)
    x, w = draw(rng, (4, 1, 32), "bf16"), draw(rng, (4, 1, 32), "bf16")
    grad = np.zeros_like(x)
    for idx in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[idx] = 0.5
        grad[idx] = (w * (L.turn(x + e, cc, ss, 0, interleaved) -
                          L.turn(x - e, cc, ss, 0, interleaved))).sum()
    g = dev16(w, "bf16")
    A.attn_rope(A.make_rope_params(dtype="bf16", k=g, rope_cos=cos, rope_sin=sin, inverse=True,
                                   interleaved=interleaved))
    tol = turn_tolerance(grad, np.abs(w).max(), "bf16", 1.1) + 2.0 ** -40
    assert (np.abs(g.double().cpu().numpy() - grad) <= tol).all()
