"""Seeded paged caches for the tests: host arrays for the oracle and device
tensors for the library, with NaN wherever nothing may be read."""
from __future__ import annotations

import numpy as np
import torch

from bwd_tcgen05_tma_gb300 import attn as A
from bwd_tcgen05_tma_gb300 import inputs as I
from oracle import paged_ref as P

UNIT = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}  # half a step, relative
TORCH = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp8_e4m3": torch.float8_e4m3fn}
VALUES = P.e4m3_values()


class Paged:
    """new[s] new tokens behind ctx[s] cached ones for each sequence.

    layout "hnd" keeps a page as [Hkv, page, dim], "nhd" as [page, Hkv, dim],
    "packed" leaves room for another cache between pages and behind dims;
    fused: q, k_new, v_new are slices of one projection; pad: rows behind the
    last sequence; one: no offsets (one new token each)."""

    def __init__(self, new, ctx, *, seed, Hq=4, Hkv=2, d_qk=128, d_v=128, page=16, dtype="bf16",
                 cache="fp8_e4m3", rot=None, interleaved=False, layout="hnd", fused=False, pad=0,
                 one=False, spare=2, pos_shift=None, grow=1.0, std=1.0, device="cuda"):
        rng = np.random.default_rng(seed)
        self.new, self.ctx, self.page, self.dtype, self.cache = new, ctx, page, dtype, cache
        self.Hq, self.Hkv, self.d_qk, self.d_v = Hq, Hkv, d_qk, d_v
        self.lens = [a + b for a, b in zip(new, ctx)]
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(int).tolist()
        self.T = self.cu[-1] + pad
        self.interleaved, self.device = interleaved, device
        used = [-(-n // page) for n in self.lens]
        width = max(max(used), 1) + 1
        pages = sum(used) + spare
        ids = rng.permutation(pages)
        # entries behind a sequence's pages are never to be used
        self.table = np.full((len(new), width), 2 ** 31 - 1, np.int64)
        at = 0
        for s, u in enumerate(used):
            self.table[s, :u] = ids[at:at + u]
            at += u
        self.host = {}
        for name, d in (("k", d_qk), ("v", d_v)):
            if cache == "fp8_e4m3":
                codes = rng.integers(0, 127, (pages, Hkv, page, d)) | (
                    rng.integers(0, 2, (pages, Hkv, page, d)) << 7)
                vals = VALUES[codes]
                scale = 2.0 ** rng.integers(-9, -6, (pages, Hkv))
            else:
                vals, scale = I.round_to(std * rng.standard_normal((pages, Hkv, page, d)),
                                         cache).astype(np.float64), None
            keep = np.zeros((pages, page), bool)
            listed = np.zeros(pages, bool)
            for s in range(len(new)):
                listed[self.table[s, :used[s]]] = True
                for j in range(ctx[s]):
                    keep[self.table[s, j // page], j % page] = True
            vals = np.where(keep[:, None, :, None], vals, np.nan)
            if scale is not None:
                scale = np.where(listed[:, None], scale, np.nan)
            self.host[name] = [vals, scale]
        shape = ((self.T, Hq, d_qk), (self.T, Hkv, d_qk), (self.T, Hkv, d_v))
        self.q, self.k_new, self.v_new = (
            I.round_to(std * rng.standard_normal(s), dtype).astype(np.float64) for s in shape)
        self.k_new[::3] = I.round_to(self.k_new[::3] * grow, dtype)
        self.rot = d_qk if rot is None else rot
        self.pos_shift = pos_shift
        rope_len = width * page + (pos_shift or 0)
        ang = np.arange(rope_len)[:, None] * 10000.0 ** (-np.arange(self.rot // 2) /
                                                        max(1, self.rot // 2))
        self.cos, self.sin = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)

        def dev16(x):
            return torch.from_numpy(x).to(device).to(TORCH[dtype])

        t = self.t = {}
        if fused:
            flat = np.concatenate([x.reshape(self.T, -1) for x in (self.q, self.k_new, self.v_new)],
                                  1)
            t["qkv"] = dev16(flat)
            a, b = Hq * d_qk, Hq * d_qk + Hkv * d_qk
            t["q"] = t["qkv"][:, :a].unflatten(1, (Hq, d_qk))
            t["k_new"] = t["qkv"][:, a:b].unflatten(1, (Hkv, d_qk))
            t["v_new"] = t["qkv"][:, b:].unflatten(1, (Hkv, d_v))
        else:
            t["q"], t["k_new"], t["v_new"] = dev16(self.q), dev16(self.k_new), dev16(self.v_new)
        for name in ("k", "v"):
            vals, scale = self.host[name]
            x = torch.from_numpy(vals).to(device)
            x = x.float().to(TORCH[cache])
            d = x.shape[3]
            if layout == "packed":  # K and V of a page side by side
                both = torch.zeros(pages, 2, *x.shape[1:3], max(d_qk, d_v), dtype=torch.uint8,
                                   device=device)
                if cache != "fp8_e4m3":
                    both = both.to(torch.int16)
                side = both[:, 0 if name == "k" else 1, :, :, :d]
                side.copy_(x.view(both.dtype))
                x = both.view(TORCH[cache])[:, 0 if name == "k" else 1, :, :, :d]
            elif layout == "nhd":
                x = x.view(torch.uint8 if cache == "fp8_e4m3" else torch.int16)
                x = x.transpose(1, 2).contiguous().view(TORCH[cache]).transpose(1, 2)
            t[name + "_cache"] = x
            t[name + "_scale"] = None if scale is None else torch.from_numpy(scale).float().to(device)
        t["q_rot"] = torch.full((self.T, Hq, d_qk), float("nan"), dtype=TORCH[dtype], device=device)
        i32 = dict(dtype=torch.int32, device=device)
        t["table"] = torch.tensor(self.table, **i32)
        t["lens"] = torch.tensor(self.lens, **i32)
        t["cu"] = None if one else torch.tensor(self.cu, **i32)
        t["status"] = torch.zeros(1, **i32)
        t["cos"], t["sin"] = (torch.from_numpy(x).to(device) for x in (self.cos, self.sin))
        t["pos"] = None
        if pos_shift is not None:
            pos = np.zeros(self.T, np.int32)
            for _, row, p in P.new_rows(self.lens, self.cu):
                pos[row] = p + pos_shift
            t["pos"] = torch.from_numpy(pos).to(device)
        self.one = one

    # ------------------------------------------------------------ the library
    def params(self, **kw):
        t = self.t
        d = dict(dtype=self.dtype, cache_dtype=self.cache, q=t["q"], k_new=t["k_new"],
                 v_new=t["v_new"], q_rot=t["q_rot"], k_cache=t["k_cache"], v_cache=t["v_cache"],
                 k_scale=t["k_scale"], v_scale=t["v_scale"], page_table=t["table"],
                 seq_lens=t["lens"], cu_seqlens_q=t["cu"], max_q_len=max(1, max(self.new)),
                 rope_cos=t["cos"] if self.rot else None, rope_sin=t["sin"] if self.rot else None,
                 rope_pos=t["pos"], rope_interleaved=self.interleaved, status=t["status"])
        d.update(kw)
        return A.make_paged_params(**d)

    def fresh_outputs(self):
        o = torch.full((self.T, self.Hq, self.d_v), float("nan"), dtype=TORCH[self.dtype],
                       device=self.device)
        lse = torch.full((self.Hq, self.T), float("nan"), dtype=torch.float32, device=self.device)
        return o, lse

    def attend(self, p, stream=None):
        o, lse = self.fresh_outputs()
        # whatever the workspace holds has no influence
        ws = torch.full((A.attn_paged_workspace_size(p),), 255, dtype=torch.uint8,
                        device=self.device)
        A.attn_paged_fwd(p, o, lse, ws, stream)
        return o, lse

    def status(self):
        torch.cuda.synchronize()
        return int(self.t["status"].item())

    def cache_host(self, name):
        """Device cache as float64 code values / values, and scales."""
        x = self.t[name + "_cache"].float().double().cpu().numpy()
        s = self.t[name + "_scale"]
        return x, None if s is None else s.double().cpu().numpy()

    # -------------------------------------------------------------- the oracle
    def rotated(self, x):
        y = np.array(x)
        if self.rot:
            for _, row, pos in P.new_rows(self.lens, self.cu):
                r = pos + (self.pos_shift or 0)
                y[row] = P.rotate(x[row], self.cos[r].astype(np.float64),
                                  self.sin[r].astype(np.float64), self.interleaved)
        return y

    def oracle_append(self):
        for name, x in (("k", self.rotated(self.k_new)), ("v", self.v_new)):
            P.append(*self.host[name], self.table, self.page, self.lens, self.cu, x)

    def oracle_attend(self, q, from_device=True, **kw):
        """The attention of `q` (float64) over the cache as the device holds it
        (so that only the attention is compared) or as the oracle does."""
        src = {n: self.cache_host(n) if from_device else self.host[n] for n in ("k", "v")}

        def of(name):
            return lambda s: P.gather(*src[name], self.table[s], self.page, self.lens[s])

        kw.setdefault("scale", self.d_qk ** -0.5)
        return P.attend(q, of("k"), of("v"), self.lens, self.cu, **kw)


def written_slots(c):
    """Bool [pages, page]: slots of the new tokens."""
    w = np.zeros((c.host["k"][0].shape[0], c.page), bool)
    for s, _, pos in P.new_rows(c.lens, c.cu):
        w[c.table[s, pos // c.page], pos % c.page] = True
    return w


def check_attend(c, o, lse, ref, cache=None):
    """Error bounds, element by element.  With u the half step of a type:
    O is rounded once (u_out |O|); each P_ij is rounded to the MMA's type
    (fp16, or bf16 with a bf16 cache: u_p A, A = sum_j P |V|); a score is a
    fp32 sum of d + 1 terms and a few products, off by at most
    delta = (d + 8) 2^-24 D with D = max_j scale sum |q k| (+ 2^-22 of the
    score for the exponent's argument), which moves P and the normaliser by
    that much relatively each; 2^-17 covers the exponentials and the fp32 sums
    of P V over the lengths used here."""
    ro, rl, rA, rD = ref
    rows = slice(0, c.cu[-1])
    got, gl = o.double().cpu().numpy(), lse.double().cpu().numpy()
    u_out, u_p = UNIT[c.dtype], UNIT["bf16" if (cache or c.cache) == "bf16" else "fp16"]
    delta = (c.d_qk + 16) * 2.0 ** -24 * rD
    tol = u_out * np.abs(ro) + (u_p + 2.0 ** -17 + 2 * delta[..., None]) * rA * (1 + u_out) + 1e-7
    if c.dtype == "fp16":
        tol += 2.0 ** -25
    err = np.abs(got - ro)[rows]
    assert np.isfinite(got[rows]).all()
    assert (err <= tol[rows]).all(), float((err / tol[rows]).max())
    fin = np.isfinite(rl[:, rows])
    assert np.array_equal(fin, np.isfinite(gl[:, rows]))
    assert np.array_equal(gl[:, rows][~fin], rl[:, rows][~fin])
    lt = delta.T + 2.0 ** -20 * (1 + np.abs(np.where(np.isfinite(rl), rl, 0)))
    assert (np.abs(gl - rl)[:, rows][fin] <= lt[:, rows][fin]).all()
    # rows behind the last sequence are left as they were
    assert np.isnan(got[c.cu[-1]:]).all() and np.isnan(gl[:, c.cu[-1]:]).all()
