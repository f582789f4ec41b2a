"""Seeded latent caches for the tests: host arrays for the oracle and device
tensors for the library, with NaN wherever nothing may be read."""
from __future__ import annotations

import numpy as np
import torch

from bwd_tcgen05_tma_gb300 import attn as A
from bwd_tcgen05_tma_gb300 import inputs as I
from oracle import latent_ref as L
from oracle import paged_ref as P
from paged_util import TORCH, UNIT

SCALE = 192 ** -0.5


def dev16(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda().to(TORCH[dtype])


class Latent:
    """new[s] new tokens behind ctx[s] cached ones for each sequence.

    layout "rows" keeps a page as [page, d], "wide" leaves room behind every row,
    "slots" as [page][pages][d]; by_head: queries as [H, tokens, dim]; fused:
    c_new and k_rope are slices of one projection, q_rope of another; pad: rows
    behind the last sequence; one: no offsets (one new token each)."""

    def __init__(self, new, ctx, *, seed, H=16, d_c=512, page=64, dtype="bf16", interleaved=False,
                 layout="rows", by_head=False, fused=False, pad=0, one=False, spare=2,
                 pos_shift=None, std=1.0):
        rng = np.random.default_rng(seed)
        self.new, self.ctx, self.page, self.dtype, self.cache = new, ctx, page, dtype, dtype
        self.H = self.Hq = H
        self.d_c, self.d_v, self.d_r, self.d_qk = d_c, d_c, 64, d_c + 64
        self.lens = [a + b for a, b in zip(new, ctx)]
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(int).tolist()
        self.T = self.cu[-1] + pad
        self.interleaved, self.one, self.pos_shift = interleaved, one, pos_shift
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
        vals = I.round_to(std * rng.standard_normal((pages, page, self.d_qk)), dtype)
        vals = vals.astype(np.float64)
        keep = np.zeros((pages, page), bool)
        for s in range(len(new)):
            for j in range(ctx[s]):
                keep[self.table[s, j // page], j % page] = True
        self.host = np.where(keep[..., None], vals, np.nan)
        T = self.T
        self.c_new, self.k_rope, self.q_rope, self.q_lat = (
            I.round_to(std * rng.standard_normal(s), dtype).astype(np.float64)
            for s in ((T, d_c), (T, 64), (T, H, 64), (T, H, d_c)))
        ang = L.rope_table(width * page + (pos_shift or 0), L.frequencies(64))
        self.cos, self.sin = (x.astype(np.float32) for x in ang)
        t = self.t = {}
        if fused:
            both = dev16(np.concatenate([self.c_new, self.k_rope], 1), dtype)
            t["c_new"], t["k_rope"] = both[:, :d_c], both[:, d_c:]
            wide = dev16(np.concatenate([rng.standard_normal((T, H, 128)), self.q_rope], 2), dtype)
            t["q_rope"] = wide[..., 128:]
        else:
            t["c_new"], t["k_rope"] = dev16(self.c_new, dtype), dev16(self.k_rope, dtype)
            t["q_rope"] = self._queries(self.q_rope, by_head)
        t["q_lat"] = self._queries(self.q_lat, by_head)
        t["q_rot"] = torch.full_like(t["q_rope"], float("nan")) if not by_head else torch.full(
            (H, T, 64), float("nan"), dtype=TORCH[dtype], device="cuda").transpose(0, 1)
        x = dev16(self.host, dtype)
        if layout == "wide":
            pool = torch.full((pages, page, self.d_qk + 24), float("nan"), dtype=x.dtype,
                              device="cuda")
            pool[..., :self.d_qk] = x
            x = pool[..., :self.d_qk]
        elif layout == "slots":
            x = x.transpose(0, 1).contiguous().transpose(0, 1)
        t["cache"] = x
        i32 = dict(dtype=torch.int32, device="cuda")
        t["table"] = torch.tensor(self.table, **i32)
        t["lens"] = torch.tensor(self.lens, **i32)
        t["cu"] = None if one else torch.tensor(self.cu, **i32)
        t["status"] = torch.zeros(1, **i32)
        t["cos"], t["sin"] = (torch.from_numpy(x).cuda() for x in (self.cos, self.sin))
        t["pos"] = None
        if pos_shift is not None:
            pos = np.zeros(T, np.int32)
            for _, row, p in P.new_rows(self.lens, self.cu):
                pos[row] = p + pos_shift
            t["pos"] = torch.from_numpy(pos).cuda()

    def _queries(self, x, by_head):
        if by_head:
            return dev16(x.transpose(1, 0, 2), self.dtype).transpose(0, 1)
        return dev16(x, self.dtype)

    # ------------------------------------------------------------ the library
    def params(self, **kw):
        t = self.t
        d = dict(dtype=self.dtype, cache=t["cache"], d_c=self.d_c, page_table=t["table"],
                 seq_lens=t["lens"], c_new=t["c_new"], k_rope=t["k_rope"], q_rope=t["q_rope"],
                 q_lat=t["q_lat"], q_rot=t["q_rot"], cu_seqlens_q=t["cu"],
                 max_q_len=max(1, max(self.new)), rope_cos=t["cos"], rope_sin=t["sin"],
                 rope_pos=t["pos"], rope_interleaved=self.interleaved, scale=SCALE,
                 status=t["status"])
        d.update(kw)
        return A.make_latent_params(**d)

    def fresh_outputs(self):
        o = torch.full((self.T, self.H, self.d_c), float("nan"), dtype=TORCH[self.dtype],
                       device="cuda")
        lse = torch.full((self.H, self.T), float("nan"), dtype=torch.float32, device="cuda")
        return o, lse

    def attend(self, p, stream=None):
        o, lse = self.fresh_outputs()
        # whatever the workspace holds has no influence
        ws = torch.full((A.attn_latent_workspace_size(p),), 255, dtype=torch.uint8, device="cuda")
        A.attn_latent_fwd(p, o, lse, ws, stream)
        return o, lse

    def append_and_attend(self, **kw):
        A.attn_latent_append(self.params())
        return self.attend(self.params(**kw))

    def status(self):
        torch.cuda.synchronize()
        return int(self.t["status"].item())

    def cache_host(self):
        return self.t["cache"].double().cpu().numpy()

    # -------------------------------------------------------------- the oracle
    def angles(self, rows):
        return self.cos[rows].astype(np.float64), self.sin[rows].astype(np.float64)

    def rotated(self, x):
        """x [tokens, heads, 64] turned; padding rows as they are."""
        y = np.array(x)
        for _, row, pos in P.new_rows(self.lens, self.cu):
            c, s = self.angles([pos + (self.pos_shift or 0)])
            y[row] = L.turn(x[row][None], c, s, interleaved=self.interleaved)[0]
        return y

    def queries(self):
        """The queries the attention is given, as the device holds them."""
        return np.concatenate([self.q_lat, self.t["q_rot"].double().cpu().numpy()], -1)

    def oracle_attend(self, **kw):
        """The attention over the cache and the queries as the device holds them
        (so that only the attention is compared)."""
        host = self.cache_host()

        def rows_of(s):
            j = np.arange(min(self.lens[s], self.table.shape[1] * self.page))
            return host[self.table[s, j // self.page], j % self.page]

        kw.setdefault("scale", SCALE)
        return L.attend(self.queries(), rows_of, self.d_c, self.lens, self.cu, **kw)


def written_slots(c):
    """Bool [pages, page]: slots of the new tokens."""
    w = np.zeros(c.host.shape[:2], bool)
    for s, _, pos in P.new_rows(c.lens, c.cu):
        w[c.table[s, pos // c.page], pos % c.page] = True
    return w


def turn_tolerance(exact, big, dtype, magnitude=1.0):
    """A turned value is rounded once (half a step) after two fp32 products and a
    sum, each rounded: 3 * 2^-24 of |a cos| + |b sin| <= 2 `big`."""
    sub = 2.0 ** -25 if dtype == "fp16" else 0.0
    f32 = 6 * 2.0 ** -24 * big * magnitude
    return (UNIT[dtype] * np.abs(exact) + f32) * (1 + UNIT[dtype]) + sub
