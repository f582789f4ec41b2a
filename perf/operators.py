"""Workloads of the paged KV cache: appending new tokens and attending to them.

Two operators are measured, each over its range of uses:

* ``append``: the new tokens' queries and keys are rotated by their positions,
  and the keys and values are written into the pages of a cache.  An E4M3 cache
  keeps one power-of-two scale for each page and head; a page whose scale has
  to grow has its earlier codes rounded again under the new one.
* ``attend``: the new tokens' queries attend to everything their sequence has
  in the cache (softmax over the keys that the causal mask and the window keep,
  with an optional sink logit), straight from the pages.

``run`` computes either the plain form (elementary torch operations, fp32) or,
where ``own`` is true, the library's calls.  ``exact`` is the definition in 64
bits.
"""
import math
import random

import torch

own = False

ROPE_BASE = 10000.0
MIN_EXP = -64  # smallest exponent of a page's scale


def _case(name, op, **kw):
    c = dict(name=name, op=op, seqs=1, q_min=1, q_max=1, ctx_min=0, ctx_max=0, Hq=32, Hkv=8,
             d_qk=128, d_v=128, page=64, dtype="bf16", cache="fp8_e4m3", rot=128,
             interleaved=False, window=-1, sink=False, lens=1)
    c.update(kw)
    return c


def listed():
    return [
        # one user's decode step: the latency of a single token
        _case("append_decode_1", "append", ctx_min=2001, ctx_max=2001),
        # a decode step of a server's batch, sequences of all lengths
        _case("append_decode_64", "append", seqs=64, ctx_min=1, ctx_max=2048, lens=2),
        # a packed prefill batch of the THD sizes: 16 prompts of 64 to 2048 tokens
        _case("append_prefill_thd", "append", seqs=16, q_min=64, q_max=2048, ctx_max=1000,
              lens=3),
        # prefill into a 16-bit cache, 192-wide keys with rotation of a part of
        # the head (pairs side by side), small pages
        _case("append_prefill_192", "append", seqs=3, q_min=500, q_max=2048, Hq=16, Hkv=16,
              d_qk=192, page=16, cache="bf16", rot=64, interleaved=True, lens=4),
        # one user's decode step over a short context
        _case("attend_decode_1", "attend", ctx_min=1000, ctx_max=1000),
        # many short chats: the batch is wide, the contexts are a few pages
        _case("attend_decode_256_short", "attend", seqs=256, ctx_min=0, ctx_max=255, lens=5),
        # a server's decode batch with ragged contexts up to the THD row length
        _case("attend_decode_32", "attend", seqs=32, ctx_min=63, ctx_max=8191, lens=6),
        # long documents: four contexts of up to 131072 tokens, 8 query heads to a
        # KV head as in the long-context workload
        _case("attend_decode_long", "attend", seqs=4, ctx_min=100000, ctx_max=131071, Hq=64,
              lens=7),
        # checking four drafted tokens at a time in fp16, 64-wide heads with sink
        # logits and a sliding window
        _case("attend_verify_window", "attend", seqs=16, q_min=2, q_max=5, ctx_min=500,
              ctx_max=8000, Hq=16, Hkv=4, d_qk=64, d_v=64, rot=64, dtype="fp16", window=4095,
              sink=True, page=32, lens=8),
        # decode from a 16-bit cache, 192-wide keys, as many KV heads as query heads
        _case("attend_decode_192_bf16", "attend", seqs=16, ctx_min=100, ctx_max=4095, Hq=16,
              Hkv=16, d_qk=192, page=16, cache="bf16", rot=64, interleaved=True, lens=9),
        # chunks of prompts behind a cached prefix, ragged
        _case("attend_chunks", "attend", seqs=4, q_min=129, q_max=1024, ctx_min=1000,
              ctx_max=7168, lens=10),
        # one chunk of a long document: the largest arithmetic
        _case("attend_chunk_long", "attend", seqs=1, q_min=1024, q_max=1024, ctx_min=31744,
              ctx_max=31744, Hq=64, lens=11),
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attend"])
    d_qk, d_v, rot = rng.choice([(128, 128, 128), (128, 128, 128), (64, 64, 64), (192, 128, 64)])
    hkv, group = rng.choice([(8, 4), (8, 8), (4, 4), (16, 1), (2, 7), (1, 12)])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    cache = rng.choice(["fp8_e4m3", "fp8_e4m3", dtype])
    mode = rng.choice(["decode", "verify", "chunk"])
    q_max = {"decode": 1, "verify": rng.randint(2, 8),
             "chunk": _log_uniform(rng, 16, 1024)}[mode]
    q_min = rng.randint(1, q_max)
    ctx_max = _log_uniform(rng, 16, 65536 if mode == "decode" else 16384)
    most = min(256, 262144 // (ctx_max + q_max))
    if mode == "chunk":
        most = min(most, 4096 // q_max, (1 << 30) // (q_max * (ctx_max + q_max) * hkv * group))
    seqs = _log_uniform(rng, 1, max(1, most))
    return {"op": op, "seqs": seqs, "q_min": q_min, "q_max": q_max,
            "ctx_min": rng.randint(0, ctx_max), "ctx_max": ctx_max, "Hq": hkv * group, "Hkv": hkv,
            "d_qk": d_qk, "d_v": d_v, "page": rng.choice([16, 32, 64, 128]), "dtype": dtype,
            "cache": cache, "rot": rot, "interleaved": rng.random() < 0.3,
            "window": rng.choice([-1, -1, rng.randint(0, ctx_max)]), "sink": rng.random() < 0.3,
            "lens": rng.randint(1, 1 << 20)}


# ------------------------------------------------------------------- inputs


def _lengths(case):
    """(new tokens, cached tokens) of each sequence; a function of the case."""
    r = random.Random(case["lens"])
    n = [r.randint(case["q_min"], case["q_max"]) for _ in range(case["seqs"])]
    c = [r.randint(case["ctx_min"], case["ctx_max"]) for _ in range(case["seqs"])]
    return n, c


def _type(name):
    return {"bf16": torch.bfloat16, "fp16": torch.float16,
            "fp8_e4m3": torch.float8_e4m3fn}[name]


def _page_scale(amax):
    """Smallest power of two s with amax <= 448 s, at least 2^MIN_EXP.  The
    mantissa of amax (in [1/2, 1)) decides: 448 = 0.875 * 2^9."""
    m, e = torch.frexp(amax.float())
    e = torch.where(m <= 0.875, e - 9, e - 8)
    e = torch.where(amax == 0, torch.full_like(e, MIN_EXP), e).clamp(min=MIN_EXP)
    return ((e + 127) << 23).view(torch.float32)


def _cache(gen, case, pages, width):
    """Pages full of tokens as earlier appends left them, and their scales.
    Heads differ in size, as a model's do."""
    dev = torch.device("cuda")
    hkv, page = case["Hkv"], case["page"]
    x = torch.randn(pages, hkv, page, width, generator=gen, device=dev)
    x *= torch.exp(0.5 * torch.randn(1, hkv, 1, 1, generator=gen, device=dev))
    if case["cache"] != "fp8_e4m3":
        return x.to(_type(case["cache"])), None
    scale = _page_scale(x.abs().amax(dim=(2, 3)))
    codes = (x / scale[:, :, None, None]).to(torch.float8_e4m3fn)
    return codes, scale


def prepare(case, seed):
    """What a serving loop holds before the call: the new tokens' tensors, the
    cache with its page table and lengths, the rotation tables, the outputs."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    new, ctx = _lengths(case)
    page = case["page"]
    used = [(a + b + page - 1) // page for a, b in zip(new, ctx)]
    width = (case["ctx_max"] + case["q_max"] + page - 1) // page
    pages = sum(used) + 3
    order = torch.randperm(pages, generator=gen, device=dev).int()
    rows, at = [], 0
    for u in used:
        rows.append(torch.nn.functional.pad(order[at:at + u], (0, width - u)))
        at += u
    T = sum(new)
    dt = _type(case["dtype"])
    s = {"case": case, "T": T, "table": torch.stack(rows).contiguous(), "width": width}
    s["lens"] = torch.tensor([a + b for a, b in zip(new, ctx)], dtype=torch.int32, device=dev)
    cu = [0]
    for a in new:
        cu.append(cu[-1] + a)
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
    s["k_cache"], s["k_scale"] = _cache(gen, case, pages, case["d_qk"])
    s["v_cache"], s["v_scale"] = _cache(gen, case, pages, case["d_v"])

    def randn(h, d, std):
        return (std * torch.randn(T, h, d, generator=gen, device=dev)).to(dt)

    s["q"] = randn(case["Hq"], case["d_qk"], 1.5)
    if case["op"] == "append":
        s["k_new"] = randn(case["Hkv"], case["d_qk"], 1.0)
        s["v_new"] = randn(case["Hkv"], case["d_v"], 1.0)
        s["q_rot"] = torch.empty_like(s["q"])
        half = case["rot"] // 2
        inv = ROPE_BASE ** (-torch.arange(half, device=dev, dtype=torch.float64) / half)
        ang = torch.arange(width * page, device=dev, dtype=torch.float64)[:, None] * inv
        s["cos"], s["sin"] = ang.cos().float(), ang.sin().float()
    else:
        s["sink"] = torch.randn(case["Hq"], generator=gen, device=dev) if case["sink"] else None
        s["o"] = torch.empty(T, case["Hq"], case["d_v"], dtype=dt, device=dev)
        s["lse"] = torch.empty(case["Hq"], T, dtype=torch.float32, device=dev)
    if own:
        _plan(s)
    return s


def _plan(s):
    """The parameter block and the workspace, which a serving loop keeps."""
    from bwd_tcgen05_tma_gb300 import attn as A

    c = s["case"]
    s["lib"] = A
    one = c["q_max"] == 1
    common = dict(dtype=c["dtype"], cache_dtype=c["cache"], q=s["q"], k_cache=s["k_cache"],
                  v_cache=s["v_cache"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                  page_table=s["table"], seq_lens=s["lens"],
                  cu_seqlens_q=None if one else s["cu"], max_q_len=c["q_max"])
    if c["op"] == "append":
        s["params"] = A.make_paged_params(
            k_new=s["k_new"], v_new=s["v_new"], q_rot=s["q_rot"], rope_cos=s["cos"],
            rope_sin=s["sin"], rope_interleaved=c["interleaved"], **common)
    else:
        s["params"] = A.make_paged_params(
            scale=c["d_qk"] ** -0.5, mask="CAUSAL",
            window_left=None if c["window"] < 0 else c["window"], sink=s["sink"], **common)
        s["ws"] = torch.empty(A.attn_paged_workspace_size(s["params"]), dtype=torch.uint8,
                              device="cuda")


# ----------------------------------------------------------------- the calls


def run(s):
    append = s["case"]["op"] == "append"
    if own:
        if append:
            s["lib"].attn_paged_append(s["params"])
        else:
            s["lib"].attn_paged_fwd(s["params"], s["o"], s["lse"], s["ws"])
            return {"o": s["o"], "lse": s["lse"]}
    elif append:
        _plain_append(s)
    else:
        return _plain_attend(s)
    return {"q": s["q_rot"], "k_cache": s["k_cache"], "v_cache": s["v_cache"],
            "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


# --------------------------------------------------------------- plain forms


def _tokens(s):
    """Sequence, index in the sequence's new tokens, and position of every new
    token."""
    n = (s["cu"][1:] - s["cu"][:-1]).long()
    seq = torch.repeat_interleave(torch.arange(n.numel(), device=n.device), n,
                                  output_size=s["T"])
    idx = torch.arange(s["T"], device=n.device) - s["cu"].long()[seq]
    return seq, idx, s["lens"].long()[seq] - n[seq] + idx


def _rotate(x, cos, sin, rot, interleaved):
    x = x.float()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2],
                                                                   x[..., rot // 2:rot])
    c, n = cos[:, None], sin[:, None]
    ra, rb = a * c - b * n, b * c + a * n
    turned = torch.stack([ra, rb], -1).flatten(-2) if interleaved else torch.cat([ra, rb], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_append(s):
    c = s["case"]
    seq, _, pos = _tokens(s)
    cos, sin = s["cos"][pos], s["sin"][pos]
    s["q_rot"].copy_(_rotate(s["q"], cos, sin, c["rot"], c["interleaved"]))
    page = s["table"].long()[seq, pos // c["page"]]
    slot = pos % c["page"]
    _plain_write(s["k_cache"], s["k_scale"], page, slot,
                 _rotate(s["k_new"], cos, sin, c["rot"], c["interleaved"]))
    _plain_write(s["v_cache"], s["v_scale"], page, slot, s["v_new"].float())


def _plain_write(cache, scale, page, slot, x):
    if scale is None:
        cache[page, :, slot] = x.to(cache.dtype)
        return
    amax = torch.zeros_like(scale).index_reduce_(0, page, x.abs().amax(-1), "amax")
    first = torch.full(scale.shape[:1], 1 << 30, device=x.device, dtype=torch.long)
    first = first.index_reduce_(0, page, slot, "amin")
    touched = page.unique()
    old = torch.where(first[touched, None] == 0, torch.zeros_like(scale[touched]), scale[touched])
    fit = torch.maximum(_page_scale(amax[touched]), old)
    codes = cache.view(torch.uint8)
    again = codes[touched].view(cache.dtype).float() * (old / fit)[:, :, None, None]
    kept = torch.arange(cache.shape[2], device=x.device) < first[touched, None]
    codes[touched] = torch.where(kept[:, None, :, None], again.to(cache.dtype).view(torch.uint8),
                                 codes[touched])
    scale[touched] = fit
    codes[page, :, slot] = (x / scale[page][..., None]).to(cache.dtype).view(torch.uint8)


def _plain_gather(cache, scale, table, keep):
    """A cache's tokens of every sequence in fp32: [seqs, Hkv, keys, width];
    what lies behind a sequence's end is read as zero."""
    if scale is None:
        x = cache[table].float()
    else:
        x = cache.view(torch.uint8)[table].view(cache.dtype).float()
        x = x * scale[table][..., None, None]
    x = x.transpose(1, 2).flatten(2, 3)
    return torch.where(keep[:, None, :, None], x, torch.zeros((), device=x.device))


def _plain_attend(s):
    c = s["case"]
    seqs, hq, hkv, most = c["seqs"], c["Hq"], c["Hkv"], c["q_max"]
    seq, idx, pos = _tokens(s)
    table = s["table"].long()
    key = torch.arange(table.shape[1] * c["page"], device=pos.device)
    keep = key < s["lens"][:, None]
    k = _plain_gather(s["k_cache"], s["k_scale"], table, keep)
    v = _plain_gather(s["v_cache"], s["v_scale"], table, keep)
    q = torch.zeros(seqs, most, hq, c["d_qk"], device=pos.device)
    q[seq, idx] = s["q"].float()
    at = torch.full((seqs, most), -1, device=pos.device)
    at[seq, idx] = pos
    seen = key <= at[..., None]
    if c["window"] >= 0:
        seen &= key >= at[..., None] - c["window"]
    q = q.view(seqs, most, hkv, hq // hkv, -1).permute(0, 2, 3, 1, 4).flatten(2, 3)
    sc = (q @ k.transpose(-1, -2)).mul_(c["d_qk"] ** -0.5).unflatten(2, (hq // hkv, most))
    sc.masked_fill_(~seen[:, None, None], -math.inf)
    m = sc.amax(-1, keepdim=True)
    if s["sink"] is not None:
        sink = s["sink"].view(1, hkv, hq // hkv, 1, 1)
        m = torch.maximum(m, sink)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = sc.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    if s["sink"] is not None:
        l = l + (sink - m).exp()
    o = (p.flatten(2, 3) @ v).unflatten(2, (hq // hkv, most))
    o = torch.where(l > 0, o / l, torch.zeros_like(o))
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3)[seq, idx]
    lse = (m + l.log()).squeeze(-1).permute(0, 3, 1, 2).flatten(2, 3)[seq, idx]
    s["o"].copy_(o)
    s["lse"].copy_(lse.t())
    return {"o": s["o"], "lse": s["lse"]}


# ------------------------------------------------------------------- work


def work(case):
    new, ctx = _lengths(case)
    T, hq, hkv, dqk, dv = sum(new), case["Hq"], case["Hkv"], case["d_qk"], case["d_v"]
    cb = 1 if case["cache"] == "fp8_e4m3" else 2
    if case["op"] == "append":
        byts = 2 * T * hq * dqk * 2 + T * hkv * (dqk + dv) * (2 + cb) + T * case["rot"] * 4
        flops = 3 * T * (hq + hkv) * case["rot"] + (2 * T * hkv * (dqk + dv) if cb == 1 else 0)
        return {"bytes": byts, "flops": flops}
    keys = pairs = pages = 0
    for a, b in zip(new, ctx):
        w = case["window"]
        lo = max(0, b - w) if w >= 0 else 0
        keys += a + b - lo
        pages += (a + b - 1) // case["page"] - lo // case["page"] + 1
        pairs += sum(p + 1 - (max(0, p - w) if w >= 0 else 0) for p in range(b, b + a))
    byts = keys * hkv * (dqk + dv) * cb + pages * (4 + (8 * hkv if cb == 1 else 0))
    byts += T * hq * ((dqk + dv) * 2 + 4)
    return {"bytes": byts, "flops": 2 * pairs * hq * (dqk + dv)}


# ------------------------------------------------------------- in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    new, ctx = _lengths(case)
    starts = [sum(new[:i]) for i in range(len(new))]
    if case["op"] == "attend":
        return _exact_attend(s, new, ctx, starts)
    at = torch.cat([torch.arange(b, b + a) for a, b in zip(new, ctx)]).cuda()
    cos, sin = s["cos"].double()[at], s["sin"].double()[at]
    out = {"q": _exact_turn(s["q"], cos, sin, case)}
    keys = _exact_turn(s["k_new"], cos, sin, case)
    out["k_cache"], out["k_scale"] = _exact_pages(s["k_cache"], s["k_scale"], s, new, ctx,
                                                  starts, keys)
    out["v_cache"], out["v_scale"] = _exact_pages(s["v_cache"], s["v_scale"], s, new, ctx,
                                                  starts, s["v_new"].double())
    return out


def _exact_turn(x, cos, sin, case):
    """Each pair of coordinates as a complex number times exp(i angle)."""
    rot = case["rot"]
    y = x.double().clone()
    first = torch.arange(0, rot, 2) if case["interleaved"] else torch.arange(rot // 2)
    second = first + (1 if case["interleaved"] else rot // 2)
    z = torch.complex(y[..., first], y[..., second]) * torch.complex(cos, sin)[:, None]
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_e4m3(x):
    """Nearest E4M3 value, ties to the even one: 3 bits behind the leading one,
    steps of 2^-9 below 2^-6."""
    a = x.abs()
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    return torch.sign(x) * torch.round(a / step) * step


def _exact_pages(cache, scale, s, new, ctx, starts, x):
    page = s["case"]["page"]
    val = cache.double()
    if scale is None:
        for i, (a, b) in enumerate(zip(new, ctx)):
            p = torch.arange(b, b + a, device=val.device)
            val[s["table"][i].long()[p // page], :, p % page] = x[starts[i]:starts[i] + a]
        return val, None
    table = s["table"].tolist()
    out = scale.double().clone()
    for i, (a, b) in enumerate(zip(new, ctx)):
        for j in range(b // page, (a + b - 1) // page + 1):
            lo, hi = max(b, j * page), min(a + b, (j + 1) * page)
            rows = x[starts[i] + lo - b:starts[i] + hi - b].transpose(0, 1)
            need = torch.log2(rows.abs().amax(dim=(1, 2)) / 448).ceil().clamp(min=MIN_EXP)
            need = torch.exp2(need)
            id_, cut = table[i][j], lo - j * page
            if cut:
                need = torch.maximum(need, out[id_])
                val[id_, :, :cut] = _exact_e4m3(val[id_, :, :cut] *
                                                (out[id_] / need)[:, None, None])
            val[id_, :, cut:cut + hi - lo] = _exact_e4m3(rows / need[:, None, None])
            out[id_] = need
    return val, out


def _exact_attend(s, new, ctx, starts):
    c = s["case"]
    hq, hkv, page = c["Hq"], c["Hkv"], c["page"]
    g = hq // hkv
    o = torch.zeros(s["T"], hq, c["d_v"], dtype=torch.float64, device="cuda")
    lse = torch.zeros(hq, s["T"], dtype=torch.float64, device="cuda")
    for i, (a, b) in enumerate(zip(new, ctx)):
        ids = s["table"][i].long()[:(a + b + page - 1) // page]
        rows = slice(starts[i], starts[i] + a)
        at = torch.arange(b, b + a, device="cuda")[:, None]
        key = torch.arange(a + b, device="cuda")
        seen = key <= at if c["window"] < 0 else (key <= at) & (key >= at - c["window"])
        for h in range(hkv):
            k, v = s["k_cache"][ids, h].double(), s["v_cache"][ids, h].double()
            if s["k_scale"] is not None:
                k = k * s["k_scale"][ids, h].double()[:, None, None]
                v = v * s["v_scale"][ids, h].double()[:, None, None]
            k, v = k.flatten(0, 1)[:a + b], v.flatten(0, 1)[:a + b]
            for q in range(h * g, (h + 1) * g):
                sc = s["q"][rows, q].double() @ k.t() / math.sqrt(c["d_qk"])
                sc = torch.where(seen, sc, -math.inf)
                if s["sink"] is not None:
                    sc = torch.cat([sc, s["sink"][q].double().expand(a, 1)], 1)
                lse[q, rows] = torch.logsumexp(sc, 1)
                o[rows, q] = torch.softmax(sc, 1)[:, :a + b] @ v
    return {"o": o, "lse": lse}
