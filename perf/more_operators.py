"""Workloads of rotary positions and of latent attention.

Five operators are measured, each over its range of uses:

* ``table``: cosines and sines of the rotation, fp32, for every position of a
  context, with the frequencies scaled for contexts longer than trained on.
* ``rope``: queries and keys turned by their positions (forward), or gradients
  turned back (the backward pass), in the layout the attention reads.
* ``expand``: the expanded form of latent attention, for training and prompts:
  every head's key is its own part beside one rotated part that all heads share;
  keys and values as the attention reads them.  ``back`` is the gradient.
* ``append``: new tokens' latent vectors and rotated shared key parts are written
  into a paged cache of one row a token, and the queries' parts are turned.
* ``attend``: the absorbed form.  All query heads attend to the one row a token
  has in the cache; its first part is also the value.

``run`` computes either the plain form (elementary torch operations, fp32;
angles in 64 bits) or, where ``own`` is true, the library's calls.  ``exact`` is
the definition in 64 bits.
"""
import math
import random

import torch

own = False


def _table(name, **kw):
    c = dict(name=name, op="table", rope_len=8192, rot=128, base=10000.0, scaling="NONE",
             factor=1.0, trained=8192, low=1.0, high=32.0, magnitude=1.0)
    c.update(kw)
    return c


def _rope(name, **kw):
    c = dict(name=name, op="rope", rows=1, S=2048, Hq=32, Hkv=8, d=128, start=0, rot=128,
             interleaved=False, inverse=False, packed=True, seg=2048, dtype="bf16", lens=1)
    c.update(kw)
    return c


def _expand(name, **kw):
    c = dict(name=name, op="expand", back=False, rows=1, S=4096, H=16, d_n=128, d_r=64, d_v=128,
             interleaved=False, dtype="bf16", seg=4096, lens=1)
    c.update(kw)
    return c


def _latent(name, op, **kw):
    c = dict(name=name, op=op, seqs=1, q_min=1, q_max=1, ctx_min=0, ctx_max=0, H=16, d_c=512,
             d_r=64, page=64, dtype="bf16", interleaved=False, window=-1, sink=False,
             by_head=False, scale=192 ** -0.5, lens=1)
    c.update(kw)
    return c


def listed():
    return [
        # tables of a model's usual context, made when it is loaded
        _table("table_8192"),
        # tables of a context sixteen times as long as trained on: low frequencies
        # are stretched, high ones kept
        _table("table_131072_turns", rope_len=131072, rot=64, scaling="TURNS", factor=16.0,
               magnitude=1.2772588722239782),
        # the packed THD GQA training batch: queries and keys of the fused projection
        _rope("rope_thd_gqa", rows=2, S=8192, lens=2),
        # gradients of 192-wide heads of which the last 64 dims were turned, pairs
        # side by side, fp16: the backward pass of the cross-attention sizes
        _rope("rope_back_192", rows=2, S=4096, Hq=16, Hkv=16, d=192, start=128, rot=64,
              interleaved=True, inverse=True, packed=False, dtype="fp16", lens=3),
        # keys and values of a training batch from their up-projection
        _expand("expand_train", rows=2, lens=4),
        # and their gradients: the shared part's is a sum over the heads
        _expand("expand_back", rows=2, back=True, lens=5),
        # a decode step of a server's batch
        _latent("latent_append_64", "append", seqs=64, ctx_min=1, ctx_max=2048, lens=6),
        # a packed prefill batch: 16 prompts of 64 to 2048 tokens, fp16
        _latent("latent_append_prefill", "append", seqs=16, q_min=64, q_max=2048, ctx_max=1000,
                dtype="fp16", interleaved=True, lens=7),
        # one user's decode step over a short context: latency
        _latent("latent_decode_1", "attend", ctx_min=1000, ctx_max=1000),
        # a server's decode batch with ragged contexts
        _latent("latent_decode_64", "attend", seqs=64, ctx_min=63, ctx_max=8191, lens=8),
        # long documents, 64 heads: the largest traffic
        _latent("latent_decode_long", "attend", seqs=4, ctx_min=100000, ctx_max=131071, H=64,
                lens=9),
        # chunks of prompts behind a cached prefix: the largest arithmetic
        _latent("latent_chunks", "attend", seqs=3, q_min=129, q_max=512, ctx_min=1000,
                ctx_max=16384, lens=10),
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["table", "rope", "expand", "append", "attend", "attend"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    lens = rng.randint(1, 1 << 20)
    if op == "table":
        scaling = rng.choice(["NONE", "LINEAR", "BASE", "TURNS"])
        c = _table("", rope_len=_log_uniform(rng, 100, 131072), rot=16 * rng.randint(1, 8),
                   base=rng.choice([10000.0, 500000.0, 1000000.0]), scaling=scaling,
                   factor=1.0 if scaling == "NONE" else rng.uniform(1.0, 32.0),
                   magnitude=rng.choice([1.0, rng.uniform(1.0, 1.4)]))
    elif op == "rope":
        d, start, rot = rng.choice([(128, 0, 128), (128, 0, 64), (64, 0, 64), (64, 0, 32),
                                    (192, 128, 64), (192, 0, 192)])
        hkv, group = rng.choice([(8, 4), (8, 8), (4, 4), (16, 1), (2, 7), (1, 12)])
        S = _log_uniform(rng, 1, 16384)
        c = _rope("", rows=rng.randint(1, max(1, min(4, 16384 // S))), S=S, Hq=hkv * group,
                  Hkv=hkv, d=d, start=start, rot=rot, interleaved=rng.random() < 0.4,
                  inverse=rng.random() < 0.5, packed=rng.random() < 0.5,
                  seg=_log_uniform(rng, 16, 16384), dtype=dtype, lens=lens)
        while c["rows"] * S * c["Hq"] * (d // 64) > 2 * 8192 * 40 * 2:
            c["S"] = S = max(1, S // 2)
    elif op == "expand":
        S = _log_uniform(rng, 1, 8192)
        d_n, d_r, d_v = rng.choice([(128, 64, 128), (128, 64, 128), (64, 64, 128), (64, 64, 64)])
        c = _expand("", back=rng.random() < 0.5, rows=rng.randint(1, max(1, min(4, 8192 // S))),
                    S=S, H=rng.choice([1, 4, 7, 12, 16]), d_n=d_n, d_r=d_r, d_v=d_v,
                    interleaved=rng.random() < 0.5, dtype=dtype, seg=_log_uniform(rng, 16, 8192),
                    lens=lens)
    else:
        H = rng.choice([4, 7, 8, 16, 16, 20, 32, 64])
        mode = rng.choice(["decode", "verify", "chunk"])
        q_max = {"decode": 1, "verify": rng.randint(2, 8),
                 "chunk": _log_uniform(rng, 16, 512)}[mode]
        ctx_max = _log_uniform(rng, 16, 65536 if mode == "decode" else 16384)
        most = min(256, 450000 // (ctx_max + q_max), 16384 // q_max,
                   100000000 // (q_max * H * (ctx_max + q_max)))
        if op == "append":
            most = min(most, 16384 * 16 // (q_max * H))
        d_c = rng.choice([512, 512, 256])
        c = _latent("", op, seqs=_log_uniform(rng, 1, max(1, most)), q_min=rng.randint(1, q_max),
                    q_max=q_max, ctx_min=rng.randint(0, ctx_max), ctx_max=ctx_max, H=H, d_c=d_c,
                    page=rng.choice([16, 32, 64, 128]), dtype=dtype,
                    interleaved=rng.random() < 0.5,
                    window=rng.choice([-1, -1, -1, rng.randint(0, ctx_max)]),
                    sink=rng.random() < 0.3, by_head=rng.random() < 0.3, lens=lens)
        if op == "attend" and q_max * H * (ctx_max + q_max) > 100000000:
            c["q_max"] = max(1, 100000000 // (H * (ctx_max + 512)))
            c["q_min"] = min(c["q_min"], c["q_max"])
    del c["name"]
    return c


# ------------------------------------------------------------------- inputs


def _type(name):
    return {"bf16": torch.bfloat16, "fp16": torch.float16}[name]


def _lengths(case):
    """(new tokens, cached tokens) of each sequence; a function of the case."""
    r = random.Random(case["lens"])
    n = [r.randint(case["q_min"], case["q_max"]) for _ in range(case["seqs"])]
    c = [r.randint(case["ctx_min"], case["ctx_max"]) for _ in range(case["seqs"])]
    return n, c


def _positions(case):
    """Positions of packed rows: segments of 1 to `seg` tokens, each from 0."""
    r = random.Random(case["lens"])
    out = []
    for _ in range(case["rows"]):
        row = []
        while len(row) < case["S"]:
            row.extend(range(r.randint(max(1, case["seg"] // 32), case["seg"])))
        out.extend(row[:case["S"]])
    return torch.tensor(out, dtype=torch.int32, device="cuda")


def _tables(length, rot):
    half = rot // 2
    inv = 10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    ang = torch.arange(length, device="cuda", dtype=torch.float64)[:, None] * inv
    return ang.cos().float(), ang.sin().float()


def prepare(case, seed):
    """What a training step or a serving loop holds before the call."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": case}
    if case["op"] == "table":
        # models differ in their base
        s["base"] = case["base"] * (1 + random.Random(seed).random() / 16)
        for n in ("cos", "sin"):
            s[n] = torch.empty(case["rope_len"], case["rot"] // 2, device="cuda")
    else:
        dt = _type(case["dtype"])

        def randn(*shape, std=1.0):
            return torch.randn(*shape, generator=gen, device="cuda").mul_(std).to(dt)

        {"rope": _prepare_rope, "expand": _prepare_expand}.get(case["op"], _prepare_latent)(
            s, case, randn, dt)
    if own:
        _plan(s)
    return s


def _prepare_rope(s, c, randn, dt):
    T, hq, hkv, d = c["rows"] * c["S"], c["Hq"], c["Hkv"], c["d"]
    if c["packed"]:  # slices of the fused projection
        qkv = randn(T, (hq + 2 * hkv) * d)
        s["q"] = qkv[:, :hq * d].unflatten(1, (hq, d))
        s["k"] = qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
    else:
        s["q"], s["k"] = randn(T, hq, d), randn(T, hkv, d)
    s["q_out"] = torch.empty(T, hq, d, dtype=dt, device="cuda")
    s["k_out"] = torch.empty(T, hkv, d, dtype=dt, device="cuda")
    s["pos"] = _positions(c)
    s["cos"], s["sin"] = _tables(min(c["S"], c["seg"]), c["rot"])


def _prepare_expand(s, c, randn, dt):
    T, H = c["rows"] * c["S"], c["H"]
    kv, pe = (T, H, c["d_n"] + c["d_v"]), (T, c["d_r"])
    k, v = (T, H, c["d_n"] + c["d_r"]), (T, H, c["d_v"])
    make = dict(dtype=dt, device="cuda")
    if c["back"]:
        s["k"], s["v"] = randn(*k), randn(*v)
        s["kv"], s["k_rope"] = torch.empty(*kv, **make), torch.empty(*pe, **make)
    else:
        s["kv"], s["k_rope"] = randn(*kv), randn(*pe)
        s["k"], s["v"] = torch.empty(*k, **make), torch.empty(*v, **make)
    s["pos"] = _positions(c)
    s["cos"], s["sin"] = _tables(min(c["S"], c["seg"]), c["d_r"])


def _prepare_latent(s, c, randn, dt):
    new, ctx = _lengths(c)
    page, H, d = c["page"], c["H"], c["d_c"] + c["d_r"]
    used = [(a + b + page - 1) // page for a, b in zip(new, ctx)]
    width = (c["ctx_max"] + c["q_max"] + page - 1) // page
    order = torch.randperm(sum(used) + 3, generator=_host_gen(c), device="cpu").int().cuda()
    rows, at = [], 0
    for u in used:
        rows.append(torch.nn.functional.pad(order[at:at + u], (0, width - u)))
        at += u
    T = sum(new)
    i32 = dict(dtype=torch.int32, device="cuda")
    s["T"], s["table"] = T, torch.stack(rows).contiguous()
    s["lens"] = torch.tensor([a + b for a, b in zip(new, ctx)], **i32)
    cu = [0]
    for a in new:
        cu.append(cu[-1] + a)
    s["cu"] = torch.tensor(cu, **i32)
    s["cache"] = randn(sum(used) + 3, page, d)
    if c["op"] == "append":
        s["c_new"], s["k_rope"] = randn(T, c["d_c"]), randn(T, c["d_r"])
        # the queries' part that is turned lies behind the other 128 dims of a head
        s["q_rope"] = randn(T, H, 128 + c["d_r"])[..., 128:]
        s["q_rot"] = torch.empty(T, H, c["d_r"], dtype=dt, device="cuda")
        s["cos"], s["sin"] = _tables(width * page, c["d_r"])
    else:
        # as a product by heads or by tokens leaves them
        s["q_lat"] = (randn(H, T, c["d_c"]).transpose(0, 1) if c["by_head"]
                      else randn(T, H, c["d_c"]))
        s["q_rot"] = randn(T, H, c["d_r"])
        s["sink"] = randn(H).float() if c["sink"] else None
        s["o"] = torch.empty(T, H, c["d_c"], dtype=dt, device="cuda")
        s["lse"] = torch.empty(H, T, dtype=torch.float32, device="cuda")


def _host_gen(case):
    g = torch.Generator()
    g.manual_seed(case["lens"])
    return g


def _plan(s):
    """Parameter blocks and workspaces, which a user's program keeps."""
    from bwd_tcgen05_tma_gb300 import attn as A

    c = s["case"]
    s["lib"] = A
    if c["op"] == "table":
        s["params"] = A.make_rope_table_params(
            cos=s["cos"], sin=s["sin"], base=s["base"], scaling=c["scaling"], factor=c["factor"],
            trained_len=c["trained"], turns=(c["low"], c["high"]), magnitude=c["magnitude"])
    elif c["op"] == "rope":
        s["params"] = A.make_rope_params(
            dtype=c["dtype"], q=s["q"], k=s["k"], q_out=s["q_out"], k_out=s["k_out"],
            rope_cos=s["cos"], rope_sin=s["sin"], positions=s["pos"], rot_start=c["start"],
            interleaved=c["interleaved"], inverse=c["inverse"])
    elif c["op"] == "expand":
        s["params"] = A.make_latent_expand_params(
            dtype=c["dtype"], kv=s["kv"], k_rope=s["k_rope"], k=s["k"], v=s["v"],
            rope_cos=s["cos"], rope_sin=s["sin"], positions=s["pos"],
            interleaved=c["interleaved"])
    else:
        common = dict(dtype=c["dtype"], cache=s["cache"], d_c=c["d_c"], page_table=s["table"],
                      seq_lens=s["lens"], cu_seqlens_q=None if c["q_max"] == 1 else s["cu"],
                      max_q_len=c["q_max"], q_rot=s["q_rot"])
        if c["op"] == "append":
            s["params"] = A.make_latent_params(
                c_new=s["c_new"], k_rope=s["k_rope"], q_rope=s["q_rope"], rope_cos=s["cos"],
                rope_sin=s["sin"], rope_interleaved=c["interleaved"], **common)
        else:
            s["params"] = A.make_latent_params(
                q_lat=s["q_lat"], scale=c["scale"], mask="CAUSAL",
                window_left=None if c["window"] < 0 else c["window"], sink=s["sink"], **common)
            s["ws"] = torch.empty(A.attn_latent_workspace_size(s["params"]), dtype=torch.uint8,
                                  device="cuda")


# ----------------------------------------------------------------- the calls


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        if op == "table":
            s["lib"].attn_rope_table(s["params"])
        elif op == "rope":
            s["lib"].attn_rope(s["params"])
        elif op == "expand":
            (s["lib"].attn_latent_expand_bwd if c["back"] else s["lib"].attn_latent_expand)(
                s["params"])
        elif op == "append":
            s["lib"].attn_latent_append(s["params"])
        else:
            s["lib"].attn_latent_fwd(s["params"], s["o"], s["lse"], s["ws"])
    else:
        {"table": _plain_table, "rope": _plain_rope, "expand": _plain_expand,
         "append": _plain_append, "attend": _plain_attend}[op](s)
    names = {"table": ("cos", "sin"), "rope": ("q_out", "k_out"),
             "expand": ("kv", "k_rope") if c.get("back") else ("k", "v"),
             "append": ("q_rot", "cache"), "attend": ("o", "lse")}[op]
    return {n: s[n] for n in names}


# --------------------------------------------------------------- plain forms


def _plain_table(s):
    c = s["case"]
    rot, base = c["rot"], s["base"]
    p = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    if c["scaling"] == "BASE":
        base = base * c["factor"] ** (rot / (rot - 2))
    freq = torch.pow(torch.tensor(base, device="cuda", dtype=torch.float64), -2 * p / rot)
    if c["scaling"] == "LINEAR":
        freq = freq / c["factor"]
    elif c["scaling"] == "TURNS":
        turns = c["trained"] * freq / (2 * math.pi)
        w = ((turns - c["low"]) / (c["high"] - c["low"])).clamp(0, 1)
        freq = freq * (w + (1 - w) / c["factor"])
    ang = torch.arange(c["rope_len"], device="cuda", dtype=torch.float64)[:, None] * freq
    s["cos"].copy_(ang.cos() * c["magnitude"])
    s["sin"].copy_(ang.sin() * c["magnitude"])


def _turn(x, cos, sin, interleaved):
    """x: [tokens, heads, rot] fp32; cos, sin: [tokens, rot / 2]."""
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else x.chunk(2, -1)
    c, n = cos[:, None], sin[:, None]
    ra, rb = a * c - b * n, b * c + a * n
    return torch.stack([ra, rb], -1).flatten(-2) if interleaved else torch.cat([ra, rb], -1)


def _plain_rope(s):
    c = s["case"]
    pos, lo, hi = s["pos"].long(), c["start"], c["start"] + c["rot"]
    cos, sin = s["cos"][pos], s["sin"][pos]
    if c["inverse"]:
        sin = -sin
    for n in ("q", "k"):
        x = s[n].float()
        y = torch.cat([x[..., :lo], _turn(x[..., lo:hi], cos, sin, c["interleaved"]), x[..., hi:]],
                      -1)
        s[n + "_out"].copy_(y)


def _plain_expand(s):
    c = s["case"]
    pos, d_n = s["pos"].long(), c["d_n"]
    cos, sin = s["cos"][pos], s["sin"][pos]
    if c["back"]:
        s["kv"].copy_(torch.cat([s["k"][..., :d_n].float(), s["v"].float()], -1))
        pe = s["k"][..., d_n:].float().sum(1, keepdim=True)
        s["k_rope"].copy_(_turn(pe, cos, -sin, c["interleaved"])[:, 0])
        return
    pe = _turn(s["k_rope"].float()[:, None], cos, sin, c["interleaved"])
    s["k"].copy_(torch.cat([s["kv"][..., :d_n].float(), pe.expand(-1, c["H"], -1)], -1))
    s["v"].copy_(s["kv"][..., d_n:])


def _tokens(s):
    """Sequence, index in the sequence's new tokens, and position of every new
    token."""
    n = (s["cu"][1:] - s["cu"][:-1]).long()
    seq = torch.repeat_interleave(torch.arange(n.numel(), device=n.device), n,
                                  output_size=s["T"])
    idx = torch.arange(s["T"], device=n.device) - s["cu"].long()[seq]
    return seq, idx, s["lens"].long()[seq] - n[seq] + idx


def _plain_append(s):
    c = s["case"]
    seq, _, pos = _tokens(s)
    cos, sin = s["cos"][pos], s["sin"][pos]
    s["q_rot"].copy_(_turn(s["q_rope"].float(), cos, sin, c["interleaved"]))
    pe = _turn(s["k_rope"].float()[:, None], cos, sin, c["interleaved"])[:, 0]
    row = torch.cat([s["c_new"].float(), pe], -1).to(s["cache"].dtype)
    s["cache"][s["table"].long()[seq, pos // c["page"]], pos % c["page"]] = row


def _plain_attend(s):
    c = s["case"]
    seqs, H, d_c, most = c["seqs"], c["H"], c["d_c"], c["q_max"]
    seq, idx, pos = _tokens(s)
    table = s["table"].long()
    key = torch.arange(table.shape[1] * c["page"], device="cuda")
    x = s["cache"][table].flatten(1, 2).float()
    x = torch.where((key < s["lens"][:, None])[..., None], x, torch.zeros((), device="cuda"))
    q = torch.zeros(seqs, most, H, d_c + c["d_r"], device="cuda")
    q[seq, idx] = torch.cat([s["q_lat"], s["q_rot"]], -1).float()
    at = torch.full((seqs, most), -1, device="cuda")
    at[seq, idx] = pos
    seen = key <= at[..., None]
    if c["window"] >= 0:
        seen &= key >= at[..., None] - c["window"]
    sc = (q.flatten(1, 2) @ x.transpose(-1, -2)).mul_(c["scale"]).unflatten(1, (most, H))
    sc.masked_fill_(~seen[:, :, None], -math.inf)
    m = sc.amax(-1, keepdim=True)
    if s["sink"] is not None:
        m = torch.maximum(m, s["sink"].view(1, 1, H, 1))
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = sc.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    if s["sink"] is not None:
        l = l + (s["sink"].view(1, 1, H, 1) - m).exp()
    o = (p.flatten(1, 2) @ x[..., :d_c]).unflatten(1, (most, H))
    o = torch.where(l > 0, o / l, torch.zeros_like(o))
    s["o"].copy_(o[seq, idx])
    s["lse"].copy_((m + l.log())[..., 0][seq, idx].t())


# ------------------------------------------------------------------- work


def work(case):
    op = case["op"]
    if op == "table":
        n = case["rope_len"] * case["rot"] // 2
        return {"bytes": 8 * n, "flops": 4 * n}
    if op in ("rope", "expand"):
        T = case["rows"] * case["S"]
        seen = min(T, case["S"], case["seg"])  # rows of the tables, each read once
        if op == "rope":
            heads, rot = case["Hq"] + case["Hkv"], case["rot"]
            return {"bytes": 4 * T * heads * case["d"] + 4 * T + 4 * seen * rot,
                    "flops": 3 * T * heads * rot}
        H, d_n, d_r, d_v = case["H"], case["d_n"], case["d_r"], case["d_v"]
        b = 2 * T * (H * (2 * d_n + 2 * d_v + d_r) + d_r) + 4 * T + 4 * seen * d_r
        return {"bytes": b, "flops": 3 * T * d_r + (T * (H - 1) * d_r if case["back"] else 0)}
    new, ctx = _lengths(case)
    T, H, d_c, d_r = sum(new), case["H"], case["d_c"], case["d_r"]
    if op == "append":
        return {"bytes": 4 * T * (H * d_r + d_c + d_r) + 4 * T * d_r,
                "flops": 3 * T * (H + 1) * d_r}
    keys = pairs = pages = 0
    w = case["window"]
    for a, b in zip(new, ctx):
        lo = max(0, b - w) if w >= 0 else 0
        keys += a + b - lo
        pages += (a + b - 1) // case["page"] - lo // case["page"] + 1
        pairs += sum(p + 1 - (max(0, p - w) if w >= 0 else 0) for p in range(b, b + a))
    byts = 2 * keys * (d_c + d_r) + 4 * pages + T * H * (2 * (2 * d_c + d_r) + 4)
    return {"bytes": byts, "flops": 2 * pairs * H * (2 * d_c + d_r)}


# ------------------------------------------------------------- in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return {"table": _exact_table, "rope": _exact_rope, "expand": _exact_expand,
            "append": _exact_append, "attend": _exact_attend}[case["op"]](s, case)


def _exact_table(s, c):
    """Powers of a unit complex number by the angle of each frequency."""
    rot, cols = c["rot"], []
    for p in range(rot // 2):
        lb = math.log(s["base"])
        if c["scaling"] == "BASE":
            lb += math.log(c["factor"]) * rot / (rot - 2)
        f = math.exp(-lb * 2 * p / rot)
        if c["scaling"] == "LINEAR":
            f /= c["factor"]
        if c["scaling"] == "TURNS":
            t = c["trained"] / (2 * math.pi / f)
            if t <= c["low"]:
                f = f / c["factor"]
            elif t < c["high"]:
                w = (t - c["low"]) / (c["high"] - c["low"])
                f = (1 - w) * f / c["factor"] + w * f
        cols.append(f)
    ang = torch.outer(torch.arange(c["rope_len"], dtype=torch.float64, device="cuda"),
                      torch.tensor(cols, dtype=torch.float64, device="cuda"))
    z = torch.polar(torch.full_like(ang, c["magnitude"]), ang)
    return {"cos": z.real, "sin": z.imag}


def _exact_turn(x, cos, sin, interleaved, back=False):
    """Each pair of coordinates as a complex number times exp(i angle)."""
    rot = 2 * cos.shape[1]
    y = x.double().clone()
    first = torch.arange(0, rot, 2) if interleaved else torch.arange(rot // 2)
    second = first + (1 if interleaved else rot // 2)
    z = torch.complex(y[..., first], y[..., second])
    w = torch.complex(cos, sin)[:, None]
    z = z * (w.conj() if back else w)
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _angles(s, pos):
    return s["cos"].double()[pos], s["sin"].double()[pos]


def _exact_rope(s, c):
    cos, sin = _angles(s, s["pos"].long())
    part = slice(c["start"], c["start"] + c["rot"])
    out = {}
    for n in ("q", "k"):
        y = s[n].double()
        y[..., part] = _exact_turn(s[n][..., part], cos, sin, c["interleaved"], c["inverse"])
        out[n + "_out"] = y
    return out


def _exact_expand(s, c):
    cos, sin = _angles(s, s["pos"].long())
    d_n, H, T = c["d_n"], c["H"], c["rows"] * c["S"]
    if c["back"]:
        kv = torch.zeros(T, H, d_n + c["d_v"], dtype=torch.float64, device="cuda")
        kv[..., :d_n], kv[..., d_n:] = s["k"][..., :d_n].double(), s["v"].double()
        # the sum over heads of each one's gradient turned back
        g = _exact_turn(s["k"][..., d_n:], cos, sin, c["interleaved"], True)
        return {"kv": kv, "k_rope": torch.einsum("thd->td", g)}
    k = torch.zeros(T, H, d_n + c["d_r"], dtype=torch.float64, device="cuda")
    k[..., :d_n] = s["kv"][..., :d_n].double()
    k[..., d_n:] = _exact_turn(s["k_rope"][:, None], cos, sin, c["interleaved"])
    return {"k": k, "v": s["kv"][..., d_n:].double()}


def _exact_append(s, c):
    new, ctx = _lengths(c)
    at = torch.cat([torch.arange(b, b + a) for a, b in zip(new, ctx)]).cuda()
    cos, sin = _angles(s, at)
    pe = _exact_turn(s["k_rope"][:, None], cos, sin, c["interleaved"])[:, 0]
    out, row, page = s["cache"].double(), 0, c["page"]
    for i, (a, b) in enumerate(zip(new, ctx)):
        p = torch.arange(b, b + a, device="cuda")
        ids, slot = s["table"][i].long()[p // page], p % page
        out[ids, slot, :c["d_c"]] = s["c_new"][row:row + a].double()
        out[ids, slot, c["d_c"]:] = pe[row:row + a]
        row += a
    return {"q_rot": _exact_turn(s["q_rope"], cos, sin, c["interleaved"]), "cache": out}


def _exact_attend(s, c):
    new, ctx = _lengths(c)
    H, d_c, page, row = c["H"], c["d_c"], c["page"], 0
    o = torch.zeros(s["T"], H, d_c, dtype=torch.float64, device="cuda")
    lse = torch.zeros(H, s["T"], dtype=torch.float64, device="cuda")
    for i, (a, b) in enumerate(zip(new, ctx)):
        ids = s["table"][i].long()[:(a + b + page - 1) // page]
        x = s["cache"][ids].double().flatten(0, 1)[:a + b]
        at = torch.arange(b, b + a, device="cuda")[:, None]
        key = torch.arange(a + b, device="cuda")
        seen = key <= at if c["window"] < 0 else (key <= at) & (key >= at - c["window"])
        rows = slice(row, row + a)
        for h in range(H):
            sc = s["q_lat"][rows, h].double() @ x[:, :d_c].t()
            sc = (sc + s["q_rot"][rows, h].double() @ x[:, d_c:].t()) * c["scale"]
            sc = torch.where(seen, sc, -math.inf)
            if s["sink"] is not None:
                sc = torch.cat([sc, s["sink"][h].double().expand(a, 1)], 1)
            lse[h, rows] = torch.logsumexp(sc, 1)
            o[rows, h] = torch.softmax(sc, 1)[:, :a + b] @ x[:, :d_c]
        row += a
    return {"o": o, "lse": lse}
