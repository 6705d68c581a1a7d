"""Cases that measure the cache and attention calls of the target pass.

Between scheduling and verification a round runs the target model over the
admitted tokens: request b brings its last committed token and ell[b] admitted
draft tokens.  Three groups of calls do that pass's own work beside the
model's matrix products:

  plan    dspark_cache_plan / dspark_cache_commit: the round's block tables,
          slot map, positions and key lengths from the admitted lengths, and
          after verification the pages behind the accepted tokens given back;
  norm    dspark_qk_norm_rope (with dspark_cache_read): the norm of every
          query and key head, the position rotation, and the write of keys and
          values into the 4-bit cache, in one pass;
  attend  dspark_cache_attention: the queries of every request against its
          4-bit pages, causal inside the block, optionally windowed.

`own` selects the framework's calls; otherwise run() computes the same in
elementary torch operations.

Cache format (both forms read and write it): cache [n_pages, Hkv, R] bytes, a
record of R = P * D * 9 / 8 bytes for the P tokens of one page and head:
  K codes [D/32][P][16], K scales [P][D/16], V codes and V scales the same.
A byte of codes holds dims (2j, 2j+1) of its 32-dim chunk as e2m1 (low nibble
first); a scale byte is the e4m3 scale of 16 dims; a value is
code * scale * (k_scale or v_scale).
"""
import math

import torch

own = False

PAGE_DTYPE = torch.uint8
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------- cases
def listed():
    return [
        # A handful of requests: only the latency of the two calls counts.
        {"name": "plan_small", "op": "plan", "B": 4, "G": 5, "P": 64, "ctx": 2000},
        # The high-concurrency round of the benchmark.
        {"name": "plan_headline", "op": "plan", "B": 256, "G": 5, "P": 64, "ctx": 4096},
        # The saturated engine: 1024 requests, blocks of 8, small pages.
        {"name": "plan_saturated", "op": "plan", "B": 1024, "G": 8, "P": 16, "ctx": 8192},
        # The largest batch the library takes.
        {"name": "plan_largest", "op": "plan", "B": 4096, "G": 3, "P": 32, "ctx": 4096},
        # One request, no admitted draft: a plain decoding step.
        {"name": "norm_one", "op": "norm", "B": 1, "G": 0, "Hq": 32, "Hkv": 8, "D": 128, "rot": 128, "inter": False,
         "P": 64, "dtype": "bf16", "ctx": 1000, "write": True},
        # The high-concurrency round, 64 query heads over 8 key heads.
        {"name": "norm_headline", "op": "norm", "B": 256, "G": 5, "Hq": 64, "Hkv": 8, "D": 128, "rot": 128,
         "inter": False, "P": 64, "dtype": "bf16", "ctx": 4096, "write": True},
        # fp32 rows, half of each head rotated in interleaved pairs, no cache: keys come back as rows.
        {"name": "norm_fp32_rows", "op": "norm", "B": 37, "G": 12, "Hq": 10, "Hkv": 10, "D": 64, "rot": 32,
         "inter": True, "P": 16, "dtype": "f32", "ctx": 70000, "write": False},
        # The saturated engine: up to 9 tokens of 1024 requests.
        {"name": "norm_saturated", "op": "norm", "B": 1024, "G": 8, "Hq": 32, "Hkv": 8, "D": 128, "rot": 64,
         "inter": False, "P": 16, "dtype": "bf16", "ctx": 1024, "write": True},
        # One request, one token: a plain decoding step over a short context.
        {"name": "attend_one", "op": "attend", "B": 1, "G": 0, "Hq": 32, "Hkv": 8, "D": 128, "P": 16, "ctx": 1000,
         "window": 0},
        # The high-concurrency round: 256 requests of up to 6 tokens, ragged contexts.
        {"name": "attend_headline", "op": "attend", "B": 256, "G": 5, "Hq": 64, "Hkv": 8, "D": 128, "P": 64,
         "ctx": 4096, "window": 0},
        # Long blocks over a 128-token sliding window, heads of 64.
        {"name": "attend_window", "op": "attend", "B": 128, "G": 16, "Hq": 24, "Hkv": 8, "D": 64, "P": 32,
         "ctx": 3001, "window": 128},
        # A few very long contexts: the key axis has to be split over the machine.
        {"name": "attend_long", "op": "attend", "B": 4, "G": 8, "Hq": 32, "Hkv": 8, "D": 128, "P": 64, "ctx": 131072,
         "window": 0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("plan", "norm", "attend", "attend"))
    if op == "plan":
        B = _log(rng, 1, 4096)
        return {"op": op, "B": B, "G": rng.randint(0, min(16, 16384 // B - 1)), "P": rng.choice((16, 32, 64, 128)),
                "ctx": _log(rng, 1, 8192)}
    D = rng.choice((64, 128))
    Hkv = rng.choice((1, 2, 3, 4, 8, 10))
    P = rng.choice((16, 32, 64, 128))
    if op == "norm":
        B = _log(rng, 1, 1024)
        return {"op": op, "B": B, "G": rng.randint(0, min(16, 9216 // B - 1)), "Hq": Hkv * rng.randint(1, 40 // Hkv),
                "Hkv": Hkv, "D": D, "rot": rng.choice([r for r in (0, 32, 64, 128) if r <= D]),
                "inter": rng.random() < 0.3, "P": P, "dtype": rng.choice(("bf16", "bf16", "f32")),
                "ctx": _log(rng, 1, min(131072, (1 << 20) // B)), "write": rng.random() < 0.7}
    B = _log(rng, 1, 256)
    Hkv = min(Hkv, 8)
    group = rng.choice((1, 2, 3, 4, 5, 8))
    # no more keys, and no more scores, than the largest listed case
    top = max(64, min(131072, 256 * 4096 // B, 256 * 4096 * 8 * 128 // (B * Hkv * D)))
    return {"op": op, "B": B, "G": rng.randint(0, 5 if B > 64 else 16), "Hq": Hkv * group, "Hkv": Hkv, "D": D,
            "P": P, "ctx": _log(rng, 1, top), "window": rng.choice((0, 0, 128, 1000))}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 11)
    return g


def _int(g, lo, hi, shape):
    return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=torch.int32)


def _lengths(case, g):
    """Ragged contexts (a quarter of `ctx` to all of it) and admitted lengths (survival decays along the block)."""
    B, G, top = case["B"], case["G"], case["ctx"]
    ctx = _int(g, max(1, top // 4) - 1, top, (B,)) if top > 1 else _int(g, 0, 2, (B,))
    keep = torch.rand((B, G + 1), generator=g, device="cuda") < 0.85
    ell = keep[:, :G].to(torch.int32).cumprod(1).sum(1).to(torch.int32) if G else torch.zeros_like(ctx)
    return ctx, ell


def _pages(n, P):
    return (n + P - 1) // P


def _ws(nbytes):
    return torch.zeros((nbytes + 255) // 256 * 256, dtype=torch.uint8, device="cuda")


def prepare(case, seed):
    g = _gen(seed)
    ctx, ell = _lengths(case, g)
    B, G, P = case["B"], case["G"], case["P"]
    max_pages = _pages(case["ctx"] + G + 1, P)
    s = {"case": case, "ctx": ctx, "ell": ell, "P": P, "G": G, "B": B, "T": B * (G + 1)}
    i32 = dict(dtype=torch.int32, device="cuda")
    if case["op"] == "plan":
        # Every request holds the pages of its context; the rest of the pool is free, in no order.
        n_pages = B * max_pages + 7
        perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
        held = _pages(ctx, P).to(torch.int32)
        first = held.cumsum(0) - held
        col = torch.arange(max_pages, device="cuda")[None, :]
        idx = (first[:, None] + col).clamp(max=n_pages - 1)
        s["table"] = torch.where(col < held[:, None], perm[idx], -1).to(torch.int32).contiguous()
        s["held"] = held.contiguous()
        used = held.sum()
        s["free_list"] = perm.roll(-int(used)).contiguous()
        s["free_count"] = (n_pages - used).to(torch.int32).reshape(1)
        s["free_list"][int(s["free_count"]):] = -1
        u = torch.rand((B,), generator=g, device="cuda")
        s["nout"] = (1 + (u * (ell + 1).float()).int()).clamp(max=ell + 1).to(torch.int32)
        s |= {"q_start": torch.zeros(B + 1, **i32), "kv_len": torch.zeros(B, **i32), "ctx_out": torch.zeros(B, **i32),
              "slot": torch.zeros(s["T"], **i32), "pos": torch.zeros(s["T"], **i32), "ws": _ws(256)}
        return s
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    n = ell + 1
    s["q_start"] = torch.zeros(B + 1, **i32)
    s["q_start"][1:] = n.cumsum(0)
    T, R = s["T"], P * D * 9 // 8
    dt = torch.float32 if case.get("dtype") == "f32" else torch.bfloat16
    qkv = torch.randn((T, Hq + 2 * Hkv, D), generator=g, device="cuda") * 2.0
    s["qkv"] = qkv.to(dt)
    s["q"], s["k"], s["v"] = s["qkv"].split([Hq, Hkv, Hkv], 1)
    n_pages = B * max_pages + 1                                               # one that no request holds
    s["table"] = torch.randperm(n_pages - 1, generator=g, device="cuda").to(torch.int32).reshape(B, max_pages).contiguous()
    if case["op"] == "norm":
        row = torch.arange(T, device="cuda")
        b = torch.searchsorted(s["q_start"][1:].contiguous(), row.int(), right=True).clamp(max=B - 1)
        pos = ctx[b] + row.int() - s["q_start"][b]
        live = row < s["q_start"][B]
        page = s["table"][b, (pos // P).clamp(max=max_pages - 1).long()]
        s["pos"] = torch.where(live, pos, -1).to(torch.int32)
        s["slot"] = torch.where(live, page * P + pos % P, -1).to(torch.int32)
        s["n_rows"] = s["q_start"][B:]
        s["wq"] = (1.0 + 0.1 * torch.randn((D,), generator=g, device="cuda")).to(dt)
        s["wk"] = (1.0 + 0.1 * torch.randn((D,), generator=g, device="cuda")).to(dt)
        half = max(1, case["rot"] // 2)
        freq = (10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)).float()
        s["inv_freq"] = freq[:case["rot"] // 2].contiguous()
        s["q_out"] = torch.zeros((T, Hq, D), dtype=dt, device="cuda")
        if case["write"]:
            s["cache"] = torch.zeros((n_pages, Hkv, R), dtype=PAGE_DTYPE, device="cuda")
            s["k_val"] = torch.zeros((T, Hkv, D), dtype=torch.bfloat16, device="cuda")
            s["v_val"] = torch.zeros_like(s["k_val"])
        else:
            s["k_out"] = torch.zeros((T, Hkv, D), dtype=dt, device="cuda")
        s["ws"] = _ws(256)
        return s
    # A pool of quantised pages of normal keys and values, dealt over the cache.
    pool = min(256, n_pages)
    kv = torch.randn((2, pool, Hkv, P, D), generator=g, device="cuda")
    parts = []
    for x in (kv[0], kv[1]):
        codes, scale = _quantise(x)
        parts += [_pack(codes).reshape(pool, Hkv, -1), scale.view(PAGE_DTYPE).reshape(pool, Hkv, -1)]
    pool_bytes = torch.cat(parts, 2)
    s["cache"] = pool_bytes[torch.randint(0, pool, (n_pages,), generator=g, device="cuda")].contiguous()
    s["kv_len"] = (ctx + n).to(torch.int32)
    s["out"] = torch.zeros((T, Hq, D), dtype=torch.bfloat16, device="cuda")
    s["scale"] = D ** -0.5
    s["ws"] = _ws(16 << 20)
    return s


# ------------------------------------------------------- the 4-bit format
def _quantise(x):
    """fp32 [..., D] -> (codes uint8 [..., D] of e2m1, scales e4m3 [..., D/16]); ties go to the even code."""
    y = x.reshape(*x.shape[:-1], -1, 16)
    scale = (y.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    sf = scale.float()[..., None]
    a = torch.where(sf > 0, y / sf, 0.0)
    m = a.abs()
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0))
    return (code + 8 * (a < 0)).to(torch.uint8).reshape(x.shape), scale


def _pack(codes):
    """codes [..., P, D] -> bytes [..., D/32, P, 16]."""
    b = codes[..., 0::2] | (codes[..., 1::2] << 4)
    return b.reshape(*b.shape[:-1], -1, 16).transpose(-3, -2).contiguous()


def _unpack(rec, P, D):
    """One half of records [..., P * D * 9 / 16] -> fp32 values [..., P, D]."""
    codes = rec[..., :P * D // 2].reshape(*rec.shape[:-1], D // 32, P, 16).transpose(-3, -2)
    nib = torch.stack((codes & 15, codes >> 4), -1).reshape(*rec.shape[:-1], P, D)
    lut = torch.tensor(GRID + tuple(-v for v in GRID), device=rec.device)
    scale = rec[..., P * D // 2:].contiguous().view(torch.float8_e4m3fn).reshape(*rec.shape[:-1], P, D // 16)
    val = lut[nib.int()].reshape(*rec.shape[:-1], P, D // 16, 16)
    return (val * scale.float()[..., None]).reshape(*rec.shape[:-1], P, D)


# -------------------------------------------------------------- plain forms
def _plain_plan(s):
    """One round's plan and commit on the state's tables, in place."""
    P, G, T = s["P"], s["G"], s["T"]
    table, held, free, ctx = s["table"], s["held"].long(), s["free_list"], s["ctx"].long()
    B, max_pages = table.shape
    count = s["free_count"].long()
    n = torch.minimum(s["ell"].long() + 1, max_pages * P - ctx).clamp(min=0)
    need = (_pages(ctx + n, P) - held).clamp(min=0)
    first = need.cumsum(0) - need
    fits = (need == 0) | (first + need <= count)
    n = torch.where(fits, n, torch.minimum(n, held * P - ctx).clamp(min=0))
    need = torch.where(fits, need, 0)
    start = torch.cat((torch.zeros_like(n[:1]), n.cumsum(0)))
    col = torch.arange(max_pages, device="cuda")[None, :]
    at = count - 1 - (first[:, None] + col - held[:, None])
    new = (col >= held[:, None]) & (col < (held + need)[:, None])
    table.copy_(torch.where(new, free[at.clamp(0, free.numel() - 1)], table))
    row = torch.arange(T, device="cuda")
    b = torch.searchsorted(start[1:].contiguous(), row, right=True).clamp(max=B - 1)
    live = row < start[B]
    pos = torch.where(live, ctx[b] + row - start[b], -1)
    page = table[b, (pos // P).clamp(0, max_pages - 1)].long()
    s["slot"].copy_(torch.where(live, page * P + pos % P, -1))
    s["pos"].copy_(pos)
    s["q_start"].copy_(start)
    s["kv_len"].copy_(ctx + n)
    held, count = held + need, count - need.sum()
    # commit
    out = ctx + torch.minimum(s["nout"].long(), n)
    keep = _pages(out, P)
    rel = (held - keep).clamp(min=0)
    last = rel.cumsum(0)
    total = last[-1]
    i = torch.arange(free.numel(), device="cuda")
    r = total - 1 - (i - count)
    pushed = (i >= count) & (r >= 0)
    rb = torch.searchsorted(last, r.clamp(min=0), right=True).clamp(max=B - 1)
    back = table[rb, (keep[rb] + r - (last - rel)[rb]).clamp(0, max_pages - 1)]
    free.copy_(torch.where(pushed, back, free))
    table.copy_(torch.where((col >= keep[:, None]) & (col < held[:, None]), -1, table))
    s["held"].copy_(torch.minimum(held, keep))
    s["free_count"].copy_(count + total)
    s["ctx_out"].copy_(out)


def _plan_outputs(s):
    # The list above free_count is spare room: only what is free counts.
    return {k: s[k] for k in ("table", "held", "free_list", "free_count", "q_start", "kv_len", "slot", "pos", "ctx_out")}


def _plain_norm_rows(x, w, eps, cos, sin, rot, inter):
    x = x.float()
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w.float()
    if rot == 0:
        return x
    if inter:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).reshape(*x.shape[:-1], rot)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        r = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((r, x[..., rot:]), -1)


EPS = 1e-6


def _plain_norm(s):
    case, P = s["case"], s["P"]
    D, rot, Hkv = case["D"], case["rot"], case["Hkv"]
    live = (s["pos"] >= 0)[:, None, None]
    ang = (s["pos"].clamp(min=0).double()[:, None] * s["inv_freq"].double())[:, None, :]
    cos, sin = ang.cos().float(), ang.sin().float()
    q = _plain_norm_rows(s["q"], s["wq"], EPS, cos, sin, rot, case["inter"])
    k = _plain_norm_rows(s["k"], s["wk"], EPS, cos, sin, rot, case["inter"])
    s["q_out"].copy_(torch.where(live, q.to(s["q_out"].dtype), s["q_out"]))
    if not case["write"]:
        s["k_out"].copy_(torch.where(live, k.to(s["k_out"].dtype), s["k_out"]))
        return {"q": s["q_out"], "k": s["k_out"]}
    # Scatter each token's bytes into its record; rows without a slot go to the page that no request holds.
    cache = s["cache"]
    slot = s["slot"].long()
    page, off = torch.where(slot >= 0, slot // P, cache.shape[0] - 1), slot % P
    h = torch.arange(Hkv, device="cuda")
    rec = cache.shape[2]
    base = ((page[:, None] * Hkv + h) * rec)[..., None]
    flat = cache.view(-1)
    vals = {}
    for part, (name, x) in enumerate((("k", k), ("v", s["v"].float()))):
        codes, scale = _quantise(x)
        packed = (codes[..., 0::2] | (codes[..., 1::2] << 4))
        d = torch.arange(D // 2, device="cuda")
        at = base + part * (rec // 2) + (d // 16) * (P * 16) + off[:, None, None] * 16 + d % 16
        e = torch.arange(D // 16, device="cuda")
        at_s = base + part * (rec // 2) + P * D // 2 + off[:, None, None] * (D // 16) + e
        ok = (slot >= 0)[:, None, None]
        flat[at] = packed
        flat[at_s] = scale.view(PAGE_DTYPE)
        lut = torch.tensor(GRID + tuple(-v for v in GRID), device="cuda")
        got = flat[at]
        nib = torch.stack((got & 15, got >> 4), -1).reshape(*x.shape)
        sc = flat[at_s].view(torch.float8_e4m3fn).float()
        val = (lut[nib.int()].reshape(*x.shape[:-1], D // 16, 16) * sc[..., None]).reshape(x.shape)
        vals[name] = torch.where(ok, val, 0.0).to(torch.bfloat16)
    s["k_val"].copy_(vals["k"])
    s["v_val"].copy_(vals["v"])
    return {"q": s["q_out"], "k": s["k_val"], "v": s["v_val"]}


def _plain_attend(s):
    case, P = s["case"], s["P"]
    B, G, Hq, Hkv, D = case["B"], case["G"], case["Hq"], case["Hkv"], case["D"]
    T, N, group = s["T"], G + 1, case["Hq"] // case["Hkv"]
    rec = s["cache"][s["table"].long()].transpose(1, 2)                       # [B, Hkv, pages, R]
    S = s["table"].shape[1] * P
    half = rec.shape[-1] // 2
    K = _unpack(rec[..., :half], P, D).reshape(B, Hkv, S, D)
    V = _unpack(rec[..., half:], P, D).reshape(B, Hkv, S, D)
    start, kv_len = s["q_start"].long(), s["kv_len"].long()
    j = torch.arange(N, device="cuda")[None, :]
    n = (start[1:] - start[:-1])[:, None]
    row = (start[:-1, None] + j).clamp(max=T - 1)                             # [B, N] rows of q
    q = s["q"][row].float().reshape(B, N, Hkv, group, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, group * N, D)
    pos = kv_len[:, None] - n + j                                             # [B, N]
    key = torch.arange(S, device="cuda")
    see = (key <= pos[..., None]) & (key < kv_len[:, None, None])
    if case["window"] > 0:
        see &= key > (pos - case["window"])[..., None]
    x = (q @ K.transpose(-1, -2)).mul_(s["scale"]).reshape(B, Hkv, group, N, S)
    x.masked_fill_(~see[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = x.sum(-1, keepdim=True)
    o = (x.reshape(B, Hkv, group * N, S) @ V).reshape(B, Hkv, group, N, D)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4).reshape(B * N, Hq, D).to(torch.bfloat16)
    # Back to packed rows: packed row t comes from (its request, its place in the block).
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(start[1:].contiguous(), t, right=True).clamp(max=B - 1)
    live = (t < start[B])[:, None, None]
    s["out"].copy_(torch.where(live, o[(b * N + t - start[b]).clamp(0, B * N - 1)], s["out"]))
    return s["out"]


def run(s):
    op = s["case"]["op"]
    if not own:
        if op == "plan":
            _plain_plan(s)
            return _plan_outputs(s)
        return _plain_norm(s) if op == "norm" else _plain_attend(s)
    from speculative_decoding_draft_rank_b200 import _lib
    if op == "plan":
        _lib.dspark_cache_plan(s["ctx"], s["ell"], s["G"], s["table"], s["held"], s["free_list"], s["free_count"],
                               s["P"], s["ws"], s["q_start"], s["kv_len"], s["slot"], s["pos"])
        _lib.dspark_cache_commit(s["ctx"], s["q_start"], s["nout"], None, s["table"], s["held"], s["free_list"],
                                 s["free_count"], s["P"], s["ws"], s["ctx_out"])
        return _plan_outputs(s)
    if op == "norm":
        case = s["case"]
        if case["write"]:
            _lib.dspark_qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], EPS, s["pos"], s["inv_freq"], case["inter"],
                                     s["n_rows"], s["q_out"], None, s["ws"], v=s["v"], cache=s["cache"],
                                     slot=s["slot"], page=s["P"])
            _lib.dspark_cache_read(s["cache"], s["slot"], s["P"], s["k_val"], s["v_val"], s["ws"])
            return {"q": s["q_out"], "k": s["k_val"], "v": s["v_val"]}
        _lib.dspark_qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], EPS, s["pos"], s["inv_freq"], case["inter"],
                                 s["n_rows"], s["q_out"], s["k_out"], s["ws"])
        return {"q": s["q_out"], "k": s["k_out"]}
    _lib.dspark_cache_attention(s["q"], s["cache"], s["table"], s["q_start"], s["kv_len"], s["P"], s["scale"],
                                s["case"]["window"], s["ws"], s["out"])
    return s["out"]


# --------------------------------------------------------------------- work
def work(case):
    """Expected bytes and operations of one pass (lengths average as _lengths draws them)."""
    B, G, P = case["B"], case["G"], case["P"]
    n = 1 + sum(0.85 ** (i + 1) for i in range(G))        # mean tokens of a request
    ctx = max(0.5, 0.625 * case["ctx"])
    if case["op"] == "plan":
        # lengths in and out, slots and positions, and about one table entry and one free page a request
        return {"bytes": 4 * B * (2 * (G + 1) + 12), "flops": 0}
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if case["op"] == "norm":
        e = 4 if case["dtype"] == "f32" else 2
        rows = B * n
        byt = rows * D * e * 2 * Hq + rows * 8
        if case["write"]:   # keys and values in, their records out, the records read back as bf16 rows
            byt += rows * Hkv * D * (2 * e + 2 * 0.5625 * 2 + 2 * 2)
        else:
            byt += rows * Hkv * D * 2 * e
        return {"bytes": byt, "flops": rows * (Hq + Hkv) * D * 8}
    keys = ctx + n
    if case["window"] > 0:
        keys = min(keys, case["window"] + n)
    return {"bytes": B * keys * Hkv * D * 1.125 + 4 * B * n * Hq * D + 4 * B * keys / P,
            "flops": 4 * B * n * Hq * D * (min(keys, case["window"]) if case["window"] > 0 else keys)}


# -------------------------------------------------------------------- exact
def exact(case, seed):
    s = prepare(case, seed)
    return {"plan": _exact_plan, "norm": _exact_norm, "attend": _exact_attend}[case["op"]](s)


def _exact_plan(s):
    """The tables as a serving loop on the host would keep them: lists, one request at a time."""
    P, T = s["P"], s["T"]
    r = {k: s[k].tolist() for k in ("ctx", "ell", "nout", "table", "held", "free_list", "free_count")}
    width, count = len(r["table"][0]), r["free_count"][0]
    start, slot, pos, kv_len, full = [0], [], [], [], False
    for b, (c, e) in enumerate(zip(r["ctx"], r["ell"])):
        n = max(0, min(e + 1, width * P - c))
        need = max(0, -(-(c + n) // P) - r["held"][b])
        full = full or need > count
        if need and full:
            n, need = max(0, min(n, r["held"][b] * P - c)), 0
        for _ in range(need):
            count -= 1
            r["table"][b][r["held"][b]] = r["free_list"][count]
            r["held"][b] += 1
        for p in range(c, c + n):
            pos.append(p)
            slot.append(r["table"][b][p // P] * P + p % P)
        start.append(start[-1] + n)
        kv_len.append(c + n)
    back, out = [], []
    for b, c in enumerate(r["ctx"]):
        out.append(c + min(r["nout"][b], start[b + 1] - start[b]))
        keep = -(-out[b] // P)
        for j in range(keep, r["held"][b]):
            back.append(r["table"][b][j])
            r["table"][b][j] = -1
        r["held"][b] = min(keep, r["held"][b])
    for page in reversed(back):
        r["free_list"][count] = page
        count += 1
    pad = [-1] * (T - len(slot))
    put = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    return {"table": put(r["table"]), "held": put(r["held"]), "free_list": put(r["free_list"]),
            "free_count": put([count]), "q_start": put(start), "kv_len": put(kv_len), "slot": put(slot + pad),
            "pos": put(pos + pad), "ctx_out": put(out)}


def _nearest(x):
    """Values of 16-dim groups in 64 bits: every dim goes to the nearest of the 15 grid points times the scale."""
    y = x.reshape(*x.shape[:-1], -1, 16)
    scale = (y.abs().amax(-1, keepdim=True) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn).double()
    grid = torch.tensor(GRID, dtype=torch.float64, device=x.device)
    # Order the candidates so that on a tie the even code comes first.
    order = torch.tensor([0, 2, 4, 6, 1, 3, 5, 7], device=x.device)
    gap = (y.abs()[..., None] - grid[order] * scale[..., None]).abs()
    val = grid[order][gap.argmin(-1)] * scale
    return torch.where(y < 0, -val, val).reshape(x.shape)


def _exact_norm(s):
    case = s["case"]
    D, rot, m = case["D"], case["rot"], int(s["q_start"][-1])
    half = rot // 2
    ang = s["pos"][:m].double()[:, None] * s["inv_freq"].double()
    turn = torch.polar(torch.ones_like(ang), ang)[:, None, :]                 # e^{i angle}

    def rows(x, w):
        x = x[:m].double()
        x = x / (x.square().sum(-1, keepdim=True) / D + EPS).sqrt() * w.double()
        if not rot:
            return x
        lo, hi = (slice(0, rot, 2), slice(1, rot, 2)) if case["inter"] else (slice(0, half), slice(half, rot))
        z = torch.complex(x[..., lo], x[..., hi]) * turn
        x[..., lo], x[..., hi] = z.real, z.imag
        return x

    def whole(x, like):
        r = like.double()
        r[:m] = x
        return r

    q, k = whole(rows(s["q"], s["wq"]), s["q_out"]), rows(s["k"], s["wk"])
    if not case["write"]:
        return {"q": q, "k": whole(k, s["k_out"])}
    return {"q": q, "k": whole(_nearest(k), s["k_val"]), "v": whole(_nearest(s["v"][:m].double()), s["v_val"])}


def _minifloat(bits, man, bias):
    """Integer bits (sign dropped) of a float with `man` mantissa bits -> float64."""
    e, m = (bits >> man).double(), (bits & ((1 << man) - 1)).double() / (1 << man)
    return torch.where(e > 0, (1 + m) * torch.exp2(e - bias), m * 2.0 ** (1 - bias))


def _values(half, P, D):
    """One half of records [pages, Hkv, P * D * 9 / 16] -> float64 [Hkv, pages * P, D], from the bits."""
    n, h = half.shape[:2]
    code = half[..., :P * D // 2].reshape(n, h, D // 32, P, 16).int()
    code = torch.stack((code % 16, code // 16), -1)                           # [n, h, D/32, P, 16, 2]
    val = _minifloat(code % 8, 1, 1) * (1 - 2 * (code // 8)).double()
    val = val.permute(1, 0, 3, 2, 4, 5).reshape(h, n * P, D // 16, 16)
    scale = _minifloat(half[..., P * D // 2:].int() % 128, 3, 7).reshape(n, h, P, D // 16)
    return (val * scale.transpose(0, 1).reshape(h, n * P, D // 16, 1)).reshape(h, n * P, D)


def _exact_attend(s):
    case, P, D = s["case"], s["P"], s["case"]["D"]
    Hkv, group = case["Hkv"], case["Hq"] // case["Hkv"]
    out = s["out"].double()
    start, lens = s["q_start"].tolist(), s["kv_len"].tolist()
    half = s["cache"].shape[2] // 2
    for b, (n, L) in enumerate(zip((y - x for x, y in zip(start, start[1:])), lens)):
        lo = max(0, L - n - case["window"] + 1) // P * P if case["window"] > 0 else 0
        rec = s["cache"][s["table"][b, lo // P:_pages(L, P)].long()]          # [pages, Hkv, R]
        K, V = (_values(r, P, D)[:, :L - lo] for r in (rec[..., :half], rec[..., half:]))
        q = s["q"][start[b]:start[b + 1]].double().reshape(n, Hkv, group, D)
        x = torch.einsum("nhgd,hsd->hgns", q, K) * s["scale"]
        i = torch.arange(n, device="cuda")[:, None] + (L - n)
        key = torch.arange(lo, L, device="cuda")[None, :]
        hide = (key > i) | ((key <= i - case["window"]) if case["window"] > 0 else False)
        p = torch.softmax(x.masked_fill(hide, -math.inf), -1)
        out[start[b]:start[b + 1]] = torch.einsum("hgns,hsd->nhgd", p, V).reshape(n, Hkv * group, D)
    return out
