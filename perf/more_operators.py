"""Cases for the tally of attention weight, the eviction it decides, and the norm
with rotation by positions of several axes.

Operators (include/pkv.h, reached through paged_kv_decode_bind_gb300):

  decode  decode attention over the paged cache that adds every cached token's
          attention weight to a running tally (pkv_tally_decode_layer)
  prompt  the weight that a chunk's last queries give every token of its context,
          added to the tally (pkv_tally_extend)
  evict   requests past a limit cut to a budget of tokens for each layer and KV
          head, by the tally, their rows moved together in place (pkv_tally_evict)
  step    a decode step on a full cache: bind, attention with the tally, eviction
  axes    RMS norm of every query and key head with a rotation whose pairs follow
          the positions of several axes (pkv_qk_norm_rope_axes)

The tally of a token and KV head is the sum of its weights exp(s - lse) over the
group's query heads and the queries so far; a new token starts at its first
weights.  `origin` is the count of tokens its request held before it, evicted ones
included.  Kept are the tokens whose origin is among the first `sinks` or the last
`recent`, then those of the largest tally, the lowest index first among equals.
Kept tokens past the budget move, in order, into the free places below it.
"""
import math
import random

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases ----
def listed():
    return [
        # the smallest decode batch: one request, latency only
        dict(name="decode_single_d64", op="decode", batch=1, hq=8, hkv=2, d=64, page=16, lo=128,
             hi=128, spread="uniform", lens_seed=1),
        # token-level indices (page size 1), lengths from one token to 8192
        dict(name="decode_flat_b16", op="decode", batch=16, hq=32, hkv=8, d=128, page=1, lo=1,
             hi=8192, spread="log", lens_seed=3),
        # a full decode batch, groups of eight query heads
        dict(name="decode_sweep_b64", op="decode", batch=64, hq=16, hkv=2, d=128, page=16, lo=1024,
             hi=4096, spread="uniform", lens_seed=4),
        # long contexts before their first eviction
        dict(name="decode_long_b4", op="decode", batch=4, hq=32, hkv=8, d=128, page=16, lo=65536,
             hi=65536, spread="uniform", lens_seed=5),
        # a prefill chunk on cached prefixes, all its queries observed
        dict(name="prompt_chunk_b4", op="prompt", batch=4, hq=32, hkv=8, d=128, page=16, lo=512,
             hi=2048, spread="uniform", new=256, window=256, lens_seed=7),
        # the last chunk of a long prompt, whose queries decide what stays
        dict(name="prompt_last_32k", op="prompt", batch=1, hq=32, hkv=8, d=128, page=16, lo=32768,
             hi=32768, spread="uniform", new=64, window=64, lens_seed=8),
        # a whole prompt in one pass, every query observed
        dict(name="prompt_whole_8k", op="prompt", batch=1, hq=32, hkv=8, d=128, page=16, lo=0, hi=0,
             spread="uniform", new=8192, window=8192, lens_seed=9),
        # a batch of prompts cut to a common budget
        dict(name="evict_sweep_b64", op="evict", layers=4, batch=64, hq=16, hkv=2, d=128, page=16,
             lo=1024, hi=4096, spread="uniform", budget=1024, sinks=4, recent=256, lens_seed=10),
        # long contexts cut to an eighth
        dict(name="evict_long_b4", op="evict", layers=1, batch=4, hq=32, hkv=8, d=128, page=16,
             lo=65536, hi=65536, spread="uniform", budget=8192, sinks=4, recent=1024, lens_seed=11),
        # a decode step on a cache at its budget: one token in, one out
        dict(name="step_full_b16", op="step", layers=1, batch=16, hq=32, hkv=8, d=128, page=16,
             lo=2048, hi=2048, spread="uniform", budget=2048, sinks=4, recent=512, lens_seed=12),
        # a decode step's queries and keys behind images and evictions
        dict(name="axes_step_b64", op="axes", tokens=64, hq=16, hkv=2, d=128, rot=128,
             layout="turns", interleaved=False, norm=True, packed=True, step=True),
        # a prompt of text and images in one pass
        dict(name="axes_prompt_16k", op="axes", tokens=16384, hq=32, hkv=8, d=128, rot=128,
             layout="sections", interleaved=False, norm=True, packed=True, step=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "prompt", "prompt", "evict", "evict", "step", "axes"])
    hkv = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 4, 8, 16] if hkv <= 2 else [1, 2, 4])
    c = dict(op=op, hq=hkv * group, hkv=hkv, d=rng.choice([64, 128]))
    if op == "axes":
        c.update(tokens=_log(rng, 1, 16384), rot=rng.choice([32, 64, c["d"]]),
                 layout=rng.choice(["sections", "turns", "one"]), interleaved=rng.random() < 0.5,
                 norm=rng.random() < 0.8, packed=rng.random() < 0.5, step=rng.random() < 0.5)
        return c
    c["page"] = rng.choice([1, 5, 8, 16, 16, 32, 48, 64])
    c.update(spread=rng.choice(["uniform", "log"]), lens_seed=rng.randrange(1 << 20))
    if op == "prompt":
        new = _log(rng, 1, 2048)
        hi = _log(rng, 1, 8192) if rng.random() < 0.8 else 0
        # rows: below half of the whole prompt's scores
        batch = max(1, min(16, (1 << 30) // (c["hq"] * new * (hi + new))))
        c.update(batch=rng.randint(1, batch), lo=hi // 2, hi=hi, new=new,
                 window=rng.choice([new, rng.randint(1, new)]))
        return c
    layers = 1 if op == "decode" else rng.choice([1, 2, 3])
    batch = _log(rng, 1, 64)
    budget = 2_000_000 // (hkv * batch * layers)  # rows: below the longest listed case
    hi = max(2, min(65536, _log(rng, 64, max(65, budget))))
    c.update(batch=batch, lo=rng.choice([0, 1, hi // 2]), hi=hi)
    if op != "decode":
        keep = rng.randint(max(1, hi // 8), hi - 1)
        recent = rng.randint(0, keep // 2)
        c.update(layers=layers, budget=keep, recent=recent, sinks=rng.randint(0, min(8, keep - recent)))
    if op == "step":
        c.update(lo=c["budget"], hi=c["budget"])
    return c


def _lens(case):
    """Cached tokens of every request before the pass."""
    r = random.Random(case["lens_seed"])
    lo, hi = case["lo"], case["hi"]
    if case["spread"] == "log" and hi > 0:
        a = max(1, lo)
        lens = [int(round(math.exp(r.uniform(math.log(a), math.log(hi))))) for _ in
                range(case["batch"])]
        lens[0] = lo  # a request of the least length (0 where the range starts there)
        lens[-1] = hi
        return lens
    return [r.randint(lo, hi) for _ in range(case["batch"])]


def _new(case):
    """New tokens of every request (`prompt`)."""
    r = random.Random(case["lens_seed"] + 1)
    return [case["new"]] + [r.randint(max(1, case["new"] // 2), case["new"])
                            for _ in range(case["batch"] - 1)]


def _moves(case, n):
    """Rows that move when a request of n tokens is cut to the budget, if its tally
    says nothing about its tokens' places."""
    keep, recent, sinks = case["budget"], case["recent"], case["sinks"]
    if n <= keep:
        return 0
    late = max(0, n - keep - recent)  # unprotected tokens past the budget
    return min(recent, n - keep) + (keep - recent - sinks) * late / max(1, n - recent - sinks)


def work(case):
    hkv, hq, d = case["hkv"], case["hq"], case["d"]
    if case["op"] == "axes":
        rows = case["tokens"] * (hq + hkv)
        return {"bytes": rows * d * 4 + case["tokens"] * (case["rot"] * 4 + 12) + 4 * d,
                "flops": rows * (4 * d + 3 * case["rot"])}
    lens = _lens(case)
    if case["op"] == "prompt":
        new = _new(case)
        seen = [min(case["window"], n) for n in new]
        pairs = sum(w * (a + n) - w * (w - 1) / 2 for a, n, w in zip(lens, new, seen))
        return {"bytes": sum(lens) * hkv * (2 * d + 8) + sum(new) * hkv * (2 * d + 8)
                + sum(seen) * hq * (2 * d + 4), "flops": 2 * d * hq * pairs}
    layers = case.get("layers", 1)
    attn = {"bytes": sum(lens) * hkv * (4 * d + 8) + case["batch"] * hq * (4 * d + 4),
            "flops": 4 * sum(lens) * hq * d}
    if case["op"] == "decode":
        return attn
    if case["op"] == "step":
        move = sum(_moves(case, n + 1) for n in lens)
        return {"bytes": layers * (attn["bytes"] + hkv * (8 * sum(lens) + move * (8 * d + 16))),
                "flops": layers * attn["flops"]}
    move = sum(_moves(case, n) for n in lens)
    cut = sum(n for n in lens if n > case["budget"])
    return {"bytes": 8 * case["batch"] + layers * hkv * (8 * cut + move * (8 * d + 16)),
            "flops": layers * hkv * cut}


# ----------------------------------------------------------------- inputs ----
def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 7 + 3)


def _axis_of_pair(case):
    """Axis (0 time, 1 height, 2 width) of each rotated pair: an eighth, then three
    eighths twice and the rest to time; in turns over the first three quarters; or one axis."""
    n = case["rot"] // 2
    if case["layout"] == "one":
        return [0] * n
    if case["layout"] == "turns":
        return [i % 3 if i < n * 3 // 4 else 0 for i in range(n)]
    a, b = n // 4, (n - n // 4) // 2
    return [0] * a + [1] * b + [2] * (n - a - b)


def _image_positions(tokens, start):
    """Positions [3, tokens] of 64 tokens of text and an image of 32 x 32 in turns."""
    i = torch.arange(tokens, device=DEV)
    r = i % 1088
    base = start + i // 1088 * 96
    j = r - 64
    text = j < 0
    place = [torch.zeros_like(j), j // 32, j % 32]
    return torch.stack([torch.where(text, base + r, base + 64 + p) for p in place]).int()


def _prepare_axes(case, seed):
    g = _generator(seed)
    H, D, Hq, T, rot = case["hkv"], case["d"], case["hq"], case["tokens"], case["rot"]
    st = {"case": case}
    width = (Hq + 2 * H) * D if case["packed"] else Hq * D
    x = (torch.randn((T, width), generator=g, device=DEV) * 2).bfloat16()
    st["q"] = x[:, :Hq * D]
    st["k"] = x[:, Hq * D:(Hq + H) * D] if case["packed"] else \
        (torch.randn((T, H * D), generator=g, device=DEV) * 2).bfloat16()
    span = 32768
    start = int(torch.randint(0, span // 2, (1,), generator=g, device=DEV))
    st["axis"] = _axis_of_pair(case)
    n_axes = max(st["axis"]) + 1
    st["rows"] = st["evicted"] = st["delta"] = None
    if case["step"]:
        # one token a request: its index in the cache on every axis, moved by what
        # was evicted before it and by its images (which take fewer positions than tokens)
        i32 = dict(generator=g, device=DEV, dtype=torch.int32)
        st["positions"] = torch.randint(4096, 8192, (T,), **i32)
        st["rows"] = torch.randperm(2 * T, generator=g, device=DEV)[:T].int()
        st["evicted"] = torch.randint(0, 16384, (2 * T,), **i32)
        st["delta"] = torch.randint(-4096, 1, (2 * T,), **i32)
    else:
        st["positions"] = _image_positions(T, start)[:n_axes].contiguous()
    w = [(1 + 0.1 * torch.randn(D, generator=g, device=DEV)).bfloat16() for _ in range(2)]
    st["q_weight"], st["k_weight"] = w if case["norm"] else (None, None)
    inv = 10000.0 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
    ang = torch.arange(span, device=DEV, dtype=torch.float64)[:, None] * inv[None]
    st["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()
    st["eps"] = 1e-6
    st["q_out"] = torch.zeros((T, Hq, D), dtype=torch.bfloat16, device=DEV)
    st["k_out"] = torch.zeros((T, H, D), dtype=torch.bfloat16, device=DEV)
    st["pair_axis"] = torch.tensor(st["axis"], device=DEV)
    if own:
        import paged_kv_decode_bind_gb300 as pkv
        st["rope"] = pkv.QkNormRopeAxes(
            n_q_heads=Hq, n_kv_heads=H, head_dim=D, rot_dim=rot, cos_sin=st["cos_sin"],
            q_weight=st["q_weight"], k_weight=st["k_weight"], eps=st["eps"],
            interleaved=case["interleaved"], axis_of_pair=st["axis"], rows=st["rows"],
            evicted=st["evicted"], delta=st["delta"])
    return st


def prepare(case, seed):
    if case["op"] == "axes":
        return _prepare_axes(case, seed)
    g = _generator(seed)
    op, H, D, Hq, P = case["op"], case["hkv"], case["d"], case["hq"], case["page"]
    NL = case.get("layers", 1)
    lens = _lens(case)
    B = len(lens)
    new = _new(case) if op == "prompt" else [0] * B
    # the lengths that the pass meets: decode's with their newest token
    total = [a + b for a, b in zip(lens, new)]
    room = [n + (op == "step") for n in total]
    per = [max(1, -(-n // P)) for n in room]
    pages = sum(per) + max(4, sum(per) // 8)
    cols = max(per)
    perm = torch.randperm(pages, generator=g, device=DEV).int()
    rows = torch.randperm(2 * B, generator=g, device=DEV)[:B].int()
    table = torch.full((2 * B, cols), -1, dtype=torch.int32, device=DEV)
    off = 0
    for b, r in enumerate(rows.tolist()):
        table[r, :per[b]] = perm[off:off + per[b]]
        off += per[b]
    i32 = dict(dtype=torch.int32, device=DEV)
    st = dict(case=case, table=table, rows=rows, most=max(room), scale=D ** -0.5,
              lens=torch.tensor(total, **i32))
    pool = (NL, pages * P, H, D)
    for side in ("k_pool", "v_pool"):
        st[side] = torch.empty(pool, dtype=torch.bfloat16, device=DEV)
        for layer in range(NL):  # a layer at a time: drawn in 32 bits
            st[side][layer] = torch.randn(pool[1:], generator=g, device=DEV)
    # the tally in one buffer: weights, origins (their bits), evicted counts
    n = NL * pages * H * P
    st["book"] = torch.zeros(2 * n + 2 * B, **i32)
    shape = (NL, pages, H, P)
    st["weight"] = st["book"][:n].view(torch.float32).view(shape)
    st["origin"] = st["book"][n:2 * n].view(shape)
    st["evicted"] = st["book"][2 * n:]
    st["weight"].copy_(torch.exp(1.5 * torch.randn(shape, generator=g, device=DEV)))
    gone = 1000 if op == "step" else 0  # tokens behind the sinks, evicted earlier
    st["evicted"][rows.long()] = gone
    tok = torch.arange(cols * P, device=DEV)[None].expand(B, -1)
    held = tok < st["lens"][:, None]
    page, at = _at(st, _slots(st, tok)[held])
    born = torch.where(tok < case.get("sinks", 0), tok, tok + gone).int()[held]
    st["origin"].permute(1, 3, 0, 2)[page, at] = born[:, None, None].expand(-1, NL, H)
    if op == "prompt":
        T = sum(new)
        st["qo_indptr"] = torch.tensor([sum(new[:b]) for b in range(B + 1)], **i32)
        st["n_rows"], st["max_new"] = T, max(new)
        st["q"] = torch.randn((T, Hq, D), generator=g, device=DEV).bfloat16()
        st["lse"] = _prompt_lse(st, lens, new)
    elif op in ("decode", "step"):
        st["q"] = torch.randn((NL, B, Hq, D), generator=g, device=DEV).bfloat16()
        st["k_new"] = torch.randn((NL, B, H, D), generator=g, device=DEV).bfloat16()
        st["v_new"] = torch.randn((NL, B, H, D), generator=g, device=DEV).bfloat16()
    if op == "evict":  # what every pass starts from
        st["book0"] = st["book"].clone()
    if op in ("evict", "step"):
        st["seq_lens"] = st["lens"].clone()
    if own:
        import paged_kv_decode_bind_gb300 as pkv
        S = 64 if op in ("decode", "step") else 1
        ws = pkv.Workspace(n_layers=NL, pool_slots=pages * P, n_q_heads=Hq, n_kv_heads=H,
                           head_dim=D, page_size=P, max_batch=B, max_reqs=2 * B,
                           max_pages_per_req=cols, max_splits=S,
                           max_total_tokens=sum(room) if P == 1 else 0)
        ws.page_table.copy_(table)
        ws.req_pool_indices.copy_(rows)
        ws.seq_lens.copy_(st["lens"])
        for side in ("k_pool", "v_pool"):
            getattr(ws, side).copy_(st[side])
            st[side] = getattr(ws, side)
        pkv.pkv_bind_step(ws, B, pkv.PKV_BIND_REBUILD)
        sms = torch.cuda.get_device_properties(0).multi_processor_count
        st["splits"] = pkv.pkv_choose_pieces(ws, B, max(room), sum(room), sms)
        st["tally"] = pkv.Tally(ws, weight=st["weight"], origin=st["origin"],
                                evicted=st["evicted"])
        st["ws"], st["out"], st["lse_out"] = ws, ws.out_bf16(B), ws.lse[:B]
        if op in ("evict", "step"):
            st["seq_lens"] = ws.seq_lens
    return st


def _prompt_lse(st, lens, new):
    """Log-sum-exp of every new token's scores, as the chunk's attention leaves it."""
    c = st["case"]
    H, G = c["hkv"], c["hq"] // c["hkv"]
    lse = torch.empty((st["n_rows"], c["hq"]), device=DEV)
    at = 0
    for b, (a, n) in enumerate(zip(lens, new)):
        tok = torch.arange(a + n, device=DEV)
        k = st["k_pool"][0][_slots(st, tok[None].expand(c["batch"], -1))[b]].float()
        late = tok[None] > a + torch.arange(n, device=DEV)[:, None]
        for h in range(H):
            q = st["q"][at:at + n, h * G:(h + 1) * G].float().transpose(0, 1)
            s = (q @ k[:, h].T) * st["scale"]
            lse[at:at + n, h * G:(h + 1) * G] = torch.logsumexp(
                s.masked_fill_(late[None], -math.inf), -1).T
        at += n
    return lse


# ------------------------------------------------------------ plain forms ----
def _slots(st, tok):
    """Pool slots of token positions tok [B, n]."""
    P = st["case"]["page"]
    page = st["table"][st["rows"].long()[:, None], tok // P].clamp_min(0).long()
    return page * P + tok % P


def _by_slot(st, name, layer):
    """A layer's tally as [slots, H] (a view where it can be written through)."""
    x = st[name][layer]
    return x.permute(0, 2, 1)  # [pages, P, H]


def _at(st, slots):
    P = st["case"]["page"]
    return slots // P, slots % P


def _plain_decode(st, layer, lens):
    """Append at the last token, attention and tally of one layer."""
    c = st["case"]
    B, H, D = c["batch"], c["hkv"], c["d"]
    k_pool, v_pool = st["k_pool"][layer], st["v_pool"][layer]
    last = _slots(st, (lens.long() - 1).clamp_min(0)[:, None])[:, 0]
    some = lens > 0
    for pool, x in ((k_pool, st["k_new"][layer]), (v_pool, st["v_new"][layer])):
        pool[last] = torch.where(some[:, None, None], x, pool[last])
    tok = torch.arange(st["most"], device=DEV)
    live = tok[None] < lens[:, None]  # [B, L]
    slots = _slots(st, tok[None].expand(live.shape))
    q = st["q"][layer].float().view(B, H, -1, D)
    k = k_pool[slots].float().permute(0, 2, 3, 1)
    s = torch.matmul(q, k) * st["scale"]  # [B, H, G, L]
    del k
    s = s.masked_fill(~live[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True).clamp_min(-3e38)
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    p = p / total.clamp_min(1e-38)
    o = torch.matmul(p, v_pool[slots].float().permute(0, 2, 1, 3))
    lse = torch.where(some[:, None, None, None], m + torch.log(total), -math.inf)
    w = p.sum(2).permute(0, 2, 1)  # [B, L, H]
    weight, origin = _by_slot(st, "weight", layer), _by_slot(st, "origin", layer)
    page, at = _at(st, slots[live])
    newest = (tok[None] == lens[:, None] - 1)[live]
    old = torch.where(newest[:, None], torch.zeros_like(w[live]), weight[page, at])
    weight[page, at] = old + w[live]
    page, at = _at(st, last[some])
    born = lens - 1 + st["evicted"][st["rows"].long()]
    origin[page, at] = born[some][:, None].expand(-1, H)
    return o.reshape(B, c["hq"], D).bfloat16(), lse.reshape(B, c["hq"])


def _plain_prompt(st):
    c = st["case"]
    B, H, D = c["batch"], c["hkv"], c["d"]
    G = c["hq"] // H
    ind, lens = st["qo_indptr"].long(), st["lens"].long()
    n = ind[1:] - ind[:-1]
    i = torch.arange(min(c["window"], st["max_new"]), device=DEV)[None]
    first = (n - c["window"]).clamp_min(0)[:, None]  # the first observed query
    live_q = first + i < n[:, None]  # [B, W]
    row = (ind[:-1, None] + first + i).clamp_max(st["n_rows"] - 1)
    tok = torch.arange(st["most"], device=DEV)[None]
    live_k = tok < lens[:, None]
    slots = _slots(st, tok.expand(live_k.shape))
    q = st["q"][row].float().view(B, -1, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, -1, D)
    k = st["k_pool"][0][slots].float().permute(0, 2, 3, 1)
    s = torch.matmul(q, k).mul_(st["scale"]).view(B, H, G, -1, tok.shape[1])
    s -= st["lse"][row].view(B, -1, H, G).permute(0, 2, 3, 1)[..., None]
    sees = (tok[:, None] <= (lens - n)[:, None, None] + (first + i)[..., None]) & \
        live_q[..., None] & live_k[:, None]  # [B, W, L]
    w = s.masked_fill_(~sees[:, None, None], -math.inf).exp_().sum((2, 3)).permute(0, 2, 1)
    old = tok < (lens - n)[:, None]
    weight, origin = _by_slot(st, "weight", 0), _by_slot(st, "origin", 0)
    page, at = _at(st, slots[live_k])
    was = torch.where(old[live_k][:, None], weight[page, at], torch.zeros_like(w[live_k]))
    weight[page, at] = was + w[live_k]
    fresh = live_k & ~old
    page, at = _at(st, slots[fresh])
    born = (tok + st["evicted"].long()[st["rows"].long()][:, None])[fresh].int()
    origin[page, at] = born[:, None].expand(-1, H)


def _plain_evict(st):
    c = st["case"]
    NL, B, H, keep = c["layers"], c["batch"], c["hkv"], c["budget"]
    rows = st["rows"].long()
    lens = st["seq_lens"]
    total = (lens + st["evicted"][rows])[:, None]
    tok = torch.arange(st["most"], device=DEV)[None]
    slots = _slots(st, tok.expand(B, -1))
    page, at = _at(st, slots)
    cut = (lens > keep)[:, None]
    live = (tok < lens[:, None]) & cut  # [B, L]
    # [NL, B, L, H] -> [NL, B, H, L]
    weight = st["weight"].permute(1, 3, 0, 2)[page, at].permute(2, 0, 3, 1)
    origin = st["origin"].permute(1, 3, 0, 2)[page, at].permute(2, 0, 3, 1)
    safe = (origin < c["sinks"]) | (origin >= (total - c["recent"])[:, None])
    key = torch.where(safe, math.inf, weight.double())
    key = torch.where(live[:, None], key, -math.inf)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :keep]
    kept = torch.zeros(key.shape, dtype=torch.bool, device=DEV).scatter_(-1, order, True)
    kept &= live[:, None]
    # the j-th kept token past the budget takes the j-th free place below it
    src = (kept & (tok >= keep)).nonzero()
    dst = (~kept & (tok < keep) & live[:, None]).nonzero()
    layer, b, h = src[:, 0], src[:, 1], src[:, 2]
    a, z = slots[b, src[:, 3]], slots[b, dst[:, 3]]
    for side in ("k_pool", "v_pool"):
        st[side][layer, z, h] = st[side][layer, a, h]
    for name in ("weight", "origin"):
        x = st[name].permute(0, 1, 3, 2)
        x[(layer, *_at(st, z), h)] = x[(layer, *_at(st, a), h)]
    gone = torch.where(cut[:, 0], lens - keep, 0)
    st["evicted"][rows] += gone
    st["seq_lens"].sub_(gone)


def _plain_axes(st):
    c = st["case"]
    rot, T = c["rot"], c["tokens"]
    pos = st["positions"].long()
    if c["step"]:
        rows = st["rows"].long()
        pos = (pos + st["evicted"].long()[rows] + st["delta"].long()[rows])[None].expand(3, -1)
    pair = torch.arange(rot // 2, device=DEV)
    line = pos[st["pair_axis"]].T  # [T, pairs]
    cos, sin = st["cos_sin"][line, pair][:, None], st["cos_sin"][line, pair + rot // 2][:, None]

    def one(x, w):
        x = x.float().view(T, -1, c["d"])
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + st["eps"]) * w.float()
        if c["interleaved"]:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([y, x[..., rot:]], -1).bfloat16()

    return {"q": one(st["q"], st["q_weight"]), "k": one(st["k"], st["k_weight"])}


def run(st):
    c = st["case"]
    op, B = c["op"], c.get("batch", 0)
    if own:
        import paged_kv_decode_bind_gb300 as pkv
        if op == "axes":
            pkv.pkv_qk_norm_rope_axes(st["rope"], c["tokens"], st["q"], st["k"], st["positions"],
                                      st["q_out"], st["k_out"])
            return {"q": st["q_out"], "k": st["k_out"]}
        ws, tally = st["ws"], st["tally"]
        if op == "prompt":
            pkv.pkv_tally_extend(ws, tally, B, 0, st["qo_indptr"], st["max_new"], st["n_rows"],
                                 c["window"], st["q"], st["lse"], st["scale"])
            return {"weight": st["weight"], "origin": st["origin"]}
        if op == "decode":
            pkv.pkv_tally_decode_layer(ws, tally, B, 0, st["q"], st["k_new"], st["v_new"],
                                       st["scale"], st["splits"])
            return {"out": st["out"], "lse": st["lse_out"], "weight": st["weight"],
                    "origin": st["origin"], "k_pool": st["k_pool"], "v_pool": st["v_pool"]}
    elif op == "axes":
        return _plain_axes(st)
    elif op == "prompt":
        _plain_prompt(st)
        return {"weight": st["weight"], "origin": st["origin"]}
    elif op == "decode":
        out, lse = _plain_decode(st, 0, st["lens"])
        return {"out": out, "lse": lse, "weight": st["weight"], "origin": st["origin"],
                "k_pool": st["k_pool"], "v_pool": st["v_pool"]}
    state = {k: st[k] for k in ("weight", "origin", "evicted", "seq_lens", "k_pool", "v_pool")}
    if op == "evict":
        # every pass meets lengths and a tally as the attention before it left them
        st["book"].copy_(st["book0"])
        st["seq_lens"].copy_(st["lens"])
        if own:
            pkv.pkv_tally_evict(ws, tally, B, st["most"], c["budget"], c["budget"], c["sinks"],
                                c["recent"])
        else:
            _plain_evict(st)
        return state
    if own:
        pkv.pkv_bind_step(ws, B, pkv.PKV_BIND_STEADY)
        for layer in range(c["layers"]):
            pkv.pkv_tally_decode_layer(ws, tally, B, layer, st["q"][layer], st["k_new"][layer],
                                       st["v_new"][layer], st["scale"], st["splits"])
        pkv.pkv_tally_evict(ws, tally, B, st["most"], c["budget"], c["budget"], c["sinks"],
                            c["recent"])
        return dict(state, out=st["out"], lse=st["lse_out"])
    st["seq_lens"].add_(1)
    for layer in range(c["layers"]):
        out, lse = _plain_decode(st, layer, st["seq_lens"])
    _plain_evict(st)
    return dict(state, out=out, lse=lse)


# ---------------------------------------------------------- in 64 bits -------
def _slots64(st, b, n):
    P = st["case"]["page"]
    t = torch.arange(n, device=DEV)
    line = st["table"][int(st["rows"][b])].long()
    return line[torch.div(t, P, rounding_mode="floor")] * P + torch.remainder(t, P)


def _record64(st, name):
    """A tally's values in 64 bits as [NL, slots, H], and how to lay them out again."""
    x = st[name]
    NL, pages, H, P = x.shape
    y = x.double() if name == "weight" else x.long()
    back = lambda z: z.view(NL, pages, P, H).transpose(2, 3).contiguous()  # noqa: E731
    return y.transpose(2, 3).reshape(NL, pages * P, H).contiguous(), back


def _decode64(st, layer, b, n, weight, origin):
    """Request b's token n - 1 appended, its attention and tally, in place."""
    c = st["case"]
    H, G = c["hkv"], c["hq"] // c["hkv"]
    slot = _slots64(st, b, n)
    st["k_pool"][layer, slot[-1]] = st["k_new"][layer, b]
    st["v_pool"][layer, slot[-1]] = st["v_new"][layer, b]
    k, v = (st[x][layer][slot].double() for x in ("k_pool", "v_pool"))
    out, lse = [], []
    weight[layer, slot[-1]] = 0
    origin[layer, slot[-1]] = n - 1 + int(st["evicted"][int(st["rows"][b])])
    for h in range(H):
        s = st["q"][layer, b, h * G:(h + 1) * G].double() @ k[:, h].T * st["scale"]
        p = torch.softmax(s, -1)
        out.append(p @ v[:, h])
        lse.append(torch.logsumexp(s, -1))
        weight[layer, slot, h] += p.sum(0)
    return torch.cat(out), torch.cat(lse)


def _evict64(st, b, n, weight, origin):
    """The kept tokens of request b by one sort of (protected, tally, index) for each
    layer and head."""
    c = st["case"]
    keep, total = c["budget"], n + int(st["evicted"][int(st["rows"][b])])
    slot = _slots64(st, b, n)
    for layer in range(c["layers"]):
        for h in range(c["hkv"]):
            w, o = weight[layer, slot, h].clone(), origin[layer, slot, h]
            w[(o < c["sinks"]) | (o >= total - c["recent"])] = math.inf
            kept = torch.argsort(-w, stable=True)[:keep].sort().values
            movers = kept[kept >= keep]
            free = torch.ones(keep, dtype=torch.bool, device=DEV)
            free[kept[kept < keep]] = False
            to, frm = slot[free.nonzero()[:, 0]], slot[movers]
            for x in (weight, origin, st["k_pool"], st["v_pool"]):
                x[layer, to, h] = x[layer, frm, h]


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    H, D, Hq, op = case["hkv"], case["d"], case["hq"], case["op"]
    G = Hq // H
    if op == "axes":
        T, rot = case["tokens"], case["rot"]
        pos = st["positions"].long()
        if case["step"]:
            pos = pos + (st["evicted"].long() + st["delta"].long())[st["rows"].long()]
        got = {}
        for name, heads in (("q", Hq), ("k", H)):
            x = st[name].double().reshape(T, heads, D)
            if case["norm"]:
                x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / D + st["eps"])
                x = x * st[name + "_weight"].double()
            y = x.clone()
            for i, axis in enumerate(st["axis"]):
                line = st["cos_sin"].double()[pos if case["step"] else pos[axis]]
                cos, sin = line[:, i, None], line[:, rot // 2 + i, None]
                lo, hi = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + rot // 2)
                y[..., lo] = x[..., lo] * cos - x[..., hi] * sin
                y[..., hi] = x[..., hi] * cos + x[..., lo] * sin
            got[name] = y
        return got
    weight, lay = _record64(st, "weight")
    origin, lay_int = _record64(st, "origin")
    lens = st["lens"].tolist()
    if op == "prompt":
        ind = st["qo_indptr"].tolist()
        for b, n in enumerate(lens):
            slot, m = _slots64(st, b, n), ind[b + 1] - ind[b]
            k = st["k_pool"][0][slot].double()
            weight[0, slot[n - m:]] = 0
            origin[0, slot[n - m:]] = torch.arange(n - m, n, device=DEV)[:, None]
            a = max(0, m - case["window"])
            place = torch.arange(n - m + a, n, device=DEV)  # the observed queries' positions
            for h in range(H):
                for x in range(h * G, (h + 1) * G):
                    s = st["q"][ind[b] + a:ind[b + 1], x].double() @ k[:, h].T * st["scale"]
                    p = torch.exp(s - st["lse"][ind[b] + a:ind[b + 1], x].double()[:, None])
                    p = torch.where(torch.arange(n, device=DEV)[None] <= place[:, None], p, 0)
                    weight[0, slot, h] += p.sum(0)
        return {"weight": lay(weight), "origin": lay_int(origin)}
    got = {}
    if op in ("decode", "step"):
        got["out"] = torch.zeros((case["batch"], Hq, D), dtype=torch.float64, device=DEV)
        got["lse"] = torch.full((case["batch"], Hq), -math.inf, dtype=torch.float64, device=DEV)
        for layer in range(case.get("layers", 1)):
            for b, n in enumerate(lens):
                if n + (op == "step") > 0:
                    got["out"][b], got["lse"][b] = _decode64(st, layer, b, n + (op == "step"),
                                                             weight, origin)
    if op in ("evict", "step"):
        for b, n in enumerate(lens):
            n += op == "step"
            if n > case["budget"]:
                _evict64(st, b, n, weight, origin)
                st["evicted"][int(st["rows"][b])] += n - case["budget"]
                lens[b] = case["budget"]
        got.update(evicted=st["evicted"], seq_lens=torch.tensor(lens, device=DEV))
    got.update(weight=lay(weight), origin=lay_int(origin), k_pool=st["k_pool"],
               v_pool=st["v_pool"])
    return got
