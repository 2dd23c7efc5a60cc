"""Cases for the 8-bit KV cache operators and the query / key norm with rotation.

Operators (include/pkv.h, reached through paged_kv_decode_bind_gb300):

  attn    decode attention over a paged cache of 8-bit codes with one scale for
          each block of tokens and KV head (pkv_kv8_decode_layer)
  append  new K/V rows quantised into that cache as they are written, one row
          per request or a chunk per request, and read back
          (pkv_kv8_append / pkv_kv8_extend_append, pkv_kv8_read)
  read    the cached rows of every request back as bf16 (pkv_kv8_read)
  rope    RMS norm of every query and key head with the position rotation in
          the same pass (pkv_qk_norm_rope)

A scale is a power of two: the smallest 2^e, e in [-100, 100], with
amax <= qmax * 2^e over the block's rows of one KV head (qmax 448 for e4m3, 127
for int8).  A block that already holds rows keeps the larger of its scale and
the new rows'; where it grows, the older codes are rounded to the new scale.
"""
import math
import random

import torch

own = False

QMAX = {"e4m3": 448.0, "int8": 127.0}
DEV = "cuda"


# ------------------------------------------------------------------ cases ----
def listed():
    return [
        # the smallest decode batch: one request, one layer, latency only
        dict(name="attn_single_d64", op="attn", batch=1, hq=8, hkv=2, d=64, page=16, block=16,
             lo=128, hi=128, spread="uniform", dtype="e4m3", lens_seed=1, outliers=0.0),
        # a small serving batch of ordinary contexts on 16-token pages
        dict(name="attn_paged_b4", op="attn", batch=4, hq=32, hkv=8, d=128, page=16, block=16,
             lo=512, hi=2048, spread="uniform", dtype="e4m3", lens_seed=2, outliers=0.01),
        # token-level indices (page size 1), lengths from one token to 8192
        dict(name="attn_flat_b16", op="attn", batch=16, hq=32, hkv=8, d=128, page=1, block=1,
             lo=1, hi=8192, spread="log", dtype="int8", lens_seed=3, outliers=0.0),
        # a full decode batch, groups of eight query heads
        dict(name="attn_sweep_b64", op="attn", batch=64, hq=16, hkv=2, d=128, page=16, block=16,
             lo=1024, hi=4096, spread="uniform", dtype="e4m3", lens_seed=4, outliers=0.0),
        # long contexts: 64 Ki tokens each, outlier keys
        dict(name="attn_long_b4", op="attn", batch=4, hq=32, hkv=8, d=128, page=16, block=16,
             lo=65536, hi=65536, spread="uniform", dtype="int8", lens_seed=5, outliers=0.01),
        # one decode step's rows of a full batch, into blocks partly filled
        dict(name="append_decode_b64", op="append", batch=64, hq=16, hkv=2, d=128, page=16,
             block=16, lo=1024, hi=4096, spread="uniform", new=1, chunk=False, dtype="e4m3",
             lens_seed=6),
        # a prefill chunk on cached prefixes, and the context back as bf16
        dict(name="append_chunk_b4", op="append", batch=4, hq=32, hkv=8, d=128, page=16, block=16,
             lo=512, hi=2048, spread="uniform", new=256, chunk=True, dtype="int8", lens_seed=7),
        # ragged contexts on token-level indices read back
        dict(name="read_flat_b16", op="read", batch=16, hq=32, hkv=8, d=128, page=1, block=1,
             lo=1, hi=8192, spread="log", dtype="int8", lens_seed=8),
        # one long prefix read back before a chunk attends it
        dict(name="read_prefix_32k", op="read", batch=1, hq=32, hkv=8, d=128, page=16, block=16,
             lo=32832, hi=32832, spread="uniform", dtype="e4m3", lens_seed=9),
        # the decode step's queries and keys of a small batch
        dict(name="rope_decode_b4", op="rope", tokens=4, hq=32, hkv=8, d=128, rot=128,
             interleaved=False, norm=True, packed=True, span=2048),
        # a chunk, head size 64, half of it rotated in adjacent pairs
        dict(name="rope_chunk_d64", op="rope", tokens=1024, hq=16, hkv=2, d=64, rot=32,
             interleaved=True, norm=True, packed=True, span=4096),
        # a long prompt in one pass
        dict(name="rope_prompt_32k", op="rope", tokens=32768, hq=32, hkv=8, d=128, rot=128,
             interleaved=False, norm=True, packed=True, span=65536),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "append", "read", "rope"])
    hkv = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 4, 8, 16] if hkv <= 2 else [1, 2, 4])
    c = dict(op=op, hq=hkv * group, hkv=hkv, d=rng.choice([64, 128]))
    if op == "rope":
        c.update(tokens=_log(rng, 1, 16384), rot=rng.choice([16, 32, 64, c["d"]]),
                 interleaved=rng.random() < 0.5, norm=rng.random() < 0.8,
                 packed=rng.random() < 0.5, span=_log(rng, 16384, 131072))
        return c
    page = rng.choice([1, 5, 8, 16, 16, 32, 48, 64])
    block = rng.choice([x for x in (1, 2, 4, 5, 8, 16, 24, 32, 64) if page % x == 0])
    batch = _log(rng, 1, 64)
    # rows: below the longest listed case (what is read back moves three times the bytes)
    budget = (2_000_000 if op == "attn" else 600_000) // (hkv * batch)
    hi = max(1, min(65536, _log(rng, max(1, min(64, budget // 2)), max(2, budget))))
    c.update(batch=batch, page=page, block=block, lo=rng.choice([0, 1, max(1, hi // 2)]), hi=hi,
             spread=rng.choice(["uniform", "log"]), dtype=rng.choice(["e4m3", "int8"]),
             lens_seed=rng.randrange(1 << 20))
    if op == "attn":
        c["outliers"] = rng.choice([0.0, 0.01])
    if op == "append":
        c["chunk"] = rng.random() < 0.6
        c["new"] = _log(rng, 1, min(512, max(2, budget // 4))) if c["chunk"] else 1
    return c


def _lens(case):
    """Cached tokens of every request (before the append, for `append`)."""
    r = random.Random(case["lens_seed"])
    lo, hi = case["lo"], max(case["lo"], case["hi"])
    if case["spread"] == "log":
        a = max(1, lo)
        lens = [int(round(math.exp(r.uniform(math.log(a), math.log(max(a, hi)))))) for _ in
                range(case["batch"])]
        lens[0] = lo  # a request of the least length (0 where the range starts there)
        lens[-1] = hi
        return lens
    return [r.randint(lo, hi) for _ in range(case["batch"])]


def _new(case):
    """New tokens of every request (`append`)."""
    if not case["chunk"]:
        return [1] * case["batch"]
    r = random.Random(case["lens_seed"] + 1)
    return [case["new"]] + [r.randint(max(1, case["new"] // 2), case["new"])
                            for _ in range(case["batch"] - 1)]


def _read_starts(case, lens, new):
    """First token read back: the start of the first block that changes for the
    rows of a decode step, the whole context for a chunk."""
    if case["chunk"]:
        return [0] * len(lens)
    return [n // case["block"] * case["block"] for n in lens]


def work(case):
    hkv, d = case["hkv"], case["d"]
    if case["op"] == "rope":
        rows = case["tokens"] * (case["hq"] + hkv)
        return {"bytes": rows * d * 4 + case["tokens"] * (case["rot"] * 4 + 4) + 4 * d,
                "flops": rows * (4 * d + 3 * case["rot"])}
    lens, blk = _lens(case), case["block"]
    code = lambda ns: sum(ns) * hkv * d * 2 + sum(-(-n // blk) for n in ns) * hkv * 8  # noqa: E731
    if case["op"] == "attn":
        rows = case["batch"] * case["hq"]
        return {"bytes": code(lens) + rows * (d * 4 + 4), "flops": 4 * sum(lens) * case["hq"] * d}
    if case["op"] == "read":
        return {"bytes": code(lens) + sum(lens) * hkv * d * 4, "flops": 2 * sum(lens) * hkv * d}
    new = _new(case)
    # codes written, and read back as bf16: what changes a row's bytes only once
    starts = _read_starts(case, lens, new)
    back = [a + b - s for a, b, s in zip(lens, new, starts)]
    return {"bytes": sum(new) * hkv * d * 4 + code(new) + code([x - y for x, y in zip(back, new)])
            + sum(back) * hkv * d * 4, "flops": 4 * (sum(new) + sum(back)) * hkv * d}


# ----------------------------------------------------------------- inputs ----
def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 7 + 3)


def _exponent(amax, dtype):
    """Smallest e in [-100, 100] with amax <= qmax * 2^e."""
    m, x = torch.frexp(amax)  # amax = m * 2^x, m in [1/2, 1)
    top, shift = (0.875, 9) if dtype == "e4m3" else (0.9921875, 7)  # qmax = top * 2^shift
    e = torch.where(m <= top, x - shift, x - shift + 1)
    return torch.where(amax > 0, e, torch.full_like(e, -100)).clamp(-100, 100)


def _power(e):
    """2^e in 32 bits, for whole e in the exponent's range."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _encode(y, dtype):
    """Codes (as bytes) of values already divided by their scale."""
    if dtype == "e4m3":
        return y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return y.round().clamp(-127, 127).to(torch.int8).view(torch.uint8)


def _decode(codes, dtype):
    return codes.view(torch.float8_e4m3fn if dtype == "e4m3" else torch.int8).float()


def _cache(g, pages, case, outliers):
    """Codes [1, slots, hkv, d] and scales [1, pages, hkv, page / block] of one pool
    of normal rows, rounded to bf16 as a model's are."""
    P, blk, H, D = case["page"], case["block"], case["hkv"], case["d"]
    x = torch.randn((pages * P, H, D), generator=g, device=DEV)
    if outliers:
        x *= torch.where(torch.rand((pages * P, 1, 1), generator=g, device=DEV) < outliers, 8., 1.)
    x = x.bfloat16().float().view(pages, P // blk, blk, H, D)
    e = _exponent(x.abs().amax(dim=(2, 4)), case["dtype"])  # [pages, P / blk, H]
    s = _power(e)
    codes = _encode(x / s[:, :, None, :, None], case["dtype"])
    return codes.view(1, pages * P, H, D), s.permute(0, 2, 1).contiguous().view(1, pages, H, P // blk)


def prepare(case, seed):
    g = _generator(seed)
    H, D, Hq = case["hkv"], case["d"], case["hq"]
    st = {"case": case}
    if case["op"] == "rope":
        T, rot = case["tokens"], case["rot"]
        width = (Hq + 2 * H) * D if case["packed"] else Hq * D
        x = (torch.randn((T, width), generator=g, device=DEV) * 2).bfloat16()
        st["q"] = x[:, :Hq * D]
        st["k"] = x[:, Hq * D:(Hq + H) * D] if case["packed"] else \
            (torch.randn((T, H * D), generator=g, device=DEV) * 2).bfloat16()
        start = int(torch.randint(0, case["span"] - T + 1, (1,), generator=g, device=DEV))
        st["positions"] = torch.arange(start, start + T, device=DEV, dtype=torch.int32)
        w = [(1 + 0.1 * torch.randn(D, generator=g, device=DEV)).bfloat16() for _ in range(2)]
        st["q_weight"], st["k_weight"] = w if case["norm"] else (None, None)
        inv = 10000.0 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
        ang = torch.arange(case["span"], device=DEV, dtype=torch.float64)[:, None] * inv[None]
        st["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()
        st["eps"] = 1e-6
        st["q_out"] = torch.zeros((T, Hq, D), dtype=torch.bfloat16, device=DEV)
        st["k_out"] = torch.zeros((T, H, D), dtype=torch.bfloat16, device=DEV)
        if own:
            import paged_kv_decode_bind_gb300 as pkv
            st["rope"] = pkv.QkNormRope(
                n_q_heads=Hq, n_kv_heads=H, head_dim=D, rot_dim=rot, cos_sin=st["cos_sin"],
                q_weight=st["q_weight"], k_weight=st["k_weight"], eps=st["eps"],
                interleaved=case["interleaved"])
        return st
    lens = _lens(case)
    new = _new(case) if case["op"] == "append" else [0] * len(lens)
    B, P, blk = len(lens), case["page"], case["block"]
    total = [a + b for a, b in zip(lens, new)]
    per = [max(1, -(-n // P)) for n in total]
    pages = sum(per) + max(4, sum(per) // 8)
    cols = max(per)
    perm = torch.randperm(pages, generator=g, device=DEV).int()
    rows = torch.randperm(2 * B, generator=g, device=DEV)[:B].int()
    table = torch.full((2 * B, cols), -1, dtype=torch.int32, device=DEV)
    off = 0
    for b, r in enumerate(rows.tolist()):
        table[r, :per[b]] = perm[off:off + per[b]]
        off += per[b]
    st.update(table=table, rows=rows, pages=pages,
              lens=torch.tensor(total, dtype=torch.int32, device=DEV))
    outliers = case.get("outliers", 0.0)
    st["k_pool"], st["k_scale"] = _cache(g, pages, case, outliers)
    st["v_pool"], st["v_scale"] = _cache(g, pages, case, 0.0)
    i32 = dict(dtype=torch.int32, device=DEV)
    if case["op"] == "attn":
        st["q"] = torch.randn((B, Hq, D), generator=g, device=DEV).bfloat16()
        st["scale"] = D ** -0.5
        st["most"] = max(total)
    else:
        starts = _read_starts(case, lens, new) if case["op"] == "append" else [0] * B
        back = [a - s for a, s in zip(total, starts)]
        st["starts"] = torch.tensor(starts, **i32)
        st["dst"] = torch.tensor([sum(back[:b]) for b in range(B + 1)], **i32)
        st["n_back"] = sum(back)
        st["k_out"] = torch.zeros((sum(back), H, D), dtype=torch.bfloat16, device=DEV)
        st["v_out"] = torch.zeros_like(st["k_out"])
    if case["op"] == "append":
        T = sum(new)
        st["qo_indptr"] = torch.tensor([sum(new[:b]) for b in range(B + 1)], **i32)
        st["n_new"], st["max_new"] = T, max(new)
        # later rows are now and then larger than what their block has seen
        big = torch.exp(torch.randn((2, T, 1, 1), generator=g, device=DEV) * 0.7)
        x = (torch.randn((2, T, H, D), generator=g, device=DEV) * big).bfloat16()
        st["k_new"], st["v_new"] = x[0].contiguous(), x[1].contiguous()
    if own:
        import paged_kv_decode_bind_gb300 as pkv
        flat = P == 1
        S = 1
        ws = pkv.Workspace(n_layers=1, pool_slots=pages * P, n_q_heads=Hq, n_kv_heads=H,
                           head_dim=D, page_size=P, max_batch=B, max_reqs=2 * B,
                           max_pages_per_req=cols, max_splits=256 if case["op"] == "attn" else 1,
                           max_total_tokens=sum(total) if flat else 0, pools=False)
        ws.page_table.copy_(table)
        ws.req_pool_indices.copy_(rows)
        ws.seq_lens.copy_(st["lens"])
        pkv.pkv_bind_step(ws, B, pkv.PKV_BIND_REBUILD)
        if case["op"] == "attn":
            sms = torch.cuda.get_device_properties(0).multi_processor_count
            S = pkv.pkv_choose_pieces(ws, B, max(total), sum(total), sms)
        st["cache"] = pkv.Kv8Cache(ws, dtype=case["dtype"], scale_block=blk,
                                   k_pool=st["k_pool"], v_pool=st["v_pool"],
                                   k_scale=st["k_scale"], v_scale=st["v_scale"])
        st["ws"], st["splits"] = ws, S
        st["out"], st["lse"] = ws.out_bf16(B), ws.lse[:B]
    return st


# ------------------------------------------------------------ plain forms ----
def _slots(st, tok, req=None):
    """Pool slots of token positions tok [B, n] (or [n] of requests req [n])."""
    P = st["case"]["page"]
    rows = st["rows"].long() if req is None else st["rows"].long()[req]
    page = st["table"][rows[:, None] if req is None else rows, tok // P].clamp_min(0).long()
    return page * P + tok % P


def _scales(st, scale, slots):
    """Scale of every (slot, head): slots [...] -> [..., H]."""
    P, blk = st["case"]["page"], st["case"]["block"]
    return scale[0].permute(0, 2, 1)[slots // P, slots % P // blk]


def _rows(st, side, slots):
    """Dequantised rows [..., H, D] in 32 bits."""
    return _decode(st[side + "_pool"][0][slots], st["case"]["dtype"]) * \
        _scales(st, st[side + "_scale"], slots)[..., None]


def _plain_attn(st):
    c = st["case"]
    tok = torch.arange(max(1, st["most"]), device=DEV)
    live = tok[None] < st["lens"][:, None]  # [B, L]
    slots = _slots(st, tok[None].expand(live.shape).clamp_max((st["table"].shape[1]) * c["page"] - 1))
    k = _rows(st, "k", slots)
    q = st["q"].float().view(c["batch"], c["hkv"], -1, c["d"])
    s = torch.matmul(q, k.permute(0, 2, 3, 1)) * st["scale"]  # [B, H, G, L]
    del k
    s = s.masked_fill(~live[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m.clamp_min(-3e38))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, _rows(st, "v", slots).permute(0, 2, 1, 3)) / total.clamp_min(1e-38)
    o = torch.where(total > 0, o, torch.zeros_like(o))
    return {"out": o.reshape(c["batch"], c["hq"], c["d"]).bfloat16(),
            "lse": (m + torch.log(total)).reshape(c["batch"], c["hq"])}


def _plain_read(st):
    row = torch.arange(st["n_back"], device=DEV)
    req = torch.searchsorted(st["dst"].long(), row, right=True) - 1
    tok = row - st["dst"].long()[req] + st["starts"].long()[req]
    slots = _slots(st, tok, req)
    return {"k": _rows(st, "k", slots).bfloat16(), "v": _rows(st, "v", slots).bfloat16()}


def _plain_append(st):
    """New rows into the cache: every block that gets rows, in one padded array
    [blocks, block, H, D] of older codes and new rows."""
    c = st["case"]
    P, blk, dtype = c["page"], c["block"], c["dtype"]
    row = torch.arange(st["n_new"], device=DEV)
    ind = st["qo_indptr"].long()
    req = torch.searchsorted(ind, row, right=True) - 1
    first = st["lens"].long()[req] - (ind[req + 1] - ind[req])  # tokens cached before
    tok = first + row - ind[req]
    slots = _slots(st, tok, req)
    blocks, at = torch.unique(slots // blk, return_inverse=True)
    inside = slots % blk
    n = blocks.numel()
    began = torch.full((n,), blk, device=DEV).scatter_reduce(0, at, inside, "amin")
    place = torch.arange(blk, device=DEV)
    held = place[None] < began[:, None]  # older rows of the block
    of_block = blocks[:, None] * blk + place[None]
    for side in ("k", "v"):
        pool, scale = st[side + "_pool"][0], st[side + "_scale"][0]
        x = st[side + "_new"].float()
        amax = torch.zeros((n, x.shape[1]), device=DEV).scatter_reduce(
            0, at[:, None].expand(-1, x.shape[1]), x.abs().amax(-1), "amax")
        want = _power(_exponent(amax, dtype))
        page, sub = blocks * blk // P, blocks * blk % P // blk
        old = scale[page, :, sub]  # [n, H]
        new = torch.where((began > 0)[:, None], torch.maximum(old, want), want)
        codes = pool[of_block]
        again = _encode(_decode(codes, dtype) * (old / new)[:, None, :, None], dtype)
        pool[of_block] = torch.where(held[..., None, None], again, codes)
        pool[slots] = _encode(x / new[at][..., None], dtype)
        scale[page, :, sub] = new


def _plain_rope(st):
    c = st["case"]
    rot, T = c["rot"], c["tokens"]
    cs = st["cos_sin"][st["positions"].long()][:, None]
    cos, sin = cs[..., :rot // 2], cs[..., rot // 2:]

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
    op = c["op"]
    if own:
        import paged_kv_decode_bind_gb300 as pkv
        B = c.get("batch", 0)
        if op == "attn":
            pkv.pkv_kv8_decode_layer(st["ws"], st["cache"], B, 0, st["q"], None, None,
                                     st["scale"], st["splits"], pkv.PKV_FLAG_WRITE_LSE)
            return {"out": st["out"], "lse": st["lse"]}
        if op == "rope":
            pkv.pkv_qk_norm_rope(st["rope"], c["tokens"], st["q"], st["k"], st["positions"],
                                 st["q_out"], st["k_out"])
            return {"q": st["q_out"], "k": st["k_out"]}
        if op == "append" and c["chunk"]:
            pkv.pkv_kv8_extend_append(st["ws"], st["cache"], B, 0, st["qo_indptr"],
                                      st["max_new"], st["k_new"], st["v_new"])
        elif op == "append":
            pkv.pkv_kv8_append(st["ws"], st["cache"], B, 0, 1, st["k_new"], st["v_new"])
        pkv.pkv_kv8_read(st["ws"], st["cache"], B, 0, st["starts"], st["dst"], st["n_back"],
                         st["k_out"], st["v_out"])
        got = {"k": st["k_out"], "v": st["v_out"]}
    elif op == "attn":
        return _plain_attn(st)
    elif op == "rope":
        return _plain_rope(st)
    else:
        if op == "append":
            _plain_append(st)
        got = _plain_read(st)
    if op == "append":
        got.update(k_scale=st["k_scale"], v_scale=st["v_scale"])
    return got


# ---------------------------------------------------------- in 64 bits -------
def _powers64(lo, hi):
    """2^lo .. 2^hi; a device's pow is not exact."""
    return torch.tensor([2.0 ** e for e in range(lo, hi + 1)], dtype=torch.float64, device=DEV)


def _value64(codes, dtype):
    """What a code stands for, from its bits."""
    c = codes.long()
    if dtype == "int8":
        return torch.where(c > 127, c - 256, c).double()
    mag, man = (c >> 3) & 15, (c & 7).double()
    v = torch.where(mag > 0, (8 + man) * _powers64(-10, 5)[mag], man * 2.0 ** -9)
    v = torch.where((c & 127) == 127, torch.full_like(v, math.nan), v)
    return torch.where(c > 127, -v, v)


def _nearest64(y, dtype):
    """The value of the code nearest to y (ties to the even one), saturating."""
    if dtype == "int8":
        return torch.round(y).clamp(-127, 127)
    # |y| = m * 2^x, m in [1/2, 1): steps of 2^(x - 4), of 2^-9 below the normal range
    x = torch.frexp(y.abs().clamp(2.0 ** -6, 448))[1].long()
    step = _powers64(-9, 5)[x - 4 + 9]
    return (torch.round(y / step) * step).clamp(-448, 448)


def _at64(st, b, tok):
    """Slots and (page, block in page) of request b's tokens, by its table row."""
    P, blk = st["case"]["page"], st["case"]["block"]
    line = st["table"][int(st["rows"][b])].long()
    page = line[torch.div(tok, P, rounding_mode="floor")]
    return page * P + tok % P, page, torch.div(tok % P, blk, rounding_mode="floor")


def _request64(st, side, b, tok):
    slot, page, sub = _at64(st, b, tok)
    s = st[side + "_scale"][0][page, :, sub].double()
    return _value64(st[side + "_pool"][0][slot], st["case"]["dtype"]) * s[..., None]


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    H, D = case["hkv"], case["d"]
    if case["op"] == "rope":
        pos, rot = st["positions"].long(), case["rot"]
        cos = st["cos_sin"].double()[pos, :rot // 2].unsqueeze(1)
        sin = st["cos_sin"].double()[pos, rot // 2:].unsqueeze(1)
        got = {}
        for name, heads in (("q", case["hq"]), ("k", H)):
            x = st[name].double().reshape(case["tokens"], heads, D)
            if case["norm"]:
                x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / D + st["eps"])
                x = x * st[name + "_weight"].double()
            i = torch.arange(rot // 2, device=DEV)
            lo, hi = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + rot // 2)
            y = x.clone()
            y[..., lo] = x[..., lo] * cos - x[..., hi] * sin
            y[..., hi] = x[..., hi] * cos + x[..., lo] * sin
            got[name] = y
        return got
    lens = st["lens"].tolist()
    if case["op"] == "attn":
        out = torch.zeros((len(lens), case["hq"], D), dtype=torch.float64, device=DEV)
        lse = torch.full((len(lens), case["hq"]), -math.inf, dtype=torch.float64, device=DEV)
        G = case["hq"] // H
        for b, n in enumerate(lens):
            if n == 0:
                continue
            tok = torch.arange(n, device=DEV)
            k, v = _request64(st, "k", b, tok), _request64(st, "v", b, tok)
            for h in range(H):
                q = st["q"][b, h * G:(h + 1) * G].double()
                s = (q @ k[:, h].T) * st["scale"]
                lse[b, h * G:(h + 1) * G] = torch.logsumexp(s, -1)
                out[b, h * G:(h + 1) * G] = torch.softmax(s, -1) @ v[:, h]
        return {"out": out, "lse": lse}
    starts, dst = st["starts"].tolist(), st["dst"].tolist()
    got = {s: torch.zeros((st["n_back"], H, D), dtype=torch.float64, device=DEV) for s in "kv"}
    scales = {s: st[s + "_scale"].double().clone() for s in "kv"}
    powers = _powers64(-100, 100)
    qo = st["qo_indptr"].tolist() if case["op"] == "append" else None
    blk, dtype = case["block"], case["dtype"]
    for b, n in enumerate(lens):
        tok = torch.arange(n, device=DEV)
        if n == 0:
            continue
        for side in "kv":
            x = _request64(st, side, b, tok)
            if qo is not None:
                before = n - (qo[b + 1] - qo[b])
                x[before:] = st[side + "_new"][qo[b]:qo[b + 1]].double()
                # whole blocks from the first that changes on, padded with zeros
                a = before // blk * blk
                pad = -(n - a) % blk
                z = torch.cat([x[a:], x.new_zeros((pad, H, D))]).view(-1, blk, H, D)
                fresh = torch.cat([tok[a:] >= before, tok.new_zeros(pad, dtype=torch.bool)])
                fresh = fresh.view(-1, blk, 1, 1)
                amax = torch.where(fresh, z.abs(), torch.zeros_like(z)).amax(dim=(1, 3))
                want = powers[torch.searchsorted(powers * QMAX[dtype], amax).clamp_max(200)]
                _, page, sub = _at64(st, b, tok[a::blk])
                if before > a:
                    want[0] = torch.maximum(want[0], scales[side][0][page[0], :, sub[0]])
                scales[side][0][page, :, sub] = want
                x[a:] = (_nearest64(z / want[:, None, :, None], dtype) *
                         want[:, None, :, None]).view(-1, H, D)[:n - a]
            got[side][dst[b]:dst[b + 1]] = x[starts[b]:]
    if qo is not None:
        got.update(k_scale=scales["k"], v_scale=scales["v"])
    return got
