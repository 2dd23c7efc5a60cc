"""The 8-bit cache's operators on the GPU against the 64-bit oracle: append (one
row, chunks), read-back and decode attention.

Codes, scales and read-back values are compared bit for bit: every scale is a
power of two, so the values that are rounded are exact.  Attention is held to
the bounds of Problem.attention (derived from the roundings it makes)."""
import numpy as np
import pytest
import torch

import oracle.kv8 as K8
import oracle.ref as R
import pkv_inputs as W
from kv8_problem import K8_values, Problem, check_attention
from paged_kv_decode_bind_gb300 import _abi as A

pytestmark = pytest.mark.gpu

BF16, F32 = 2.0 ** -8, 2.0 ** -24

# (page size, scale block): one block a page, several, one token each, odd
# sizes, blocks over several 16-token pieces, token-level indices
PAGES = [(16, 16), (16, 4), (32, 32), (8, 8), (5, 5), (12, 3), (48, 24), (64, 64), (128, 128),
         (1, 1)]


def _problem(lens, dtype="e4m3", page=16, block=16, heads=(8, 2), d=128, layers=1, steps=0,
             seed=7, outlier=0.0):
    p = W.make_problem(batch=len(lens), n_layers=layers, n_q_heads=heads[0], n_kv_heads=heads[1],
                       head_dim=d, page_size=page, seq_lens=lens, steps=steps, seed=seed,
                       pool_factor=1.3, outlier_frac=outlier)
    return Problem(p, dtype, block)


def _same(cache, prob):
    torch.cuda.synchronize()
    for got, want in ((cache.k_pool, prob.k.codes), (cache.v_pool, prob.v.codes),
                      (cache.k_scale, prob.k.scales), (cache.v_scale, prob.v.scales)):
        assert np.array_equal(got.cpu().numpy(), want)


def _rows(shape, seed, spread=1.5):
    """bf16 rows whose sizes differ, so that some make their block's scale grow."""
    g = torch.Generator().manual_seed(seed)
    size = torch.exp(torch.randn(shape[:-1] + (1,), generator=g) * spread)
    return (torch.randn(shape, generator=g) * size).bfloat16()


def _attend(prob, ws, cache, q, S, lens, flags=0, new=(None, None), layer=0, what=""):
    B = prob.p.batch
    f32 = flags & A.PKV_FLAG_OUT_F32
    A.pkv_kv8_decode_layer(ws, cache, B, layer, q, *new, prob.p.scale, S,
                           flags | A.PKV_FLAG_WRITE_LSE)
    torch.cuda.synchronize()
    got = (ws.out_f32(B) if f32 else ws.out_bf16(B)).double().cpu().numpy()
    check_attention(got, ws.lse[:B].double().cpu().numpy(),
                    prob.attention(layer, q.cpu(), lens), what, F32 if f32 else BF16)
    assert int(ws.err.item()) == 0
    assert int(ws.split_counters.abs().sum()) == 0
    return got


# ------------------------------------------------------------------ append ----
@pytest.mark.parametrize("dtype", ["e4m3", "int8"])
@pytest.mark.parametrize("page,block", PAGES)
@pytest.mark.parametrize("d", [64, 128])
def test_append_rows(cuda, dtype, page, block, d):
    lens = [1, 2, page, page + 1, 3 * page + 2, 37]
    prob = _problem(lens, dtype, page, block, d=d, layers=2)
    ws, cache = prob.device()
    k, v = _rows((2, len(lens), 2, d), 1), _rows((2, len(lens), 2, d), 2)
    A.pkv_kv8_append(ws, cache, len(lens), 0, 2, k.cuda(), v.cuda())
    for layer in range(2):
        for b, n in enumerate(lens):
            for side, x in ((prob.k, k), (prob.v, v)):
                side.append(layer, prob.slots(b, n - 1, n), K8_values(x[layer, b:b + 1]))
    _same(cache, prob)
    assert int(ws.err.item()) == 0


@pytest.mark.parametrize("dtype", ["e4m3", "int8"])
@pytest.mark.parametrize("hkv", [1, 3, 40])
def test_append_head_counts(cuda, dtype, hkv):
    # 40 heads: more rows than one pass of the block holds
    lens = [5, 20]
    prob = _problem(lens, dtype, heads=(hkv, hkv))
    ws, cache = prob.device()
    k, v = _rows((1, 2, hkv, 128), 3), _rows((1, 2, hkv, 128), 4)
    A.pkv_kv8_append(ws, cache, 2, 0, 1, k.cuda(), v.cuda())
    for b, n in enumerate(lens):
        prob.k.append(0, prob.slots(b, n - 1, n), K8_values(k[0, b:b + 1]))
        prob.v.append(0, prob.slots(b, n - 1, n), K8_values(v[0, b:b + 1]))
    _same(cache, prob)


SPECIAL = [0.0, -0.0, float("inf"), float("-inf"), float("nan"), 3e38, -3e38, 1e-38, 448.0, 449.0,
           127.0, 127.5, 2.0 ** -9, 2.0 ** -10, -2.0 ** -10, 1e-30]


@pytest.mark.parametrize("dtype", ["e4m3", "int8"])
@pytest.mark.parametrize("fill", ["mixed", "zero", "nan", "inf", "huge", "tiny"])
def test_append_special_values(cuda, dtype, fill):
    lens = [1, 9, 16]
    prob = _problem(lens, dtype)
    ws, cache = prob.device()
    k = torch.zeros((1, 3, 2, 128))
    if fill == "mixed":
        k[...] = torch.tensor(SPECIAL * 8)
    else:
        k += {"zero": 0.0, "nan": float("nan"), "inf": float("-inf"), "huge": 3e38,
              "tiny": 1e-39}[fill]
    k = k.bfloat16()
    v = -k
    A.pkv_kv8_append(ws, cache, 3, 0, 1, k.cuda(), v.cuda())
    with np.errstate(invalid="ignore", over="ignore"):
        for b, n in enumerate(lens):
            prob.k.append(0, prob.slots(b, n - 1, n), K8_values(k[0, b:b + 1]))
            prob.v.append(0, prob.slots(b, n - 1, n), K8_values(v[0, b:b + 1]))
    torch.cuda.synchronize()
    for got, want in ((cache.k_pool, prob.k.codes), (cache.v_pool, prob.v.codes)):
        got = got.cpu().numpy()
        if dtype == "e4m3":  # the sign of a NaN is not kept by the conversion
            got, want = np.where(got == 0xff, 0x7f, got), np.where(want == 0xff, 0x7f, want)
        assert np.array_equal(got, want)
    assert np.array_equal(cache.k_scale.cpu().numpy(), prob.k.scales)
    assert np.array_equal(cache.v_scale.cpu().numpy(), prob.v.scales)


@pytest.mark.parametrize("dtype", ["e4m3", "int8"])
@pytest.mark.parametrize("page,block", PAGES)
@pytest.mark.parametrize("d", [64, 128])
def test_append_chunks(cuda, dtype, page, block, d):
    before = [0, 1, page - 1, page, 2 * page + 3, 40]
    new = [3 * page + 1, 1, 2, 0, 5, 70]
    lens = [a + b for a, b in zip(before, new)]
    prob = _problem(lens, dtype, page, block, d=d, layers=2)
    ws, cache = prob.device()
    T = sum(new)
    qo = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    k, v = _rows((T, 2, d), 5), _rows((T, 2, d), 6)
    A.pkv_kv8_extend_append(ws, cache, len(lens), 1, torch.from_numpy(qo).cuda(), max(new),
                            k.cuda(), v.cuda())
    for b in range(len(lens)):
        s = prob.slots(b, before[b], lens[b])
        i = 0
        while i < len(s):  # the oracle takes runs of consecutive slots of a block
            n = min(len(s) - i, block - int(s[i]) % page % block)
            prob.k.append(1, s[i:i + n], K8_values(k[qo[b] + i:qo[b] + i + n]))
            prob.v.append(1, s[i:i + n], K8_values(v[qo[b] + i:qo[b] + i + n]))
            i += n
    _same(cache, prob)
    assert int(ws.err.item()) == 0


# --------------------------------------------------------------- read-back ----
@pytest.mark.parametrize("dtype", ["e4m3", "int8"])
@pytest.mark.parametrize("page,block", PAGES)
@pytest.mark.parametrize("d,hkv", [(64, 1), (128, 3)])
@pytest.mark.parametrize("f32", [False, True])
def test_read(cuda, dtype, page, block, d, hkv, f32):
    lens = [0, 1, page, 3 * page + 1, 75]
    starts = [0, 0, 1, page, 75]
    prob = _problem(lens, dtype, page, block, heads=(hkv, hkv), d=d, layers=2)
    ws, cache = prob.device()
    rows = [n - s for n, s in zip(lens, starts)]
    dst = np.cumsum([3] + rows[:-1]).astype(np.int32) + 2 * np.arange(len(rows), dtype=np.int32)
    total = int(dst[-1] + rows[-1] + 4)
    dt = torch.float32 if f32 else torch.bfloat16
    k = torch.full((total, hkv, d), -7.0, dtype=dt, device="cuda")
    v = torch.full_like(k, -7.0)
    A.pkv_kv8_read(ws, cache, len(lens), 1, torch.tensor(starts, dtype=torch.int32).cuda(),
                   torch.from_numpy(dst).cuda(), total, k, v, A.PKV_FLAG_OUT_F32 if f32 else 0)
    torch.cuda.synchronize()
    for got, side in ((k, prob.k), (v, prob.v)):
        want = np.full((total, hkv, d), -7.0)  # rows that no token maps to stay
        for b in range(len(lens)):
            want[dst[b]:dst[b] + rows[b]] = side.rows(1, prob.slots(b, starts[b], lens[b]))
        assert np.array_equal(got.double().cpu().numpy(), want)
    assert int(ws.err.item()) == 0


def test_read_rounds_other_scales_once(cuda):
    # a calibrated scale need not be a power of two
    prob = _problem([20], "int8")
    prob.k.scales *= np.float32(0.7)
    ws, cache = prob.device()
    k = torch.zeros((20, 2, 128), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    A.pkv_kv8_read(ws, cache, 1, 0, None, torch.zeros(1, dtype=torch.int32).cuda(), 20, k, v)
    want = prob.k.rows(0, prob.slots(0, 0, 20))
    got = k.double().cpu().numpy()
    # code * scale to fp32, then to bf16
    assert np.all(np.abs(got - want) <= np.abs(want) * (BF16 + 2 * F32))


# --------------------------------------------------------------- attention ----
@pytest.mark.parametrize("dtype", ["e4m3", "int8"])
@pytest.mark.parametrize("heads", [(2, 2), (4, 2), (8, 2), (24, 3), (32, 2)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("S", [1, 3])
def test_attention_heads(cuda, dtype, heads, d, S):
    lens = [1, 17, 300, 0, 64, 129]
    prob = _problem(lens, dtype, heads=heads, d=d, outlier=0.02)
    ws, cache = prob.device(max_splits=S)
    q = W.normal_bf16((len(lens), heads[0], d), 11).cuda()
    _attend(prob, ws, cache, q, S, lens, what=f"{dtype} {heads} {d} {S}")


@pytest.mark.parametrize("dtype", ["e4m3", "int8"])
@pytest.mark.parametrize("page,block", PAGES)
@pytest.mark.parametrize("S", [1, 4])
def test_attention_pages(cuda, dtype, page, block, S):
    lens = [1, 15, 16, 33, page + 1, 500]
    prob = _problem(lens, dtype, page, block)
    ws, cache = prob.device(max_splits=S)
    q = W.normal_bf16((len(lens), 8, 128), 12).cuda()
    _attend(prob, ws, cache, q, S, lens, what=f"{page} {block} {S}")


@pytest.mark.parametrize("S", [1, 2, 7, 16])
def test_attention_splits_long(cuda, S):
    lens = [4097, 2000, 5]
    prob = _problem(lens, "e4m3", heads=(8, 2))
    ws, cache = prob.device(max_splits=S)
    q = W.normal_bf16((3, 8, 128), 13).cuda()
    _attend(prob, ws, cache, q, S, lens, A.PKV_FLAG_OUT_F32, what=f"S={S}")


@pytest.mark.parametrize("B", [33, 200, 257, 300, 1025])
def test_attention_batches(cuda, B):
    # past 32 and past 256 requests the split plan is made another way
    lens = [(37 * i) % 90 if i % 7 else 0 for i in range(B)]
    lens[-1] = 0
    prob = _problem(lens, "int8", heads=(2, 1), d=64)
    ws, cache = prob.device(max_splits=2)
    q = W.normal_bf16((B, 2, 64), 14).cuda()
    for S in (1, 2):
        _attend(prob, ws, cache, q, S, lens, what=f"B={B} S={S}")


@pytest.mark.parametrize("page", [16, 1])
@pytest.mark.parametrize("S", [2, 9])
def test_attention_large_batch(cuda, page, S):
    # one request far longer than the others, empty ones, bad ones among them
    B = 310
    lens = [(53 * i) % 70 for i in range(B)]
    lens[7], lens[200], lens[0] = 2500, 900, 0
    prob = _problem(lens, page=page, block=page, heads=(4, 2), d=64)
    ws, cache = prob.device(max_splits=S)
    q = W.normal_bf16((B, 4, 64), 15).cuda()
    _attend(prob, ws, cache, q, S, lens)
    bad = {3: -1, 150: prob.p.max_pages_per_req * page + 1, 309: -(2 ** 31)}
    for b, n in bad.items():
        ws.seq_lens[b], lens[b] = n, 0
    A.pkv_kv8_decode_layer(ws, cache, B, 0, q, None, None, prob.p.scale, S, A.PKV_FLAG_WRITE_LSE)
    torch.cuda.synchronize()
    assert int(ws.err.item()) == A.PKV_DEVERR_LEN and int(ws.split_counters.abs().sum()) == 0
    check_attention(ws.out_bf16(B).double().cpu().numpy(), ws.lse[:B].double().cpu().numpy(),
                    prob.attention(0, q.cpu(), lens), "the good requests", BF16)


@pytest.mark.parametrize("dtype", ["e4m3", "int8"])
def test_attention_scales_far_apart(cuda, dtype):
    # value blocks of very different sizes, zero blocks among them, and keys that
    # move the maximum from block to block
    lens = [200, 64]
    prob = _problem(lens, dtype, block=4)
    rng = np.random.default_rng(5)
    shape = prob.v.scales.shape
    prob.v.scales[...] = 2.0 ** rng.integers(-30, 31, shape)
    prob.v.codes[:, ::7] = 0
    prob.k.scales[...] = 2.0 ** rng.integers(-12, 0, shape)
    ws, cache = prob.device(max_splits=3)
    q = W.normal_bf16((2, 8, 128), 15).cuda()
    for S in (1, 3):
        _attend(prob, ws, cache, q, S, lens, A.PKV_FLAG_OUT_F32, what=f"S={S}")


@pytest.mark.parametrize("size", [2.0 ** -100, 2.0 ** -20, 2.0 ** 20, 2.0 ** 100])
def test_attention_query_sizes(cuda, size):
    # queries far outside the range of 16-bit floats, with a scale that undoes it
    lens = [100, 31]
    prob = _problem(lens)
    prob.p.scale = float(np.float32(prob.p.scale / size))
    ws, cache = prob.device(max_splits=2)
    q = (W.normal_bf16((2, 8, 128), 16).float() * size).bfloat16().cuda()
    _attend(prob, ws, cache, q, 2, lens, what=f"{size}")


def test_attention_ignores_what_no_token_holds(cuda):
    # NaN codes, and NaN and infinite scales, in every slot that no live token
    # uses, page tails included
    lens = [1, 18, 250, 0]
    prob = _problem(lens, "e4m3", block=1)
    used = np.zeros(prob.p.pool_slots, dtype=bool)
    for b, n in enumerate(lens):
        used[prob.slots(b, 0, n)] = True
    for side, bad in ((prob.k, np.nan), (prob.v, np.inf)):
        side.codes[:, ~used] = 0x7f
        free = ~used.reshape(-1, 16)
        side.scales.transpose(0, 1, 3, 2)[:, free] = bad
    ws, cache = prob.device(max_splits=3)
    q = W.normal_bf16((4, 8, 128), 17).cuda()
    for S in (1, 3):
        _attend(prob, ws, cache, q, S, lens, what=f"S={S}")


@pytest.mark.parametrize("n", [40, 600])
def test_attention_nan_reaches_its_own_request_only(cuda, n):
    lens = [n, n]  # 600: over two splits, of which one holds the NaN
    prob = _problem(lens)
    prob.k.codes[0, prob.slots(0, 7, 8)[0], 1, 3] = 0x7f
    ws, cache = prob.device(max_splits=2)
    q = W.normal_bf16((2, 8, 128), 18).cuda()
    A.pkv_kv8_decode_layer(ws, cache, 2, 0, q, None, None, prob.p.scale, 2)
    got = ws.out_bf16(2).double().cpu().numpy()
    assert np.isnan(got[0, 4:]).all()  # the heads of KV head 1
    assert np.isfinite(got[0, :4]).all()
    got[0, 4:] = 0
    o, _, bo, _ = prob.attention(0, q.cpu(), lens)
    o[0, 4:] = 0
    bo[0, 4:] = 0
    check_attention(got, None, (o, None, bo, None), "others", BF16)


def test_attention_queries_that_are_not_finite(cuda):
    # a head whose query holds NaN or an infinity is NaN, the others are as they
    # should be; a scale of zero averages the values
    lens = [70, 300]
    prob = _problem(lens)
    ws, cache = prob.device(max_splits=3)
    q = W.normal_bf16((2, 8, 128), 35)
    bad = q.clone()
    bad[0, 1, 5], bad[1, 6, 127] = float("nan"), float("inf")
    A.pkv_kv8_decode_layer(ws, cache, 2, 0, bad.cuda(), None, None, prob.p.scale, 3)
    torch.cuda.synchronize()
    got = ws.out_bf16(2).double().cpu().numpy()
    assert np.isnan(got[0, 1]).all() and np.isnan(got[1, 6]).all()
    o, _, bo, _ = prob.attention(0, q, lens)
    for x in (got, o, bo):
        x[0, 1] = x[1, 6] = 0
    check_attention(got, None, (o, None, bo, None), "finite heads", BF16)
    prob.p.scale = 0.0
    _attend(prob, ws, cache, q.cuda(), 3, lens, what="scale 0")


@pytest.mark.parametrize("seed", range(40))
def test_attention_random(cuda, seed):
    # shapes, lengths, pages and splits drawn together
    r = np.random.default_rng(900 + seed)
    hkv = int(r.choice([1, 2, 3, 5]))
    heads = (hkv * int(r.choice([1, 2, 4, 8, 16])), hkv)
    page, block = PAGES[r.integers(len(PAGES))] if seed % 4 else [(48, 3), (80, 16)][seed // 4 % 2]
    B = int(r.choice([1, 2, 5, 20, 40]))
    top = int(r.choice([3, 40, 300, 1500 if B <= 5 else 200]))
    lens = [int(x) for x in r.integers(0, top + 1, B)]
    S = int(r.choice([1, 2, 3, 9, 40]))
    d, dtype = int(r.choice([64, 128])), str(r.choice(["e4m3", "int8"]))
    prob = _problem(lens, dtype, page, block, heads=heads, d=d, seed=seed + 1)
    ws, cache = prob.device(max_splits=S, max_batch=B + 3)
    q = W.normal_bf16((B, heads[0], d), 500 + seed).cuda()
    flags = A.PKV_FLAG_OUT_F32 if seed % 3 == 0 else 0
    _attend(prob, ws, cache, q, S, lens, flags, what=f"{heads} {page} {block} {lens} S={S} {d}")


@pytest.mark.parametrize("batch", [1, 2])
def test_rows_behind_the_batch_are_left(cuda, batch):
    prob = _problem([30, 40, 50])
    ws, cache = prob.device(max_splits=2)
    q = W.normal_bf16((3, 8, 128), 19).cuda()
    ws.out.fill_(5.0)
    ws.lse.fill_(5.0)
    A.pkv_kv8_decode_layer(ws, cache, batch, 0, q, None, None, prob.p.scale, 2,
                           A.PKV_FLAG_OUT_F32 | A.PKV_FLAG_WRITE_LSE)
    torch.cuda.synchronize()
    assert torch.all(ws.out[batch:] == 5.0) and torch.all(ws.lse[batch:] == 5.0)
    assert not torch.any(ws.out[:batch] == 5.0)


# ------------------------------------------------------- the layer together ----
@pytest.mark.parametrize("dtype", ["e4m3", "int8"])
@pytest.mark.parametrize("page,block", PAGES)
def test_decode_steps(cuda, dtype, page, block):
    # bind, append and attend for several steps, across block and page ends;
    # one request starts empty
    lens, steps, layers = [0, 14, 15, 130], 5, 2
    prob = _problem(lens, dtype, page, block, layers=layers, steps=steps)
    ws, cache = prob.device(max_splits=3)
    B = len(lens)
    for step in range(steps):
        q, k, v = W.step_inputs(prob.p, step)
        k = _rows(tuple(k.shape), 100 + step, 1.0)
        A.pkv_bind_step(ws, B, A.PKV_BIND_STEADY)
        lens = [n + 1 for n in lens]
        for layer in range(layers):
            for b, n in enumerate(lens):
                prob.k.append(layer, prob.slots(b, n - 1, n), K8_values(k[layer, b:b + 1]))
                prob.v.append(layer, prob.slots(b, n - 1, n), K8_values(v[layer, b:b + 1]))
            _attend(prob, ws, cache, q[layer].cuda(), 3, lens, new=(k[layer].cuda(), v[layer].cuda()),
                    layer=layer, what=f"step {step}")
    _same(cache, prob)


def test_chunk_then_read_then_decode(cuda):
    before, new = [0, 21], [40, 9]
    lens = [a + b for a, b in zip(before, new)]
    prob = _problem(lens, "int8", steps=1)
    ws, cache = prob.device(max_splits=2)
    qo = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    k, v = _rows((49, 2, 128), 21), _rows((49, 2, 128), 22)
    A.pkv_kv8_extend_append(ws, cache, 2, 0, torch.from_numpy(qo).cuda(), 40, k.cuda(), v.cuda())
    for b in range(2):
        s = prob.slots(b, before[b], lens[b])
        i = 0
        while i < len(s):
            n = min(len(s) - i, 16 - int(s[i]) % 16)
            prob.k.append(0, s[i:i + n], K8_values(k[qo[b] + i:qo[b] + i + n]))
            prob.v.append(0, s[i:i + n], K8_values(v[qo[b] + i:qo[b] + i + n]))
            i += n
    rk = torch.zeros((sum(lens), 2, 128), dtype=torch.bfloat16, device="cuda")
    rv = torch.zeros_like(rk)
    A.pkv_kv8_read(ws, cache, 2, 0, None, ws.kv_indptr, sum(lens), rk, rv)
    want = np.concatenate([prob.k.rows(0, prob.slots(b, 0, n)) for b, n in enumerate(lens)])
    assert np.array_equal(rk.double().cpu().numpy(), want)
    q, k1, v1 = W.step_inputs(prob.p, 0)
    A.pkv_bind_step(ws, 2, A.PKV_BIND_STEADY)
    for b, n in enumerate(lens):
        prob.k.append(0, prob.slots(b, n, n + 1), K8_values(k1[0, b:b + 1]))
        prob.v.append(0, prob.slots(b, n, n + 1), K8_values(v1[0, b:b + 1]))
    _attend(prob, ws, cache, q[0].cuda(), 2, [n + 1 for n in lens],
            new=(k1[0].cuda(), v1[0].cuda()))
    _same(cache, prob)


@pytest.mark.parametrize("dtype,page,block", [("e4m3", 16, 16), ("int8", 1, 1), ("e4m3", 8, 4)])
@pytest.mark.parametrize("graph", [False, True])
def test_runner_steps(cuda, dtype, page, block, graph):
    # whole steps as a program runs them: bind, then per layer the norm with
    # rotation at the bind's positions, append and attention
    from paged_kv_decode_bind_gb300 import DecodeRunner, QkNormRope, rope_table
    lens, steps, layers, d = [3, 40, 129], 3, 2, 128
    prob = _problem(lens, dtype, page, block, layers=layers, steps=steps)
    ws, cache = prob.device(max_splits=3)
    table = rope_table(200, d)
    ropes = [QkNormRope(n_q_heads=8, n_kv_heads=2, head_dim=d, cos_sin=table,
                        q_weight=W.normal_bf16((d,), 50 + l).cuda(),
                        k_weight=W.normal_bf16((d,), 60 + l).cuda()) for l in range(layers)]
    run = DecodeRunner(ws, 3, num_splits=3, scale=prob.p.scale, cache=cache, norm_rope=ropes,
                       out_per_layer=True)
    assert run.launches_per_step == 1 + (page == 1) + 3 * layers
    if graph:
        run.capture()
    tab = table.double().cpu().numpy()
    for step in range(steps):
        q, k, v = W.step_inputs(prob.p, step)
        for dst, src in ((run.q_in, q), (run.k_in, k), (run.v_in, v)):
            dst.copy_(src)
        run.replay() if graph else run.step()
        torch.cuda.synchronize()
        lens = [n + 1 for n in lens]
        for l in range(layers):
            # the rotated rows as the kernel rounds them (its own tests bound them)
            qr = torch.zeros((3, 8, d), dtype=torch.bfloat16, device="cuda")
            kr = torch.zeros((3, 2, d), dtype=torch.bfloat16, device="cuda")
            A.pkv_qk_norm_rope(ropes[l], 3, run.q_in[l], run.k_in[l], ws.position_ids, qr, kr)
            for b in range(3):
                cos, sin = tab[lens[b] - 1, :d // 2], tab[lens[b] - 1, d // 2:]
                want = K8.norm_rope(K8_values(k[l, b]), K8_values(ropes[l].k_weight.cpu()), cos,
                                    sin, float(np.float32(1e-6)), False)
                assert np.abs(kr[b].double().cpu().numpy() - want).max() <= 2.0 ** -7 * \
                    np.abs(want).max()
                s = prob.slots(b, lens[b] - 1, lens[b])
                prob.k.append(l, s, K8_values(kr[b:b + 1].cpu()))
                prob.v.append(l, s, K8_values(v[l, b:b + 1]))
            check_attention(run.outs[l].double().cpu().numpy(), None,
                            prob.attention(l, qr.cpu(), lens), f"step {step} layer {l}", BF16)
    _same(cache, prob)
    assert int(ws.err.item()) == 0 and int(ropes[0].err.item()) == 0


@pytest.mark.parametrize("eight_bit", [True, False])
def test_runner_reports_positions_past_the_table(cuda, eight_bit):
    from paged_kv_decode_bind_gb300 import DecodeRunner, QkNormRope, Workspace, rope_table
    lens, steps = [20, 7], 3
    prob = _problem(lens, layers=2, steps=steps)
    if eight_bit:
        ws, cache = prob.device()
    else:
        ws, cache = Workspace.from_problem(prob.p), None
    rope = QkNormRope(n_q_heads=8, n_kv_heads=2, head_dim=128, cos_sin=rope_table(21, 128))
    run = DecodeRunner(ws, 2, scale=prob.p.scale, cache=cache, norm_rope=rope)
    run.step()
    assert int(ws.err.item()) == 0  # position 20, the last of the table
    run.step()
    assert int(ws.err.item()) == A.PKV_DEVERR_POSITION


@pytest.mark.parametrize("dtype,page,block,d", [("e4m3", 16, 16, 128), ("int8", 1, 1, 128),
                                                ("int8", 12, 4, 64)])
@pytest.mark.parametrize("S", [1, 3])
def test_extender(cuda, dtype, page, block, d, S):
    from paged_kv_decode_bind_gb300 import Kv8Extender
    before, new = [0, 130, 700], [90, 1, 33]
    lens = [a + b for a, b in zip(before, new)]
    prob = _problem(lens, dtype, page, block, d=d, layers=2)
    ws, cache = prob.device()
    ext = Kv8Extender(ws, cache, 3, max_new=96, max_context=740, scale=prob.p.scale, num_splits=S)
    T = sum(new)
    qo = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    for layer in range(2):
        q, k, v = W.normal_bf16((T, 8, d), 70), _rows((T, 2, d), 71), _rows((T, 2, d), 72)
        out = torch.zeros((T, 8, d), dtype=torch.float32, device="cuda")
        ext.layer(layer, torch.from_numpy(qo).cuda(), 90, q.cuda(), k.cuda(), v.cuda(), out,
                  A.PKV_FLAG_OUT_F32)
        torch.cuda.synchronize()
        got = out.double().cpu().numpy()
        for b in range(3):
            s = prob.slots(b, before[b], lens[b])
            i = 0
            while i < len(s):
                n = min(len(s) - i, block - int(s[i]) % page % block)
                prob.k.append(layer, s[i:i + n], K8_values(k[qo[b] + i:qo[b] + i + n]))
                prob.v.append(layer, s[i:i + n], K8_values(v[qo[b] + i:qo[b] + i + n]))
                i += n
            kk, vv = (x.rows(layer, prob.slots(b, 0, lens[b])) for x in (prob.k, prob.v))
            for t in range(new[b]):
                n = before[b] + t + 1
                o, _, _, _, _ = K8.attention(K8_values(q[qo[b] + t]), kk[:n], vv[:n], prob.p.scale)
                # the bound of the extend kernel's own tests, relative to the
                # values' size (P is applied as bf16 high and low parts)
                assert np.abs(got[qo[b] + t] - o).max() <= 1e-3 * np.abs(vv[:n]).max()
    _same(cache, prob)
    assert int(ws.err.item()) == 0


@pytest.mark.parametrize("full", [False, True])
@pytest.mark.parametrize("warp", [False, True])
@pytest.mark.parametrize("S", [1, 2])
def test_extender_passes_flags_on(cuda, full, warp, S):
    # PKV_FLAG_EXTEND_FULL: a chunk's first row sees its last one's token too
    from paged_kv_decode_bind_gb300 import Kv8Extender
    lens, new = [70, 33], [20, 33]
    prob = _problem(lens)
    ws, cache = prob.device()
    ext = Kv8Extender(ws, cache, 2, max_new=33, max_context=80, scale=prob.p.scale, num_splits=S)
    qo = torch.tensor([0, 20, 53], dtype=torch.int32).cuda()
    q, k, v = W.normal_bf16((53, 8, 128), 90), _rows((53, 2, 128), 91), _rows((53, 2, 128), 92)
    out = torch.zeros((53, 8, 128), dtype=torch.float32, device="cuda")
    ext.layer(0, qo, 33, q.cuda(), k.cuda(), v.cuda(), out, A.PKV_FLAG_OUT_F32 |
              A.PKV_FLAG_PLAN_EARLY | full * A.PKV_FLAG_EXTEND_FULL |
              warp * A.PKV_FLAG_EXTEND_WARP_MMA)
    torch.cuda.synchronize()
    got = out.double().cpu().numpy()
    kr, vr = (x[0].double().cpu().numpy() for x in (ext.k_rows, ext.v_rows))
    for b, n in enumerate(lens):
        at = int(ext.first_row[b])
        kk, vv = kr[at:at + n], vr[at:at + n]
        for t in range(new[b]):
            m = n if full else n - new[b] + t + 1
            o = K8.attention(K8_values(q[int(qo[b]) + t]), kk[:m], vv[:m], prob.p.scale)[0]
            assert np.abs(got[int(qo[b]) + t] - o).max() <= 1e-3 * np.abs(vv[:m]).max()
    assert int(ws.err.item()) == 0


def test_extender_refuses_longer_contexts(cuda):
    # a context past max_context: its request is skipped, its neighbour's rows
    # are its own
    from paged_kv_decode_bind_gb300 import Kv8Extender
    lens = [60, 30]
    prob = _problem(lens)
    ws, cache = prob.device()
    ext = Kv8Extender(ws, cache, 2, max_new=4, max_context=40, scale=prob.p.scale)
    q, k, v = W.normal_bf16((4, 8, 128), 80), _rows((4, 2, 128), 81), _rows((4, 2, 128), 82)
    out = torch.full((4, 8, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    qo = torch.tensor([0, 2, 4], dtype=torch.int32).cuda()
    ext.layer(0, qo, 2, q.cuda(), k.cuda(), v.cuda(), out)
    torch.cuda.synchronize()
    assert int(ws.err.item()) == A.PKV_DEVERR_LEN
    s = prob.slots(1, 28, 30)
    prob.k.append(0, s, K8_values(k[2:]))
    prob.v.append(0, s, K8_values(v[2:]))
    _same(cache, prob)
    assert torch.all(out[:2] == 5.0)
    kk, vv = (x.rows(0, prob.slots(1, 0, 30)) for x in (prob.k, prob.v))
    o, _, _, _, _ = K8.attention(K8_values(q[3]), kk, vv, prob.p.scale)
    got = out[3].double().cpu().numpy()
    assert np.abs(got - o).max() <= 1e-3 * np.abs(vv).max() + BF16 * np.abs(o).max()


def test_graph_replay_and_other_stream(cuda):
    lens = [33, 500]
    prob = _problem(lens, steps=4)
    ws, cache = prob.device(max_splits=4)
    q, k, v = (x[0].cuda() for x in W.step_inputs(prob.p, 0))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()

    def step(stream):
        A.pkv_bind_step(ws, 2, A.PKV_BIND_STEADY, stream=stream)
        A.pkv_kv8_decode_layer(ws, cache, 2, 0, q, k, v, prob.p.scale, 4, A.PKV_FLAG_WRITE_LSE,
                               stream=stream)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        step(torch.cuda.current_stream())
    for n in range(2):  # replayed, then eagerly on a stream of its own
        g.replay()
    torch.cuda.synchronize()
    step(side)
    torch.cuda.synchronize()
    for n in range(1, 4):
        for b in range(2):
            s = prob.slots(b, lens[b] + n - 1, lens[b] + n)
            prob.k.append(0, s, K8_values(k[b:b + 1].cpu()))
            prob.v.append(0, s, K8_values(v[b:b + 1].cpu()))
    _same(cache, prob)
    got = ws.out_bf16(2).double().cpu().numpy()
    check_attention(got, ws.lse[:2].double().cpu().numpy(),
                    prob.attention(0, q.cpu(), [n + 3 for n in lens]), "graph", BF16)
    assert int(ws.err.item()) == 0


# ------------------------------------------------------------ device errors ----
def _bad_page(ws, prob, b, col, value):
    ws.page_table[int(prob.p.req_pool_indices[b]), col] = value


@pytest.mark.parametrize("page", [16, 8])
@pytest.mark.parametrize("value", [-1, 1 << 30])
@pytest.mark.parametrize("S", [1, 3])
def test_attention_bad_page(cuda, page, value, S):
    lens = [200, 150]
    prob = _problem(lens, page=page, block=8)
    ws, cache = prob.device(max_splits=S)
    _bad_page(ws, prob, 0, 3, value)
    q = W.normal_bf16((2, 8, 128), 23).cuda()
    A.pkv_kv8_decode_layer(ws, cache, 2, 0, q, None, None, prob.p.scale, S, A.PKV_FLAG_WRITE_LSE)
    torch.cuda.synchronize()
    assert int(ws.err.item()) == A.PKV_DEVERR_PAGE
    assert int(ws.split_counters.abs().sum()) == 0
    got, lse = ws.out_bf16(2).double().cpu().numpy(), ws.lse[:2].double().cpu().numpy()
    assert np.isfinite(got).all()
    if S == 1:
        assert (got[0] == 0).all() and np.isneginf(lse[0]).all()
    ref = prob.attention(0, q.cpu(), lens)
    check_attention(got[1:], lse[1:], tuple(x[1:] for x in ref), "the other request", BF16)


@pytest.mark.parametrize("S", [1, 2])
def test_attention_bad_lengths_and_rows(cuda, S):
    prob = _problem([50, 60, 70, 80])
    ws, cache = prob.device(max_splits=S)
    ws.seq_lens[0] = -3
    ws.seq_lens[1] = prob.p.max_pages_per_req * 16 + 1
    ws.req_pool_indices[2] = prob.p.max_reqs
    q = W.normal_bf16((4, 8, 128), 24).cuda()
    A.pkv_kv8_decode_layer(ws, cache, 4, 0, q, None, None, prob.p.scale, S, A.PKV_FLAG_WRITE_LSE)
    torch.cuda.synchronize()
    assert int(ws.err.item()) == A.PKV_DEVERR_LEN | A.PKV_DEVERR_PAGE
    got, lse = ws.out_bf16(4).double().cpu().numpy(), ws.lse[:4].double().cpu().numpy()
    assert (got[:3] == 0).all() and np.isneginf(lse[:3]).all()
    ref = prob.attention(0, q.cpu(), [0, 0, 0, 80])
    check_attention(got, lse, ref, "the good request", BF16)


def test_flat_bad_slot_and_total(cuda):
    prob = _problem([30, 40, 50], page=1, block=1)
    ws, cache = prob.device(max_splits=2)
    ws.kv_indices[35] = prob.p.pool_slots  # token 5 of request 1
    ws.struct.max_total_tokens = 100       # request 2 ends at 120
    q = W.normal_bf16((3, 8, 128), 25).cuda()
    A.pkv_kv8_decode_layer(ws, cache, 3, 0, q, None, None, prob.p.scale, 1, A.PKV_FLAG_WRITE_LSE)
    torch.cuda.synchronize()
    assert int(ws.err.item()) == A.PKV_DEVERR_SLOT | A.PKV_DEVERR_TOTAL
    got, lse = ws.out_bf16(3).double().cpu().numpy(), ws.lse[:3].double().cpu().numpy()
    assert (got[1:] == 0).all() and np.isneginf(lse[1:]).all()
    ref = prob.attention(0, q.cpu(), [30, 0, 0])
    check_attention(got, lse, ref, "the good request", BF16)


@pytest.mark.parametrize("S", [1, 2])
def test_bounded_wait_runs_out(cuda, S):
    # the hook leaves every warp's first copy unissued: the waits run out (~1 s),
    # the outputs are empty, and the next launch is as it should be
    lens = [300, 40]
    prob = _problem(lens)
    ws, cache = prob.device(max_splits=S)
    q = W.normal_bf16((2, 8, 128), 33).cuda()
    A.pkv_kv8_decode_layer(ws, cache, 2, 0, q, None, None, prob.p.scale, S,
                           A.PKV_FLAG_TEST_SKIP_FIRST_TILE | A.PKV_FLAG_WRITE_LSE)
    torch.cuda.synchronize()
    assert int(ws.err.item()) == A.PKV_DEVERR_TIMEOUT
    assert torch.all(ws.out_bf16(2) == 0) and torch.all(torch.isneginf(ws.lse[:2]))
    assert int(ws.split_counters.abs().sum()) == 0
    ws.err.zero_()
    _attend(prob, ws, cache, q, S, lens, what="after a timeout")


@pytest.mark.parametrize("page", [16, 8])
def test_early_start(cuda, page):
    # layers after the first of a step may start before the previous ends: the
    # same results as without the flag, over several steps
    lens, layers = [700, 45, 0], 3
    prob = _problem(lens, page=page, block=8, layers=layers)
    ws, cache = prob.device(max_splits=4)
    q = W.normal_bf16((layers, 3, 8, 128), 34).cuda()
    for rep in range(3):
        for flag in (0, A.PKV_FLAG_PLAN_EARLY):
            outs = []
            A.pkv_bind_step(ws, 3, A.PKV_BIND_REBUILD)
            for layer in range(layers):
                A.pkv_kv8_decode_layer(ws, cache, 3, layer, q[layer], None, None, prob.p.scale, 4,
                                       A.PKV_FLAG_WRITE_LSE | (flag if layer else 0))
                outs.append((ws.out_bf16(3).clone(), ws.lse[:3].clone()))
            torch.cuda.synchronize()
            for layer, (o, l) in enumerate(outs):
                check_attention(o.double().cpu().numpy(), l.double().cpu().numpy(),
                                prob.attention(layer, q[layer].cpu(), lens), "early", BF16)
    assert int(ws.err.item()) == 0


@pytest.mark.parametrize("page,block", [(16, 16), (64, 64), (16, 2), (1, 1), (12, 4)])
def test_early_start_with_append(cuda, page, block):
    # every layer appends and starts early: the appended block (its older rows
    # rounded again) is the one that is attended, over many quick layers
    lens, layers, steps = [700, 47, 0, 15], 6, 4
    prob = _problem(lens, page=page, block=block, layers=layers, steps=steps)
    ws, cache = prob.device(max_splits=4)
    for step in range(steps):
        q, k, v = (x.cuda() for x in W.step_inputs(prob.p, step))
        k = k * (4.0 ** step)  # every step's rows make their block grow
        outs = []
        A.pkv_bind_step(ws, 4, A.PKV_BIND_STEADY)
        for layer in range(layers):
            A.pkv_kv8_decode_layer(ws, cache, 4, layer, q[layer], k[layer], v[layer],
                                   prob.p.scale, 4, A.PKV_FLAG_WRITE_LSE |
                                   (A.PKV_FLAG_PLAN_EARLY if layer else 0))
            outs.append((ws.out_bf16(4).clone(), ws.lse[:4].clone()))
        torch.cuda.synchronize()
        lens = [n + 1 for n in lens]
        for layer, (o, l) in enumerate(outs):
            for b, n in enumerate(lens):
                s = prob.slots(b, n - 1, n)
                prob.k.append(layer, s, K8_values(k[layer, b:b + 1].cpu()))
                prob.v.append(layer, s, K8_values(v[layer, b:b + 1].cpu()))
            check_attention(o.double().cpu().numpy(), l.double().cpu().numpy(),
                            prob.attention(layer, q[layer].cpu(), lens), "early", BF16)
    _same(cache, prob)
    assert int(ws.err.item()) == 0


@pytest.mark.parametrize("page,block", [(64, 16), (16, 16), (16, 2), (12, 4), (1, 1)])
def test_early_start_behind_a_long_layer(cuda, page, block):
    # a graph of layers in which request 0 keeps the previous layer running while
    # the next one's blocks already load the short requests' older blocks, whose
    # scales lie in the same sectors as the one that the append is about to change
    lens, layers, steps = [20000, 47, 30, 250], 3, 3
    p = W.make_problem(batch=4, n_layers=layers, n_q_heads=8, n_kv_heads=2, head_dim=128,
                       page_size=page, seq_lens=lens, steps=steps, seed=11, pool_factor=1.1)
    got = []
    for flag in (0, A.PKV_FLAG_PLAN_EARLY):
        from paged_kv_decode_bind_gb300 import Kv8Cache, Workspace
        ws = Workspace(n_layers=layers, pool_slots=p.pool_slots, n_q_heads=8, n_kv_heads=2,
                       head_dim=128, page_size=page, max_batch=4, max_reqs=p.max_reqs,
                       max_pages_per_req=p.max_pages_per_req, max_splits=64,
                       max_total_tokens=4 * p.max_pages_per_req if page == 1 else 0,
                       index_mode=p.index_mode, pools=False)
        ws.page_table.copy_(p.page_table)
        ws.req_pool_indices[:4].copy_(p.req_pool_indices)
        ws.seq_lens[:4].copy_(p.seq_lens)
        g = torch.Generator(device="cuda").manual_seed(3)
        shape = (layers, p.pool_slots, 2, 128)
        pool = lambda: torch.randint(0, 120, shape, generator=g, dtype=torch.uint8,  # noqa: E731
                                     device="cuda")
        cache = Kv8Cache(ws, scale_block=block, k_pool=pool(), v_pool=pool())
        cache.k_scale.fill_(2.0 ** -9), cache.v_scale.fill_(2.0 ** -9)
        q, k, v = (torch.zeros_like(x.cuda()) for x in W.step_inputs(p, 0))
        outs = [torch.zeros((4, 8, 128), dtype=torch.bfloat16, device="cuda")
                for _ in range(layers)]

        def step():
            A.pkv_bind_step(ws, 4, A.PKV_BIND_STEADY)
            for l in range(layers):
                view = A.PkvWorkspace.from_buffer_copy(ws.struct)
                view.out = outs[l].data_ptr()
                A.pkv_kv8_decode_layer(view, cache, 4, l, q[l], k[l], v[l], p.scale, 64,
                                       flag if l else 0)

        graph = torch.cuda.CUDAGraph()
        ws.seq_lens[:4] -= 1  # the call that loads the kernels appends nothing that stays
        keep = [t.clone() for t in (cache.k_pool, cache.v_pool, cache.k_scale, cache.v_scale)]
        step()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            step()
        for t, was in zip((cache.k_pool, cache.v_pool, cache.k_scale, cache.v_scale), keep):
            t.copy_(was)
        ws.seq_lens[:4].copy_(p.seq_lens)
        run = []
        for i in range(steps):
            for dst, src in zip((q, k, v), W.step_inputs(p, i)):
                dst.copy_(src)
            k.mul_(4.0 ** (i + 1))  # every step's rows make their block grow
            v.mul_(4.0 ** (i + 1))
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            run += [x.clone() for x in outs]
        run += [cache.k_pool, cache.v_pool, cache.k_scale, cache.v_scale]
        got.append(run)
        assert int(ws.err.item()) == 0
    for a, b in zip(*got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("S", [1, 3])
def test_padded_batch_raises_nothing(cuda, S):
    # empty requests beside others: no row, no error, zeros
    lens = [0, 39, 0, 130]
    prob = _problem(lens, layers=1, steps=1)
    ws, cache = prob.device(max_splits=S)
    q, k, v = W.step_inputs(prob.p, 0)
    for b in (1, 3):  # position lens - 1 again: the row of the newest token
        s = prob.slots(b, lens[b] - 1, lens[b])
        prob.k.append(0, s, K8_values(k[0, b:b + 1]))
        prob.v.append(0, s, K8_values(v[0, b:b + 1]))
    got = _attend(prob, ws, cache, q[0].cuda(), S, lens, new=(k[0].cuda(), v[0].cuda()))
    assert (got[[0, 2]] == 0).all()
    _same(cache, prob)
    # the append on its own has a row for every entry
    A.pkv_kv8_append(ws, cache, 4, 0, 1, k.cuda(), v.cuda())
    assert int(ws.err.item()) == A.PKV_DEVERR_SLOT


def test_rows_never_written_count_as_zeros(cuda):
    # a new cache under lengths that nothing wrote (a program's first, empty run)
    from paged_kv_decode_bind_gb300 import Kv8Cache
    prob = _problem([5, 70, 333])
    ws, _ = prob.device(max_splits=2)
    q, k, v = (x.cuda() for x in W.step_inputs(_problem([5, 70, 333], steps=1).p, 0))
    for dtype in ("e4m3", "int8"):
        cache = Kv8Cache(ws, dtype=dtype)
        A.pkv_kv8_decode_layer(ws, cache, 3, 0, q[0], None, None, 0.1, 2, A.PKV_FLAG_WRITE_LSE)
        assert torch.all(ws.out_bf16(3) == 0)
        n = torch.tensor([5.0, 70.0, 333.0], device="cuda").log()[:, None]
        assert (ws.lse[:3] - n).abs().max() <= 1e-4  # log n; its terms of 74 .. 80 are in steps of 2^-17
        # one row written: the others weigh in as zeros
        A.pkv_kv8_decode_layer(ws, cache, 3, 0, q[0], k[0], v[0], 0.1, 2)
        assert torch.all(torch.isfinite(ws.out_bf16(3))) and int(ws.err.item()) == 0


@pytest.mark.parametrize("page,block", [(16, 16), (64, 16), (1, 1), (12, 4)])
def test_read_starts_early(cuda, page, block):
    # a chunk's append and the read-back that starts while it runs, many times in
    # a graph: as call by call without the flag
    lens, new, times, most = [3000, 40, 0, 517], [64, 7, 0, 30], 6, 3100
    prob = _problem(lens, page=page, block=block)
    total = sum(new)
    qo = torch.tensor([0, 64, 71, 71, 101], dtype=torch.int32, device="cuda")
    rows = [(_rows((total, 2, 128), 70 + i) * 4.0 ** i).cuda() for i in range(times)]
    dst = torch.arange(4, dtype=torch.int32, device="cuda") * most
    got = []
    for flag in (0, A.PKV_FLAG_PLAN_EARLY):
        ws, cache = prob.device()
        outs = torch.zeros((times, 2, 4 * most, 2, 128), dtype=torch.bfloat16, device="cuda")

        def run():
            for i in range(times):
                A.pkv_kv8_extend_append(ws, cache, 4, 0, qo, 64, rows[i], rows[-1 - i])
                A.pkv_kv8_read(ws, cache, 4, 0, None, dst, 4 * most, outs[i, 0], outs[i, 1], flag)

        if flag:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                run()
            graph.replay()
        else:
            run()
        torch.cuda.synchronize()
        assert int(ws.err.item()) == 0
        got.append((outs, cache.k_pool, cache.k_scale, cache.v_scale))
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert got[0][0][-1, 0, :3000].any() and not got[0][0][:, :, 3000:most].any()


def test_read_of_no_rows(cuda):
    prob = _problem([0, 20])
    ws, cache = prob.device()
    dst = torch.zeros(2, dtype=torch.int32, device="cuda")
    A.pkv_kv8_read(ws, cache, 1, 0, None, dst, 0, None, None)
    assert int(ws.err.item()) == 0
    starts = torch.full((2,), 20, dtype=torch.int32, device="cuda")
    A.pkv_kv8_read(ws, cache, 2, 0, starts, dst, 0, None, None)
    assert int(ws.err.item()) == 0
    A.pkv_kv8_read(ws, cache, 2, 0, None, dst, 0, None, None)  # 20 rows, room for none
    assert int(ws.err.item()) == A.PKV_DEVERR_TOTAL


def test_append_bad_slot(cuda):
    prob = _problem([20, 30, 40])
    ws, cache = prob.device()
    ws.out_loc[0], ws.out_loc[2] = -1, prob.p.pool_slots
    k, v = _rows((1, 3, 2, 128), 26), _rows((1, 3, 2, 128), 27)
    A.pkv_kv8_append(ws, cache, 3, 0, 1, k.cuda(), v.cuda())
    prob.k.append(0, prob.slots(1, 29, 30), K8_values(k[0, 1:2]))
    prob.v.append(0, prob.slots(1, 29, 30), K8_values(v[0, 1:2]))
    _same(cache, prob)
    assert int(ws.err.item()) == A.PKV_DEVERR_SLOT


def test_chunk_bad_requests(cuda):
    lens, new = [20, 30, 40, 50], [4, 40, 5, 20]  # request 1: more new tokens than it has
    prob = _problem(lens)
    ws, cache = prob.device()
    _bad_page(ws, prob, 3, 2, -5)  # tokens 32 .. 47; new ones are 30 .. 49
    qo = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    k, v = _rows((69, 2, 128), 28), _rows((69, 2, 128), 29)
    A.pkv_kv8_extend_append(ws, cache, 4, 0, torch.from_numpy(qo).cuda(), 40, k.cuda(), v.cuda())
    for b, a, n, at in ((0, 16, 4, 0), (2, 35, 5, 44), (3, 30, 2, 49), (3, 48, 2, 67)):
        s = prob.slots(b, a, a + n)
        prob.k.append(0, s, K8_values(k[at:at + n]))
        prob.v.append(0, s, K8_values(v[at:at + n]))
    _same(cache, prob)
    assert int(ws.err.item()) == A.PKV_DEVERR_LEN | A.PKV_DEVERR_PAGE


def test_read_bad_requests(cuda):
    lens = [20, 30, 40, 17, 9]
    prob = _problem(lens)
    ws, cache = prob.device()
    _bad_page(ws, prob, 1, 1, 1 << 20)      # tokens 16 .. 29
    ws.req_pool_indices[3] = -1
    starts = torch.tensor([-1, 0, 0, 0, 3], dtype=torch.int32).cuda()
    dst = torch.tensor([0, 20, 62, 50, 67], dtype=torch.int32).cuda()  # request 2 past the end
    k = torch.full((80, 2, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    v = torch.full_like(k, 3.0)
    A.pkv_kv8_read(ws, cache, 5, 0, starts, dst, 80, k, v)
    torch.cuda.synchronize()
    want = np.full((80, 2, 128), 3.0)
    want[20:36] = prob.k.rows(0, prob.slots(1, 0, 16))
    want[36:50] = 0
    want[50:67] = 0
    want[67:73] = prob.k.rows(0, prob.slots(4, 3, 9))
    assert np.array_equal(k.double().cpu().numpy(), want)
    assert int(ws.err.item()) == A.PKV_DEVERR_LEN | A.PKV_DEVERR_TOTAL | A.PKV_DEVERR_PAGE


def test_read_many_requests(cuda):
    # more requests than are laid out at a time, most of them short
    lens = [(17 * i) % 41 for i in range(600)]
    prob = _problem(lens, "int8", heads=(1, 1), d=64)
    ws, cache = prob.device()
    n = sum(lens)
    k = torch.zeros((n, 1, 64), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    A.pkv_kv8_read(ws, cache, 600, 0, None, ws.kv_indptr, n, k, v)
    torch.cuda.synchronize()
    for got, side in ((k, prob.k), (v, prob.v)):
        want = np.concatenate([side.rows(0, prob.slots(b, 0, m)) for b, m in enumerate(lens)])
        assert np.array_equal(got.double().cpu().numpy(), want)
    assert int(ws.err.item()) == 0


def test_offsets_past_32_bits(cuda):
    # 3 layers of 2^21 slots x 8 heads x 128 bytes: layer 2 starts at 2^32 bytes
    from paged_kv_decode_bind_gb300 import Kv8Cache, Workspace
    slots = 1 << 21
    ws = Workspace(n_layers=3, pool_slots=slots, n_q_heads=8, n_kv_heads=8, head_dim=128,
                   page_size=16, max_batch=1, max_reqs=1, max_pages_per_req=2, pools=False)
    cache = Kv8Cache(ws, dtype="int8", scale_block=16)
    ws.page_table[0] = torch.tensor([slots // 16 - 1, slots // 16 - 2], dtype=torch.int32)
    ws.seq_lens[0] = 19
    A.pkv_bind_step(ws, 1, A.PKV_BIND_REBUILD)
    k, v = _rows((19, 8, 128), 30, 0.1), _rows((19, 8, 128), 31, 0.1)
    qo = torch.tensor([0, 19], dtype=torch.int32).cuda()
    A.pkv_kv8_extend_append(ws, cache, 1, 2, qo, 19, k.cuda(), v.cuda())
    rk = torch.zeros((19, 8, 128), dtype=torch.bfloat16, device="cuda")
    rv = torch.zeros_like(rk)
    A.pkv_kv8_read(ws, cache, 1, 2, None, ws.kv_indptr, 19, rk, rv)
    q = W.normal_bf16((1, 8, 128), 32)
    A.pkv_kv8_decode_layer(ws, cache, 1, 2, q.cuda(), None, None, 0.1, 1, A.PKV_FLAG_OUT_F32)
    torch.cuda.synchronize()
    # every written element is within half an int8 step of its block's scale
    for x, y in ((k, rk), (v, rv)):
        x, y = x.double().numpy(), y.double().cpu().numpy()
        for a, e in ((0, 16), (16, 19)):
            amax = np.abs(x[a:e]).max(axis=(0, 2), keepdims=True)
            s = np.vectorize(lambda m: K8.need(m, "int8"))(amax)
            assert np.all(np.abs(x[a:e] - y[a:e]) <= s / 2)
    o, _, mass, _, _ = K8.attention(K8_values(q)[0], rk.double().cpu().numpy(),
                                 rv.double().cpu().numpy(), float(np.float32(0.1)))
    got = ws.out_f32(1).double().cpu().numpy()[0]
    assert np.all(np.abs(got - o) <= 2.0 ** -10 * mass + 1e-6)
    # nothing outside the two pages of layer 2
    lo = int(torch.count_nonzero(cache.k_pool[:2])) + int(torch.count_nonzero(
        cache.k_pool[2, :slots - 32]))
    assert lo == 0 and int(ws.err.item()) == 0


def _rising_scores(lens, hq, tail, zero):
    """Requests whose scores lie 5.5 (7.9 in powers of two, just under what moves the
    reference) above those of their first 128 tokens, value scales `zero` (codes 0
    there) but for ordinary values in the last block where `tail`.  One KV head,
    D = 64, int8."""
    prob = _problem(lens, "int8", heads=(hq, 1), d=64)
    prob.k.codes[...] = 0
    prob.k.scales[...] = 1.0
    tail_codes, tail_scales = prob.v.codes.copy(), prob.v.scales.copy()
    prob.v.codes[...] = 0
    prob.v.scales[...] = zero
    for b, n in enumerate(lens):
        s = prob.slots(b, 0, n)
        prob.k.codes[0, s[128:], 0, 0] = 127
        if tail:
            last = s[(n - 1) // 16 * 16:]
            prob.v.codes[0, last] = tail_codes[0, last]
            prob.v.scales[0, last[0] // 16] = tail_scales[0, last[0] // 16]
    q = torch.zeros((len(lens), hq, 64), dtype=torch.bfloat16)
    q[:, :, 0] = 5.5 / 127 / prob.p.scale
    return prob, q


def _far(scale):
    """What lse may be off besides Problem.attention's bound where the value scales lie far
    from 1.  The reference r is as large as far = 8 + |log2 scale| + 8 (place, scale,
    scores): the subtraction x - r rounds by half a step of that, and so do both terms of
    lse = r ln 2 + log(sum): ln 2 itself and the product (1.5 half steps), the logarithm
    (2 half steps)."""
    return 5 * F32 * (16 + abs(np.log2(max(scale, 2.0 ** -80)))) * np.log(2)


@pytest.mark.parametrize("n,hq", [(20000, 2), (20000, 16), (150000, 2)])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("S", [1, 2, 5])
def test_attention_long_runs_of_zero_values(cuda, n, hq, tail, S):
    # rows of zeros carry the smallest scale: the sum of their weights stays finite
    # within a warp (150000: over 9000 tokens each), a unit and a merge
    prob, q = _rising_scores([n, 40], hq, tail, 2.0 ** -100)
    ws, cache = prob.device(max_splits=S)
    A.pkv_kv8_decode_layer(ws, cache, 2, 0, q.cuda(), None, None, prob.p.scale, S,
                           A.PKV_FLAG_WRITE_LSE | A.PKV_FLAG_OUT_F32)
    torch.cuda.synchronize()
    got = ws.out_f32(2).double().cpu().numpy()
    o, l, bo, bl = prob.attention(0, q, [n, 40])
    check_attention(got, ws.lse[:2].double().cpu().numpy(), (o, l, bo, bl + _far(2.0 ** -100)),
                    f"{n} S={S}", F32)
    assert got.any() == tail and int(ws.err.item()) == 0


@pytest.mark.parametrize("zero", [2.0 ** -100, 2.0 ** -81, 2.0 ** -80, 2.0 ** -60, 2.0 ** 100])
@pytest.mark.parametrize("S", [1, 3])
def test_attention_values_at_the_scale_limits(cuda, zero, S):
    # ordinary codes under the smallest and largest scales
    lens = [3000, 50]
    prob, q = _rising_scores(lens, 2, False, zero)
    g = np.random.default_rng(8)
    prob.v.codes[...] = g.integers(0, 256, prob.v.codes.shape)
    prob.v.codes[prob.v.codes == 128] = 127  # -128 is no code
    ws, cache = prob.device(max_splits=S)
    A.pkv_kv8_decode_layer(ws, cache, 2, 0, q.cuda(), None, None, prob.p.scale, S,
                           A.PKV_FLAG_WRITE_LSE | A.PKV_FLAG_OUT_F32)
    torch.cuda.synchronize()
    o, l, bo, bl = prob.attention(0, q, lens)
    bl += _far(zero)
    if zero < 2.0 ** -80:
        # the reference counts these scales as 2^-80, so a warp's largest weight is at
        # least 2^8 zero / 2^-80, and a weight below fp16's normal range is cut off at
        # 2^-24: over all tokens 2^-24 / (2^88 zero) of the largest p_t v_scale_t, times
        # sum_t |code_t| (2 %: the query is rounded, the scores rise by 5.5 / 2^8 more)
        codes = [np.abs(prob.v.rows(0, prob.slots(b, 0, n)) / zero).sum(0) for b, n in
                 enumerate(lens)]
        for b, n in enumerate(lens):
            x = np.where(np.arange(n) < 128, 0, 5.5)
            top = zero / np.exp(x - x.max()).sum()  # the largest p_t v_scale_t
            bo[b] += 2.0 ** -24 / (2.0 ** 88 * zero) * 1.02 * top * codes[b]
    check_attention(ws.out_f32(2).double().cpu().numpy() / zero,
                    ws.lse[:2].double().cpu().numpy(), (o / zero, l, bo / zero, bl),
                    f"{zero} S={S}", F32)
    assert int(ws.err.item()) == 0


@pytest.mark.parametrize("dtype", ["e4m3", "int8"])
@pytest.mark.parametrize("chunk", [False, True])
@pytest.mark.parametrize("page,block", [(16, 16), (48, 24)])
def test_append_to_blocks_of_other_scales(cuda, dtype, chunk, page, block):
    # a calibrated cache is appended to: kept scales that are no powers of two, and rows
    # whose quotients are ties between two codes, or so near to one that the quotient's
    # own rounding to fp32 makes it one; then rows that make such blocks grow
    ties = {"e4m3": [17.0, 8.5, 19.0, 25.0, 304.0, 2.125], "int8": [0.5, 2.5, 7.5, 12.5, 99.5, 126.5]}[dtype]
    r = np.random.default_rng(12)
    B, H, new = 24, 2, 3 if chunk else 1
    before = [int(x) for x in r.integers(1, block - new + 1, B)]
    lens = [n + new for n in before]
    prob = _problem(lens, dtype, page, block, heads=(H, H))
    k, v = torch.zeros((B * new, H, 128)), torch.zeros((B * new, H, 128))
    for side, x in ((prob.k, k), (prob.v, v)):
        for b in range(B):
            s = prob.slots(b, 0, block)
            pg = s[0] // page
            for h in range(H):
                t = ties[r.integers(len(ties))]
                if b % 3 == 0:  # exact ties: x = t * 240, t * 224
                    scale, x0 = [(240.0, 240 * t), (224.0, 224 * t)][b // 3 % 2]
                    if (torch.tensor(x0).bfloat16().double() != x0).any():
                        x0 = scale * ties[1]
                else:
                    x0 = float(torch.tensor(r.uniform(1, 2) * 2.0 ** r.integers(-40, 40)).bfloat16())
                    scale = np.float32(x0 / t)
                rows = x0 * 2.0 ** -r.integers(0, 8, (new, 128)).astype(np.float64)
                if b % 3 == 2:  # grows to `top`: older codes of 101 or 208 land at a tie
                    top = 2.0 ** np.floor(np.log2(x0))
                    c, t = (101, 12.5) if dtype == "int8" else (0x75, 17.0)
                    scale = np.float32(t * top / K8.TABLE[dtype][c])
                    side.codes[0, s, h, ::2] = c
                    rows[0, 0] = x0
                    rows *= 0.75 * K8.QMAX[dtype] * top / x0
                side.scales[0, pg, h, s[0] % page // block] = scale
                x[b * new:(b + 1) * new, h] = torch.from_numpy(
                    rows * r.choice([-1, 1], (new, 128))).float()
    k, v = k.bfloat16(), v.bfloat16()
    ws, cache = prob.device()
    if chunk:
        qo = torch.arange(0, B * new + 1, new, dtype=torch.int32).cuda()
        A.pkv_kv8_extend_append(ws, cache, B, 0, qo, new, k.cuda(), v.cuda())
    else:
        A.pkv_kv8_append(ws, cache, B, 0, 1, k.cuda(), v.cuda())
    kept = grown = 0
    for b in range(B):
        s = prob.slots(b, before[b], lens[b])
        for side, x in ((prob.k, k), (prob.v, v)):
            at = (0, s[0] // page, slice(None), s[0] % page // block)
            was = side.scales[at].copy()
            side.append(0, s, K8_values(x[b * new:(b + 1) * new]))
            kept += int((side.scales[at] == was).sum())
            grown += int((side.scales[at] > was).sum())
    assert kept >= B and grown >= B // 2
    _same(cache, prob)
    assert int(ws.err.item()) == 0


@pytest.mark.parametrize("dtype", ["e4m3", "int8"])
@pytest.mark.parametrize("hkv,d", [(33, 128), (40, 128), (65, 64)])
@pytest.mark.parametrize("f32", [False, True])
def test_read_wide_rows(cuda, dtype, hkv, d, f32):
    # rows of more than 256 words of 16 codes: a thread takes several columns
    lens = [19, 5]
    prob = _problem(lens, dtype, heads=(hkv, hkv), d=d)
    ws, cache = prob.device()
    dt = torch.float32 if f32 else torch.bfloat16
    k = torch.full((24, hkv, d), -7.0, dtype=dt, device="cuda")
    v = torch.full_like(k, -7.0)
    A.pkv_kv8_read(ws, cache, 2, 0, None, ws.kv_indptr, 24, k, v, A.PKV_FLAG_OUT_F32 if f32 else 0)
    torch.cuda.synchronize()
    for got, side in ((k, prob.k), (v, prob.v)):
        want = np.concatenate([side.rows(0, prob.slots(b, 0, n)) for b, n in enumerate(lens)])
        assert np.array_equal(got.double().cpu().numpy(), want)
    assert int(ws.err.item()) == 0


@pytest.mark.parametrize("lens", [[20000], [20000, 300, 7], [9000] * 6])
@pytest.mark.parametrize("page", [16, 1])
@pytest.mark.parametrize("S", [2, 3, 4, 8])
def test_splits_share_a_request_out(cuda, lens, page, S):
    # with a query of zeros a partial's log-sum-exp is the logarithm of its tokens: few
    # splits cut the longest request into about S equal parts, not S - 1
    prob = _problem(lens, page=page, block=page, heads=(4, 2), d=64)
    ws, cache = prob.device(max_splits=S)
    B = len(lens)
    ws.ml_part.zero_()
    q = torch.zeros((B, 4, 64), dtype=torch.bfloat16, device="cuda")
    A.pkv_kv8_decode_layer(ws, cache, B, 0, q, None, None, prob.p.scale, S, A.PKV_FLAG_WRITE_LSE)
    torch.cuda.synchronize()
    n = ws.ml_part[:B].double().cpu().numpy()
    n = np.where(n[..., 1] > 0, np.exp(n[..., 0]), 0)  # [B, Hq, S]
    whole = np.exp(ws.lse[:B].double().cpu().numpy())
    assert np.abs(whole - np.array(lens)[:, None]).max() <= 0.1
    # (a request in one piece has no partials)
    assert np.all((np.abs(n.sum(-1) - whole) <= 0.1) | (n.sum(-1) == 0)) and n[0].all(0).any()
    assert n[0].max() <= lens[0] / S + 16 * 20  # rounding to pages, a start's share
    _attend(prob, ws, cache, W.normal_bf16((B, 4, 64), 77).cuda(), S, lens, what=f"{lens} {S}")


@pytest.mark.parametrize("form", ["fused", "unfused", "planned"])
@pytest.mark.parametrize("page", [16, 1])
@pytest.mark.parametrize("S", [1, 3])
@pytest.mark.parametrize("graph", [False, True])
def test_runner_norm_rope_on_the_bf16_cache(cuda, form, page, S, graph):
    # whole steps with the norm and rotation in front of the bf16 cache's layers, which
    # (fused) may start while the kernel before them runs
    from paged_kv_decode_bind_gb300 import DecodeRunner, QkNormRope, Workspace, rope_table
    lens, steps, layers, d = [3, 40, 700, 0], 3, 3, 128
    B = len(lens)
    p = W.make_problem(batch=B, n_layers=layers, n_q_heads=8, n_kv_heads=2, head_dim=d,
                       page_size=page, seq_lens=lens, steps=steps, seed=21)
    ws = Workspace.from_problem(p, max_splits=S)
    table = rope_table(800, d)
    ropes = [QkNormRope(n_q_heads=8, n_kv_heads=2, head_dim=d, cos_sin=table,
                        q_weight=W.normal_bf16((d,), 50 + l).cuda(),
                        k_weight=W.normal_bf16((d,), 60 + l).cuda()) for l in range(layers)]
    run = DecodeRunner(ws, B, num_splits=S, scale=p.scale, norm_rope=ropes, out_per_layer=True,
                       flags=A.PKV_FLAG_OUT_F32, fused=form != "unfused", plan=form == "planned")
    if graph:
        run.capture()
    pools = {n: x.clone() for n, x in (("k", p.k_pool), ("v", p.v_pool))}
    for step in range(steps):
        q, k, v = W.step_inputs(p, step)
        for dst, src in ((run.q_in, q), (run.k_in, k), (run.v_in, v)):
            dst.copy_(src)
        run.replay() if graph else run.step()
        torch.cuda.synchronize()
        lens = [n + 1 for n in lens]
        for l in range(layers):
            # the rotated rows as the kernel rounds them (its own tests bound them)
            qr = torch.zeros((B, 8, d), dtype=torch.bfloat16, device="cuda")
            kr = torch.zeros((B, 2, d), dtype=torch.bfloat16, device="cuda")
            A.pkv_qk_norm_rope(ropes[l], B, run.q_in[l], run.k_in[l], ws.position_ids, qr, kr)
            torch.cuda.synchronize()
            got = run.outs[l].double().cpu().numpy()
            for b, n in enumerate(lens):
                row = p.page_table[int(p.req_pool_indices[b])].long()
                t = torch.arange(n)
                s = row[t // page] * page + t % page
                pools["k"][l, s[-1]], pools["v"][l, s[-1]] = kr[b].cpu(), v[l, b]
                kk, vv = (K8_values(pools[x][l, s]) for x in "kv")
                o, _, mass, size, _ = K8.attention(K8_values(qr[b].cpu()), kk, vv, p.scale)
                # scores as in Problem.attention; weights as bf16 high and low parts, 2^-17
                dw = 2.0 ** -17 + 2 * (d + 8) * F32 * size + 2.0 ** -20
                tol = 2 * dw[:, None] * mass + F32 * np.abs(o)
                assert (np.abs(got[b] - o) - tol).max() <= 0
    for name, pool in (("k", ws.k_pool), ("v", ws.v_pool)):
        assert torch.equal(pool.cpu(), pools[name])
    assert int(ws.err.item()) == 0 and ws.seq_lens[:B].tolist() == lens


@pytest.mark.parametrize("sign", [1, -1])
def test_attention_scores_at_their_limit(cuda, sign):
    # scores near 2^26 (in powers of two), a few tokens tied at the top of each request
    # whose value scales lie far apart: their average.  (One split: several are weighed
    # by log-sum-exps that fp32 holds in steps of 4 here.)
    lens = [900, 70]
    prob = _problem(lens, "int8", heads=(2, 1), d=64)
    prob.k.codes[...] = 0
    prob.k.scales[...] = 2.0 ** 21
    prob.v.scales[...] = 2.0 ** np.random.default_rng(6).integers(-30, 31, prob.v.scales.shape)
    for b, n in enumerate(lens):
        s = prob.slots(b, 0, n)
        prob.k.codes[0, s, 0, 0] = 0x81  # -127
        prob.k.codes[0, s[[3, n // 2, n - 2]], 0, 0] = 127 if sign > 0 else 0x82  # -126
    prob.p.scale = 0.125
    q = torch.zeros((2, 2, 64), dtype=torch.bfloat16)
    q[:, :, 0] = 1.0
    ws, cache = prob.device()
    A.pkv_kv8_decode_layer(ws, cache, 2, 0, q.cuda(), None, None, prob.p.scale, 1,
                           A.PKV_FLAG_OUT_F32)
    torch.cuda.synchronize()
    got = ws.out_f32(2).double().cpu().numpy()
    for b, n in enumerate(lens):
        s = prob.slots(b, 0, n)
        o, _, mass, _, floor = K8.attention(K8_values(q)[b], prob.k.rows(0, s), prob.v.rows(0, s),
                                            prob.p.scale, prob.v.scale_of(0, s))
        # equal scores are equal in fp32 too, so the weights are off by their two fp16
        # parts alone; r is in steps of 4, so the largest weight is at least 2^4 and the
        # smallest step 2^-24 at most 2^-28 of it
        tol = 2 * 2.0 ** -20 * mass + 2.0 ** -28 * floor + 4 * F32 * np.abs(o)
        assert (np.abs(got[b] - o) - tol).max() <= 0
    assert int(ws.err.item()) == 0


@pytest.mark.parametrize("dtype", ["e4m3", "int8"])
@pytest.mark.parametrize("heads", [(2, 2), (4, 2), (8, 2), (16, 2), (32, 2)])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 16), (128, 1), (64, 8)])
def test_attention_weights_keep_their_low_parts(cuda, dtype, heads, d, page):
    # fp32 outputs: a weight is a high and a low fp16 part, each cut off after 11 bits
    # (2^-20 of it in all), of a smallest step 2^-24 where the largest is at least 2^8
    lens = [700, 33, 5]
    prob = _problem(lens, dtype, page, page, heads=heads, d=d, outlier=0.01)
    prob.v.scales[...] *= 2.0 ** np.random.default_rng(3).integers(-3, 4, prob.v.scales.shape)
    ws, cache = prob.device(max_splits=3)
    q = W.normal_bf16((3, heads[0], d), 88)
    for S in (1, 3):
        A.pkv_kv8_decode_layer(ws, cache, 3, 0, q.cuda(), None, None, prob.p.scale, S,
                               A.PKV_FLAG_OUT_F32)
        torch.cuda.synchronize()
        got = ws.out_f32(3).double().cpu().numpy()
        for b, n in enumerate(lens):
            s = prob.slots(b, 0, n)
            o, _, mass, size, floor = K8.attention(
                K8_values(q)[b], prob.k.rows(0, s), prob.v.rows(0, s), prob.p.scale,
                prob.v.scale_of(0, s))
            # scores and exponentials as in Problem.attention; the sums of n products in
            # fp32 (n / 16 of them in a row, then the warps')
            dw = 2.0 ** -20 + 2 * (d + 8) * F32 * size + 2.0 ** -20 + (n / 16 + 16) * F32
            tol = 2 * dw[:, None] * mass + 2.0 ** -32 * floor + F32 * np.abs(o)
            assert (np.abs(got[b] - o) - tol).max() <= 0
    assert int(ws.err.item()) == 0


@pytest.mark.parametrize("page,block", [(16, 16), (1, 1)])
def test_extender_captured_on_another_stream(cuda, page, block):
    # one chunk captured on a stream of its own and replayed with other rows: as call by call
    from paged_kv_decode_bind_gb300 import Kv8Extender
    lens, qo = [70, 45], torch.tensor([0, 20, 53], dtype=torch.int32).cuda()
    rows = [[x.cuda() for x in (W.normal_bf16((53, 8, 128), 90 + i), _rows((53, 2, 128), 93 + i),
                                _rows((53, 2, 128), 96 + i))] for i in range(2)]
    got = []
    for graph in (False, True):
        prob = _problem(lens, page=page, block=block)
        ws, cache = prob.device()
        ext = Kv8Extender(ws, cache, 2, max_new=33, max_context=80, scale=prob.p.scale)
        q, k, v = (x.clone() for x in rows[0])
        out = torch.zeros((53, 8, 128), dtype=torch.bfloat16, device="cuda")
        torch.cuda.synchronize()
        outs = []
        if graph:
            side = torch.cuda.Stream()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                ext.layer(0, qo, 33, q, k, v, out)
        for i in range(2):
            for dst, src in zip((q, k, v), rows[i]):
                dst.copy_(src)
            g.replay() if graph else ext.layer(0, qo, 33, q, k, v, out)
            torch.cuda.synchronize()
            outs.append(out.clone())
        got.append(outs + [cache.k_pool, cache.v_pool, cache.k_scale, cache.v_scale])
        assert int(ws.err.item()) == 0 and outs[0].any() and not torch.equal(*outs)
    for a, b in zip(*got):
        assert torch.equal(a, b)
