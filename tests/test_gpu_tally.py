"""The tally of attention weight and the eviction on the GPU against the 64-bit oracle.

Weights are held to tally_problem.weight_bound (derived from the roundings they pass).
An eviction moves bits: pools, weights, origins and lengths are compared exactly, with the
oracle's ranks taken from the weights that the device holds."""
import numpy as np
import pytest
import torch

import oracle.kv8 as K8
import oracle.ref as R
import oracle.tally as T
import tally_problem as P
from paged_kv_decode_bind_gb300 import (DecodeRunner, Eviction, QkNormRopeAxes, Tally,
                                        TallyExtender, Workspace, rope_table)
from paged_kv_decode_bind_gb300 import _abi as A

pytestmark = pytest.mark.gpu

HEADS = [(2, 2), (4, 2), (8, 2), (16, 2), (16, 1), (12, 3)]
LENS = [0, 1, 15, 16, 17, 63, 64, 65, 129, 700]


def _bf16(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).bfloat16()


# ------------------------------------------------------------------ decode ----
def _decode_reference(p, ws, tally, layer, q, lens, appended):
    """Expected (weight, origin) by slot and the bound, from the device's state before."""
    w0, o0 = P.by_slot(tally.weight).astype(np.float64), P.by_slot(tally.origin).copy()
    bound = np.zeros_like(w0)
    pool, qf = P.f64(ws.k_pool[layer]), P.f64(q)
    ev = tally.evicted.cpu().numpy()
    for b, n in enumerate(lens):
        if n == 0:
            continue
        s = P.slots(p, b, n)
        k = pool[s]
        lse = T.log_sum_exp(qf[b:b + 1], k, p.scale, [n - 1])
        w, err = T.weights(qf[b:b + 1], k, lse, p.scale, [n - 1])
        size = np.abs(lse).max()
        if appended:
            w0[layer, s[-1]] = 0
            o0[layer, s[-1]] = n - 1 + ev[int(p.req_pool_indices[b])]
        w0[layer, s] += w
        # the device's lse is its own: its error is a score's, at the largest
        worst = (2 * p.head_dim + 16) * P.EPS32 * (
            np.abs(k[:, :, None]) * np.abs(qf[b].reshape(k.shape[1], -1, p.head_dim))[None]
        ).sum(-1).max() * p.scale + 2.0 ** -20 + 8 * P.EPS32 * size
        bound[layer, s] = P.weight_bound(w, err, qf.shape[1] // k.shape[1], size, p.head_dim,
                                         worst)
    return w0, o0, bound + 2 * P.EPS32 * w0


def _check_tally(tally, ref, what=""):
    w, o, bound = ref
    got = P.by_slot(tally.weight).astype(np.float64)
    assert np.array_equal(P.by_slot(tally.origin), o), what
    err = np.abs(got - w) - bound
    assert err.max() <= 0, f"{what}: {err.max():.3e} past the bound"
    assert np.array_equal(got[bound == 2 * P.EPS32 * w], w[bound == 2 * P.EPS32 * w]), what


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 5, 1])
@pytest.mark.parametrize("splits", [1, 5])
def test_decode(cuda, heads, d, page, splits):
    p = P.problem(LENS, page=page, heads=heads, d=d, layers=2, steps=1)
    ws, tally = P.device(p, max_splits=splits)
    # the same layer without the tally, on a workspace of its own
    ws2, _ = P.device(p, max_splits=splits)
    B, q = p.batch, _bf16((p.batch, heads[0], d), 1, 2.0).cuda()
    k, v = (_bf16((p.batch, heads[1], d), s).cuda() for s in (2, 3))
    A.pkv_decode_layer(ws2, B, 1, q, k, v, p.scale, splits, A.PKV_FLAG_WRITE_LSE)
    # the oracle's view: the pools behind the append, the tally in front of it
    ws.k_pool.copy_(ws2.k_pool)
    ref = _decode_reference(p, ws, tally, 1, q, LENS, True)
    ws.k_pool.copy_(p.k_pool)
    A.pkv_tally_decode_layer(ws, tally, B, 1, q, k, v, p.scale, splits)
    torch.cuda.synchronize()
    _check_tally(tally, ref)
    for name in ("k_pool", "v_pool", "lse"):
        assert torch.equal(getattr(ws, name), getattr(ws2, name)), name
    assert torch.equal(ws.out_bf16(B), ws2.out_bf16(B))
    assert int(ws.err.item()) == 0 and int(ws.split_counters.abs().sum()) == 0


@pytest.mark.parametrize("page", [32, 8, 1, 48])
def test_decode_without_append_adds(cuda, page):
    p = P.problem([1, 130, 33], page=page, heads=(8, 4))
    ws, tally = P.device(p, max_splits=2)
    q = _bf16((3, 8, 128), 5).cuda()
    ref = _decode_reference(p, ws, tally, 0, q, [1, 130, 33], False)
    A.pkv_tally_decode_layer(ws, tally, 3, 0, q, None, None, p.scale, 2,
                             A.PKV_FLAG_OUT_F32 | A.PKV_FLAG_FORCE_GATHER)
    torch.cuda.synchronize()
    _check_tally(tally, ref)
    # every head's weights sum to one
    s = P.slots(p, 1, 130)
    ref2 = P.by_slot(tally.weight).astype(np.float64)[0, s].sum(0)
    A.pkv_tally_decode_layer(ws, tally, 3, 0, q, None, None, p.scale, 2)
    torch.cuda.synchronize()
    grown = P.by_slot(tally.weight).astype(np.float64)[0, s].sum(0) - ref2
    assert np.allclose(grown, 2, atol=1e-4)


@pytest.mark.parametrize("batch", [33, 300])
def test_decode_many_requests(cuda, batch):
    lens = [(7 * b) % 90 for b in range(batch)]
    p = P.problem(lens, heads=(4, 2), d=64)
    ws, tally = P.device(p, max_splits=3)
    q = _bf16((batch, 4, 64), 5).cuda()
    ref = _decode_reference(p, ws, tally, 0, q, lens, False)
    A.pkv_tally_decode_layer(ws, tally, batch, 0, q, None, None, p.scale, 3)
    torch.cuda.synchronize()
    _check_tally(tally, ref)


def test_decode_values_that_are_not_finite(cuda):
    """A NaN key empties its split; the other splits' tokens weigh as if it were not
    there.  NaN rows behind the last token and in the tally change nothing else."""
    lens = [512, 40]
    p = P.problem(lens, heads=(4, 2), d=64)
    ws, tally = P.device(p, max_splits=4)
    s0, s1 = P.slots(p, 0, 512), P.slots(p, 1, 48)
    q = _bf16((2, 4, 64), 5).cuda()
    ws.k_pool[0, s1[40:]] = float("nan")
    ws.v_pool[0, s1[40:]] = float("nan")
    ws.k_pool[0, s0[500], 1] = float("nan")  # KV head 1, the last of four splits
    before = P.by_slot(tally.weight).astype(np.float64)
    A.pkv_tally_decode_layer(ws, tally, 2, 0, q, None, None, p.scale, 4, A.PKV_FLAG_FIXED_CHUNK)
    torch.cuda.synchronize()
    grown = P.by_slot(tally.weight).astype(np.float64)[0] - before[0]
    assert np.isfinite(grown).all()
    assert np.allclose(grown[s0, 0].sum(), 2, atol=1e-4)
    assert np.allclose(grown[s1[:40]].sum(0), 2, atol=1e-4)
    assert np.all(grown[s1[40:]] == 0)
    # KV head 1: tokens of the last split gain nothing, the others sum to one a head
    assert np.all(grown[s0[384:], 1] == 0)
    assert np.allclose(grown[s0[:384], 1].sum(), 2, atol=1e-4)


def test_decode_bad_page_weighs_nothing(cuda):
    p = P.problem([200, 64], heads=(4, 2), d=64)
    ws, tally = P.device(p, max_splits=2)
    row = int(p.req_pool_indices[0])
    ws.page_table[row, 3] = 10 ** 6
    before = P.by_slot(tally.weight).astype(np.float64)
    A.pkv_tally_decode_layer(ws, tally, 2, 0, _bf16((2, 4, 64), 5).cuda(), None, None, p.scale, 1)
    torch.cuda.synchronize()
    assert int(ws.err.item()) == A.PKV_DEVERR_PAGE
    grown = P.by_slot(tally.weight).astype(np.float64)[0] - before[0]
    s1 = P.slots(p, 1, 64)
    assert np.allclose(grown[s1].sum(0), 2, atol=1e-4)
    grown[s1] = 0
    assert np.all(grown == 0)


def test_decode_bounded_wait_weighs_nothing(cuda):
    p = P.problem([200], heads=(4, 2), d=64)
    ws, tally = P.device(p)
    before = tally.weight.clone()
    A.pkv_tally_decode_layer(ws, tally, 1, 0, _bf16((1, 4, 64), 5).cuda(), None, None, p.scale, 1,
                             A.PKV_FLAG_TEST_SKIP_FIRST_TILE)
    torch.cuda.synchronize()
    assert int(ws.err.item()) == A.PKV_DEVERR_TIMEOUT
    assert torch.equal(tally.weight, before)


# ------------------------------------------------------------------ extend ----
def _extend_reference(p, ws, tally, layer, q, lse, lens, new, window, skip=()):
    w0, o0 = P.by_slot(tally.weight).astype(np.float64), P.by_slot(tally.origin).copy()
    bound = np.zeros_like(w0)
    pool, qf, l = P.f64(ws.k_pool[layer]), P.f64(q), lse.double().cpu().numpy()
    ev = tally.evicted.cpu().numpy()
    at = 0
    for b, (L, n) in enumerate(zip(lens, new)):
        if n and b not in skip:
            s = P.slots(p, b, L)
            i0 = max(0, n - window)
            pos = np.arange(L - n + i0, L)
            w, err = T.weights(qf[at + i0:at + n], pool[s], l[at + i0:at + n], p.scale, pos)
            w0[layer, s[L - n:]] = 0
            o0[layer, s[L - n:]] = (np.arange(L - n, L) + ev[int(p.req_pool_indices[b])])[:, None]
            w0[layer, s] += w
            fin = l[at + i0:at + n][np.isfinite(l[at + i0:at + n])]
            bound[layer, s] = P.weight_bound(
                w, err, (n - i0) * qf.shape[1] // pool.shape[1],
                np.abs(fin).max() if fin.size else 0, p.head_dim)
        at += n
    return w0, o0, bound + 2 * P.EPS32 * w0


def _extend(p, lens, new, *, window=10 ** 6, layer=0, scale_q=1.5, lse=None, spoil=None, splits=1):
    """Run pkv_tally_extend with the oracle's lse; (tally, reference, workspace)."""
    ws, tally = P.device(p)
    T_ = sum(new)
    q = _bf16((max(1, T_), p.n_q_heads, p.head_dim), 11, scale_q)
    if lse is None:
        rows, at = [], 0
        pool, qf = P.f64(ws.k_pool[layer]), P.f64(q)
        for b, (L, n) in enumerate(zip(lens, new)):
            rows.append(T.log_sum_exp(qf[at:at + n], pool[P.slots(p, b, L)], p.scale,
                                      list(range(L - n, L))))
            at += n
        lse = torch.from_numpy(np.concatenate(rows)).float()
    if spoil:
        spoil(ws, q, lse)
    qo = torch.tensor([sum(new[:b]) for b in range(len(new) + 1)], dtype=torch.int32).cuda()
    ref = _extend_reference(p, ws, tally, layer, q, lse, lens, new, window)
    q, lse = q.cuda(), lse.cuda().contiguous()
    A.pkv_tally_extend(ws, tally, len(new), layer, qo, max(new), T_, window, q, lse, p.scale)
    torch.cuda.synchronize()
    return ws, tally, ref, (qo, q, lse)


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 5, 1])
def test_extend(cuda, heads, d, page):
    lens = [1, 128, 129, 300, 0, 77, 5, 256]
    new = [1, 128, 1, 45, 0, 77, 0, 33]
    p = P.problem(lens, page=page, heads=heads, d=d, layers=2)
    ws, tally, ref, _ = _extend(p, lens, new, layer=1)
    _check_tally(tally, ref)
    assert int(ws.err.item()) == 0


def test_extend_one_row(cuda):
    """One new token: fewer rows than a query tile, on a context of one, of a tile's edge."""
    for L in (1, 128, 129, 257):
        p = P.problem([L], heads=(2, 2), d=64)
        ws, tally, ref, _ = _extend(p, [L], [1])
        _check_tally(tally, ref)


@pytest.mark.parametrize("window", [1, 7, 64, 130])
@pytest.mark.parametrize("heads", [(2, 2), (8, 2), (16, 1)])
def test_extend_window(cuda, window, heads):
    lens, new = [400, 131, 64], [200, 131, 1]
    p = P.problem(lens, heads=heads, d=64)
    ws, tally, ref, _ = _extend(p, lens, new, window=window)
    _check_tally(tally, ref)


@pytest.mark.parametrize("window", [40, 100, 150])  # one query tile, two, three
@pytest.mark.parametrize("d,page", [(128, 16), (64, 5)])
def test_extend_more_units_than_ctas(cuda, window, d, page):
    """Every CTA takes several units, whose key and query tiles follow one another through
    the same shared memory."""
    lens, new = [2600, 2500, 900, 2300, 130], [150, 149, 150, 20, 130]
    p = P.problem(lens, page=page, heads=(32, 8), d=d)
    ws, tally, ref, _ = _extend(p, lens, new, window=window)
    assert int(ws.err.item()) == 0
    _check_tally(tally, ref)


def test_extend_sums_to_the_observed_queries(cuda):
    """A whole prompt: every observed query's weights sum to one a head, whatever the
    tiles; a long context of several key tiles and query tiles a unit."""
    lens, new = [1500], [700]
    p = P.problem(lens, heads=(8, 2))
    ws, tally, ref, again = _extend(p, lens, new, window=500)
    _check_tally(tally, ref)
    first = tally.weight.clone()
    ws2, tally2, _, _ = _extend(p, lens, new, window=500)
    assert torch.equal(first, tally2.weight)  # the order of the sums is fixed


def test_extend_masked_and_not_finite_values(cuda):
    lens, new = [200, 140], [70, 30]

    def spoil(ws, q, lse):
        s0, s1 = P.slots(p, 0, 208), P.slots(p, 1, 144)
        ws.k_pool[0, s0[200:]] = float("nan")   # behind the last token
        ws.k_pool[0, s1[140:]] = float("inf")
        ws.k_pool[0, s0[199], 0] = float("nan")  # masked for all queries but the last
        ws.k_pool[0, s1[3], 1] = float("nan")    # a token that every query sees
        ws.k_pool[0, s1[5], 0] = float("inf")
        q[10, 2] = float("nan")                  # one query of one head
        lse[20] = -float("inf")
        lse[21] = float("nan")
        lse[22] = float("inf")

    p = P.problem(lens, heads=(4, 2), d=64)
    ws, tally, ref, _ = _extend(p, lens, new, spoil=spoil)
    _check_tally(tally, ref)
    assert torch.isfinite(tally.weight).all()


def test_extend_negative_and_zero_scale(cuda):
    for scale in (-0.3, 0.0):
        lens, new = [150], [40]
        p = P.problem(lens, heads=(4, 2), d=64)
        p.scale = scale
        ws, tally, ref, _ = _extend(p, lens, new)
        _check_tally(tally, ref)


def test_extend_many_requests(cuda):
    """More requests than one launch takes."""
    n = 1100
    lens = [1 + (5 * b) % 40 for b in range(n)]
    new = [1 + (3 * b) % L for b, L in enumerate(lens)]
    p = P.problem(lens, page=8, heads=(2, 1), d=64)
    ws, tally, ref, _ = _extend(p, lens, new)
    _check_tally(tally, ref)


def test_extend_device_errors_leave_the_rest(cuda):
    """A bad length, a table row out of range and too few rows skip their request; a bad
    page keeps the entries of its 128-token tile."""
    lens, new = [300, 40, 60, 20, 50], [30, 10, 20, 20, 50]
    p = P.problem(lens, heads=(4, 2), d=64)
    for case in ("len", "row", "page", "rows"):
        ws, tally = P.device(p)
        q = _bf16((sum(new), 4, 64), 11)
        lse = torch.zeros(sum(new), 4) + 3
        n_rows, err, skip = sum(new), A.PKV_DEVERR_LEN, (1,)
        if case == "len":
            ws.seq_lens[1] = 5  # fewer tokens than new ones
        elif case == "row":
            ws.req_pool_indices[1] = 10 ** 6
            err = A.PKV_DEVERR_PAGE
        elif case == "page":
            ws.page_table[int(p.req_pool_indices[0]), 9] = -1  # token 144: tile 1 of request 0
            err, skip = A.PKV_DEVERR_PAGE, ()
        else:
            n_rows, skip = sum(new) - 1, (4,)
        ref = _extend_reference(p, ws, tally, 0, q, lse, lens, new, 100, skip)
        if case == "page":
            s = P.slots(p, 0, 256)[128:]
            old = P.by_slot(tally.weight).astype(np.float64)
            ref[0][0, s], ref[1][0, s] = old[0, s], P.by_slot(tally.origin)[0, s]
        qo = torch.tensor([sum(new[:b]) for b in range(6)], dtype=torch.int32).cuda()
        A.pkv_tally_extend(ws, tally, 5, 0, qo, max(new), n_rows, 100, q.cuda(), lse.cuda(),
                           p.scale)
        torch.cuda.synchronize()
        assert int(ws.err.item()) == err, case
        _check_tally(tally, ref, case)


@pytest.mark.parametrize("page,flags", [(16, 0), (16, A.PKV_FLAG_EXTEND_WARP_MMA), (1, 0)])
@pytest.mark.parametrize("splits", [1, 3])
def test_extender(cuda, page, flags, splits):
    """Append, attention and tally: outputs as pkv_extend_attn gives them, weights within
    the bound of the oracle's, with the device's own log-sum-exps."""
    lens, new = [300, 90, 8], [100, 90, 1]
    p = P.problem(lens, page=page, heads=(8, 2))
    ws, tally = P.device(p)
    N = sum(new)
    q, k, v = _bf16((N, 8, 128), 11), _bf16((N, 2, 128), 12), _bf16((N, 2, 128), 13)
    qo = torch.tensor([0, 100, 190, 191], dtype=torch.int32).cuda()
    ext = TallyExtender(ws, tally, 3, max_new=100, scale=p.scale, window=64, num_splits=splits)
    out = torch.zeros((N, 8, 128), dtype=torch.bfloat16, device="cuda")
    before = (tally.weight.clone(), tally.origin.clone())
    ext.layer(0, qo, 100, q.cuda(), k.cuda(), v.cuda(), out, flags)
    torch.cuda.synchronize()
    now = (tally.weight.clone(), tally.origin.clone())
    tally.weight.copy_(before[0])
    tally.origin.copy_(before[1])
    w, o, bound = _extend_reference(p, ws, tally, 0, q, ext.lse[:N], lens, new, 64)
    tally.weight.copy_(now[0])
    tally.origin.copy_(now[1])
    _check_tally(tally, (w, o, bound))
    slots = [P.slots(p, b, n) for b, n in enumerate(lens)]
    got = out.double().cpu().numpy()
    ref = R.extend_attention(R.tensor_bits(q), R.tensor_bits(ws.k_pool.cpu()),
                             R.tensor_bits(ws.v_pool.cpu()), 0, slots, new, p.scale, 2)
    ref = ref[0] if isinstance(ref, tuple) else ref
    assert np.abs(got - np.asarray(ref).reshape(got.shape)).max() <= 1e-2
    assert int(ws.err.item()) == 0


def test_extend_weights_past_fp32(cuda):
    """A log-sum-exp far below its scores gives weights past fp32: they add nothing, the
    other queries' weights of the same tokens count."""
    lens, new = [200, 140], [70, 30]

    def spoil(ws, q, lse):
        lse[5, 1] = -1000.0  # past 64 bits too
        lse[40] = -300.0     # e^300: past fp32 alone
        lse[90, 0] = -700.0

    p = P.problem(lens, heads=(4, 2), d=64)
    ws, tally, ref, _ = _extend(p, lens, new, spoil=spoil)
    _check_tally(tally, ref)
    assert torch.isfinite(tally.weight).all()


@pytest.mark.parametrize("window", [10 ** 6, 20])
def test_extend_a_key_that_is_not_finite_changes_no_other(cuda, window):
    """NaN and infinite keys weigh nothing, and every other token's weight keeps its bits."""
    lens, new = [300, 140], [70, 30]
    p = P.problem(lens, heads=(8, 2), d=64)
    _, clean, _, (_, _, lse) = _extend(p, lens, new, window=window)
    s0, s1 = P.slots(p, 0, 300), P.slots(p, 1, 140)

    def spoil(ws, q, lse):
        ws.k_pool[0, s0[3], 0] = float("nan")
        ws.k_pool[0, s0[250], 1] = float("inf")  # a new token, masked for some queries
        ws.k_pool[0, s1[70], 1] = float("nan")

    _, tally, ref, _ = _extend(p, lens, new, window=window, lse=lse.cpu(), spoil=spoil)
    _check_tally(tally, ref)
    a, b = (P.by_slot(x.weight).view(np.int32)[0].copy() for x in (clean, tally))
    for slot, h in ((s0[3], 0), (s0[250], 1), (s1[70], 1)):
        a[slot, h] = b[slot, h] = 0
    assert np.array_equal(a, b)


@pytest.mark.parametrize("window", [500, 40])
def test_extend_every_query_weighs_one(cuda, window):
    """From a tally of zeros each KV head holds the group's heads times the observed
    queries, within the sum of its tokens' bounds and of fp32's lse."""
    lens, new = [1500, 129], [700, 60]
    p = P.problem(lens, heads=(8, 2))
    ws, tally, ref, (qo, q, lse) = _extend(p, lens, new, window=window)
    tally.weight.zero_()
    A.pkv_tally_extend(ws, tally, 2, 0, qo, 700, sum(new), window, q, lse, p.scale)
    torch.cuda.synchronize()
    got = P.by_slot(tally.weight).astype(np.float64)[0]
    for b, (L, n) in enumerate(zip(lens, new)):
        s = P.slots(p, b, L)
        count = 4 * min(n, window)
        off = ref[2][0, s].sum(0) + 2 * P.EPS32 * float(lse.abs().max()) * count
        assert np.all(np.abs(got[s].sum(0) - count) <= off)


# ------------------------------------------------------------------- evict ----
def _evict_reference(p, ws, tally, lens, budget, limit, sinks, recent, skip=()):
    state = {n: P.by_slot(getattr(tally, n)).copy() for n in ("weight", "origin")}
    state.update({n: getattr(ws, n).view(torch.int16).cpu().numpy().copy()
                  for n in ("k_pool", "v_pool")})
    ev, out = tally.evicted.cpu().numpy().copy(), list(lens)
    for b, n in enumerate(lens):
        if n <= limit or b in skip:
            continue
        row = int(p.req_pool_indices[b])
        s = P.slots(p, b, n)
        for layer in range(p.n_layers):
            for h in range(p.n_kv_heads):
                kept = T.keep(state["weight"][layer, s, h], state["origin"][layer, s, h],
                              n + int(ev[row]), budget, sinks, recent)
                pairs = T.moves(kept, budget)
                if pairs:
                    frm, to = (s[list(x)] for x in zip(*pairs))
                    for x in state.values():
                        x[layer, to, h] = x[layer, frm, h]
        ev[row] += n - budget
        out[b] = budget
    return state, ev, out


def _check_evict(p, ws, tally, ref):
    state, ev, lens = ref
    torch.cuda.synchronize()
    assert ws.seq_lens[:p.batch].tolist() == lens
    assert np.array_equal(tally.evicted.cpu().numpy(), ev)
    for n in ("weight", "origin"):
        got = P.by_slot(getattr(tally, n))
        assert np.array_equal(got.view(np.int32), state[n].view(np.int32)), n
    for n in ("k_pool", "v_pool"):
        assert np.array_equal(getattr(ws, n).view(torch.int16).cpu().numpy(), state[n]), n
    assert int(ws.split_counters.abs().sum()) == 0


def _set_tally(p, ws, tally, kind, seed=5):
    g = torch.Generator().manual_seed(seed)
    shape = tally.weight.shape
    if kind == "random":
        w = torch.exp(1.5 * torch.randn(shape, generator=g))
    elif kind == "ties":  # few values, both zeros
        w = torch.randint(0, 4, shape, generator=g).float() * 0.5
        w = torch.where((w == 0) & (torch.rand(shape, generator=g) < 0.5), -w, w)
    elif kind == "equal":
        w = torch.full(shape, 0.25)
    else:  # not finite, negative, tiny
        pick = torch.randint(0, 7, shape, generator=g)
        vals = torch.tensor([float("nan"), float("inf"), -float("inf"), -1.0, 0.0, 1e-42, 2.0])
        w = vals[pick]
    tally.weight.copy_(w)
    # origins: the index, moved by what was evicted behind the first ones
    ev = tally.evicted.cpu().numpy()
    o = P.by_slot(tally.origin)
    for b, n in enumerate(p.seq_lens.tolist()):
        e = ev[int(p.req_pool_indices[b])]
        t = np.arange(n)
        o[:, P.slots(p, b, n)] = np.where(t < 3, t, t + e)[None, :, None]
    NL, pages, H, Pg = shape
    tally.origin.copy_(torch.from_numpy(
        np.ascontiguousarray(o.reshape(NL, pages, Pg, H).transpose(0, 1, 3, 2))))


@pytest.mark.parametrize("kind", ["random", "ties", "equal", "odd"])
@pytest.mark.parametrize("page,d,heads", [(16, 128, (8, 2)), (5, 64, (3, 3)), (1, 128, (4, 1)),
                                          (64, 64, (4, 4))])
@pytest.mark.parametrize("budget,limit,sinks,recent", [(100, 100, 4, 32), (100, 150, 0, 0),
                                                       (1, 1, 0, 0), (64, 64, 32, 32)])
def test_evict(cuda, kind, page, d, heads, budget, limit, sinks, recent):
    lens = [0, 1, 64, 100, 101, 150, 151, 700, 333]
    p = P.problem(lens, page=page, heads=heads, d=d, layers=2)
    ws, tally = P.device(p)
    _set_tally(p, ws, tally, kind)
    ref = _evict_reference(p, ws, tally, lens, budget, limit, sinks, recent)
    A.pkv_tally_evict(ws, tally, p.batch, 700, limit, budget, sinks, recent)
    _check_evict(p, ws, tally, ref)
    assert int(ws.err.item()) == 0


@pytest.mark.parametrize("kind", ["random", "ties", "equal", "odd"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("budget,sinks,recent", [(1, 0, 0), (1, 1, 0), (100, 4, 32), (100, 100, 0),
                                                 (100, 0, 100), (3000, 4, 100)])
def test_evict_one_token(cuda, kind, d, budget, sinks, recent):
    """A request one token over: the token that ranks last goes, whatever the others do."""
    lens = [budget + 1, budget, budget + 2, budget + 1, 0]
    p = P.problem(lens, page=16 if d == 64 else 5, heads=(6, 3), d=d, layers=2)
    ws, tally = P.device(p)
    _set_tally(p, ws, tally, kind)
    ref = _evict_reference(p, ws, tally, lens, budget, budget, sinks, recent)
    A.pkv_tally_evict(ws, tally, p.batch, budget + 2, budget, budget, sinks, recent)
    _check_evict(p, ws, tally, ref)
    assert int(ws.err.item()) == 0


def test_evict_one_token_bad_page(cuda):
    p = P.problem([51, 51], heads=(4, 2), d=64, layers=2)
    ws, tally = P.device(p)
    _set_tally(p, ws, tally, "random")
    ws.page_table[int(p.req_pool_indices[1]), 2] = -4
    ref = _evict_reference(p, ws, tally, [51, 51], 50, 50, 2, 10, (1,))
    A.pkv_tally_evict(ws, tally, 2, 51, 50, 50, 2, 10)
    _check_evict(p, ws, tally, ref)
    assert int(ws.err.item()) == A.PKV_DEVERR_PAGE


@pytest.mark.parametrize("kind", ["random", "ties"])
@pytest.mark.parametrize("lens,max_len,budget", [
    ([5000, 2049], 5000, 1025),      # clusters for idle SMs
    ([20000], 20000, 3001),          # segments past one CTA's
    ([3000, 17], 393216, 2900),      # a bound far past the lengths (the table's row counts)
    ([70000], 70000, 69999),         # one token out
    ([66000, 65], 66000, 64)])
def test_evict_long(cuda, kind, lens, max_len, budget):
    p = P.problem(lens, heads=(2, 1), d=64)
    ws, tally = P.device(p)
    _set_tally(p, ws, tally, kind)
    ref = _evict_reference(p, ws, tally, lens, budget, budget, 4, min(50, budget - 4))
    A.pkv_tally_evict(ws, tally, p.batch, max_len, budget, budget, 4, min(50, budget - 4))
    _check_evict(p, ws, tally, ref)


def test_evict_largest_segments(cuda):
    """A bound that gives a cluster's CTAs their largest segments."""
    n = A.PKV_TALLY_MAX_LEN
    p = P.problem([n], heads=(1, 1), d=64, page=64)
    ws, tally = P.device(p)
    _set_tally(p, ws, tally, "random")
    ref = _evict_reference(p, ws, tally, [n], 200000, 200000, 4, 1000)
    A.pkv_tally_evict(ws, tally, 1, n, 200000, 200000, 4, 1000)
    _check_evict(p, ws, tally, ref)


def test_evict_rows_far_into_a_pool(cuda):
    """Row offsets past 2^31 bytes and 2^32 elements of the pools."""
    H, D, slots = 8, 128, 2 ** 22 + 4096  # 2^32 elements and more a pool
    ws = Workspace(n_layers=1, pool_slots=slots, n_q_heads=8, n_kv_heads=H, head_dim=D,
                   page_size=16, max_batch=1, max_reqs=1, max_pages_per_req=20)
    tally = Tally(ws)
    last = slots // 16
    ws.page_table.copy_(torch.arange(last - 20, last, dtype=torch.int32).flip(0)[None])
    ws.seq_lens.fill_(300)
    near = torch.arange(slots - 320, slots, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn((320, H, D), generator=g, device="cuda").bfloat16()
    ws.k_pool[0, near], ws.v_pool[0, near] = x, -x
    tally.weight[:, last - 20:] = torch.rand((1, 20, H, 16), generator=g, device="cuda")
    w = tally.weight.clone()
    A.pkv_tally_evict(ws, tally, 1, 300, 40, 40, 0, 0)
    torch.cuda.synchronize()
    t = np.arange(300)
    slot = (last - 1 - t // 16) * 16 + t % 16
    wt = P.by_slot(w[:, last - 20:])[0, slot - (slots - 320)]
    got_k, got_v = ws.k_pool[0, near], ws.v_pool[0, near]
    for h in range(H):
        kept = T.keep(wt[:, h], np.zeros(300) + 5, 300, 40, 0, 0)
        where = np.arange(300)
        for a, b in T.moves(kept, 40):
            where[b] = a
        src = torch.from_numpy(slot[where] - (slots - 320)).cuda()
        dst = torch.from_numpy(slot - (slots - 320)).cuda()
        assert torch.equal(got_k[dst, h], x[src, h]) and torch.equal(got_v[dst, h], -x[src, h])


def test_evict_device_errors_leave_the_request(cuda):
    lens = [300, 200, 250, 260]
    for case in ("page", "row", "len", "bound"):
        p = P.problem(lens, heads=(4, 2), d=64, layers=2)
        ws, tally = P.device(p)
        _set_tally(p, ws, tally, "random")
        err, max_len = A.PKV_DEVERR_PAGE, 300
        if case == "page":
            ws.page_table[int(p.req_pool_indices[1]), 11] = 10 ** 6
        elif case == "row":
            ws.req_pool_indices[1] = -1
        elif case == "len":
            ws.seq_lens[1] = -7
            err = A.PKV_DEVERR_LEN
        else:
            max_len, err = 260, A.PKV_DEVERR_LEN
        skip = (0,) if case == "bound" else (1,)
        ref = _evict_reference(p, ws, tally, lens, 50, 50, 2, 10, skip)
        if case == "len":
            ref[2][1] = -7
        A.pkv_tally_evict(ws, tally, 4, max_len, 50, 50, 2, 10)
        _check_evict(p, ws, tally, ref)
        assert int(ws.err.item()) == err, case


# ------------------------------------------------------------ in one step ----
def _axes_rope(ws, tally, Hq, H, D, span=600):
    delta = torch.zeros(ws.shape["max_reqs"], dtype=torch.int32, device="cuda")
    for b, r in enumerate(ws.req_pool_indices.tolist()):
        delta[r] = -3 * b
    return QkNormRopeAxes(n_q_heads=Hq, n_kv_heads=H, head_dim=D, cos_sin=rope_table(span, D),
                          q_weight=_bf16((D,), 41).cuda(), k_weight=_bf16((D,), 42).cuda(),
                          sections=(D // 8, 3 * D // 16, 3 * D // 16), rows=ws.req_pool_indices,
                          evicted=tally.evicted, delta=delta)


@pytest.mark.parametrize("page", [16, 1])
def test_prompt_evictions_and_steps(cuda, page):
    """A prompt, its eviction, and decode steps that evict, with the norm and a rotation
    by three axes in front: every stage against the oracle, from the device's state in
    front of that stage."""
    NL, Hq, H, D, B = 2, 8, 2, 64, 3
    lens, new = [150, 40, 97], [150, 40, 97]
    p = P.problem(lens, page=page, heads=(Hq, H), d=D, layers=NL, steps=12)
    ws, tally = P.device(p, max_splits=3)
    tally.take_rows(ws.req_pool_indices)
    N = sum(new)
    qo = torch.tensor([0, 150, 190, 287], dtype=torch.int32).cuda()
    ext = TallyExtender(ws, tally, B, max_new=150, scale=p.scale, window=32)
    out = torch.zeros((N, Hq, D), dtype=torch.bfloat16, device="cuda")
    for layer in range(NL):
        q, k, v = (_bf16((N, h, D), 20 + 3 * layer + i).cuda() for i, h in enumerate((Hq, H, H)))
        ext.layer(layer, qo, 150, q, k, v, out)
    ev = Eviction(budget=64, sinks=4, recent=16)
    ref = _evict_reference(p, ws, tally, lens, 64, 64, 4, 16)
    A.pkv_tally_evict(ws, tally, B, 160, ev.limit, ev.budget, ev.sinks, ev.recent)
    _check_evict(p, ws, tally, ref)
    lens = [ev.length(n) for n in lens]
    total = list(new)  # all tokens so far
    rows = ws.req_pool_indices.tolist()
    rope = _axes_rope(ws, tally, Hq, H, D)
    tab = rope.norm.cos_sin.cpu().double().numpy()
    run = DecodeRunner(ws, B, num_splits=3, scale=p.scale, norm_rope=rope, tally=tally, evict=ev,
                       out_per_layer=True)
    for step in range(4):
        for i, x in enumerate((run.q_in, run.k_in, run.v_in)):
            x.copy_(_bf16(tuple(x.shape), 60 + 3 * step + i))
        run.bind()
        lens = [n + 1 for n in lens]
        for layer in range(NL):
            before = (tally.weight.clone(), tally.origin.clone())
            run.layer(layer)
            torch.cuda.synchronize()
            after = (tally.weight.clone(), tally.origin.clone())
            # the heads behind the norm and the rotation, by the count of all tokens
            for b in range(B):
                row = tab[total[b] - 3 * b]
                for x, w, used in ((run.q_in, rope.norm.q_weight, run.q_use),
                                   (run.k_in, rope.norm.k_weight, run.k_use)):
                    y = K8.norm_rope(P.f64(x[layer, b]), P.f64(w), row[:D // 2], row[D // 2:],
                                     1e-6, False)
                    # one rounding to bf16, and fp32 steps of values below 64
                    assert np.all(np.abs(P.f64(used[b]) - y) <= 2.0 ** -8 * np.abs(y) + 1e-4)
                s = P.slots(p, b, lens[b])
                assert torch.equal(ws.k_pool[layer, s[-1]], run.k_use[b])
                assert torch.equal(ws.v_pool[layer, s[-1]], run.v_in[layer, b])
            tally.weight.copy_(before[0])
            tally.origin.copy_(before[1])
            ref = _decode_reference(p, ws, tally, layer, run.q_use, lens, True)
            tally.weight.copy_(after[0])
            tally.origin.copy_(after[1])
            _check_tally(tally, ref)
        ref = _evict_reference(p, ws, tally, lens, 64, 64, 4, 16)
        A.pkv_tally_evict(ws, tally, B, run.evict_len, ev.limit, ev.budget, ev.sinks, ev.recent)
        _check_evict(p, ws, tally, ref)
        assert int(ws.err.item()) == 0
        lens = [ev.length(n) for n in lens]
        total = [n + 1 for n in total]
        for b, r in enumerate(rows):
            assert lens[b] + int(tally.evicted[r]) == total[b]


def test_graph_replays_as_eager(cuda):
    """Two layers with the early start, captured and replayed, as the same steps run
    eagerly: bit for bit, attention, tally and evictions."""
    got = []
    for graph, plan in ((False, False), (True, False), (True, True)):
        p = P.problem([500, 70, 130], heads=(8, 2), layers=3, steps=8)
        ws, tally = P.device(p, max_splits=4)
        run = DecodeRunner(ws, 3, num_splits=4, scale=p.scale, tally=tally, plan=plan,
                           norm_rope=_axes_rope(ws, tally, 8, 2, 128, 1000),
                           evict=Eviction(budget=72, limit=75, sinks=2, recent=8, max_len=501),
                           out_per_layer=True)
        for i, x in enumerate((run.q_in, run.k_in, run.v_in)):
            x.copy_(_bf16(tuple(x.shape), 70 + i))
        if graph:
            run.capture()
        for _ in range(6):
            run.replay() if graph else run.step()
        torch.cuda.synchronize()
        assert int(ws.err.item()) == 0
        got.append([x.clone() for x in (run.outs.view(torch.int16), tally.weight, tally.origin,
                                        tally.evicted, ws.seq_lens, ws.k_pool.view(torch.int16),
                                        ws.v_pool.view(torch.int16))])
    for other in got[1:]:
        for a, b in zip(got[0], other):
            assert torch.equal(a, b)


def test_prompt_captured_and_replayed_with_other_inputs(cuda):
    """TallyExtender and the eviction in one graph, replayed on other rows, lengths and
    new-token counts, as the same calls run eagerly."""
    p = P.problem([300, 200], heads=(8, 2), d=64, layers=2, steps=0)
    lens, new = [[300, 200], [257, 130], [300, 1]], [[100, 64], [33, 100], [1, 1]]
    got = []
    for graph in (False, True):
        ws, tally = P.device(p)
        ext = TallyExtender(ws, tally, 2, max_new=100, scale=p.scale, window=50)
        q = torch.zeros((200, 8, 64), dtype=torch.bfloat16, device="cuda")
        k, v = (torch.zeros((200, 2, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        out, qo = torch.zeros_like(q), torch.zeros(3, dtype=torch.int32, device="cuda")

        def calls():
            for layer in range(2):
                ext.layer(layer, qo, 100, q, k, v, out)
            A.pkv_tally_evict(ws, tally, 2, 300, 150, 120, 4, 16)

        st = torch.cuda.Stream()
        g = None
        for i in range(3):
            q.copy_(_bf16(tuple(q.shape), 80 + i))
            k.copy_(_bf16(tuple(k.shape), 90 + i))
            v.copy_(_bf16(tuple(v.shape), 95 + i))
            ws.seq_lens.copy_(torch.tensor(lens[i], dtype=torch.int32))
            qo.copy_(torch.tensor([0, new[i][0], sum(new[i])], dtype=torch.int32))
            torch.cuda.synchronize()
            if not graph:
                calls()
            else:
                if g is None:
                    g = torch.cuda.CUDAGraph()
                    with torch.cuda.stream(st), torch.cuda.graph(g, stream=st):
                        calls()
                g.replay()
            torch.cuda.synchronize()
            assert int(ws.err.item()) == 0
            got.append([x.clone() for x in (tally.weight, tally.origin, tally.evicted, ws.seq_lens,
                                            ws.k_pool.view(torch.int16), out.view(torch.int16))])
    for a, b in zip(got[:3], got[3:]):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


@pytest.mark.parametrize("page,heads", [(16, (8, 2)), (1, (16, 8)), (5, (2, 2))])
@pytest.mark.parametrize("lens", [[70], [900, 3, 260, 64], [400] * 40])
@pytest.mark.parametrize("turns", [False, True])
def test_decode_back_to_back(cuda, page, heads, lens, turns):
    """Decode layers with nothing between them, each reading early the weights that the one
    before stores: bit for bit as the same calls with a wait behind each.  turns: every
    other call takes the first request alone, so that other blocks come to its tokens."""
    calls, B = 24, len(lens)
    qs = [_bf16((B, heads[0], 64), 300 + i).cuda() for i in range(calls)]
    got = []
    for wait in (True, False):
        for layers in (1, 3):
            p = P.problem(lens, page=page, heads=heads, d=64, layers=layers)
            ws, tally = P.device(p, max_splits=3)
            torch.cuda.synchronize()
            for i, q in enumerate(qs):
                early = A.PKV_FLAG_PLAN_EARLY if i > 0 else 0
                n = 1 if turns and i % 2 else B
                A.pkv_tally_decode_layer(ws, tally, n, i % layers, q, None, None, p.scale, 3, early)
                if wait:
                    torch.cuda.synchronize()
            torch.cuda.synchronize()
            assert int(ws.err.item()) == 0
            got.append((tally.weight.clone(), ws.lse.clone()))
    for a, b in zip(got[:2], got[2:]):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_decode_back_to_back_sums_to_the_calls(cuda):
    """The same against the oracle: weights of many calls, from one layer's tally of zeros."""
    lens, calls = [260, 900, 1], 20
    p = P.problem(lens, page=1, heads=(16, 8), d=64)
    ws, tally = P.device(p, max_splits=3)
    tally.weight.zero_()
    qs = [_bf16((3, 16, 64), 300 + i).cuda() for i in range(calls)]
    torch.cuda.synchronize()
    for q in qs:
        A.pkv_tally_decode_layer(ws, tally, 3, 0, q, None, None, p.scale, 3)
    torch.cuda.synchronize()
    got = P.by_slot(tally.weight).astype(np.float64)
    tally.weight.zero_()
    w, bound = 0.0, 0.0
    for q in qs:
        one = _decode_reference(p, ws, tally, 0, q, lens, False)
        w, bound = w + one[0], bound + one[2]
    # and an addition's rounding for each call
    assert np.all(np.abs(got - w) <= bound + calls * P.EPS32 * w)


@pytest.mark.parametrize("page", [16, 1])
def test_decode_right_behind_an_eviction(cuda, page):
    """A layer whose lengths, weights and rows the launch before it wrote, without and with
    a wait between the two."""
    lens, got = [300, 90, 700], []
    q = _bf16((3, 8, 128), 5).cuda()
    for wait in (True, False):
        p = P.problem(lens, page=page, heads=(8, 4))
        ws, tally = P.device(p, max_splits=3)
        _set_tally(p, ws, tally, "random")
        torch.cuda.synchronize()
        for budget in (200, 120, 64):
            A.pkv_tally_evict(ws, tally, 3, 700, budget, budget, 4, 16)
            if wait:
                torch.cuda.synchronize()
            A.pkv_tally_decode_layer(ws, tally, 3, 0, q, None, None, p.scale, 3)
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        assert ws.seq_lens.tolist() == [64, 64, 64] and int(ws.err.item()) == 0
        got.append((tally.weight.clone(), tally.origin.clone(), ws.out_bf16(3).clone()))
    for a, b in zip(*got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("seed", range(24))
def test_random_shapes(cuda, seed):
    """Seeded combinations of everything: a prompt's tally, a decode layer's, an eviction."""
    r = np.random.default_rng(1000 + seed)
    H = int(r.choice([1, 2, 3, 5, 8]))
    heads, d = (H * int(r.choice([1, 2, 4, 8])), H), int(r.choice([64, 128]))
    page, B = int(r.choice([1, 3, 7, 16, 24, 32, 80])), int(r.integers(1, 9))
    lens = [int(x) for x in r.integers(0, 400, B)]
    new = [int(r.integers(0, n + 1)) for n in lens]
    if not sum(new):
        lens[0], new[0] = 9, 4
    p = P.problem(lens, page=page, heads=heads, d=d, layers=2)
    layer = int(r.integers(0, 2))
    ws, tally, ref, _ = _extend(p, lens, new, window=int(r.integers(1, 300)), layer=layer)
    _check_tally(tally, ref, "prompt")
    S = int(r.integers(1, 4))
    ws, tally = P.device(p, max_splits=S)
    q = _bf16((B, heads[0], d), seed).cuda()
    k, v = (_bf16((B, H, d), seed + s).cuda() for s in (100, 200))
    add = bool(r.integers(0, 2))
    if add:  # the oracle's view of the pool
        old = ws.k_pool.clone()
        for b, n in enumerate(lens):
            if n:
                ws.k_pool[layer, P.slots(p, b, n)[-1]] = k[b]
    ref = _decode_reference(p, ws, tally, layer, q, lens, add)
    if add:
        ws.k_pool.copy_(old)
    A.pkv_tally_decode_layer(ws, tally, B, layer, q, k if add else None, v if add else None,
                             p.scale, S)
    torch.cuda.synchronize()
    _check_tally(tally, ref, "decode")
    _set_tally(p, ws, tally, ["random", "ties", "odd"][seed % 3], seed)
    budget = int(r.integers(1, 300))
    sinks = int(r.integers(0, min(5, budget) + 1))
    recent = int(r.integers(0, budget - sinks + 1))
    limit = budget + int(r.integers(0, 50))
    ref = _evict_reference(p, ws, tally, lens, budget, limit, sinks, recent)
    A.pkv_tally_evict(ws, tally, B, int(r.integers(400, 9000)), limit, budget, sinks, recent)
    _check_evict(p, ws, tally, ref)
    assert int(ws.err.item()) == 0


def test_another_stream(cuda):
    """Calls on a stream of their own, ordered with their inputs by it alone."""
    lens = [300, 100]
    p = P.problem(lens, heads=(8, 2), steps=1)
    ws, tally = P.device(p, max_splits=2)
    q = _bf16((2, 8, 128), 5)
    ref = _decode_reference(p, ws, tally, 0, q, lens, False)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        dq = torch.zeros((2, 8, 128), dtype=torch.bfloat16, device="cuda")
        dq.copy_(q.pin_memory(), non_blocking=True)
        A.pkv_tally_decode_layer(ws, tally, 2, 0, dq, None, None, p.scale, 2)
        mid = (tally.weight.clone(), tally.origin.clone(), tally.evicted.clone())
        A.pkv_tally_evict(ws, tally, 2, 300, 120, 120, 4, 20, stream=st)
    st.synchronize()
    now = (tally.origin.clone(), tally.evicted.clone())
    for x, y in zip((tally.weight, tally.origin, tally.evicted), mid):
        x.copy_(y)  # the state in front of the eviction, for the oracle
    _check_tally(tally, ref)
    assert ws.seq_lens.tolist() == [120, 100]
    want = _evict_reference(p, ws, tally, lens, 120, 120, 4, 20)
    assert np.array_equal(P.by_slot(now[0]), want[0]["origin"])
    assert np.array_equal(now[1].cpu().numpy(), want[1])
