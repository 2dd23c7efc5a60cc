"""The tally's oracle pinned, its entry points' refusals, and its owners on the host."""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle.tally as T
import paged_kv_decode_bind_gb300 as pkv
from paged_kv_decode_bind_gb300 import _abi as A


# ------------------------------------------------------------------ oracle ----
def test_weights_by_hand():
    # two heads of one KV head over two tokens: scores (0, ln 3) and (0, 0)
    q = np.array([[[math.log(3.0)], [0.0]]])
    k = np.array([[[0.0]], [[1.0]]])
    lse = T.log_sum_exp(q, k, 1.0, [1])
    assert np.allclose(lse, [[math.log(4.0), math.log(2.0)]])
    w, _ = T.weights(q, k, lse, 1.0, [1])
    assert np.allclose(w, [[0.25 + 0.5], [0.75 + 0.5]])
    # a query that sees the first token only, and one without a softmax
    w, _ = T.weights(np.repeat(q, 2, 0), k, np.array([[0.0, 0.0], [-np.inf, np.nan]]), 1.0, [0, 1])
    assert np.allclose(w, [[2.0], [0.0]])


def test_weights_past_fp32_are_nothing():
    q, k = np.array([[[1.0]], [[1.0]], [[1.0]], [[1.0]]]), np.array([[[0.0]], [[1.0]]])
    lse = np.array([[-80.0], [-89.0], [-1000.0], [1.0]])  # fp32 ends at e^88.7
    w, _ = T.weights(q, k, lse, 1.0, [1] * 4)
    assert np.allclose(w, [[math.exp(80.0)], [math.exp(81.0)]], rtol=1e-12)


def test_keep_and_moves_by_hand():
    w = np.array([0.5, 3.0, np.nan, 0.5, 0.5, 0.1, 0.2])
    o = np.array([0, 9, 10, 11, 12, 13, 14])
    # total 15: origin 0 (sink) and 14 (recent) stay, then 3.0, then the first 0.5
    kept = T.keep(w, o, 15, 4, 1, 1)
    assert kept == [0, 1, 3, 6]
    assert T.moves(kept, 4) == [(6, 2)]
    # all but one: the NaN goes
    assert T.keep(w, o, 15, 6, 0, 0) == [0, 1, 3, 4, 5, 6]
    assert T.keep(np.zeros(5), np.arange(5) + 3, 100, 2, 0, 0) == [0, 1]


@pytest.mark.parametrize("mistake", ["ties", "protected", "order"])
def test_planted_mistakes_show(mistake):
    """The hand-worked case above tells a wrong rule from the right one."""
    w = np.array([0.5, 3.0, np.nan, 0.5, 0.5, 0.1, 0.2])
    o = np.array([0, 9, 10, 11, 12, 13, 14])
    if mistake == "ties":  # the last of equals
        kept = sorted(sorted(range(7), key=lambda t: (not (o[t] < 1 or o[t] >= 14),
                                                      -np.nan_to_num(w[t], nan=-1), -t))[:4])
    elif mistake == "protected":
        kept = T.keep(w, o, 15, 4, 0, 0)
    else:
        kept = T.keep(w, np.roll(o, 1), 15, 4, 1, 1)  # origins of the wrong tokens
    assert kept != [0, 1, 3, 6]


# ---------------------------------------------------------------- C entries ----
def _ws(**kw):
    """A workspace struct whose pointers look right; no call below gets to launch."""
    d = dict(n_layers=2, pool_slots=64, n_q_heads=8, n_kv_heads=2, head_dim=64, page_size=16,
             index_mode=0, max_batch=4, max_reqs=4, max_pages_per_req=4, max_splits=2,
             max_total_tokens=0, max_seq_len=0)
    d.update({n: 4096 for n in ("k_pool", "v_pool", "req_pool_indices", "page_table", "seq_lens",
                                "position_ids", "kv_indptr", "out_loc", "o_part", "ml_part", "out",
                                "lse", "err", "split_counters")})
    d.update(kw)
    return A.PkvWorkspace(**d)


def _t(**kw):
    d = dict(weight=4096, origin=4096, evicted=4096, score=4096, score_tokens=64, reserved=0)
    d.update(kw)
    return A.PkvTally(**d)


def test_struct_layout():
    assert ctypes.sizeof(A.PkvTally) == 4 * 8 + 8
    assert ctypes.sizeof(A.PkvRopeAxes) == 8 + 3 * 8 + 128


def test_tally_bytes():
    ws, t = _ws(), _t()
    for n in ("weight", "origin"):
        assert A.pkv_tally_bytes(ws, t, n) == 2 * 64 * 2 * 4
    assert A.pkv_tally_bytes(ws, t, "evicted") == 16
    assert A.pkv_tally_bytes(ws, t, "score") == 4 * 8 * 64 * 4
    assert A.pkv_tally_bytes(ws, t, "other") == 0


BAD_TALLY = [dict(weight=None), dict(origin=None), dict(evicted=None), dict(reserved=1),
             dict(weight=4098), dict(origin=4097)]


@pytest.mark.parametrize("ws,t,batch,layer,splits,flags,status", [
    *[({}, kw, 1, 0, 1, 0, A.PKV_ERR_INVALID) for kw in BAD_TALLY],
    ({}, dict(score=None), 1, 0, 1, 0, A.PKV_ERR_INVALID),
    ({}, dict(score=4100), 1, 0, 1, 0, A.PKV_ERR_INVALID),
    ({}, dict(score_tokens=63), 1, 0, 1, 0, A.PKV_ERR_CAPACITY),
    (dict(max_seq_len=63), dict(score_tokens=63), 0, 0, 1, 0, A.PKV_OK),
    (dict(lse=None), {}, 1, 0, 1, 0, A.PKV_ERR_INVALID),
    (dict(lse=4100), {}, 1, 0, 1, 0, A.PKV_ERR_INVALID),
    ({}, {}, 1, 0, 1, A.PKV_FLAG_FORCE_SIMT, A.PKV_ERR_INVALID),
    (dict(head_dim=256), {}, 1, 0, 1, 0, A.PKV_ERR_UNSUPPORTED),
    (dict(n_q_heads=6), {}, 1, 0, 1, 0, A.PKV_ERR_UNSUPPORTED),
    ({}, {}, 5, 0, 1, 0, A.PKV_ERR_CAPACITY),
    ({}, {}, 1, 2, 1, 0, A.PKV_ERR_CAPACITY),
    ({}, {}, 1, 0, 3, 0, A.PKV_ERR_CAPACITY),
    ({}, {}, -1, 0, 1, 0, A.PKV_ERR_INVALID),
    (dict(split_counters=None), {}, 1, 0, 2, 0, A.PKV_ERR_INVALID),
    ({}, {}, 0, 0, 1, 0, A.PKV_OK),
])
def test_decode_refusals(ws, t, batch, layer, splits, flags, status):
    assert A.pkv_tally_decode_layer(_ws(**ws), _t(**t), batch, layer, 4096, None, None, 1.0,
                                    splits, flags, stream=0, check=False) == status


def test_decode_refuses_half_an_append():
    for k, v in ((4096, None), (None, 4096), (4100, 4096)):
        assert A.pkv_tally_decode_layer(_ws(), _t(), 1, 0, 4096, k, v, 1.0, stream=0,
                                        check=False) == A.PKV_ERR_INVALID


@pytest.mark.parametrize("ws,t,kw,status", [
    *[({}, kw, {}, A.PKV_ERR_INVALID) for kw in BAD_TALLY],
    ({}, {}, dict(qo=None), A.PKV_ERR_INVALID),
    ({}, {}, dict(window=0), A.PKV_ERR_INVALID),
    ({}, {}, dict(scale=math.nan), A.PKV_ERR_INVALID),
    ({}, {}, dict(scale=-math.inf), A.PKV_ERR_INVALID),
    ({}, {}, dict(n_rows=-1), A.PKV_ERR_INVALID),
    ({}, {}, dict(max_qo=-1), A.PKV_ERR_INVALID),
    ({}, {}, dict(batch=-1), A.PKV_ERR_INVALID),
    ({}, {}, dict(batch=5), A.PKV_ERR_CAPACITY),
    ({}, {}, dict(layer=2), A.PKV_ERR_CAPACITY),
    ({}, {}, dict(q=None), A.PKV_ERR_INVALID),
    ({}, {}, dict(q=4104), A.PKV_ERR_INVALID),
    ({}, {}, dict(lse=None), A.PKV_ERR_INVALID),
    (dict(k_pool=None), {}, {}, A.PKV_ERR_INVALID),
    (dict(head_dim=32), {}, {}, A.PKV_ERR_UNSUPPORTED),
    (dict(n_q_heads=24), {}, {}, A.PKV_ERR_UNSUPPORTED),
    ({}, dict(score=None, score_tokens=0), dict(batch=0), A.PKV_OK),
    ({}, {}, dict(n_rows=0, q=None, lse=None), A.PKV_OK),
    ({}, {}, dict(max_qo=0), A.PKV_OK),
])
def test_extend_refusals(ws, t, kw, status):
    d = dict(batch=1, layer=0, qo=4096, max_qo=4, n_rows=4, window=4, q=4096, lse=4096, scale=1.0)
    d.update(kw)
    assert A.pkv_tally_extend(_ws(**ws), _t(**t), d["batch"], d["layer"], d["qo"], d["max_qo"],
                              d["n_rows"], d["window"], d["q"], d["lse"], d["scale"], stream=0,
                              check=False) == status


@pytest.mark.parametrize("ws,t,kw,status", [
    *[({}, kw, {}, A.PKV_ERR_INVALID) for kw in BAD_TALLY],
    ({}, {}, dict(budget=0), A.PKV_ERR_INVALID),
    ({}, {}, dict(limit=9), A.PKV_ERR_INVALID),
    ({}, {}, dict(sinks=-1), A.PKV_ERR_INVALID),
    ({}, {}, dict(recent=-1), A.PKV_ERR_INVALID),
    ({}, {}, dict(sinks=5, recent=6), A.PKV_ERR_INVALID),
    ({}, {}, dict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1), A.PKV_ERR_INVALID),
    ({}, {}, dict(max_len=-1), A.PKV_ERR_INVALID),
    ({}, {}, dict(max_len=A.PKV_TALLY_MAX_LEN + 1), A.PKV_ERR_UNSUPPORTED),
    ({}, {}, dict(batch=-1), A.PKV_ERR_INVALID),
    ({}, {}, dict(batch=5), A.PKV_ERR_CAPACITY),
    (dict(head_dim=32), {}, {}, A.PKV_ERR_UNSUPPORTED),
    (dict(k_pool=None), {}, {}, A.PKV_ERR_INVALID),
    (dict(v_pool=4104), {}, {}, A.PKV_ERR_INVALID),
    (dict(split_counters=None), {}, {}, A.PKV_ERR_INVALID),
    (dict(page_table=None), {}, {}, A.PKV_ERR_INVALID),
    ({}, dict(score=None, score_tokens=0), dict(batch=0), A.PKV_OK),
])
def test_evict_refusals(ws, t, kw, status):
    d = dict(batch=1, max_len=64, limit=10, budget=10, sinks=0, recent=0)
    d.update(kw)
    assert A.pkv_tally_evict(_ws(**ws), _t(**t), d["batch"], d["max_len"], d["limit"], d["budget"],
                             d["sinks"], d["recent"], stream=0, check=False) == status


def test_axes_refusals():
    lib = A.load()
    args = A.PkvQkNormRopeArgs(n_q_heads=2, n_kv_heads=0, head_dim=64, rot_dim=64,
                               max_positions=8, interleaved=0, eps=1e-6, reserved=0,
                               cos_sin=4096, err=4096)

    def call(axes, stride=0, tokens=1, positions=4096):
        return lib.pkv_qk_norm_rope_axes(args, axes, tokens, 4096, 128, None, 0, positions, stride,
                                         4096, 128, None, 0, None)

    def axes(axis=(), **kw):
        d = dict(n_axes=1, n_rows=0)
        d.update(kw)
        return A.PkvRopeAxes(**d, axis=(ctypes.c_uint8 * 128)(*axis))

    assert call(None) == A.PKV_ERR_INVALID
    for a in (axes(n_axes=0), axes(n_axes=5), axes(n_rows=-1), axes((0, 1)), axes((3,), n_axes=3),
              axes(rows=4096), axes(evicted=4096, n_rows=4), axes(delta=4096, rows=4096)):
        assert call(a) == A.PKV_ERR_INVALID
    assert call(axes(n_axes=2), stride=3, tokens=4) == A.PKV_ERR_INVALID
    assert call(axes(n_axes=2), stride=-1) == A.PKV_ERR_INVALID
    assert call(axes(), positions=None) == A.PKV_ERR_INVALID
    assert call(axes(), tokens=0) == A.PKV_OK
    # an axis past rot_dim / 2 pairs is not looked at
    assert call(axes([0] * 32 + [9]), tokens=0) == A.PKV_OK


# ------------------------------------------------------------------- owners ----
def _workspace(**kw):
    d = dict(n_layers=2, pool_slots=64, n_q_heads=8, n_kv_heads=2, head_dim=64, page_size=16,
             max_batch=4, max_reqs=4, max_pages_per_req=4, max_splits=2, device="cpu")
    d.update(kw)
    return pkv.Workspace(**d)


def test_tally_owner():
    ws = _workspace()
    t = pkv.Tally(ws)
    assert t.weight.shape == (2, 4, 2, 16) and t.score.shape == (4, 2, 64, 4)
    for n in ("weight", "origin", "evicted", "score"):
        assert A.pkv_tally_bytes(ws, t, n) == getattr(t, n).numel() * 4
    given = torch.ones(2, 4, 2, 16)
    assert pkv.Tally(ws, weight=given).weight is given
    for bad in (given[:1], given.double(), given.transpose(1, 3).contiguous().transpose(1, 3)):
        with pytest.raises(ValueError):
            pkv.Tally(ws, weight=bad)
    t.evicted.fill_(3)
    t.take_rows([1, 2])
    assert t.evicted.tolist() == [3, 0, 0, 3]


def test_a_tally_of_other_shapes_is_refused():
    t = pkv.Tally(_workspace())
    for kw in (dict(pool_slots=128), dict(n_layers=1), dict(page_size=8), dict(max_reqs=5),
               dict(n_q_heads=4)):
        ws = _workspace(**kw)
        with pytest.raises(ValueError):
            A.pkv_tally_evict(ws, t, 0, 64, 10, 10)
        with pytest.raises(ValueError):
            A.pkv_tally_extend(ws, t, 0, 0, None, 0, 0, 1, None, None, 1.0)
        with pytest.raises(ValueError):
            pkv.TallyExtender(ws, t, 1, max_new=4, scale=1.0)
    # a bare struct, and more requests than the scratch holds
    big = _workspace(max_batch=8)
    with pytest.raises(ValueError):
        A.pkv_tally_decode_layer(big, t, 5, 0, None, None, None, 1.0)
    with pytest.raises(ValueError):
        A.pkv_tally_evict(_workspace(max_reqs=5).struct, t, 0, 64, 10, 10)
    assert A.pkv_tally_evict(_workspace().struct, t, 0, 64, 10, 10) == A.PKV_OK


def test_eviction():
    e = pkv.Eviction(budget=10, sinks=4, recent=6)
    assert (e.limit, e.length(10), e.length(11)) == (10, 10, 10)
    e = pkv.Eviction(budget=10, limit=20)
    assert (e.length(20), e.length(21)) == (20, 10)
    for kw in (dict(budget=0), dict(budget=5, limit=4), dict(budget=5, sinks=3, recent=3),
               dict(budget=5, sinks=-1), dict(budget=5, recent=-1), dict(budget=5, max_len=5),
               dict(budget=5, max_len=A.PKV_TALLY_MAX_LEN + 1)):
        with pytest.raises(ValueError):
            pkv.Eviction(**kw)


def test_bind_tracker_follows_an_eviction():
    t = pkv.BindTracker()
    e = pkv.Eviction(budget=10, limit=12)
    assert t.mode([1, 2], [12, 5]) == A.PKV_BIND_REBUILD
    assert t.mode([1, 2], [13, 6]) == A.PKV_BIND_STEADY
    t.evicted(e)  # the step left 10 and 6
    assert t.mode([1, 2], [11, 7]) == A.PKV_BIND_STEADY


def test_an_eviction_leaves_requests_past_its_bound():
    """As the device does: those longer than max_len stay as they are."""
    e = pkv.Eviction(budget=10, limit=12, max_len=20)
    assert [e.length(n) for n in (12, 13, 20, 21, 500)] == [12, 10, 10, 21, 500]
    t = pkv.BindTracker()
    t.mode([1, 2], [20, 21])
    t.evicted(e)
    assert t.mode([1, 2], [11, 22]) == A.PKV_BIND_STEADY
    e = pkv.Eviction(budget=10)
    assert e.length(A.PKV_TALLY_MAX_LEN) == 10
    assert e.length(A.PKV_TALLY_MAX_LEN + 1) == A.PKV_TALLY_MAX_LEN + 1


def test_extender_refusals():
    ws = _workspace()
    t = pkv.Tally(ws)
    for kw in (dict(max_new=0), dict(max_new=4, window=0), dict(max_new=4, num_splits=0)):
        with pytest.raises(ValueError):
            pkv.TallyExtender(ws, t, 1, scale=1.0, **kw)
    for batch in (0, 5):
        with pytest.raises(ValueError):
            pkv.TallyExtender(ws, t, batch, max_new=4, scale=1.0)
    ext = pkv.TallyExtender(ws, t, 2, max_new=4, scale=1.0)
    x = torch.zeros(1)
    for kw in (dict(max_qo_len=5), dict(flags=A.PKV_FLAG_EXTEND_FULL), dict(v_new=None)):
        a = dict(layer=0, qo_indptr=x, max_qo_len=4, q=x, k_new=x, v_new=x, out=x)
        a.update(kw)
        with pytest.raises(ValueError):
            ext.layer(**a)


def test_runner_refusals():
    ws = _workspace()
    t, e = pkv.Tally(ws), pkv.Eviction(budget=8)
    table = torch.zeros(8, 64)
    heads = dict(n_q_heads=8, n_kv_heads=2, head_dim=64, cos_sin=table)
    axes = dict(rows=ws.req_pool_indices, evicted=t.evicted, **heads)
    assert pkv.DecodeRunner(ws, 2, tally=t, evict=e).evict_len == 64
    assert pkv.DecodeRunner(ws, 2, tally=t, evict=pkv.Eviction(8, max_len=9)).evict_len == 9
    pkv.DecodeRunner(ws, 2, tally=t, evict=e, norm_rope=pkv.QkNormRopeAxes(**axes))
    other = dict(axes, rows=ws.req_pool_indices.clone())
    loose = dict(axes, evicted=t.evicted.clone())
    for kw in (dict(evict=e), dict(tally=t, fused=False),
               dict(tally=t, cache=pkv.Kv8Cache(ws)),
               dict(tally=pkv.Tally(_workspace(max_reqs=5))),
               # positions that do not follow the evictions
               dict(tally=t, evict=e, norm_rope=pkv.QkNormRope(**heads)),
               dict(tally=t, evict=e, norm_rope=pkv.QkNormRopeAxes(**loose)),
               dict(tally=t, evict=e, norm_rope=pkv.QkNormRopeAxes(**other)),
               dict(norm_rope=pkv.QkNormRopeAxes(**dict(heads, n_kv_heads=1)))):
        with pytest.raises(ValueError):
            pkv.DecodeRunner(ws, 2, **kw)


def test_axes_owner():
    table = torch.zeros(8, 64)
    base = dict(n_q_heads=2, n_kv_heads=1, head_dim=64, cos_sin=table)
    r = pkv.QkNormRopeAxes(sections=(8, 12, 12), **base)
    assert list(r.axes.axis)[:32] == [0] * 8 + [1] * 12 + [2] * 12 and r.axes.n_axes == 3
    assert pkv.QkNormRopeAxes(**base).axes.n_axes == 1
    i = torch.zeros(4, dtype=torch.int32)
    for kw in (dict(sections=(8, 12)), dict(axis_of_pair=[0] * 31), dict(axis_of_pair=[4] * 32),
               dict(sections=(32,), axis_of_pair=[0] * 32), dict(rows=i), dict(evicted=i),
               dict(rows=i.long(), delta=i), dict(rows=i, evicted=i, delta=i[:3].clone()),
               dict(rows=i[::2], evicted=i)):
        with pytest.raises(ValueError):
            pkv.QkNormRopeAxes(**base, **kw)


def test_axes_tensors_are_checked():
    table = torch.zeros(8, 64)
    i = torch.zeros(4, dtype=torch.int32)
    r = pkv.QkNormRopeAxes(n_q_heads=2, n_kv_heads=1, head_dim=64, cos_sin=table,
                           sections=(16, 16), rows=i, delta=i)
    q, k = torch.zeros(9, 128).bfloat16(), torch.zeros(9, 64).bfloat16()
    good = torch.zeros(2, 4, dtype=torch.int32)
    for n, pos, qq in ((5, torch.zeros(2, 5, dtype=torch.int32), q),  # rows hold four tokens
                       (4, good.long(), q), (4, good[:, :3], q), (4, good[:1], q),
                       (4, torch.zeros(4, 2, dtype=torch.int32).T, q), (4, good, q.float()),
                       (4, good, q[:3]), (4, torch.zeros(3, 4, dtype=torch.int32), q)):
        with pytest.raises(ValueError):
            A.pkv_qk_norm_rope_axes(r, n, qq, k, pos, q, k)
    with pytest.raises(AttributeError):  # the plain call's arguments have no axes
        A.pkv_qk_norm_rope_axes(r.norm, 1, q, k, good, q, k)
    with pytest.raises((AttributeError, ctypes.ArgumentError)):
        A.pkv_qk_norm_rope(r, 1, q, k, good[0], q, k)


def test_axes_take_one_row_for_every_axis():
    """An expanded row is the same as the row itself: no elements between the axes."""
    one = torch.arange(5, dtype=torch.int32)[1:]
    assert A._axis_positions(one.expand(2, 4), 4, 2) == A._axis_positions(one, 4, 2) == \
        (one.data_ptr(), 0)
    with pytest.raises(ValueError):
        A._axis_positions(one.expand(2, 4), 5, 2)
