"""Norm and rotation of query and key heads on the GPU against the 64-bit
oracle.

Bound: the fp32 sum of D squares, the root and the products put the value a few
fp32 steps off (at most D + 16 of them, relative to the pair's size), then one
rounding to bf16."""
import numpy as np
import pytest
import torch

import oracle.kv8 as K8
from kv8_problem import K8_values
from paged_kv_decode_bind_gb300 import QkNormRope, rope_table
from paged_kv_decode_bind_gb300 import _abi as A

pytestmark = pytest.mark.gpu


def _bf16(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).bfloat16()


def _expect(x, w, table, pos, rot, eps, interleaved):
    """[T, heads, D] in float64 and the size of each element's pair."""
    T = x.shape[0]
    out, size = np.zeros(x.shape), np.zeros(x.shape)
    for t in range(T):
        row = table[pos[t]] if rot else np.zeros(0)
        cos, sin = row[:rot // 2], row[rot // 2:]
        out[t] = K8.norm_rope(x[t], w, cos, sin, eps, interleaved)
        one, zero = np.ones(rot // 2), np.zeros(rot // 2)
        y = np.abs(K8.norm_rope(x[t], w, one, zero, eps, interleaved))
        size[t] = y
        for i in range(rot // 2):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
            size[t][:, a] = size[t][:, b] = y[:, a] + y[:, b]
    return out, size


def _check(got, ref, D):
    o, size = ref
    got = got.double().cpu().numpy()
    tol = np.abs(o) * 2.0 ** -8 + size * (D + 16) * 2.0 ** -24 * (1 + 2.0 ** -8)
    # an element below bf16's normal range is off by half its smallest step
    assert np.all(np.isfinite(got))
    assert np.all(np.abs(got - o) <= tol + 2.0 ** -134)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv", [(1, 0), (1, 1), (8, 2), (7, 3), (32, 8)])
@pytest.mark.parametrize("rot", [0, 16, 48, 64])
@pytest.mark.parametrize("interleaved", [False, True])
def test_heads(cuda, d, hq, hkv, rot, interleaved):
    T, span = 5, 300
    x = _bf16((T, (hq + 2 * hkv) * d), 1, 3.0)
    q, k = x[:, :hq * d], x[:, hq * d:(hq + hkv) * d]
    wq, wk = _bf16((d,), 2), _bf16((d,), 3)
    table = rope_table(span, rot, device="cpu") if rot else None
    pos = torch.tensor([0, 299, 7, 7, 123], dtype=torch.int32)
    args = QkNormRope(n_q_heads=hq, n_kv_heads=hkv, head_dim=d, rot_dim=rot,
                      cos_sin=table.cuda() if rot else None, q_weight=wq.cuda(),
                      k_weight=wk.cuda(), eps=1e-5, interleaved=interleaved)
    xc = x.cuda()
    qo = torch.zeros((T, hq, d), dtype=torch.bfloat16, device="cuda")
    ko = torch.zeros((T, max(hkv, 1), d), dtype=torch.bfloat16, device="cuda")
    A.pkv_qk_norm_rope(args, T, xc[:, :hq * d], xc[:, hq * d:(hq + hkv) * d] if hkv else None,
                       pos.cuda(), qo, ko if hkv else None)
    torch.cuda.synchronize()
    tab = table.double().numpy() if rot else None
    eps = float(np.float32(1e-5))
    p = pos.tolist()
    _check(qo, _expect(K8_values(q.reshape(T, hq, d)), K8_values(wq), tab, p, rot, eps,
                       interleaved), d)
    if hkv:
        _check(ko, _expect(K8_values(k.reshape(T, hkv, d)), K8_values(wk), tab, p, rot, eps,
                           interleaved), d)
    assert torch.equal(xc.cpu(), x) and int(args.err.item()) == 0


@pytest.mark.parametrize("T", [1, 2, 63, 1000])
@pytest.mark.parametrize("norm", ["both", "q", "none"])
def test_tokens_and_missing_weights(cuda, T, norm):
    d, hq, hkv, rot = 128, 4, 2, 128
    q, k = _bf16((T, hq, d), 4), _bf16((T, hkv, d), 5)
    w = _bf16((d,), 6)
    table = rope_table(5000, rot, base=500000.0, device="cpu")
    pos = torch.arange(3999, 3999 + T, dtype=torch.int32) % 5000
    wq, wk = (w if norm != "none" else None), (w if norm == "both" else None)
    args = QkNormRope(n_q_heads=hq, n_kv_heads=hkv, head_dim=d, cos_sin=table.cuda(),
                      q_weight=None if wq is None else wq.cuda(),
                      k_weight=None if wk is None else wk.cuda())
    qc, kc = q.cuda(), k.cuda()
    A.pkv_qk_norm_rope(args, T, qc, kc, pos.cuda(), qc, kc)  # in place
    torch.cuda.synchronize()
    eps, tab = float(np.float32(1e-6)), table.double().numpy()
    for got, x, ww in ((qc, q, wq), (kc, k, wk)):
        _check(got, _expect(K8_values(x), None if ww is None else K8_values(ww), tab,
                            pos.tolist(), rot, eps, False), d)


@pytest.mark.parametrize("size", [0.0, 1e-30, 1e-12, 1e15])
def test_sizes(cuda, size):
    # zero heads stay zero (eps keeps the root finite); large ones stay finite
    d = 128
    q = _bf16((3, 2, d), 7, size)
    table = rope_table(16, d, device="cpu")
    w = _bf16((d,), 8)
    args = QkNormRope(n_q_heads=2, n_kv_heads=0, head_dim=d, cos_sin=table.cuda(),
                      q_weight=w.cuda())
    out = torch.ones((3, 2, d), dtype=torch.bfloat16, device="cuda")
    A.pkv_qk_norm_rope(args, 3, q.cuda(), None, torch.tensor([1, 2, 3], dtype=torch.int32).cuda(),
                       out, None)
    torch.cuda.synchronize()
    _check(out, _expect(K8_values(q), K8_values(w), table.double().numpy(), [1, 2, 3], d,
                        float(np.float32(1e-6)), False), d)


def test_strided_output_and_bad_positions(cuda):
    d, T = 64, 6
    q, k = _bf16((T, 2, d), 9), _bf16((T, 1, d), 10)
    table = rope_table(50, 32, device="cpu")
    args = QkNormRope(n_q_heads=2, n_kv_heads=1, head_dim=d, rot_dim=32, cos_sin=table.cuda(),
                      q_weight=_bf16((d,), 11).cuda(), k_weight=_bf16((d,), 12).cuda())
    pos = torch.tensor([0, 49, 50, -1, 3, 2 ** 31 - 1], dtype=torch.int32)
    out = torch.full((T, 4 * d), 9.0, dtype=torch.bfloat16, device="cuda")
    A.pkv_qk_norm_rope(args, T, q.cuda(), k.cuda(), pos.cuda(), out[:, :2 * d],
                       out[:, 2 * d:3 * d])
    torch.cuda.synchronize()
    assert int(args.err.item()) == A.PKV_DEVERR_POSITION
    bad = [2, 3, 5]
    assert torch.all(out[bad, :3 * d] == 0) and torch.all(out[:, 3 * d:] == 9.0)
    good = [0, 1, 4]
    p = pos[good].tolist()
    eps, tab = float(np.float32(1e-6)), table.double().numpy()
    _check(out[good, :2 * d].reshape(3, 2, d),
           _expect(K8_values(q[good]), K8_values(args.q_weight.cpu()), tab, p, 32, eps, False), d)
    _check(out[good, 2 * d:3 * d].reshape(3, 1, d),
           _expect(K8_values(k[good]), K8_values(args.k_weight.cpu()), tab, p, 32, eps, False), d)


def test_an_empty_request_is_no_error(cuda):
    d, pos = 128, torch.tensor([4, -1, 0], dtype=torch.int32)
    q, k = _bf16((3, 4, d), 21).cuda(), _bf16((3, 2, d), 22).cuda()
    args = QkNormRope(n_q_heads=4, n_kv_heads=2, head_dim=d, cos_sin=rope_table(5, d))
    A.pkv_qk_norm_rope(args, 3, q, k, pos.cuda(), q, k)
    assert int(args.err.item()) == 0
    assert torch.all(q[1] == 0) and torch.all(k[1] == 0) and q[0].any() and k[2].any()
    A.pkv_qk_norm_rope(args, 3, q, k, (pos - 1).cuda(), q, k)
    assert int(args.err.item()) == A.PKV_DEVERR_POSITION


def test_norm_alone_needs_no_positions(cuda):
    d = 128
    q, w = _bf16((4, 3, d), 15), _bf16((d,), 16)
    args = QkNormRope(n_q_heads=3, n_kv_heads=0, head_dim=d, rot_dim=0, q_weight=w.cuda())
    out = torch.zeros((4, 3, d), dtype=torch.bfloat16, device="cuda")
    A.pkv_qk_norm_rope(args, 4, q.cuda(), None, None, out, None)
    torch.cuda.synchronize()
    _check(out, _expect(K8_values(q), K8_values(w), None, [0] * 4, 0, float(np.float32(1e-6)),
                        False), d)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_heads_that_are_not_finite(cuda, bad):
    # a head with NaN or an infinity is its own affair
    d = 64
    q, w = _bf16((5, 4, d), 17), _bf16((d,), 18)
    dirty = q.clone()
    dirty[2, 1, 40] = bad
    table = rope_table(8, d, device="cpu")
    args = QkNormRope(n_q_heads=4, n_kv_heads=0, head_dim=d, cos_sin=table.cuda(), q_weight=w.cuda())
    out = torch.zeros((5, 4, d), dtype=torch.bfloat16, device="cuda")
    pos = torch.arange(5, dtype=torch.int32)
    A.pkv_qk_norm_rope(args, 5, dirty.cuda(), None, pos.cuda(), out, None)
    torch.cuda.synchronize()
    assert torch.isnan(out[2, 1]).any()
    out[2, 1] = 0
    o, size = _expect(K8_values(q), K8_values(w), table.double().numpy(), pos.tolist(), d,
                      float(np.float32(1e-6)), False)
    o[2, 1] = size[2, 1] = 0
    _check(out, (o, size), d)


def test_rows_behind_the_last_token_are_left(cuda):
    d = 128
    args = QkNormRope(n_q_heads=4, n_kv_heads=1, head_dim=d, cos_sin=rope_table(64, d))
    q, k = _bf16((8, 4, d), 13).cuda(), _bf16((8, 1, d), 14).cuda()
    qo, ko = torch.full_like(q, 2.0), torch.full_like(k, 2.0)
    A.pkv_qk_norm_rope(args, 3, q, k, torch.arange(8, dtype=torch.int32).cuda(), qo, ko)
    torch.cuda.synchronize()
    assert torch.all(qo[3:] == 2.0) and torch.all(ko[3:] == 2.0)


def test_rope_table_keeps_far_angles():
    # position * frequency in 64 bits, rounded once: a 32-bit angle of 1e5 radians
    # would be off by 2^-8
    t = rope_table(100001, 16, device="cpu").double().numpy()
    i = np.arange(0, 16, 2)
    a = 100000 * 10000.0 ** (-i / 16)
    assert np.abs(t[100000] - np.concatenate([np.cos(a), np.sin(a)])).max() <= 2.0 ** -24
