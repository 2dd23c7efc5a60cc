"""Norm and rotation by positions of several axes on the GPU against the 64-bit oracle.
Bound: as in test_gpu_qk_norm_rope.py (the arithmetic is the same, the rows of the table
differ by pair)."""
import numpy as np
import pytest
import torch

import oracle.kv8 as K8
from kv8_problem import K8_values
from paged_kv_decode_bind_gb300 import QkNormRope, QkNormRopeAxes, rope_table
from paged_kv_decode_bind_gb300 import _abi as A
from test_gpu_qk_norm_rope import _bf16, _check

pytestmark = pytest.mark.gpu

SPAN = 300


def _expect(x, w, table, pos, axis, rot, eps, interleaved):
    """[T, heads, D] in float64 and the size of each element's pair; pos [axes, T], a token
    of position -1 on every axis is zeros."""
    out, size = np.zeros(x.shape), np.zeros(x.shape)
    half = rot // 2
    i = np.arange(half)
    lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    for t in range(x.shape[0]):
        if half and all(pos[a][t] < 0 for a in set(axis)):
            continue
        line = [table[pos[a][t]] for a in axis]
        cos = np.array([r[j] for j, r in enumerate(line)])
        sin = np.array([r[half + j] for j, r in enumerate(line)])
        out[t] = K8.norm_rope(x[t], w, cos, sin, eps, interleaved)
        y = np.abs(K8.norm_rope(x[t], w, np.ones(half), np.zeros(half), eps, interleaved))
        size[t] = y
        size[t][:, lo] = size[t][:, hi] = y[:, lo] + y[:, hi]
    return out, size


LAYOUTS = {
    "one": lambda n: [0] * n,
    "sections": lambda n: [0] * (n // 4) + [1] * ((n - n // 4) // 2) +
    [2] * (n - n // 4 - (n - n // 4) // 2),
    "odd": lambda n: [min(3, i // 5) for i in range(n)],
    "turns": lambda n: [i % 3 for i in range(n)],
    "last": lambda n: [3] * n,  # axes 0 to 2 in no pair
}


@pytest.mark.parametrize("layout", sorted(LAYOUTS))
@pytest.mark.parametrize("d,rot", [(64, 16), (64, 64), (128, 128), (128, 48), (256, 256)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens", [1, 5, 67])
def test_axes(cuda, layout, d, rot, interleaved, tokens):
    hq, hkv, n = 6, 2, rot // 2
    axis = LAYOUTS[layout](n)
    x = _bf16((tokens, (hq + 2 * hkv) * d), 1, 3.0)
    q, k = x[:, :hq * d], x[:, hq * d:(hq + hkv) * d]
    wq, wk = _bf16((d,), 2), _bf16((d,), 3)
    table = rope_table(SPAN, rot, device="cpu")
    g = torch.Generator().manual_seed(9)
    n_axes = max(axis) + 1
    pos = torch.randint(0, SPAN, (n_axes, tokens + 3), generator=g, dtype=torch.int32)
    rope = QkNormRopeAxes(n_q_heads=hq, n_kv_heads=hkv, head_dim=d, rot_dim=rot,
                          cos_sin=table.cuda(), q_weight=wq.cuda(), k_weight=wk.cuda(),
                          axis_of_pair=axis, interleaved=interleaved)
    dx = x.cuda()
    qo = torch.zeros((tokens, hq, d), dtype=torch.bfloat16, device="cuda")
    ko = torch.zeros((tokens, hkv, d), dtype=torch.bfloat16, device="cuda")
    A.pkv_qk_norm_rope_axes(rope, tokens, dx[:, :hq * d], dx[:, hq * d:(hq + hkv) * d],
                            pos.cuda(), qo, ko)
    torch.cuda.synchronize()
    assert int(rope.err.item()) == 0
    tab, pn = table.double().numpy(), pos.numpy()
    for got, src, w, h in ((qo, q, wq, hq), (ko, k, wk, hkv)):
        ref = _expect(K8_values(src.contiguous()).reshape(tokens, h, d), K8_values(w), tab, pn,
                      axis, rot, 1e-6, interleaved)
        _check(got, ref, d)


@pytest.mark.parametrize("norm", [False, True])
def test_one_axis_is_the_plain_rotation(cuda, norm):
    """Bit for bit, with shifts that add up to the plain call's positions."""
    T, hq, hkv, d = 33, 8, 2, 128
    q, k = _bf16((T, hq, d), 1).cuda(), _bf16((T, hkv, d), 2).cuda()
    w = _bf16((d,), 3).cuda() if norm else None
    common = dict(n_q_heads=hq, n_kv_heads=hkv, head_dim=d, cos_sin=rope_table(SPAN, d),
                  q_weight=w, k_weight=w)
    g = torch.Generator().manual_seed(5)
    rows = torch.randperm(2 * T, generator=g)[:T].int()
    ev = torch.randint(0, 100, (2 * T,), generator=g, dtype=torch.int32)
    dl = torch.randint(-50, 1, (2 * T,), generator=g, dtype=torch.int32)
    pos = torch.randint(50, 200, (T,), generator=g, dtype=torch.int32)
    plain, axes = QkNormRope(**common), QkNormRopeAxes(
        rows=rows.cuda(), evicted=ev.cuda(), delta=dl.cuda(), **common)
    outs = [[torch.zeros_like(x) for x in (q, k)] for _ in range(2)]
    moved = pos + ev[rows.long()] + dl[rows.long()]
    A.pkv_qk_norm_rope(plain, T, q, k, moved.cuda(), *outs[0])
    A.pkv_qk_norm_rope_axes(axes, T, q, k, pos.cuda(), *outs[1])
    torch.cuda.synchronize()
    assert int(plain.err.item()) == 0 and int(axes.err.item()) == 0
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_one_row_of_positions_for_every_axis(cuda):
    """[tokens], the same row expanded, and a copy of it for each axis: the same bits."""
    T, hq, hkv, d = 9, 4, 2, 64
    q, k = _bf16((T, hq, d), 1).cuda(), _bf16((T, hkv, d), 2).cuda()
    rope = QkNormRopeAxes(n_q_heads=hq, n_kv_heads=hkv, head_dim=d, sections=(8, 12, 12),
                          cos_sin=rope_table(SPAN, d))
    pos = torch.randint(0, SPAN, (T,), generator=torch.Generator().manual_seed(5)).int().cuda()
    outs = []
    for x in (pos, pos.expand(3, T), pos.expand(3, T).contiguous()):
        outs.append([torch.zeros_like(y) for y in (q, k)])
        A.pkv_qk_norm_rope_axes(rope, T, q, k, x, *outs[-1])
    torch.cuda.synchronize()
    assert int(rope.err.item()) == 0
    for other in outs[1:]:
        for a, b in zip(outs[0], other):
            assert torch.equal(a, b)


def test_positions_outside_the_table(cuda):
    """Zeros and an error for a position of an axis in use, or a row, that is out of range;
    zeros alone for an empty request; no look at an axis that no pair follows."""
    T, hq, d = 7, 2, 64
    q = _bf16((T, hq, d), 1).cuda()
    axis = [0] * 16 + [2] * 16
    rows = torch.tensor([0, 1, 2, 3, 0, 0, 9], dtype=torch.int32).cuda()
    ev = torch.tensor([0, 5, -400, 2 ** 31 - 1], dtype=torch.int32).cuda()
    rope = QkNormRopeAxes(n_q_heads=hq, n_kv_heads=0, head_dim=d, cos_sin=rope_table(SPAN, d),
                          axis_of_pair=axis, rows=rows, evicted=ev)
    pos = torch.tensor([[3, 294, 100, 1, -1, 4, 5],
                        [10 ** 6] * T,
                        [7, 295, 100, 1, -1, SPAN, 5]], dtype=torch.int32).cuda()
    want = [True, False, False, False, False, False, False]
    for t in range(T):
        rope.err.zero_()
        out = torch.full_like(q[:1], 5.0)
        one = QkNormRopeAxes(n_q_heads=hq, n_kv_heads=0, head_dim=d, cos_sin=rope.norm.cos_sin,
                             axis_of_pair=axis, rows=rows[t:t + 1].contiguous(), evicted=ev)
        A.pkv_qk_norm_rope_axes(one, 1, q[t:t + 1], None, pos[:, t:t + 1].contiguous(), out, None)
        torch.cuda.synchronize()
        assert bool((out != 0).any()) == want[t], t
        assert int(one.err.item()) == (0 if want[t] or t == 4 else A.PKV_DEVERR_POSITION), t


def test_in_place_many_tokens(cuda):
    """A prompt's tokens in place, in one pass, as token by token."""
    T, hq, hkv, d = 3000, 4, 2, 128
    x = _bf16((T, (hq + hkv) * d), 1).cuda()
    g = torch.Generator().manual_seed(5)
    pos = torch.randint(0, SPAN, (3, T), generator=g, dtype=torch.int32).cuda()
    rope = QkNormRopeAxes(n_q_heads=hq, n_kv_heads=hkv, head_dim=d, cos_sin=rope_table(SPAN, d),
                          sections=(16, 24, 24))
    y, z = x.clone(), x.clone()
    A.pkv_qk_norm_rope_axes(rope, T, y[:, :hq * d], y[:, hq * d:], pos, y[:, :hq * d],
                            y[:, hq * d:])
    for t in (0, 1, 1499, T - 1):
        one = z[t:t + 1].clone()
        A.pkv_qk_norm_rope_axes(rope, 1, one[:, :hq * d], one[:, hq * d:],
                                pos[:, t:t + 1].contiguous(), one[:, :hq * d], one[:, hq * d:])
        torch.cuda.synchronize()
        assert torch.equal(one[0], y[t])
    assert int(rope.err.item()) == 0
