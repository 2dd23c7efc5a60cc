"""Shared set-up of the tally's tests: a paged bf16 problem with a tally on a device, the
oracle's view of it, and bounds."""
from __future__ import annotations

import numpy as np
import torch

import oracle.ref as R
import oracle.tally as T
import pkv_inputs as W

EPS32 = 2.0 ** -24  # half a step of fp32, relative


def f64(t):
    return R.bf16_bits_to_f64(R.tensor_bits(t.cpu()))


def problem(lens, *, page=16, heads=(8, 2), d=128, layers=1, steps=0, seed=7):
    return W.make_problem(batch=len(lens), n_layers=layers, n_q_heads=heads[0],
                          n_kv_heads=heads[1], head_dim=d, page_size=page, seq_lens=lens,
                          steps=steps, seed=seed, pool_factor=1.3)


def slots(p, b, n):
    row = p.page_table[int(p.req_pool_indices[b])].numpy()
    t = np.arange(n)
    return row[t // p.page_size].astype(np.int64) * p.page_size + t % p.page_size


def by_slot(x):
    """[NL, pages, H, P] -> [NL, slots, H]."""
    x = x.cpu().numpy() if isinstance(x, torch.Tensor) else x
    NL, pages, H, P = x.shape
    return np.ascontiguousarray(x.transpose(0, 1, 3, 2)).reshape(NL, pages * P, H)


def device(p, *, max_splits=1, seed=3, max_batch=None, dev="cuda"):
    """(workspace, tally) of the problem, bound as it is; every entry of the tally holds
    something before, and every table row an evicted count."""
    from paged_kv_decode_bind_gb300 import Tally, Workspace
    from paged_kv_decode_bind_gb300 import _abi as A
    ws = Workspace(n_layers=p.n_layers, pool_slots=p.pool_slots, n_q_heads=p.n_q_heads,
                   n_kv_heads=p.n_kv_heads, head_dim=p.head_dim, page_size=p.page_size,
                   max_batch=max_batch or p.batch, max_reqs=p.max_reqs,
                   max_pages_per_req=p.max_pages_per_req, max_splits=max_splits,
                   max_total_tokens=(p.batch * p.max_pages_per_req if p.page_size == 1 else 0),
                   index_mode=p.index_mode, device=dev)
    ws.load(p)
    tally = Tally(ws)
    g = torch.Generator().manual_seed(seed)
    tally.weight.copy_(torch.exp(torch.randn(tally.weight.shape, generator=g)))
    tally.origin.copy_(torch.randint(0, 1000, tally.origin.shape, generator=g, dtype=torch.int32))
    tally.evicted.copy_(torch.randint(0, 100, tally.evicted.shape, generator=g,
                                      dtype=torch.int32))
    if ws.device.type == "cuda":
        A.pkv_bind_step(ws, p.batch, A.PKV_BIND_REBUILD)
    return ws, tally


def weight_bound(w, err, count, lse_size, D, lse_err=0.0):
    """Bound on a computed weight sum.  A score: 2 D fp32 roundings of its products' sum
    (tensor cores may cut a sum off instead of rounding it, a whole step each) and a few
    of its scaling, relative to sum |q k|; the subtraction of lse in log2 units: a few
    steps of |lse| and of the exponent; the exponential 2^-20; `count` additions."""
    # |s| <= |size|, so the exponent is at most |s| + |lse| in size
    per = 2.0 ** -20 + lse_err + 8 * EPS32 * lse_size + count * 2 * EPS32
    return (2 * D + 16) * EPS32 * err + per * w
