"""Shared set-up of the 8-bit cache tests: a paged problem whose bf16 pools are
quantised by the oracle, its workspace and cache on a device, and bounds."""
from __future__ import annotations

import numpy as np
import torch

import oracle.kv8 as K8
import oracle.ref as R
import pkv_inputs as W

EPS32 = 2.0 ** -24  # half a step of fp32, relative


def quantise_pool(pool, P, block, dtype):
    """Oracle codes and scales of a bf16 pool [NL, slots, H, D]."""
    NL, slots, H, D = pool.shape
    x = K8_values(pool).reshape(NL, slots // block, block, H, D)
    amax = np.abs(x).max(axis=(2, 4))  # [NL, slots / block, H]
    need = np.vectorize(lambda a: K8.need(a, dtype))(amax)
    codes = K8.encode(x / need[:, :, None, :, None], dtype).reshape(NL, slots, H, D)
    s = need.reshape(NL, slots // P, P // block, H).transpose(0, 1, 3, 2)
    return codes, np.ascontiguousarray(s).astype(np.float32)


def K8_values(t):
    return R.bf16_bits_to_f64(R.tensor_bits(t))


class Problem:
    """A DecodeProblem with 8-bit pools: self.k, self.v are oracle caches."""

    def __init__(self, p: W.DecodeProblem, dtype, block):
        self.p, self.dtype, self.block = p, dtype, block
        self.k, self.v = (K8.Cache(*quantise_pool(x, p.page_size, block, dtype), p.page_size,
                                   block, dtype) for x in (p.k_pool, p.v_pool))

    def slots(self, b, lo, hi):
        p = self.p
        row = p.page_table[int(p.req_pool_indices[b])].numpy()
        t = np.arange(lo, hi)
        return row[t // p.page_size].astype(np.int64) * p.page_size + t % p.page_size

    def device(self, max_splits=1, device="cuda", max_batch=None):
        """(workspace, cache) with this problem's state, metadata bound as it is."""
        from paged_kv_decode_bind_gb300 import Kv8Cache, Workspace
        from paged_kv_decode_bind_gb300 import _abi as A
        p = self.p
        ws = Workspace(n_layers=p.n_layers, pool_slots=p.pool_slots, n_q_heads=p.n_q_heads,
                       n_kv_heads=p.n_kv_heads, head_dim=p.head_dim, page_size=p.page_size,
                       max_batch=max_batch or p.batch, max_reqs=p.max_reqs,
                       max_pages_per_req=p.max_pages_per_req, max_splits=max_splits,
                       max_total_tokens=(p.batch * p.max_pages_per_req
                                         if p.page_size == 1 else 0),
                       index_mode=p.index_mode, device=device, pools=False)
        ws.page_table.copy_(p.page_table)
        ws.req_pool_indices[:p.batch].copy_(p.req_pool_indices)
        ws.seq_lens[:p.batch].copy_(p.seq_lens)
        t = lambda x: torch.from_numpy(x.copy()).to(ws.device)  # noqa: E731
        cache = Kv8Cache(ws, dtype=self.dtype, scale_block=self.block, k_pool=t(self.k.codes),
                         v_pool=t(self.v.codes), k_scale=t(self.k.scales),
                         v_scale=t(self.v.scales))
        if ws.device.type == "cuda":
            A.pkv_bind_step(ws, p.batch, A.PKV_BIND_REBUILD)
        return ws, cache

    def attention(self, layer, q, lens):
        """Oracle outputs of every request and the bounds on their errors."""
        q = K8_values(q)
        outs, lses, bo, bl = [], [], [], []
        for b, n in enumerate(lens):
            s = self.slots(b, 0, n)
            o, lse, mass, size, floor = K8.attention(
                q[b], self.k.rows(layer, s), self.v.rows(layer, s), self.p.scale,
                self.v.scale_of(layer, s))
            # score: D products and sums in fp32 plus the two scalings; weight: the
            # exponential of a score off by that (and by a few fp32 steps of its
            # own argument, at most |score|), then one rounding to fp16
            ds = (self.p.head_dim + 8) * EPS32 * size
            dw = 2.0 ** -11 + 2 * ds + 2.0 ** -20
            outs.append(o)
            lses.append(lse)
            # numerator and denominator both carry the weights' error.  A weight
            # p_t v_scale_t below fp16's normal range is off by half its smallest
            # step, 2^-25, in a unit in which the largest weight of the warp is at
            # least 2^7 (so at most 2^-32 of the request's largest weight): over all
            # tokens that is 2^-32 max_t(p_t v_scale_t) sum_t |code_t|
            bo.append(2 * dw[:, None] * mass + 2.0 ** -32 * floor)
            bl.append(2 * ds + 2.0 ** -20 + 4 * EPS32 * np.abs(np.where(np.isfinite(lse), lse, 0)))
        return np.stack(outs), np.stack(lses), np.stack(bo), np.stack(bl)


def check_attention(got, lse, ref, what, out_step):
    """got, lse against ref = Problem.attention(...): out_step is half a step of
    the output type, relative."""
    o, l, bo, bl = ref
    err = np.abs(got - o) - (bo + out_step * (np.abs(o) + bo) + 1e-30)
    assert np.all(np.isfinite(got)), what
    assert err.max() <= 0, f"{what}: {err.max():.3e} past the bound"
    if lse is not None:
        dead = np.isneginf(l)
        assert np.array_equal(np.isneginf(lse), dead), what
        e = np.abs(np.where(dead, 0, lse) - np.where(dead, 0, l)) - bl
        assert e.max() <= 0, f"{what}: lse {e.max():.3e} past the bound"
