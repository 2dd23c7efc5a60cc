"""The tally of attention weight beside a workspace, and what it decides.

``Tally`` owns the buffers of ``pkv_tally``.  A chunk of a prompt goes through
``TallyExtender`` (append, attention, the tally of its last queries); a decode step through
``DecodeRunner(..., tally=..., evict=Eviction(...))``, which tallies in every layer and cuts
requests past the limit at its end.  The page table, and with it every attention call of the
library, stays as it is: kept tokens move together into a request's first indices.
"""
from __future__ import annotations

import dataclasses

import torch

from . import _abi


class Tally:
    """weight (fp32) and origin (int32) [NL, slots / P, Hkv, P], evicted int32 [max_reqs].

    Existing tensors of those shapes may be given; new ones start as zeros.  A request that
    takes a table row over starts with evicted[row] = 0 (``take_rows``).  The scratch of a
    decode layer's scores is sized for every request at the most it may hold: two captured
    graphs that run at the same time need a tally each, as they need a workspace each.  A
    call with a workspace of other shapes raises ValueError."""

    def __init__(self, ws, *, weight=None, origin=None, evicted=None):
        sh, st = ws.shape, ws.struct
        P, H = sh["page_size"], sh["n_kv_heads"]
        home = torch.empty(0, device=ws.device).device  # "cuda" with its index
        entries = (sh["n_layers"], sh["pool_slots"] // P, H, P)

        def own(x, shape, dt):
            if x is None:
                return torch.zeros(shape, dtype=dt, device=ws.device)
            if tuple(x.shape) != shape or x.dtype != dt or not x.is_contiguous() or \
                    x.device != home:
                raise ValueError(f"expected a dense {dt} tensor of {shape} on {ws.device}")
            return x

        self.device, self.max_batch = ws.device, sh["max_batch"]
        self.shape = (sh["n_layers"], sh["pool_slots"], sh["n_q_heads"], H, P, sh["max_reqs"])
        self.weight = own(weight, entries, torch.float32)
        self.origin = own(origin, entries, torch.int32)
        self.evicted = own(evicted, (sh["max_reqs"],), torch.int32)
        room = sh["max_pages_per_req"] * P
        if st.max_seq_len > 0:
            room = min(room, st.max_seq_len)
        self.score = torch.zeros((sh["max_batch"], H, room, sh["n_q_heads"] // H),
                                 dtype=torch.float32, device=ws.device)
        self.struct = _abi.PkvTally(weight=self.weight.data_ptr(), origin=self.origin.data_ptr(),
                                    evicted=self.evicted.data_ptr(), score=self.score.data_ptr(),
                                    score_tokens=room, reserved=0)

    def take_rows(self, rows):
        """New requests take these table rows (an int64 or int32 tensor, or a list)."""
        if not isinstance(rows, torch.Tensor):
            rows = torch.tensor(rows, device=self.evicted.device)
        self.evicted[rows.long()] = 0


def check_tally(ws, tally, batch=0):
    """Raise ValueError unless the tally is one of this workspace's shapes and device."""
    _abi._tally(ws, tally, batch)
    if isinstance(tally, Tally) and tally.weight.device != ws.err.device:
        raise ValueError(f"the tally is on {tally.weight.device}, the workspace on "
                         f"{ws.err.device}")


@dataclasses.dataclass(frozen=True)
class Eviction:
    """Requests of more than `limit` tokens (None: budget) keep `budget`: the first `sinks`
    and the last `recent` of all their tokens, then those of the largest tally.  max_len:
    a bound on the lengths that a step meets (None: what a table row holds, at most
    PKV_TALLY_MAX_LEN); longer requests are left as they are, with PKV_DEVERR_LEN.  It
    settles what the eviction's launch costs: in a decode loop give limit + 1 (24 layers, 16
    requests at their budget of 2048 in rows of 131072 tokens: 822 us a step with it, 1293
    without)."""

    budget: int
    limit: int | None = None
    sinks: int = 0
    recent: int = 0
    max_len: int | None = None

    def __post_init__(self):
        if self.limit is None:
            object.__setattr__(self, "limit", self.budget)
        if self.budget < 1 or self.limit < self.budget or self.sinks < 0 or self.recent < 0 or \
                self.sinks + self.recent > self.budget:
            raise ValueError("1 <= budget <= limit, and budget holds sinks and recent")
        if self.max_len is not None and not self.limit < self.max_len <= _abi.PKV_TALLY_MAX_LEN:
            raise ValueError("max_len is past the limit, at most PKV_TALLY_MAX_LEN")

    @property
    def bound(self) -> int:
        """The most tokens of a request that is cut."""
        return _abi.PKV_TALLY_MAX_LEN if self.max_len is None else self.max_len

    def length(self, n: int) -> int:
        """A request's tokens after the eviction."""
        return self.budget if self.limit < n <= self.bound else n


class TallyExtender:
    """A chunk of new tokens per request, layer by layer: append, causal attention, and the
    tally of the last `window` (None: all) new tokens' weights.

    Chunks hold at most max_new tokens.  Every buffer is allocated here once, so calls of
    one extender run one after the other (on one stream, or ordered by the caller)."""

    EXTEND_FLAGS = _abi.PKV_FLAG_OUT_F32 | _abi.PKV_FLAG_EXTEND_WARP_MMA

    def __init__(self, ws, tally, batch, *, max_new, scale, window=None, num_splits=1):
        sh = ws.shape
        Hq, D = sh["n_q_heads"], sh["head_dim"]
        if not 0 < batch <= sh["max_batch"]:
            raise ValueError("batch must be in 1 .. the workspace's max_batch")
        if max_new < 1 or num_splits < 1 or (window is not None and window < 1):
            raise ValueError("max_new, window and num_splits start at 1")
        check_tally(ws, tally)
        f32 = dict(dtype=torch.float32, device=ws.device)
        self.ws, self.tally, self.batch, self.max_new = ws, tally, batch, max_new
        self.scale, self.num_splits = scale, num_splits
        self.window = max_new if window is None else window
        self.lse = torch.zeros((batch * max_new, Hq), **f32)
        rows = batch * max_new * num_splits if num_splits > 1 else 1
        self.part_o = torch.zeros(rows * Hq * D, **f32)
        self.part_ml = torch.zeros(rows * Hq * 2, **f32)
        # the workspace with room for every new token's log-sum-exp and partials
        v = _abi.PkvWorkspace.from_buffer_copy(ws.struct)
        v.max_batch, v.max_splits = batch * max_new, num_splits
        v.lse, v.o_part, v.ml_part = (x.data_ptr() for x in (self.lse, self.part_o, self.part_ml))
        self.view = v

    def layer(self, layer, qo_indptr, max_qo_len, q, k_new, v_new, out, flags=0, stream=None):
        """Rows q, k_new, v_new [total, heads, D] of the new tokens (offsets qo_indptr, as
        pkv_extend_attn) into out [total, Hq, D]; ws.seq_lens count the new tokens, and
        flat indices are bound (PKV_BIND_REBUILD).  k_new and v_new None: the rows are in
        the cache.  flags: those of EXTEND_FLAGS; the permission of PKV_FLAG_PLAN_EARLY is
        not used (the launch before the attention writes rows it reads)."""
        if max_qo_len > self.max_new:
            raise ValueError("max_qo_len exceeds max_new")
        if (k_new is None) != (v_new is None):
            raise ValueError("k_new and v_new, or neither")
        flags &= ~_abi.PKV_FLAG_PLAN_EARLY
        if flags & ~self.EXTEND_FLAGS:
            raise ValueError("flags: PKV_FLAG_OUT_F32, _EXTEND_WARP_MMA")
        if k_new is not None:
            _abi.pkv_extend_append(self.view, self.batch, layer, qo_indptr, max_qo_len, k_new,
                                   v_new, stream)
        _abi.pkv_extend_attn(self.view, self.batch, layer, qo_indptr, max_qo_len, q, out,
                             self.scale, self.num_splits, flags | _abi.PKV_FLAG_WRITE_LSE, stream)
        _abi.pkv_tally_extend(self.view, self.tally, self.batch, layer, qo_indptr, max_qo_len,
                              min(q.shape[0], self.lse.shape[0]), self.window, q, self.lse,
                              self.scale, stream)
