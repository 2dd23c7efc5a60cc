"""The 8-bit KV cache beside a workspace, and the attention paths over it.

``Kv8Cache`` owns the codes and block scales of ``pkv_kv8`` for one
workspace.  A decode step appends and attends through ``pkv_kv8_decode_layer``
(``DecodeRunner(..., cache=...)`` runs whole steps).  A chunk of new tokens goes
through ``Kv8Extender``: append to the 8-bit cache, the whole context read back
as bf16 pages, and ``pkv_extend_attn`` over those pages.
"""
from __future__ import annotations

import torch

from . import _abi

DTYPES = {"e4m3": _abi.PKV_KV8_E4M3, "int8": _abi.PKV_KV8_INT8}


class Kv8Cache:
    """Codes [NL, slots, Hkv, D] and scales [NL, slots / P, Hkv, P / scale_block].

    Existing uint8 and fp32 tensors of those shapes may be given (for example
    a cache that was saved); new ones start as zeros under the
    smallest scale, so that rows never written count as zeros.  A workspace built
    with ``pools=False`` has no bf16 pools to pay for.  A call with a workspace of
    other shapes raises ValueError."""

    def __init__(self, ws, *, dtype="e4m3", scale_block=None, k_pool=None, v_pool=None,
                 k_scale=None, v_scale=None):
        if dtype not in DTYPES:
            raise ValueError(f"dtype is one of {sorted(DTYPES)}")
        sh = ws.shape
        P, H, D = sh["page_size"], sh["n_kv_heads"], sh["head_dim"]
        if scale_block is None:
            scale_block = next(b for b in (16, 8, 4, 2, 1) if P % b == 0)
        if not 1 <= scale_block <= 128 or P % scale_block:
            raise ValueError("scale_block is 1 .. 128 and divides the page size")
        home = torch.empty(0, device=ws.device).device  # "cuda" with its index
        codes = (sh["n_layers"], sh["pool_slots"], H, D)
        scales = (sh["n_layers"], sh["pool_slots"] // P, H, P // scale_block)

        def own(x, shape, dt):
            if x is None:
                return torch.full(shape, 2.0 ** -100 if dt.is_floating_point else 0, dtype=dt,
                                  device=ws.device)
            if tuple(x.shape) != shape or x.dtype != dt or not x.is_contiguous() or \
                    x.device != home:
                raise ValueError(f"expected a dense {dt} tensor of {shape} on {ws.device}")
            return x

        self.dtype, self.scale_block, self.device = dtype, scale_block, ws.device
        self.pool_shape = ws.pool_shape  # calls hold it against their workspace's
        self.k_pool, self.v_pool = (own(x, codes, torch.uint8) for x in (k_pool, v_pool))
        self.k_scale, self.v_scale = (own(x, scales, torch.float32) for x in (k_scale, v_scale))
        self.struct = _abi.PkvKv8(
            dtype=DTYPES[dtype], scale_block=scale_block, k_pool=self.k_pool.data_ptr(),
            v_pool=self.v_pool.data_ptr(), k_scale=self.k_scale.data_ptr(),
            v_scale=self.v_scale.data_ptr())


def check_cache(ws, cache):
    """Raise ValueError unless the cache is one of this workspace's shapes and device."""
    _abi._kv8(ws, cache)
    if isinstance(cache, Kv8Cache) and cache.k_pool.device != ws.err.device:
        raise ValueError(f"the cache is on {cache.k_pool.device}, the workspace on {ws.err.device}")


class Kv8Extender:
    """A chunk of new tokens per request on the 8-bit cache, layer by layer:
    append, the contexts read back as bf16 pages, causal attention over those
    (``pkv_extend_attn``).  The reading moves three times the cache's bytes:
    with the append 13 of a layer's 58 us for 4 chunks of 256 tokens on 917 to 2270.

    Contexts hold at most max_context tokens (longer ones raise PKV_DEVERR_LEN),
    chunks at most max_new.  Every buffer is allocated here once, so calls of one
    extender run one after the other (on one stream, or ordered by the caller)."""

    # Not PKV_FLAG_WRITE_LSE: ws.lse has a row per request, not per new token.
    EXTEND_FLAGS = (_abi.PKV_FLAG_OUT_F32 | _abi.PKV_FLAG_EXTEND_FULL |
                    _abi.PKV_FLAG_EXTEND_WARP_MMA)

    def __init__(self, ws, cache, batch, *, max_new, max_context, scale, num_splits=1):
        sh = ws.shape
        H, Hq, D = sh["n_kv_heads"], sh["n_q_heads"], sh["head_dim"]
        if not 0 < batch <= sh["max_batch"]:
            raise ValueError("batch must be in 1 .. the workspace's max_batch")
        if max_new < 1 or max_context < 1 or num_splits < 1:
            raise ValueError("max_new, max_context and num_splits start at 1")
        check_cache(ws, cache)
        # no context is longer than its table row
        max_context = min(max_context, sh["max_pages_per_req"] * sh["page_size"])
        dev = ws.device
        room = -(-max_context // 16) * 16  # rows per request: whole 16-token pages
        i32 = dict(dtype=torch.int32, device=dev)
        self.ws, self.cache, self.batch, self.max_new = ws, cache, batch, max_new
        self.scale, self.num_splits, self.n_rows = scale, num_splits, batch * room
        self.k_rows = torch.zeros((1, batch * room, H, D), dtype=torch.bfloat16, device=dev)
        self.v_rows = torch.zeros_like(self.k_rows)
        self.first_row = torch.arange(batch, **i32) * room
        self.table = torch.arange(batch * room // 16, **i32).view(batch, room // 16)
        self.requests = torch.arange(batch, **i32)
        rows = batch * max_new * num_splits if num_splits > 1 else 1
        self.part_o = torch.zeros(rows * Hq * D, dtype=torch.float32, device=dev)
        self.part_ml = torch.zeros(rows * Hq * 2, dtype=torch.float32, device=dev)
        # the 8-bit cache with lengths held to the room a request has
        self.read_view = _abi.PkvWorkspace.from_buffer_copy(ws.struct)
        limit = ws.struct.max_seq_len
        self.read_view.max_seq_len = min(max_context, limit) if limit > 0 else max_context
        # the rows as a bf16 pool of one layer, request b's pages in row b
        v = _abi.PkvWorkspace.from_buffer_copy(self.read_view)
        v.n_layers, v.pool_slots, v.page_size = 1, batch * room, 16
        v.index_mode, v.max_reqs, v.max_pages_per_req = _abi.PKV_IDX_PAGE_TABLE, batch, room // 16
        v.max_batch, v.max_splits = batch * max_new, num_splits
        v.k_pool, v.v_pool = self.k_rows.data_ptr(), self.v_rows.data_ptr()
        v.page_table, v.req_pool_indices = self.table.data_ptr(), self.requests.data_ptr()
        v.o_part, v.ml_part, v.lse = self.part_o.data_ptr(), self.part_ml.data_ptr(), None
        self.rows_view = v

    def layer(self, layer, qo_indptr, max_qo_len, q, k_new, v_new, out, flags=0, stream=None):
        """Rows q, k_new, v_new [total, heads, D] of the new tokens (offsets
        qo_indptr, as pkv_extend_attn) into out [total, Hq, D]; ws.seq_lens count
        the new tokens, and flat indices are bound (PKV_BIND_REBUILD).
        flags: those of EXTEND_FLAGS, with pkv_extend_attn's meaning; the permission
        of PKV_FLAG_PLAN_EARLY is not used (the launch before the attention writes
        the rows it reads)."""
        if max_qo_len > self.max_new:
            raise ValueError("max_qo_len exceeds max_new")
        flags &= ~_abi.PKV_FLAG_PLAN_EARLY
        if flags & ~self.EXTEND_FLAGS:
            raise ValueError("flags: PKV_FLAG_OUT_F32, _EXTEND_FULL, _EXTEND_WARP_MMA")
        _abi.pkv_kv8_extend_append(self.read_view, self.cache, self.batch, layer, qo_indptr,
                                   max_qo_len, k_new, v_new, stream)
        _abi.pkv_kv8_read(self.read_view, self.cache, self.batch, layer, None, self.first_row,
                          self.n_rows, self.k_rows, self.v_rows,
                          # the append, if there is one, is the previous launch
                          _abi.PKV_FLAG_PLAN_EARLY if max_qo_len else 0, stream)
        _abi.pkv_extend_attn(self.rows_view, self.batch, 0, qo_indptr, max_qo_len, q, out,
                             self.scale, self.num_splits, flags, stream)


class QkNormRope:
    """Arguments of ``pkv_qk_norm_rope`` with the tensors they point at.

    cos_sin: fp32 [positions, rot_dim], cosines then sines (``rope_table``);
    q_weight / k_weight: bf16 [D] or None (that side is not normalised)."""

    def __init__(self, *, n_q_heads, n_kv_heads, head_dim, rot_dim=None, cos_sin=None,
                 q_weight=None, k_weight=None, eps=1e-6, interleaved=False, err=None):
        rot_dim = head_dim if rot_dim is None else rot_dim
        for w in (q_weight, k_weight):
            if w is not None and (w.dtype != torch.bfloat16 or tuple(w.shape) != (head_dim,) or
                                  not w.is_contiguous()):
                raise ValueError("weights are dense bf16 [head_dim]")
        if rot_dim and (cos_sin is None or cos_sin.dtype != torch.float32 or
                        cos_sin.dim() != 2 or cos_sin.shape[1] != rot_dim or
                        not cos_sin.is_contiguous()):
            raise ValueError("cos_sin is dense fp32 [positions, rot_dim]")
        homes = {x.device for x in (cos_sin, q_weight, k_weight, err) if x is not None}
        if len(homes) > 1:
            raise ValueError(f"the tensors are on several devices: {sorted(map(str, homes))}")
        if err is None:
            err = torch.zeros(1, dtype=torch.int32, device=homes.pop() if homes else "cuda")
        elif err.dtype != torch.int32 or err.numel() < 1:
            raise ValueError("err is an int32 tensor")
        self.err = err
        self.cos_sin, self.q_weight, self.k_weight = cos_sin, q_weight, k_weight
        self.widths = (head_dim, n_q_heads * head_dim, n_kv_heads * head_dim)  # of a token's rows
        self.struct = _abi.PkvQkNormRopeArgs(
            n_q_heads=n_q_heads, n_kv_heads=n_kv_heads, head_dim=head_dim, rot_dim=rot_dim,
            max_positions=0 if not rot_dim else cos_sin.shape[0], interleaved=int(interleaved),
            eps=eps, reserved=0, q_weight=_abi._ptr(q_weight), k_weight=_abi._ptr(k_weight),
            cos_sin=_abi._ptr(cos_sin) if rot_dim else None, err=self.err.data_ptr())


class QkNormRopeAxes:
    """Arguments of ``pkv_qk_norm_rope_axes``: a QkNormRope whose pairs follow several
    axes (time, height, width).

    axis_of_pair: the axis of each of the rot_dim / 2 pairs, or sections: how many pairs
    in a row each axis has, as (16, 24, 24).  Neither: one axis.
    rows, evicted, delta: int32 device tensors; a token's positions move by
    evicted[rows[t]] + delta[rows[t]] (either may be None).  In a decode step rows is
    ws.req_pool_indices and evicted a Tally's, so that the position is the count of all the
    request's tokens; delta is what its images took from that.  Other arguments are
    QkNormRope's."""

    def __init__(self, *, axis_of_pair=None, sections=None, rows=None, evicted=None, delta=None,
                 **norm):
        self.norm = QkNormRope(**norm)
        self.args, self.err, self.widths = self.norm.struct, self.norm.err, self.norm.widths
        pairs = self.args.rot_dim // 2
        if axis_of_pair is not None and sections is not None:
            raise ValueError("axis_of_pair or sections, not both")
        if sections is not None:
            axis_of_pair = [a for a, n in enumerate(sections) for _ in range(n)]
        elif axis_of_pair is None:
            axis_of_pair = [0] * pairs
        axis_of_pair = [int(a) for a in axis_of_pair]
        if len(axis_of_pair) != pairs or any(not 0 <= a < 4 for a in axis_of_pair):
            raise ValueError(f"an axis 0 .. 3 for each of {pairs} pairs")
        shifts = [x for x in (evicted, delta) if x is not None]
        if (rows is None) != (not shifts):
            raise ValueError("rows goes with evicted or delta")
        for x in [rows] * (rows is not None) + shifts:
            if x.dtype != torch.int32 or x.dim() != 1 or not x.is_contiguous():
                raise ValueError("rows, evicted and delta are dense int32 vectors")
            if x.device != self.err.device:
                raise ValueError(f"the tensors are on {x.device} and {self.err.device}")
        if len({x.numel() for x in shifts}) > 1:
            raise ValueError("evicted and delta are of one length")
        self.rows, self.evicted, self.delta = rows, evicted, delta
        self.max_tokens = rows.numel() if rows is not None else 2 ** 31 - 1
        n_axes = len(sections) if sections is not None else max(axis_of_pair, default=0) + 1
        self.axes = _abi.PkvRopeAxes(
            n_axes=n_axes, n_rows=shifts[0].numel() if shifts else 0, rows=_abi._ptr(rows),
            evicted=_abi._ptr(evicted), delta=_abi._ptr(delta),
            axis=(_abi.ctypes.c_uint8 * 128)(*axis_of_pair))


def rope_table(positions: int, rot_dim: int, base: float = 10000.0, device="cuda"):
    """cos_sin of positions 0 .. positions - 1: angle p * base^(-2 i / rot_dim) of
    pair i, taken in 64 bits (a far position's angle loses its fraction in 32)."""
    i = torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device)
    a = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * \
        base ** (-i / rot_dim)[None]
    return torch.cat([a.cos(), a.sin()], 1).float().contiguous()
