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
    a cache that was saved); new ones start as zeros.  A workspace built with
    ``pools=False`` has no bf16 pools to pay for."""

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
        codes = (sh["n_layers"], sh["pool_slots"], H, D)
        scales = (sh["n_layers"], sh["pool_slots"] // P, H, P // scale_block)

        def own(x, shape, dt):
            if x is None:
                return torch.zeros(shape, dtype=dt, device=ws.device)
            if tuple(x.shape) != shape or x.dtype != dt or not x.is_contiguous() or \
                    x.device.type != ws.device.type:
                raise ValueError(f"expected a dense {dt} tensor of {shape} on {ws.device}")
            return x

        self.dtype, self.scale_block, self.device = dtype, scale_block, ws.device
        self.k_pool, self.v_pool = (own(x, codes, torch.uint8) for x in (k_pool, v_pool))
        self.k_scale, self.v_scale = (own(x, scales, torch.float32) for x in (k_scale, v_scale))
        self.struct = _abi.PkvKv8(
            dtype=DTYPES[dtype], scale_block=scale_block, k_pool=self.k_pool.data_ptr(),
            v_pool=self.v_pool.data_ptr(), k_scale=self.k_scale.data_ptr(),
            v_scale=self.v_scale.data_ptr())


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
        device = next((x.device for x in (cos_sin, q_weight, k_weight) if x is not None), "cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device=device) if err is None else err
        self.cos_sin, self.q_weight, self.k_weight = cos_sin, q_weight, k_weight
        self.struct = _abi.PkvQkNormRopeArgs(
            n_q_heads=n_q_heads, n_kv_heads=n_kv_heads, head_dim=head_dim, rot_dim=rot_dim,
            max_positions=0 if not rot_dim else cos_sin.shape[0], interleaved=int(interleaved),
            eps=eps, reserved=0, q_weight=_abi._ptr(q_weight), k_weight=_abi._ptr(k_weight),
            cos_sin=_abi._ptr(cos_sin) if rot_dim else None, err=self.err.data_ptr())


def rope_table(positions: int, rot_dim: int, base: float = 10000.0, device="cuda"):
    """cos_sin of positions 0 .. positions - 1: angle p * base^(-2 i / rot_dim) of
    pair i, taken in 64 bits (a far position's angle loses its fraction in 32)."""
    i = torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device)
    a = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * \
        base ** (-i / rot_dim)[None]
    return torch.cat([a.cos(), a.sin()], 1).float().contiguous()
