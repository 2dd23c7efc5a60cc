"""One decode step over every layer, as the engine's executor runs it.

Step = metadata bind once (cache.py page, bullets 25-28), then for each layer
the KV append (cache.py page, bullet 40), split-KV decode attention and the
partial merge (workspace.py page, bullets 1 and 14).  Inputs live in static
buffers owned by the runner so a whole step can be captured once into a CUDA
graph and replayed at fixed addresses (workspace.py page, bullets 6-7; one
graph per batch size, executor.py page, bullets 4-5, 7-8).
"""
from __future__ import annotations

import torch

from . import _abi
from .kv8 import QkNormRopeAxes, check_cache
from .tally import check_tally
from .workspace import Workspace


def _norm_struct(r):
    return r.args if isinstance(r, QkNormRopeAxes) else r.struct


class _AxesArgs:
    """What pkv_qk_norm_rope_axes takes of a QkNormRopeAxes, with the step's error word."""

    def __init__(self, args, axes, widths, max_tokens):
        self.args, self.axes, self.widths, self.max_tokens = args, axes, widths, max_tokens


class BindTracker:
    """Host record of the last bind (the engine's _BindState; cache.py page,
    bullets 1-4): picks STEADY when the same tasks each grew by one token."""

    def __init__(self):
        self.ids = None
        self.lens = None

    def mode(self, ids, lens):
        steady = _abi.pkv_is_steady_increment(self.ids, self.lens, list(ids), list(lens))
        self.ids, self.lens = list(ids), list(lens)
        return _abi.PKV_BIND_STEADY if steady else _abi.PKV_BIND_REBUILD

    def evicted(self, eviction):
        """The step cut its requests past the limit (an Eviction): their next lengths
        follow on the shorter ones."""
        if self.lens is not None:
            self.lens = [eviction.length(n) for n in self.lens]


class DecodeRunner:
    """Drives libpkv for one batch size on one stream."""

    def __init__(self, ws: Workspace, batch: int, *, num_splits: int = 1, flags: int = 0,
                 scale: float | None = None, stream: torch.cuda.Stream | None = None,
                 fused: bool = True, plan: bool = False, out_per_layer: bool = False,
                 cache=None, norm_rope=None, tally=None, evict=None):
        """cache: a Kv8Cache of this workspace; the layers then append to and
        attend over it instead of the bf16 pools (flags: PKV_FLAG_OUT_F32 and
        PKV_FLAG_WRITE_LSE).  norm_rope: a QkNormRope, or one per layer, applied
        to the layer's q and k at ws.position_ids before they are used (its arguments
        are copied here); a step's device errors all go to ws.err, the norm's too,
        whatever its own word is.  A QkNormRopeAxes takes ws.position_ids on every axis,
        moved by its own evicted and delta (rows: ws.req_pool_indices).
        tally: a Tally of this workspace; the layers add their attention weights to it
        (fused layers on the bf16 pools).  evict: an Eviction that ends every step; a
        norm_rope then has to be a QkNormRopeAxes with evicted=tally.evicted, as a token's
        position is no longer its index."""
        if cache is not None and (not fused or plan):
            raise ValueError("a step on the 8-bit cache has no unfused or planned form")
        if cache is not None:
            check_cache(ws, cache)
        if tally is not None and (cache is not None or not fused):
            raise ValueError("the tally is of fused layers on the bf16 pools")
        if evict is not None and tally is None:
            raise ValueError("an eviction needs a tally")
        if tally is not None:
            check_tally(ws, tally, batch)
        self.tally, self.evict = tally, evict
        self.cache = cache
        self.ws = ws
        self.batch = batch
        sh = ws.shape
        self.num_splits = num_splits
        self.flags = flags
        self.scale = scale if scale is not None else sh["head_dim"] ** -0.5
        self.stream = stream
        NL, B = sh["n_layers"], batch
        dev = ws.device
        self.q_in = torch.zeros((NL, B, sh["n_q_heads"], sh["head_dim"]), dtype=torch.bfloat16,
                                device=dev)
        self.k_in = torch.zeros((NL, B, sh["n_kv_heads"], sh["head_dim"]), dtype=torch.bfloat16,
                                device=dev)
        self.v_in = torch.zeros_like(self.k_in)
        self.norm_rope = None
        if norm_rope is not None:
            self.norm_rope = (list(norm_rope) if isinstance(norm_rope, (list, tuple))
                              else [norm_rope] * NL)
            if len(self.norm_rope) != NL or any(
                    (st.n_q_heads, st.n_kv_heads, st.head_dim) !=
                    (sh["n_q_heads"], sh["n_kv_heads"], sh["head_dim"])
                    for st in map(_norm_struct, self.norm_rope)):
                raise ValueError("norm_rope: one QkNormRope of the workspace's heads per layer")
            axes = [r for r in self.norm_rope if isinstance(r, QkNormRopeAxes)]
            if any(r.rows is not None and r.rows.data_ptr() != ws.req_pool_indices.data_ptr()
                   for r in axes):
                raise ValueError("norm_rope: rows are the workspace's req_pool_indices")
            if evict is not None and (len(axes) != NL or any(
                    r.evicted is None or r.evicted.data_ptr() != tally.evicted.data_ptr()
                    for r in axes)):
                raise ValueError("a step that evicts takes its positions by a QkNormRopeAxes with "
                                 "evicted=tally.evicted")
            if any(r.err.device != ws.err.device for r in self.norm_rope):
                raise ValueError("norm_rope: its tensors are not on the workspace's device")
            self.rope_args = []
            for r in self.norm_rope:
                args = _abi.PkvQkNormRopeArgs.from_buffer_copy(_norm_struct(r))
                args.err, args.widths = ws.err.data_ptr(), r.widths
                if isinstance(r, QkNormRopeAxes):
                    args = _AxesArgs(args, r.axes, r.widths, r.max_tokens)
                self.rope_args.append(args)
            # one layer's rows at a time: the next layer's kernel waits for this one's
            self.q_use = torch.zeros_like(self.q_in[0])
            self.k_use = torch.zeros_like(self.k_in[0])
        # out_per_layer: every layer writes its own output rows (layer l's into
        # outs[l], through a copy of the workspace struct whose `out` points
        # there), so a step leaves all its layers' results behind instead of
        # the last one's in ws.out.  bf16, or fp32 with PKV_FLAG_OUT_F32.
        self.outs = None
        self.views = None
        if out_per_layer:
            odt = torch.float32 if flags & _abi.PKV_FLAG_OUT_F32 else torch.bfloat16
            self.outs = torch.zeros((NL, B, sh["n_q_heads"], sh["head_dim"]), dtype=odt,
                                    device=dev)
            self.views = []
            for l in range(NL):
                v = _abi.PkvWorkspace.from_buffer_copy(ws.struct)
                v.out = self.outs[l].data_ptr()
                self.views.append(v)
        self.graph = None
        self.fused = fused
        flat = sh["index_mode"] == _abi.PKV_IDX_FLAT
        # kernels one step launches: bind (+ flat index build), then per layer
        # one fused kernel, or append + attention (+ merge when split)
        split = num_splits > 1
        mma = (not (flags & _abi.PKV_FLAG_FORCE_SIMT) and sh["head_dim"] in (64, 128)
               and sh["n_q_heads"] // sh["n_kv_heads"] in (1, 2, 4, 8, 16))
        # plan=True: the fused layers take the step's split plan, made once after
        # the bind (pkv_plan_step).  Off by default: with the layers pipelined by
        # programmatic dependent launch the plan saves no time, and a one-layer
        # step pays for the extra launch.
        self.use_plan = plan and fused and mma and ws.work_plan is not None
        if cache is not None or tally is not None:
            # append, attention (with its merge); or that and the weights' addition
            per_layer = 2
        else:
            per_layer = 1 if fused and mma else 2 + int(split)
        per_layer += int(self.norm_rope is not None)
        self.launches_per_step = (1 + int(flat) + int(self.use_plan and 0 < batch <= 256) +
                                  NL * per_layer + int(evict is not None))
        # the most that a request of this step may hold, for the eviction's launch
        most = evict.bound if evict is not None else _abi.PKV_TALLY_MAX_LEN
        self.evict_len = min(sh["max_pages_per_req"] * sh["page_size"], most)

    def _wsl(self, l):
        return self.views[l] if self.views is not None else self.ws

    # --- pieces -------------------------------------------------------------
    def bind(self, mode=_abi.PKV_BIND_STEADY):
        _abi.pkv_bind_step(self.ws, self.batch, mode, 0, 0, None, None, self._s())
        if self.use_plan:
            _abi.pkv_plan_step(self.ws, self.batch, self.num_splits, self.flags, self._s())

    def layer(self, l, events=None):
        """Layer l: one fused launch (append + attention + merge), or the
        three separate kernels when built with fused=False, or the 8-bit cache's
        append and attention; the norm with rotation first where there is one."""
        s = self._s()
        q, k = self.q_in[l], self.k_in[l]
        if self.norm_rope is not None:
            call = (_abi.pkv_qk_norm_rope_axes if isinstance(self.rope_args[l], _AxesArgs)
                    else _abi.pkv_qk_norm_rope)
            call(self.rope_args[l], self.batch, q, k, self.ws.position_ids, self.q_use,
                 self.k_use, s)
            q, k = self.q_use, self.k_use
        if self.cache is not None:
            if events is not None:
                events[0].record(s)
            # as below: what a layer after the first reads early is older
            early = _abi.PKV_FLAG_PLAN_EARLY if (l > 0 and events is None) else 0
            _abi.pkv_kv8_decode_layer(self._wsl(l), self.cache, self.batch, l, q, k, self.v_in[l],
                                      self.scale, self.num_splits, self.flags | early, s)
            if events is not None:
                events[1].record(s)
            return
        if self.fused:
            if events is not None:
                events[0].record(s)
            # Layers after the first read metadata the step's bind wrote two or
            # more launches earlier, so they may start before layer l-1 ends.
            early = _abi.PKV_FLAG_PLAN_EARLY if (l > 0 and events is None) else 0
            use = _abi.PKV_FLAG_USE_PLAN if self.use_plan else 0
            if self.tally is not None:
                _abi.pkv_tally_decode_layer(self._wsl(l), self.tally, self.batch, l, q, k,
                                            self.v_in[l], self.scale, self.num_splits,
                                            self.flags | early | use, s)
            else:
                _abi.pkv_decode_layer(self._wsl(l), self.batch, l, q, k, self.v_in[l], self.scale,
                                      self.num_splits, self.flags | early | use, s)
            if events is not None:
                events[1].record(s)
            return
        _abi.pkv_bind_step(self.ws, self.batch, _abi.PKV_BIND_APPEND_ONLY, l, 1, k, self.v_in[l], s)
        if events is not None:
            events[0].record(s)
        _abi.pkv_decode_attn(self._wsl(l), self.batch, l, q, self.scale, self.num_splits,
                             self.flags, s)
        if events is not None:
            events[1].record(s)
        if self.num_splits > 1:
            _abi.pkv_merge_partials(self._wsl(l), self.batch, self.num_splits, self.flags, s)

    def step(self, mode=_abi.PKV_BIND_STEADY, layer_events=None):
        """Bind, then every layer.  ``layer_events[l]`` = (start, end) CUDA
        events recorded around that layer's attention kernel."""
        self.bind(mode)
        for l in range(self.ws.shape["n_layers"]):
            self.layer(l, None if layer_events is None else layer_events[l])
        if self.evict is not None:
            e = self.evict
            _abi.pkv_tally_evict(self.ws, self.tally, self.batch, self.evict_len, e.limit, e.budget,
                                 e.sinks, e.recent, self._s())

    # --- CUDA graph -----------------------------------------------------------
    def capture(self, mode=_abi.PKV_BIND_STEADY, layer_events=None):
        """Capture one whole step (bind + all layers) into a CUDA graph.

        ``layer_events[l]`` (events made with ``external=True``) become event
        record nodes around layer l's attention kernel."""
        g = torch.cuda.CUDAGraph()
        side = torch.cuda.Stream(device=self.ws.device)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            with torch.cuda.graph(g, stream=side):
                self.step(mode, layer_events)
        torch.cuda.current_stream().wait_stream(side)
        self.graph = g
        return g

    def replay(self):
        self.graph.replay()

    def _s(self):
        if self.stream is not None:
            return self.stream
        return torch.cuda.current_stream()
