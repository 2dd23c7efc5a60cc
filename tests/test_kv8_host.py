"""The 8-bit cache and the norm with rotation on the host: struct mirrors, the
argument checks of every entry point (nothing here is launched), the Python
owners' checks, and pins of the 64-bit oracle."""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle.kv8 as K8
import paged_kv_decode_bind_gb300 as P
from paged_kv_decode_bind_gb300 import Kv8Cache, QkNormRope, Workspace, rope_table
from paged_kv_decode_bind_gb300 import _abi as A
from test_abi import _ws

F = 1 << 20  # non-null, aligned, never dereferenced


def _c(**kw):
    d = dict(dtype=0, scale_block=16, k_pool=F, v_pool=F, k_scale=F, v_scale=F)
    d.update(kw)
    return A.PkvKv8(**d)


def test_struct_layouts():
    assert ctypes.sizeof(A.PkvKv8) == 2 * 4 + 4 * 8
    assert ctypes.sizeof(A.PkvQkNormRopeArgs) == 8 * 4 + 4 * 8
    assert A.PkvQkNormRopeArgs.eps.offset == 24


def test_bytes():
    ws, c = _ws(), _c(scale_block=4)
    assert P.pkv_kv8_bytes(ws, c, "k_pool") == 2 * 64 * 2 * 128
    assert P.pkv_kv8_bytes(ws, c, "v_scale") == 2 * 64 // 4 * 2 * 4
    assert P.pkv_kv8_bytes(ws, c, "out") == 0
    assert P.pkv_kv8_bytes(ws, _c(scale_block=3), "k_scale") == 0
    assert P.pkv_kv8_bytes(ws, None, "k_scale") == 0


BAD_CACHES = [
    (dict(), dict(dtype=2), P.PKV_ERR_INVALID),
    (dict(), dict(dtype=-1), P.PKV_ERR_INVALID),
    (dict(), dict(scale_block=0), P.PKV_ERR_INVALID),
    (dict(), dict(scale_block=3), P.PKV_ERR_INVALID),
    (dict(page_size=256, pool_slots=256), dict(scale_block=256), P.PKV_ERR_INVALID),
    (dict(), dict(k_pool=F + 8), P.PKV_ERR_INVALID),
    (dict(), dict(v_pool=None), P.PKV_ERR_INVALID),
    (dict(), dict(k_scale=None), P.PKV_ERR_INVALID),
    (dict(), dict(v_scale=F + 2), P.PKV_ERR_INVALID),
    (dict(head_dim=256), dict(), P.PKV_ERR_UNSUPPORTED),
    (dict(err=None), dict(), P.PKV_ERR_INVALID),
    (dict(pool_slots=60), dict(), P.PKV_ERR_INVALID),
]


@pytest.mark.parametrize("kw,ckw,status", BAD_CACHES)
def test_every_call_checks_the_cache(kw, ckw, status):
    ws, c = _ws(**kw), _c(**ckw)
    kwargs = dict(stream=0, check=False)
    assert P.pkv_kv8_append(ws, c, 1, 0, 1, F, F, **kwargs) == status
    assert P.pkv_kv8_extend_append(ws, c, 1, 0, F, 4, F, F, **kwargs) == status
    assert P.pkv_kv8_read(ws, c, 1, 0, None, F, 4, F, F, **kwargs) == status
    assert P.pkv_kv8_decode_layer(ws, c, 1, 0, F, None, None, 0.1, **kwargs) == status


def test_null_structs():
    kwargs = dict(stream=0, check=False)
    assert P.pkv_kv8_append(_ws(), None, 1, 0, 1, F, F, **kwargs) == P.PKV_ERR_INVALID
    assert P.pkv_kv8_append(None, _c(), 1, 0, 1, F, F, **kwargs) == P.PKV_ERR_INVALID


@pytest.mark.parametrize("batch,l0,nl,k,v,kw,status", [
    (5, 0, 1, F, F, {}, P.PKV_ERR_CAPACITY),
    (-1, 0, 1, F, F, {}, P.PKV_ERR_INVALID),
    (1, 1, 2, F, F, {}, P.PKV_ERR_CAPACITY),
    (1, 0, -1, F, F, {}, P.PKV_ERR_INVALID),
    (1, 0, 1, None, F, {}, P.PKV_ERR_INVALID),
    (1, 0, 1, F, F + 4, {}, P.PKV_ERR_INVALID),
    (1, 0, 1, F, F, dict(out_loc=None), P.PKV_ERR_INVALID),
    (0, 0, 1, F, F, {}, P.PKV_OK),
    (1, 0, 0, None, None, {}, P.PKV_OK),
    (1, 2, 0, None, None, {}, P.PKV_OK),
])
def test_append_checks(batch, l0, nl, k, v, kw, status):
    got = P.pkv_kv8_append(_ws(**kw), _c(), batch, l0, nl, k, v, stream=0, check=False)
    assert got == status


@pytest.mark.parametrize("batch,layer,qo,most,k,v,kw,status", [
    (5, 0, F, 4, F, F, {}, P.PKV_ERR_CAPACITY),
    (1, 2, F, 4, F, F, {}, P.PKV_ERR_CAPACITY),
    (1, 0, None, 4, F, F, {}, P.PKV_ERR_INVALID),
    (1, 0, F, -1, F, F, {}, P.PKV_ERR_INVALID),
    (1, 0, F, 4, F + 8, F, {}, P.PKV_ERR_INVALID),
    (1, 0, F, 4, F, None, {}, P.PKV_ERR_INVALID),
    (1, 0, F, 4, F, F, dict(page_table=None), P.PKV_ERR_INVALID),
    (0, 0, F, 4, F, F, {}, P.PKV_OK),
    (1, 0, F, 0, F, F, {}, P.PKV_OK),
])
def test_extend_append_checks(batch, layer, qo, most, k, v, kw, status):
    got = P.pkv_kv8_extend_append(_ws(**kw), _c(), batch, layer, qo, most, k, v, stream=0,
                                  check=False)
    assert got == status


@pytest.mark.parametrize("batch,layer,dst,n,k,v,flags,status", [
    (5, 0, F, 4, F, F, 0, P.PKV_ERR_CAPACITY),
    (1, -1, F, 4, F, F, 0, P.PKV_ERR_INVALID),
    (1, 2, F, 4, F, F, 0, P.PKV_ERR_CAPACITY),
    (1, 0, None, 4, F, F, 0, P.PKV_ERR_INVALID),
    (1, 0, F, -4, F, F, 0, P.PKV_ERR_INVALID),
    (1, 0, F, 4, F + 2, F, 0, P.PKV_ERR_INVALID),
    (1, 0, F, 4, F, None, 0, P.PKV_ERR_INVALID),
    (1, 0, F, 4, F, F, P.PKV_FLAG_WRITE_LSE, P.PKV_ERR_INVALID),
    (0, 0, F, 4, F, F, P.PKV_FLAG_OUT_F32, P.PKV_OK),
])
def test_read_checks(batch, layer, dst, n, k, v, flags, status):
    got = P.pkv_kv8_read(_ws(), _c(), batch, layer, None, dst, n, k, v, flags, stream=0,
                         check=False)
    assert got == status


@pytest.mark.parametrize("kw,batch,layer,q,k,v,S,flags,status", [
    (dict(), 5, 0, F, None, None, 1, 0, P.PKV_ERR_CAPACITY),
    (dict(), 1, 2, F, None, None, 1, 0, P.PKV_ERR_CAPACITY),
    (dict(), 1, 0, F, None, None, 5, 0, P.PKV_ERR_CAPACITY),
    (dict(), 1, 0, F, None, None, 0, 0, P.PKV_ERR_INVALID),
    (dict(), 1, 0, None, None, None, 1, 0, P.PKV_ERR_INVALID),
    (dict(), 1, 0, F + 8, None, None, 1, 0, P.PKV_ERR_INVALID),
    (dict(), 1, 0, F, F, None, 1, 0, P.PKV_ERR_INVALID),
    (dict(), 1, 0, F, F, F + 8, 1, 0, P.PKV_ERR_INVALID),
    (dict(out_loc=None), 1, 0, F, F, F, 1, 0, P.PKV_ERR_INVALID),
    (dict(out=None), 1, 0, F, None, None, 1, 0, P.PKV_ERR_INVALID),
    (dict(o_part=None), 1, 0, F, None, None, 2, 0, P.PKV_ERR_INVALID),
    (dict(ml_part=F + 4), 1, 0, F, None, None, 2, 0, P.PKV_ERR_INVALID),
    (dict(split_counters=None), 1, 0, F, None, None, 2, 0, P.PKV_ERR_INVALID),
    (dict(lse=None), 1, 0, F, None, None, 1, P.PKV_FLAG_WRITE_LSE, P.PKV_ERR_INVALID),
    (dict(), 1, 0, F, None, None, 1, P.PKV_FLAG_FORCE_SIMT, P.PKV_ERR_INVALID),
    (dict(), 1, 0, F, None, None, 1, P.PKV_FLAG_USE_PLAN, P.PKV_ERR_INVALID),
    (dict(n_q_heads=24), 1, 0, F, None, None, 1, 0, P.PKV_ERR_UNSUPPORTED),  # G = 12
    (dict(n_q_heads=7), 1, 0, F, None, None, 1, 0, P.PKV_ERR_INVALID),
    (dict(seq_lens=None), 1, 0, F, None, None, 1, 0, P.PKV_ERR_INVALID),
    (dict(), 0, 0, F, None, None, 1, 0, P.PKV_OK),
    # the bf16 pools are not needed
    (dict(k_pool=None, v_pool=None), 0, 0, F, None, None, 1, 0, P.PKV_OK),
])
def test_decode_layer_checks(kw, batch, layer, q, k, v, S, flags, status):
    got = P.pkv_kv8_decode_layer(_ws(**kw), _c(), batch, layer, q, k, v, 0.1, S, flags, stream=0,
                                 check=False)
    assert got == status


def _rope(**kw):
    d = dict(n_q_heads=4, n_kv_heads=2, head_dim=128, rot_dim=128, max_positions=10, interleaved=0,
             eps=1e-6, reserved=0, q_weight=F, k_weight=F, cos_sin=F, err=F)
    d.update(kw)
    return A.PkvQkNormRopeArgs(**d)


@pytest.mark.parametrize("kw,status", [
    (dict(n_q_heads=0), P.PKV_ERR_INVALID), (dict(n_kv_heads=-1), P.PKV_ERR_INVALID),
    (dict(head_dim=96), P.PKV_ERR_UNSUPPORTED), (dict(rot_dim=8), P.PKV_ERR_UNSUPPORTED),
    (dict(rot_dim=144), P.PKV_ERR_UNSUPPORTED), (dict(rot_dim=-16), P.PKV_ERR_UNSUPPORTED),
    (dict(eps=-1.0), P.PKV_ERR_INVALID), (dict(eps=math.nan), P.PKV_ERR_INVALID),
    (dict(interleaved=2), P.PKV_ERR_INVALID), (dict(reserved=1), P.PKV_ERR_INVALID),
    (dict(q_weight=F + 2), P.PKV_ERR_INVALID), (dict(cos_sin=None), P.PKV_ERR_INVALID),
    (dict(cos_sin=F + 4), P.PKV_ERR_INVALID), (dict(err=None), P.PKV_ERR_INVALID),
    (dict(max_positions=-1), P.PKV_ERR_INVALID),
])
def test_rope_argument_checks(kw, status):
    got = P.pkv_qk_norm_rope(_rope(**kw), 1, F, F, F, F, F, stream=0, check=False)
    assert got == status


def test_rope_call_checks():
    lib, a = A.load(), ctypes.byref(_rope())
    call = lambda n=1, q=F, qs=512, k=F, ks=256, pos=F, qo=F, qos=512, ko=F, kos=256: \
        lib.pkv_qk_norm_rope(a, n, q, qs, k, ks, pos, qo, qos, ko, kos, None)  # noqa: E731
    bad = [dict(n=-1), dict(q=None), dict(q=F + 8), dict(qs=504), dict(qs=516), dict(k=None),
           dict(ks=248), dict(ks=260), dict(pos=None), dict(qo=None), dict(qos=0), dict(ko=F + 2),
           dict(kos=-256)]
    for kw in bad:
        assert call(**kw) == P.PKV_ERR_INVALID, kw
    assert call(n=0) == P.PKV_OK
    assert lib.pkv_qk_norm_rope(None, 0, F, 512, F, 256, F, F, 512, F, 256, None) == \
        P.PKV_ERR_INVALID


def test_rope_strides_come_from_the_tensors():
    x = torch.zeros((3, 1024), dtype=torch.bfloat16)
    assert A._heads(x[:, :512], 512, 128) == (x.data_ptr(), 1024)
    assert A._heads(x[:, 512:].view(3, 4, 128), 512, 128) == (x.data_ptr() + 1024, 1024)
    assert A._heads(None, 256, 128) == (None, 256)
    with pytest.raises(ValueError):
        A._heads(x[:, ::2], 512, 128)
    with pytest.raises(ValueError):
        A._heads(x.view(3, 8, 128).transpose(0, 1), 1024, 128)


def test_rope_strides_of_one_head_or_token():
    x = torch.zeros((6, 4, 64), dtype=torch.bfloat16)
    one = x[:, :1].transpose(0, 1)[:1]  # [1, 6, 64]: dense heads are 256 apart
    with pytest.raises(ValueError):
        A._heads(one, 384, 64)
    assert A._heads(torch.as_strided(x, (3, 1, 64), (256, 7, 1)), 64, 64)[1] == 256
    assert A._heads(torch.as_strided(x, (1, 256), (1, 1)), 256, 64)[1] == 256
    assert A._heads(torch.as_strided(x, (2, 256), (8, 1)), 256, 64)[1] == 8  # the call refuses it


def test_rope_tensors_that_do_not_fit_are_refused():
    # another type, width, head size or fewer tokens than the call has would be read,
    # or written, as something else
    r = QkNormRope(n_q_heads=4, n_kv_heads=2, head_dim=128,
                   cos_sin=rope_table(9, 128, device="cpu"))
    row = torch.zeros((3, 1024), dtype=torch.bfloat16)
    q, k, pos = row[:, :512], row[:, 512:768], torch.zeros(3, dtype=torch.int32)
    good = dict(q=q, k=k, positions=pos, q_out=q, k_out=k)

    def call(n, **kw):
        a = {**good, **kw}
        return A.pkv_qk_norm_rope(r, n, a["q"], a["k"], a["positions"], a["q_out"], a["k_out"], 0)

    assert call(0) == P.PKV_OK  # nothing is launched for no tokens
    heads = row.view(3, 8, 128)
    assert call(0, q=heads[:, :4], k_out=heads[:, 4:6]) == P.PKV_OK
    for name, n_heads in (("q", 4), ("k", 2), ("q_out", 4), ("k_out", 2)):
        w = n_heads * 128
        for bad in (row[:, :w].float(), row[:, :w].half(), row[:, :w - 128], row[:, :w + 128],
                    row.view(3, 16, 64)[:, :n_heads], row.view(3, 16, 64)[:, :2 * n_heads],
                    heads[:, :n_heads + 1], row[0, :w], row.view(3, 1, 8, 128)[:, :, :n_heads],
                    row[:, :2 * w:2]):
            with pytest.raises(ValueError):
                call(0, **{name: bad})
        with pytest.raises(ValueError):
            call(4, **{m: torch.zeros((3 if m == name else 4, x.shape[1]),
                                        dtype=torch.bfloat16)
                       for m, x in good.items() if m != "positions"},
                 positions=torch.zeros(4, dtype=torch.int32))
    for bad in (pos.long(), pos.float(), torch.zeros(6, dtype=torch.int32)[::2]):
        with pytest.raises(ValueError):
            call(0, positions=bad)
    with pytest.raises(ValueError):
        A._positions(pos, 4)
    assert A._positions(pos, 3) == pos.data_ptr() and A._positions(None, 3) is None


def test_empty_calls_need_no_buffers():
    kw = dict(stream=0, check=False)
    assert P.pkv_kv8_append(_ws(), _c(), 0, 0, 1, None, None, **kw) == P.PKV_OK
    assert P.pkv_kv8_read(_ws(), _c(), 0, 0, None, F, 0, None, None, **kw) == P.PKV_OK
    assert P.pkv_kv8_read(_ws(), _c(), 1, 0, None, F, 1, None, None, **kw) == P.PKV_ERR_INVALID
    e = torch.zeros((0, 4, 128), dtype=torch.bfloat16)
    assert P.pkv_qk_norm_rope(_rope(), 0, e, e[:, :2], None, e, e[:, :2], **kw) == P.PKV_OK


def _cpu_ws(page=16):
    return Workspace(n_layers=2, pool_slots=4 * page, n_q_heads=4, n_kv_heads=2, head_dim=64,
                     page_size=page, max_batch=2, max_reqs=2, max_pages_per_req=2,
                     max_total_tokens=64, device="cpu", pools=False)


def test_cache_owner():
    ws = _cpu_ws()
    assert ws.struct.k_pool is None
    c = Kv8Cache(ws, dtype="int8", scale_block=8)
    assert c.k_pool.shape == (2, 64, 2, 64) and c.k_scale.shape == (2, 4, 2, 2)
    assert c.struct.dtype == A.PKV_KV8_INT8 and c.struct.v_scale == c.v_scale.data_ptr()
    for name in ("k_pool", "v_pool", "k_scale", "v_scale"):
        t = getattr(c, name)
        assert t.numel() * t.element_size() == P.pkv_kv8_bytes(ws, c, name)
    assert Kv8Cache(_cpu_ws(1)).scale_block == 1 and Kv8Cache(_cpu_ws(24)).scale_block == 8
    keep = torch.zeros((2, 64, 2, 64), dtype=torch.uint8)
    assert Kv8Cache(ws, k_pool=keep).k_pool is keep
    assert not c.k_pool.any() and torch.all(c.v_scale == 2.0 ** -100)
    for kw in (dict(dtype="fp4"), dict(scale_block=3), dict(scale_block=0), dict(scale_block=32),
               dict(k_pool=keep.float()), dict(v_pool=keep[:1]), dict(v_pool=keep.to("meta")),
               dict(k_pool=keep.transpose(0, 1).contiguous().transpose(0, 1))):
        with pytest.raises(ValueError):
            Kv8Cache(ws, **kw)


def test_runner_and_extender_arguments():
    from paged_kv_decode_bind_gb300 import DecodeRunner, Kv8Extender
    ws = _cpu_ws()
    c = Kv8Cache(ws)
    assert DecodeRunner(ws, 2, cache=c).launches_per_step == 1 + 2 * 2
    for kw in (dict(fused=False), dict(plan=True)):
        with pytest.raises(ValueError):
            DecodeRunner(ws, 2, cache=c, **kw)
    r = QkNormRope(n_q_heads=4, n_kv_heads=2, head_dim=64, cos_sin=rope_table(9, 64, device="cpu"))
    assert DecodeRunner(ws, 2, norm_rope=r).launches_per_step == 1 + 2 * 2
    other = QkNormRope(n_q_heads=2, n_kv_heads=2, head_dim=64,
                       cos_sin=rope_table(9, 64, device="cpu"))
    for bad in (other, [r], [r, other]):
        with pytest.raises(ValueError):
            DecodeRunner(ws, 2, norm_rope=bad)
    e = Kv8Extender(ws, c, 2, max_new=3, max_context=20, scale=0.1, num_splits=2)
    assert e.n_rows == 64 and e.first_row.tolist() == [0, 32]
    assert e.table.tolist() == [[0, 1], [2, 3]]
    assert e.read_view.max_seq_len == 20 and e.rows_view.max_seq_len == 20
    assert e.rows_view.seq_lens == ws.struct.seq_lens and e.rows_view.err == ws.struct.err
    assert e.part_o.numel() == 2 * 3 * 2 * 4 * 64
    assert Kv8Extender(ws, c, 1, max_new=1, max_context=99, scale=0.1).read_view.max_seq_len == 32
    with pytest.raises(ValueError):
        e.layer(0, 0, 4, None, None, None, None)
    for kw in (dict(batch=3), dict(max_new=0), dict(max_context=0), dict(num_splits=0)):
        args = dict(batch=2, max_new=3, max_context=20, scale=0.1)
        args.update(kw)
        with pytest.raises(ValueError):
            Kv8Extender(ws, c, args.pop("batch"), **args)


@pytest.mark.parametrize("flag", [A.PKV_FLAG_WRITE_LSE,
                                  A.PKV_FLAG_OUT_F32 | A.PKV_FLAG_FORCE_SIMT, 1 << 20])
def test_extender_refuses_flags_it_does_not_pass_on(flag):
    from paged_kv_decode_bind_gb300 import Kv8Extender
    ws = _cpu_ws()
    e = Kv8Extender(ws, Kv8Cache(ws), 2, max_new=3, max_context=20, scale=0.1)
    with pytest.raises(ValueError):
        e.layer(0, None, 2, None, None, None, None, flag)


def test_runner_collects_position_errors():
    # whatever word the norm's arguments have, a step's errors are in ws.err
    from paged_kv_decode_bind_gb300 import DecodeRunner
    ws = _cpu_ws()
    own = torch.zeros(1, dtype=torch.int32)
    ropes = [QkNormRope(n_q_heads=4, n_kv_heads=2, head_dim=64, err=err,
                        cos_sin=rope_table(9, 64, device="cpu")) for err in (None, own)]
    run = DecodeRunner(ws, 2, norm_rope=ropes)
    for args, r in zip(run.rope_args, ropes):
        assert args.err == ws.err.data_ptr() != r.struct.err
        assert args.cos_sin == r.struct.cos_sin and args.max_positions == 9
        assert args.widths == (64, 256, 128)


@pytest.mark.parametrize("kw", [dict(n_layers=1), dict(pool_slots=32), dict(n_kv_heads=1),
                                dict(head_dim=128), dict(page_size=8, max_pages_per_req=4)])
def test_a_cache_of_other_shapes_is_refused(kw):
    # its buffers are smaller, or laid out in another way, than the workspace says
    from paged_kv_decode_bind_gb300 import DecodeRunner, Kv8Extender
    shape = dict(n_layers=2, pool_slots=64, n_q_heads=4, n_kv_heads=2, head_dim=64, page_size=16,
                 max_batch=2, max_reqs=2, max_pages_per_req=2, device="cpu", pools=False)
    ws, other = Workspace(**shape), Workspace(**{**shape, **kw})
    cache = Kv8Cache(other, scale_block=4)
    calls = [lambda w: P.pkv_kv8_append(w, cache, 0, 0, 1, F, F, 0),
             lambda w: P.pkv_kv8_extend_append(w, cache, 0, 0, F, 4, F, F, 0),
             lambda w: P.pkv_kv8_read(w, cache, 0, 0, None, F, 4, F, F, 0, 0),
             lambda w: P.pkv_kv8_decode_layer(w, cache, 0, 0, F, None, None, 0.1, 1, 0, 0),
             lambda w: DecodeRunner(w, 2, cache=cache),
             lambda w: Kv8Extender(w, cache, 2, max_new=1, max_context=9, scale=0.1)]
    for call in calls:
        with pytest.raises(ValueError):
            call(ws)
    for call in calls[:4]:  # the bare struct too
        with pytest.raises(ValueError):
            call(ws.struct)
    for w in (ctypes.byref(ws.struct), ctypes.pointer(ws.struct)):
        with pytest.raises(ValueError):
            calls[0](w)
    # its own, a copy of its struct, a reference to it
    for w in (other, A.PkvWorkspace.from_buffer_copy(other.struct), ctypes.byref(other.struct),
              ctypes.pointer(other.struct)):
        assert P.pkv_kv8_append(w, cache, 0, 0, 1, None, None, 0) == P.PKV_OK
    for call in calls[4:]:
        call(other)


def test_a_cache_on_another_device_is_refused():
    from paged_kv_decode_bind_gb300 import DecodeRunner
    ws = _cpu_ws()
    c = Kv8Cache(ws)
    c.k_pool = c.k_pool.to("meta")
    with pytest.raises(ValueError):
        DecodeRunner(ws, 2, cache=c)


def test_rope_owner():
    t = rope_table(10, 32, device="cpu")
    w = torch.ones(64, dtype=torch.bfloat16)
    r = QkNormRope(n_q_heads=2, n_kv_heads=1, head_dim=64, rot_dim=32, cos_sin=t, q_weight=w)
    assert r.struct.max_positions == 10 and r.struct.k_weight is None
    for kw in (dict(cos_sin=t.double()), dict(cos_sin=t[:, :16]), dict(cos_sin=None),
               dict(cos_sin=t, q_weight=w.float()), dict(cos_sin=t, k_weight=w[:32])):
        with pytest.raises(ValueError):
            QkNormRope(n_q_heads=2, n_kv_heads=1, head_dim=64, rot_dim=32, **kw)


def test_rope_tensors_on_several_devices_are_refused():
    # the kernel would take a host table's address for one of its own device
    from paged_kv_decode_bind_gb300 import DecodeRunner
    t = rope_table(9, 64, device="cpu")
    w = torch.ones(64, dtype=torch.bfloat16)
    kw = dict(n_q_heads=4, n_kv_heads=2, head_dim=64)
    for bad in (dict(cos_sin=t.to("meta"), q_weight=w), dict(cos_sin=t, k_weight=w.to("meta")),
                dict(cos_sin=t, err=torch.zeros(1, dtype=torch.int32, device="meta")),
                dict(cos_sin=t, err=torch.zeros(1))):
        with pytest.raises(ValueError):
            QkNormRope(**kw, **bad)
    far = QkNormRope(**kw, cos_sin=t)
    far.err = far.err.to("meta")  # as if all of it were
    with pytest.raises(ValueError):
        DecodeRunner(_cpu_ws(), 2, norm_rope=far)
    assert QkNormRope(**kw, cos_sin=t, q_weight=w).err.device == t.device


# ------------------------------------------------------------- oracle pins ----
def test_oracle_codes():
    T = K8.TABLE["e4m3"]
    assert T[0x38] == 1.0 and T[0x7e] == 448.0 and T[0x01] == 2.0 ** -9 and T[0xb8] == -1.0
    assert math.isnan(T[0x7f]) and math.isnan(T[0xff])
    # every code but NaN against torch's reading of the same bits
    codes = torch.arange(256, dtype=torch.uint8)
    ref = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(T, ref, equal_nan=True)
    # nearest, ties to even: 17 and 18 lie 1 apart from 16 and 20's midpoints
    assert K8.encode(np.array([17.0, 19.0, 465.0, -1e9, 0.0]), "e4m3").tolist() == \
        [0x58, 0x5a, 0x7e, 0xfe, 0x00]
    assert K8.encode(np.array([0.5, 1.5, -2.5, 127.4, -300.0, math.nan]), "int8").tolist() == \
        [0, 2, 254, 127, 129, 0]
    x = torch.randn(5000, generator=torch.Generator().manual_seed(1)) * 60
    want = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(K8.encode(x.double().numpy(), "e4m3"), want)


def test_oracle_need():
    assert K8.need(448.0, "e4m3") == 1.0 and K8.need(449.0, "e4m3") == 2.0
    assert K8.need(127.0, "int8") == 1.0 and K8.need(63.5, "int8") == 0.5
    assert K8.need(0.0, "int8") == 2.0 ** -100 and K8.need(3e38, "int8") == 2.0 ** 100
    assert K8.finite_max([1.0, -3.0, math.inf, math.nan]) == 3.0


def test_oracle_append_grows_a_block():
    c = K8.Cache(np.zeros((1, 4, 1, 2), np.uint8), np.zeros((1, 1, 1, 1), np.float32), 4, 4,
                 "int8")
    c.append(0, [0], np.array([[[100.0, 3.0]]]))
    c.append(0, [1], np.array([[[5.0, -400.0]]]))
    assert c.scales[0, 0, 0, 0] == 4.0
    # 3 / 4 rounds to 1; 100 = 25 * 4; 5 / 4 rounds to 1
    assert c.codes[0, :2, 0].view(np.int8).tolist() == [[25, 1], [1, -100]]
    assert c.rows(0, [0, 1])[1, 0].tolist() == [4.0, -400.0]


def test_oracle_attention_and_rope():
    k = np.array([[[0.0, 0.0]], [[2.0, 0.0]]])
    v = np.array([[[1.0, 0.0]], [[0.0, 1.0]]])
    out, lse, mass, size, _ = K8.attention(np.array([[math.log(3.0), 0.0]]), k, v, 0.5)
    assert np.allclose(out, [[0.25, 0.75]]) and np.allclose(lse, [math.log(4.0)])
    y = K8.norm_rope(np.array([[3.0, 4.0, 5.0, 0.0]]), None, np.array([0.0]), np.array([1.0]), 0,
                     False)
    assert y.tolist() == [[-4.0, 3.0, 5.0, 0.0]]
    y = K8.norm_rope(np.array([[3.0, 3.0, 3.0, 3.0]]), np.array([1.0, 2.0, 3.0, 4.0]),
                     np.array([1.0, 0.0]), np.array([0.0, 1.0]), 0, True)
    assert np.allclose(y, [[1.0, 2.0, -4.0, 3.0]])
