"""Host side of the serving operators: every refusal of their C entry points and of their classes.  No device call:
each entry point checks its arguments before it asks for a device."""
import ctypes
import math
import types

import pytest
import torch

import long_context_attention_rkv_b200 as rkv
import serving_ref as ref

INVALID = rkv.STATUS_CODE["RKV_ERR_INVALID_ARG"]
UNSUPPORTED = rkv.STATUS_CODE["RKV_ERR_UNSUPPORTED"]
WORKSPACE = rkv.STATUS_CODE["RKV_ERR_WORKSPACE"]
P = 4096                                             # an aligned address that no refused call reads


def status(call, *args):
    return getattr(rkv.lib(), call)(*args)


def at(cfg):
    return None if cfg is None else ctypes.addressof(cfg)


# --- prompt attention ----------------------------------------------------------------------

def prefill_cfg(**kw):
    names = dict(head_dim=128, n_kv_heads=2, n_q_heads=8, batch=3, q_rows=100, kv_rows=100)
    fields = {k: kw.pop(k) for k in list(kw) if k.endswith("_stride")}
    cfg = rkv.make_prefill_config(**{**names, **kw})
    for k, v in fields.items():
        setattr(cfg, k, v)
    return cfg


def prefill_status(cfg, **kw):
    a = dict(q=P, K=P, V=P, q_off=P, kv_off=None, kv_len=None, out=P, lse=None, status=P)
    a.update(kw)
    return status("rkv_prefill_attn", at(cfg), *a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(head_dim=96), UNSUPPORTED), (dict(head_dim=256), UNSUPPORTED), (dict(head_dim=0), UNSUPPORTED),
    (dict(n_kv_heads=0), INVALID), (dict(n_q_heads=0), INVALID), (dict(n_q_heads=7), INVALID),
    (dict(n_q_heads=34), UNSUPPORTED), (dict(n_kv_heads=4097, n_q_heads=4097), UNSUPPORTED),
    (dict(n_kv_heads=4096, n_q_heads=65536), UNSUPPORTED),
    (dict(batch=0), INVALID), (dict(batch=257), UNSUPPORTED), (dict(in_dtype=rkv.RKV_DTYPE_F32), UNSUPPORTED),
    (dict(in_dtype=7), INVALID), (dict(out_dtype=rkv.RKV_DTYPE_F16), INVALID), (dict(out_dtype=-1), INVALID),
    (dict(scale=-1.0), INVALID), (dict(scale=math.inf), INVALID), (dict(scale=math.nan), INVALID),
    (dict(q_rows=-1), INVALID), (dict(kv_rows=-1), INVALID), (dict(q_rows=2 ** 31), UNSUPPORTED),
    (dict(kv_rows=2 ** 31), UNSUPPORTED), (dict(q_row_stride=1020), INVALID), (dict(q_row_stride=0), INVALID),
    (dict(q_head_stride=-128), INVALID), (dict(kv_row_stride=2 ** 38), INVALID), (dict(kv_head_stride=4), INVALID),
    (dict(out_row_stride=1028), INVALID), (dict(out_head_stride=2), INVALID),
    (dict(out_dtype=rkv.RKV_DTYPE_F32, out_head_stride=2), INVALID),
    (dict(kv_padded=True, kv_plane_stride=0), INVALID), (dict(kv_padded=True, kv_plane_stride=12), INVALID),
])
def test_prefill_refuses_configurations(kw, code):
    assert prefill_status(prefill_cfg(**kw)) == code


@pytest.mark.parametrize("rows", ["q_rows", "kv_rows"])
def test_prefill_refuses_rows_next_to_31_bits(rows):
    # tokens are rounded up to tiles in 31 bits
    for n in (2 ** 31 - 255, 2 ** 31 - 1):
        assert prefill_status(prefill_cfg(**{rows: n})) == UNSUPPORTED
    assert prefill_status(prefill_cfg(**{rows: 2 ** 31 - 256}), out=None) == INVALID       # the next check


def test_prefill_refuses_pointers():
    assert prefill_status(None) == INVALID
    cfg = prefill_cfg()
    cfg.kv_padded = 2
    assert prefill_status(cfg) == INVALID
    cfg = prefill_cfg()
    for name in ("q", "K", "V", "out", "q_off", "status"):
        assert prefill_status(cfg, **{name: None}) == INVALID, name
    for name in ("q", "K", "V", "out"):
        assert prefill_status(cfg, **{name: P + 8}) == INVALID, name
    for name in ("q_off", "kv_off", "kv_len", "lse", "status"):
        assert prefill_status(cfg, **{name: P + 2}) == INVALID, name


def test_prefill_without_rows_is_done():
    assert prefill_status(prefill_cfg(q_rows=0)) == 0
    assert prefill_status(prefill_cfg(q_rows=0), q=None, out=None, q_off=None) == 0


# --- block tables --------------------------------------------------------------------------

def blocks_cfg(**kw):
    return rkv.make_blocks_config(**{**dict(batch=4, max_blocks=10, block_size=16, n_blocks=64), **kw})


EXTEND = ("lengths", "new_counts", "block_table", "free_list", "n_free", "new_off", "slot_map", "max_new", "lengths_out",
          "n_free_out", "status")
RELEASE = ("lengths", "ended", "block_table", "free_list", "n_free", "lengths_out", "n_free_out", "status")


def extend_status(cfg, **kw):
    a = {**{n: P for n in EXTEND}, "max_new": 8, **kw}
    return status("rkv_blocks_extend", at(cfg), *a.values(), None)


def release_status(cfg, **kw):
    a = {**{n: P for n in RELEASE}, **kw}
    return status("rkv_blocks_release", at(cfg), *a.values(), None)


@pytest.mark.parametrize("call", [extend_status, release_status])
@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), INVALID), (dict(max_blocks=0), INVALID), (dict(n_blocks=0), INVALID), (dict(n_blocks=-5), INVALID),
    (dict(batch=257), UNSUPPORTED), (dict(block_size=8), UNSUPPORTED), (dict(block_size=24), UNSUPPORTED),
    (dict(block_size=0), UNSUPPORTED), (dict(block_size=256), UNSUPPORTED), (dict(n_blocks=2 ** 27), UNSUPPORTED),
    (dict(max_blocks=2 ** 27), UNSUPPORTED),
])
def test_tables_refuse_configurations(call, kw, code):
    assert call(blocks_cfg(**kw)) == code


def test_tables_refuse_pointers_and_counts():
    assert extend_status(None) == INVALID and release_status(None) == INVALID
    for bad in (None, P + 1):
        for name in EXTEND:
            if name != "max_new":
                assert extend_status(blocks_cfg(), **{name: bad}) == INVALID, name
        for name in RELEASE:
            assert release_status(blocks_cfg(), **{name: bad}) == INVALID, name
    assert extend_status(blocks_cfg(), max_new=-1) == INVALID
    assert extend_status(blocks_cfg(), max_new=2 ** 31) == INVALID


# --- 8-bit block cache -----------------------------------------------------------------------

def kv8_cfg(**kw):
    names = dict(head_dim=128, n_kv_heads=2, n_q_heads=8, block_size=16, n_blocks=64, max_blocks=10, batch=4)
    fields = {k: kw.pop(k) for k in ("codes_K", "codes_V", "scale_K", "scale_V", "device_status") if k in kw}
    cfg = rkv.make_kv8_config(**{**names, **kw})
    for k in ("codes_K", "codes_V", "scale_K", "scale_V", "device_status"):
        setattr(cfg, k, fields.get(k, P))
    return cfg


def store_status(cfg, **kw):
    a = {**dict(K=P, V=P, row_stride=256, head_stride=128, slot_map=P, n_rows=5), **kw}
    return status("rkv_kv8_store", at(cfg), *a.values(), None)


def decode_status(cfg, **kw):
    a = {**dict(q=P, block_table=P, lengths=P, out=P, workspace=P, bytes=2 ** 40), **kw}
    return status("rkv_kv8_decode_attn", at(cfg), *a.values(), None)


def size_status(cfg):
    return status("rkv_kv8_workspace", at(cfg), ctypes.byref(ctypes.c_uint64()))


@pytest.mark.parametrize("call", [store_status, decode_status, size_status])
@pytest.mark.parametrize("kw,code", [
    (dict(head_dim=80), UNSUPPORTED), (dict(n_kv_heads=0), INVALID), (dict(n_q_heads=9), INVALID),
    (dict(n_q_heads=34), UNSUPPORTED), (dict(n_kv_heads=4096, n_q_heads=65536), UNSUPPORTED),
    (dict(batch=0), INVALID), (dict(batch=257), UNSUPPORTED), (dict(block_size=48), UNSUPPORTED), (dict(n_blocks=0), INVALID), (dict(max_blocks=-1), INVALID),
    (dict(n_blocks=2 ** 27), UNSUPPORTED), (dict(max_blocks=2 ** 27), UNSUPPORTED), (dict(code_type=2), INVALID),
    (dict(code_type=-1), INVALID), (dict(in_dtype=rkv.RKV_DTYPE_F32), UNSUPPORTED), (dict(in_dtype=5), INVALID),
    (dict(out_dtype=rkv.RKV_DTYPE_F16), INVALID), (dict(scale=-0.5), INVALID), (dict(scale=math.nan), INVALID),
])
def test_kv8_refuses_configurations(call, kw, code):
    assert call(kv8_cfg(**kw)) == code


@pytest.mark.parametrize("call", [store_status, decode_status, size_status])
def test_kv8_refuses_rows_next_to_31_bits(call):
    # lengths are rounded up to tiles of 64 tokens in 31 bits
    for block, most in ((16, 2 ** 27 - 4), (32, 2 ** 26 - 2), (64, 2 ** 25 - 1), (128, 2 ** 24 - 1)):
        for blocks in (most + 1, 2 ** 31 // block - 1):
            if blocks > most:
                assert call(kv8_cfg(block_size=block, max_blocks=blocks)) == UNSUPPORTED
        largest = kv8_cfg(block_size=block, max_blocks=most, **({} if call is size_status else dict(codes_K=None)))
        assert call(largest) == (0 if call is size_status else INVALID)      # the next check


@pytest.mark.parametrize("call", [store_status, decode_status])
def test_kv8_refuses_buffers(call):
    assert call(None) == INVALID
    for name, odd in (("codes_K", 8), ("codes_V", 4), ("scale_K", 2), ("scale_V", 1), ("device_status", 2)):
        assert call(kv8_cfg(**{name: None})) == INVALID, name
        assert call(kv8_cfg(**{name: P + odd})) == INVALID, name


def test_store_refuses_rows():
    cfg = kv8_cfg()
    for kw in (dict(K=None), dict(V=None), dict(slot_map=None), dict(K=P + 2), dict(V=P + 8), dict(slot_map=P + 2),
               dict(row_stride=0), dict(row_stride=-256), dict(row_stride=130), dict(head_stride=4),
               dict(head_stride=2 ** 38), dict(n_rows=-1)):
        assert store_status(cfg, **kw) == INVALID, kw
    assert store_status(cfg, n_rows=2 ** 30) == UNSUPPORTED          # rows times heads past 31 bits
    assert store_status(cfg, n_rows=2 ** 62) == UNSUPPORTED          # and past 64
    assert store_status(cfg, n_rows=0, K=None, V=None, slot_map=None) == 0


def test_decode_refuses_pointers_and_short_workspaces():
    cfg = kv8_cfg()
    for name, odd in (("q", 8), ("out", 2), ("block_table", 2), ("lengths", 1), ("workspace", 128)):
        assert decode_status(cfg, **{name: None}) == INVALID, name
        assert decode_status(cfg, **{name: P + odd}) == INVALID, name
    need = rkv.rkv_kv8_workspace(cfg)
    assert need % 256 == 0
    assert decode_status(cfg, bytes=need - 1) == WORKSPACE
    assert decode_status(cfg, bytes=0) == WORKSPACE
    assert status("rkv_kv8_workspace", at(cfg), None) == INVALID
    with pytest.raises(rkv.RkvError):
        rkv.rkv_kv8_workspace(kv8_cfg(head_dim=32))


@pytest.mark.parametrize("call,cfg", [(prefill_status, prefill_cfg), (store_status, kv8_cfg), (decode_status, kv8_cfg)])
def test_scales_whose_product_with_log2e_overflows_are_refused(call, cfg):
    for scale in (2.0 ** 127 * (1 + 2.0 ** -23), 3.4e38):
        assert call(cfg(scale=scale)) == INVALID
    largest = dict(scale=2.0 ** 127)
    if call is prefill_status:
        assert call(cfg(q_rows=0, **largest)) == 0
    elif call is store_status:
        assert call(cfg(**largest), n_rows=0) == 0
    else:
        assert call(cfg(**largest), bytes=0) == WORKSPACE          # the next check


# --- the classes -----------------------------------------------------------------------------

@pytest.fixture
def recorded(monkeypatch):
    """The raw functions replaced by a recorder, and the device check passed, so that the classes' own checks are
    what a call meets."""
    calls = []
    for name in ("rkv_prefill_attn", "rkv_blocks_extend", "rkv_blocks_release", "rkv_kv8_store", "rkv_kv8_decode_attn"):
        monkeypatch.setattr(rkv, name, lambda *a, _n=name: calls.append((_n, a)))
    monkeypatch.setattr(rkv, "_local", lambda where, tensors: ([], 0))
    monkeypatch.setattr(rkv, "_device", lambda: 0)
    return calls


def refused(call, *args, **kw):
    with pytest.raises(rkv.RkvError) as e:
        call(*args, **kw)
    assert e.value.status == INVALID


def test_prefill_class_refuses_tensors(recorded):
    op = rkv.Prefill(rkv.make_prefill_config(64, 2, 4, 2, 10, 12), device="cpu")
    bf, i32 = torch.bfloat16, torch.int32
    good = dict(q=torch.zeros(10, 4, 64, dtype=bf), K=torch.zeros(12, 2, 64, dtype=bf), V=torch.zeros(12, 2, 64, dtype=bf),
                q_off=torch.zeros(3, dtype=i32), out=torch.zeros(10, 4, 64, dtype=bf))
    more = dict(kv_off=torch.zeros(3, dtype=i32), kv_len=torch.zeros(2, dtype=i32), lse=torch.zeros(10, 4))
    op.attend(**good)
    op.attend(**good, **more)
    assert len(recorded) == 2
    for name, x in {**good, **more}.items():
        args = {**good, **more}
        refused(op.attend, **{**args, name: x.double()})
        refused(op.attend, **{**args, name: x.flatten()[:-1]})
    for name in ("q", "K", "V", "out"):                      # repeated storage: fewer elements than its shape says
        refused(op.attend, **{**good, name: good[name][:1].clone().expand(good[name].shape)})
    fused = torch.zeros(12, 8, 64, dtype=bf)                 # views of one buffer, with its strides
    strided = rkv.Prefill(rkv.make_prefill_config(64, 2, 4, 2, 12, 12, q_strides=(512, 64), kv_strides=(512, 64, 0)),
                          device="cpu")
    args = dict(q_off=good["q_off"], out=torch.zeros(12, 4, 64, dtype=bf))
    strided.attend(q=fused[:, :4], K=fused[:, 4:6], V=fused[:, 6:], **args)
    refused(strided.attend, q=fused[1:, :4], K=fused[:, 4:6], V=fused[:, 6:], **args)
    assert len(recorded) == 3


def test_tables_class_refuses_tensors(recorded):
    t = rkv.BlockTables(4, 8, 16, 20, device="cpu")
    counts, slots = torch.zeros(4, dtype=torch.int32), torch.zeros(9, dtype=torch.int32)
    t.extend(counts, slots)
    t.release(counts)
    for bad in (counts.long(), counts[:3], torch.zeros(8, dtype=torch.int32)[::2]):
        refused(t.extend, bad, slots)
        refused(t.release, bad)
    refused(t.extend, counts, slots.long())
    refused(t.extend, counts, torch.zeros(18, dtype=torch.int32)[::2])
    assert len(recorded) == 2


def test_cache_class_refuses_buffers_and_tensors(recorded, monkeypatch):
    shape = dict(head_dim=64, n_kv_heads=2, n_q_heads=4, block_size=16, n_blocks=6, max_blocks=3, batch=2)
    cfg = rkv.make_kv8_config(**shape)
    codes = torch.zeros(6, 2, 16, 64, dtype=torch.int8)
    for kw in (dict(codes_K=codes.to(torch.uint8)), dict(codes_V=codes[:5]), dict(codes_K=codes.transpose(1, 2)),
               dict(scale_K=torch.zeros(6, 2, dtype=torch.float64)), dict(scale_V=torch.zeros(2, 6)),
               dict(workspace=torch.zeros(2 ** 20)), dict(codes_K=codes.view(torch.float8_e4m3fn))):
        refused(rkv.KV8Cache, cfg, device="cpu", **kw)
    cache = rkv.KV8Cache(cfg, device="cpu")
    bf, i32 = torch.bfloat16, torch.int32
    K, slots = torch.zeros(5, 2, 64, dtype=bf), torch.zeros(5, dtype=i32)
    cache.store(K, K, slots)
    for a in ((K.half(), K.half(), slots), (K, K[:4], slots), (K[:, :1], K[:, :1], slots), (K[..., :32], K[..., :32], slots),
              (K.flatten(1), K.flatten(1), slots), (K, K, slots[:4]), (K, K, slots.long()),
              (K, torch.zeros(5, 2, 128, dtype=bf)[..., :64], slots),
              (K.transpose(1, 2).contiguous().transpose(1, 2), K.transpose(1, 2).contiguous().transpose(1, 2), slots)):
        refused(cache.store, *a)
    q, table, lens = torch.zeros(2, 4, 64, dtype=bf), torch.zeros(2, 3, dtype=i32), torch.zeros(2, dtype=i32)
    cache.decode(q, table, lens, q.clone())
    for a in ((q.half(), table, lens, q), (q[:1], table, lens, q), (q, table[:, :2], lens, q), (q, table.long(), lens, q),
              (q, table, lens[:1], q), (q, table, lens, q.float()), (q, table, lens, q[:, :2])):
        refused(cache.decode, *a)
    assert len(recorded) == 2
    monkeypatch.setattr(rkv, "_device", lambda: 1)      # another current device than the cache's
    refused(cache.store, K, K, slots)
    refused(cache.decode, q, table, lens, q)


def test_cache_class_refuses_tables_of_another_width(recorded):
    # rows of a table made for longer requests: every request after the first would be read from the wrong place
    cfg = rkv.make_kv8_config(head_dim=64, n_kv_heads=2, n_q_heads=4, block_size=16, n_blocks=6, max_blocks=3, batch=2)
    cache, i32 = rkv.KV8Cache(cfg, device="cpu"), torch.int32
    q, lens = torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.zeros(2, dtype=i32)
    for shape in ((2, 4), (3, 2), (6, 1), (2, 30), (1, 3, 4)):
        refused(cache.decode, q, torch.zeros(shape, dtype=i32), lens, q.clone())
    refused(cache.decode, q, rkv.BlockTables(2, 5, 16, 6, device="cpu").table, lens, q.clone())
    assert not recorded
    for shape in ((2, 3), (5, 3), (1, 2, 3), (6,)):        # rows behind the last request are not read
        cache.decode(q, torch.zeros(shape, dtype=i32), lens, q.clone())
    assert len(recorded) == 4


def test_classes_refuse_rows_of_other_heads(recorded):
    cfg = rkv.make_kv8_config(head_dim=64, n_kv_heads=2, n_q_heads=4, block_size=16, n_blocks=6, max_blocks=3, batch=2)
    cache, i32, bf = rkv.KV8Cache(cfg, device="cpu"), torch.int32, torch.bfloat16
    table, lens, good = torch.zeros(2, 3, dtype=i32), torch.zeros(2, dtype=i32), torch.zeros(2, 4, 64, dtype=bf)
    for shape in ((2, 8, 64), (4, 2, 64), (2, 4, 128), (2, 512), (1, 4, 2, 64)):
        refused(cache.decode, torch.zeros(shape, dtype=bf), table, lens, good.clone())
        refused(cache.decode, good, table, lens, torch.zeros(shape, dtype=bf))
    op = rkv.Prefill(rkv.make_prefill_config(64, 2, 4, 2, 10, 12), device="cpu")
    q, K, off = torch.zeros(10, 4, 64, dtype=bf), torch.zeros(12, 2, 64, dtype=bf), torch.zeros(3, dtype=i32)
    for shape in ((10, 8), (20, 2), (5, 10)):
        refused(op.attend, q, K, K, off, q.clone(), lse=torch.zeros(shape))
    assert not recorded
    for shape in ((2, 4, 64), (3, 4, 64), (2, 256), (8, 64), (512,), (2, 1, 4, 64)):
        cache.decode(torch.zeros(shape, dtype=bf), table, lens, torch.zeros(shape, dtype=bf))
    for shape in ((10, 4), (12, 4), (40,)):
        op.attend(q, K, K, off, q.clone(), lse=torch.zeros(shape))
    assert len(recorded) == 9


def test_store_class_takes_dimensions_of_one_with_any_stride(recorded):
    # one new token, or one kv-head: the stride of a dimension of one says nothing about the layout
    bf = torch.bfloat16
    shape = dict(head_dim=64, block_size=16, n_blocks=6, max_blocks=3, batch=2)
    two = rkv.KV8Cache(rkv.make_kv8_config(n_kv_heads=2, n_q_heads=4, **shape), device="cpu")
    K, V = torch.zeros(1, 2, 64, dtype=bf), torch.zeros(1, 8, 64, dtype=bf)[:, 4:6]
    slot = torch.zeros(5, dtype=torch.int32)
    two.store(K, V, slot)
    two.store(V, K, slot)
    two.store(torch.as_strided(K, (1, 2, 64), (3, 64, 1)), V, slot)
    one = rkv.KV8Cache(rkv.make_kv8_config(n_kv_heads=1, n_q_heads=4, **shape), device="cpu")
    rows = torch.zeros(5, 64, dtype=bf)
    one.store(rows.unsqueeze(1), rows.view(1, 5, 64).transpose(0, 1), slot)
    one.store(torch.as_strided(rows, (5, 1, 64), (64, 1, 1)), rows.unsqueeze(1), slot)
    one.store(rows[:1].unsqueeze(1), torch.as_strided(rows, (1, 1, 64), (5, 7, 1)), slot)
    assert [a[3:5] for _, a in recorded] == [(128, 64)] * 3 + [(64, 64)] * 3
    refused(one.store, rows.unsqueeze(1), torch.zeros(10, 64, dtype=bf)[::2].unsqueeze(1), slot)
    refused(two.store, K, torch.zeros(1, 2, 128, dtype=bf)[..., :64], slot)
    refused(two.store, K, torch.zeros(1, 3, 64, dtype=bf), slot)
    refused(two.store, K, torch.zeros(2, 64, dtype=bf), slot)


def test_raw_calls_refuse_tensors_of_another_device(monkeypatch):
    monkeypatch.setattr(rkv, "_device", lambda: 0)
    x = torch.zeros(4, dtype=torch.int32)                            # on the CPU
    cfg = rkv.make_blocks_config(4, 2, 16, 8)
    with pytest.raises(rkv.RkvError) as e:
        rkv.rkv_blocks_extend(cfg, x, x, x, x, x, x, x, 4, x, x, x)
    assert e.value.status == INVALID
    with pytest.raises(rkv.RkvError):
        rkv.rkv_kv8_store(rkv.make_kv8_config(64, 1, 1, 16, 4, 2, 1), x, x, 64, 64, x, 1)


# --- the references themselves -----------------------------------------------------------------

def test_reference_attention_by_hand():
    q = torch.tensor([[[1.0, 0.0]], [[0.0, 1.0]]])
    k = torch.tensor([[[2.0, 0.0]], [[0.0, 3.0]]])
    v = torch.tensor([[[1.0, 5.0]], [[7.0, -2.0]]])
    allowed = torch.tensor([[False, False], [True, True]])
    out, lse, _, _ = ref.attention(q, k, v, allowed, scale=1.0)
    assert (out[0] == 0).all() and lse[0].item() == -math.inf
    w = 1.0 / (1.0 + math.exp(-3.0))
    assert out[1, 0, 0].item() == pytest.approx((1 - w) * 1 + w * 7, rel=1e-12)
    assert lse[1].item() == pytest.approx(math.log(1 + math.exp(3.0)), rel=1e-12)


def test_error_word_is_taken_once():
    s = torch.tensor([5], dtype=torch.int32)
    box = types.SimpleNamespace(status=s)
    assert rkv.BlockTables.device_error(box) == 5 and rkv.BlockTables.device_error(box) == 0
