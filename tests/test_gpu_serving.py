"""GPU parity of the serving operators against their 64-bit references: prompt attention, block tables, the
8-bit block cache and its decode, alone and together as a serving loop uses them."""
import math
import random

import numpy as np
import pytest
import torch

import long_context_attention_rkv_b200 as rkv
import serving_ref as ref

pytestmark = pytest.mark.gpu

CODE = {torch.bfloat16: 0, torch.float32: 1, torch.float16: 2}
KV8 = {"int8": rkv.RKV_KV8_INT8, "e4m3": rkv.RKV_KV8_E4M3}


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def offsets(lens):
    return [0] + list(np.cumsum(lens))


def values(gen, shape, dtype, hot=2):
    x = torch.randn(shape, generator=gen)
    x[..., torch.randint(0, shape[-1], (hot,), generator=gen)] *= 8.0
    return x.to(dtype)


# --- prompt attention -------------------------------------------------------------------------

def check_prefill(q, K, V, q_off, kv_rows_of, out, lse, scale=None, in_dtype=None):
    """Every sequence of a call against the reference; kv_rows_of(b) gives its keys and values."""
    worst = 0.0
    for b in range(len(q_off) - 1):
        lo, hi = q_off[b], q_off[b + 1]
        if lo == hi:
            continue
        k, v = kv_rows_of(b)
        n, L, d = hi - lo, k.shape[0], q.shape[2]
        allowed = torch.arange(L)[None] <= (L - n + torch.arange(n))[:, None]
        want, wlse, mag, spread = ref.attention(q[lo:hi].cpu(), k.cpu(), v.cpu(), allowed, scale)
        floor = 2.0 ** -32 * float(v.abs().max()) if q.dtype is torch.float16 and L else 0.0
        tol, ltol = ref.bounds(want, mag, spread, d, L, q.dtype, out.dtype, floor)
        err = (out[lo:hi].double().cpu() - want).abs()
        assert (err <= tol).all(), f"sequence {b}: {float((err - tol).max())} over the bound {float(tol.max())}"
        worst = max(worst, float((err / tol).max()))
        if lse is not None:
            got = lse[lo:hi].double().cpu()
            none = wlse == -math.inf
            assert torch.equal(got == -math.inf, none)
            d_l = (got - wlse).abs().masked_fill(none, 0.0)
            assert (d_l <= ref.lse_bound(wlse, ltol)).all(), f"sequence {b}: log-sums"
    return worst


def prefill(q, K, V, q_off, cfg_kw=None, kv_off=None, kv_len=None, out=None, want_lse=True, expect=0, kv_padded=False):
    rows, hq, d = q.shape
    hkv = K.shape[1]
    kw = dict(head_dim=d, n_kv_heads=hkv, n_q_heads=hq, batch=len(q_off) - 1, q_rows=rows,
              kv_rows=K.shape[2] if kv_padded else K.shape[0], in_dtype=CODE[q.dtype], kv_padded=kv_padded)
    kw.update(cfg_kw or {})
    odt = {v: k for k, v in CODE.items()}[kw.get("out_dtype", kw["in_dtype"])]
    out = torch.full((rows, hq, d), 7.0, dtype=odt, device="cuda") if out is None else out
    lse = torch.full((rows, hq), 7.0, device="cuda") if want_lse else None
    op = rkv.Prefill(rkv.make_prefill_config(**kw))
    op.attend(q, K, V, ints(q_off), out, kv_off=None if kv_off is None else ints(kv_off),
              kv_len=None if kv_len is None else ints(kv_len), lse=lse)
    torch.cuda.synchronize()
    assert op.device_error() == expect
    return out, lse


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 2), (14, 2), (6, 2), (16, 1), (5, 1), (4, 4), (24, 2)])
def test_prefill_packed_lengths(dtype, d, hq, hkv):
    g = torch.Generator().manual_seed(hq * 100 + hkv + d)
    lens = [1, 0, 130, 17, 129, 300, 2, 128]
    n = sum(lens)
    q, K, V = (values(g, (n, h, d), dtype).cuda() for h in (hq, hkv, hkv))
    off = offsets(lens)
    for odt in (dtype, torch.float32):
        out, lse = prefill(q, K, V, off, dict(out_dtype=CODE[odt]))
        check_prefill(q, K, V, off, lambda b: (K[off[b]:off[b + 1]], V[off[b]:off[b + 1]]), out, lse)


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 127, 128, 129, 255, 256, 257, 511, 513, 1000, 2049])
def test_prefill_one_prompt_lengths(n):
    g = torch.Generator().manual_seed(n)
    q, K, V = (values(g, (n, h, 128), torch.bfloat16).cuda() for h in (4, 1, 1))
    out, lse = prefill(q, K, V, [0, n])
    check_prefill(q, K, V, [0, n], lambda b: (K, V), out, lse)


@pytest.mark.parametrize("d", [64, 128])
def test_prefill_chunks_over_earlier_keys(d):
    # chunks of 1 .. 200 new rows over 0 .. 700 earlier keys; a sequence with fewer keys than rows (rows that see
    # nothing) and one without any key
    g = torch.Generator().manual_seed(5)
    new, keys = [1, 200, 64, 50, 3, 33], [701, 450, 64, 20, 0, 260]
    q = values(g, (sum(new), 8, d), torch.bfloat16).cuda()
    K, V = (values(g, (sum(keys), 2, d), torch.bfloat16).cuda() for _ in range(2))
    qo, ko = offsets(new), offsets(keys)
    out, lse = prefill(q, K, V, qo, kv_off=ko)
    check_prefill(q, K, V, qo, lambda b: (K[ko[b]:ko[b + 1]], V[ko[b]:ko[b + 1]]), out, lse)
    blind = slice(qo[3], qo[3] + 30)                       # 50 rows over 20 keys: the first 30 see none
    assert (out[blind] == 0).all() and (lse[blind] == -math.inf).all()
    assert (out[qo[4]:qo[5]] == 0).all()


@pytest.mark.parametrize("dtype,out_dtype", [(torch.bfloat16, None), (torch.float16, None), (torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("hq,hkv,d,keys,new", [
    # few items over many keys (shared by 8, 4 and 2 CTAs); one, all or no key tile for some of them
    (8, 1, 128, [5000], [1]), (8, 1, 64, [1300], [37]), (7, 1, 128, [4000, 3, 900], [5, 3, 40]),
    (4, 2, 64, [2500, 0, 64, 63], [1, 2, 70, 1]), (16, 8, 128, [1500, 1601], [1, 16]), (32, 8, 64, [1700] * 4, [1, 9, 17, 0]),
    (24, 8, 128, [2600, 1300, 65, 700], [40, 1, 65, 50]), (2, 2, 128, [1025], [1025]),
])
def test_prefill_keys_shared_by_a_cluster(dtype, out_dtype, hq, hkv, d, keys, new):
    g = torch.Generator().manual_seed(hq + d + len(keys))
    q = values(g, (sum(new), hq, d), dtype).cuda()
    # gaps of 5 rows between the sequences' keys, which hold NaN
    K, V = (values(g, (sum(keys) + 5 * len(keys), hkv, d), dtype).cuda() for _ in range(2))
    starts = [o + 5 * i for i, o in enumerate(offsets(keys)[:-1])]
    for s, n in zip(starts, keys):
        K[s + n:s + n + 5] = math.nan
        V[s + n:s + n + 5] = math.nan
    off = offsets(new)
    kw = {} if out_dtype is None else dict(out_dtype=CODE[out_dtype])
    first = None
    for _ in range(3):
        out, lse = prefill(q, K, V, off, kw, kv_off=starts + [0], kv_len=keys)
        check_prefill(q, K, V, off, lambda b: (K[starts[b]:starts[b] + keys[b]], V[starts[b]:starts[b] + keys[b]]), out, lse)
        first = first or (out, lse)
        assert torch.equal(first[0], out) and torch.equal(first[1], lse)


@pytest.mark.parametrize("lens", [[450, 451, 1, 0, 300] * 11, [2049, 5, 700, 700, 64, 31, 1]])
def test_prefill_orders_of_work(lens):
    # 16 kv-heads: above 12288 tokens in all the sequences go one by one, below level by level; and with earlier keys
    g = torch.Generator().manual_seed(len(lens))
    n = sum(lens)
    q, K, V = (values(g, (n, 16, 128), torch.bfloat16).cuda() for _ in range(3))
    off = offsets(lens)
    out, lse = prefill(q, K, V, off)
    check_prefill(q, K, V, off, lambda b: (K[off[b]:off[b + 1]], V[off[b]:off[b + 1]]), out, lse)
    half = [m // 2 for m in lens]
    starts = offsets(half)
    q2 = torch.cat([q[o + m - h:o + m] for o, m, h in zip(off, lens, half)])
    out2, lse2 = prefill(q2, K, V, starts, kv_off=off)
    for b, (o, m, h) in enumerate(zip(off, lens, half)):
        rows = slice(starts[b], starts[b + 1])
        k, v = K[o:o + m].cpu(), V[o:o + m].cpu()
        allowed = torch.arange(m)[None] <= (m - h + torch.arange(h))[:, None]
        if h == 0:
            continue
        want, wlse, mag, spread = ref.attention(q2[rows].cpu(), k, v, allowed)
        tol, ltol = ref.bounds(want, mag, spread, 128, m, q.dtype, out.dtype)
        assert ((out2[rows].double().cpu() - want).abs() <= tol).all()
        assert ((lse2[rows].double().cpu() - wlse).abs() <= ref.lse_bound(wlse, ltol)).all()


def test_prefill_split_calls_on_two_streams():
    # two long single-token calls at once, repeated: no state is shared
    g = torch.Generator().manual_seed(31)
    jobs = []
    for i in range(2):
        q, K, V = (values(g, (n, h, 128), torch.bfloat16).cuda() for n, h in ((2, 8), (9000, 1), (9000, 1)))
        op = rkv.Prefill(rkv.make_prefill_config(128, 1, 8, 1, 2, 9000))
        want = torch.empty_like(q)
        op.attend(q, K, V, ints([0, 2]), want, kv_off=ints([0, 9000]))
        jobs.append((op, q, K, V, ints([0, 2]), ints([0, 9000]), want, torch.cuda.Stream(), [torch.empty_like(q) for _ in range(30)]))
    torch.cuda.synchronize()
    for r in range(30):
        for op, q, K, V, qo, ko, want, st, outs in jobs:
            with torch.cuda.stream(st):
                op.attend(q, K, V, qo, outs[r], kv_off=ko)
    torch.cuda.synchronize()
    for op, q, K, V, qo, ko, want, st, outs in jobs:
        assert op.device_error() == 0
        assert all(torch.equal(o, want) for o in outs)


def test_prefill_padded_planes_of_the_compressor_layout():
    # K, V [batch][kv_heads][max_len][d] with lengths shorter than the planes; rows behind the lengths hold NaN
    g = torch.Generator().manual_seed(6)
    lens, max_len = [200, 77, 0, 131], 211
    q = values(g, (sum(lens), 8, 128), torch.bfloat16).cuda()
    K, V = (values(g, (4, 2, max_len, 128), torch.bfloat16).cuda() for _ in range(2))
    for b, n in enumerate(lens):
        K[b, :, n:] = math.nan
        V[b, :, n:] = math.nan
    off = offsets(lens)
    out, lse = prefill(q, K, V, off, kv_padded=True)
    rows = lambda b: (K[b, :, :lens[b]].transpose(0, 1), V[b, :, :lens[b]].transpose(0, 1))  # noqa: E731
    check_prefill(q, K, V, off, rows, out, lse)
    # the same with left padding: the keys end at the plane's end
    K2, V2 = torch.full_like(K, math.inf), torch.full_like(V, math.nan)
    for b, n in enumerate(lens):
        K2[b, :, max_len - n:] = K[b, :, :n]
        V2[b, :, max_len - n:] = V[b, :, :n]
    out2, lse2 = prefill(q, K2, V2, off, kv_padded=True, kv_off=[max_len - n for n in lens] + [0], kv_len=lens)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


def test_prefill_strided_views_and_rows_left_alone():
    # q, K, V as views of one fused buffer; sequences that leave gaps; NaN in every row outside them
    g = torch.Generator().manual_seed(7)
    rows, hq, hkv, d = 400, 8, 2, 128
    fused = values(g, (rows, hq + 2 * hkv, d), torch.bfloat16).cuda()
    q, K, V = fused[:, :hq], fused[:, hq:hq + hkv], fused[:, hq + hkv:]
    lens = [150, 100]
    used = torch.zeros(rows, dtype=torch.bool)
    used[:250] = True
    fused[250:] = math.nan
    step = fused.stride(0)
    out, lse = prefill(q, K, V, [0, 150, 250], dict(q_strides=(step, d), kv_strides=(step, d, 0)))
    off = offsets(lens)
    check_prefill(q, K, V, off, lambda b: (K[off[b]:off[b + 1]], V[off[b]:off[b + 1]]), out, lse)
    assert (out[250:] == 7).all() and (lse[250:] == 7).all()
    # heads-first output
    out2 = torch.zeros((hq, rows, d), dtype=torch.bfloat16, device="cuda")
    op = rkv.Prefill(rkv.make_prefill_config(d, hkv, hq, 2, rows, rows, q_strides=(step, d), kv_strides=(step, d, 0),
                                             out_strides=(d, rows * d)))
    op.attend(q, K, V, ints([0, 150, 250]), out2)
    assert torch.equal(out2.transpose(0, 1)[:250], out[:250])


def test_prefill_scale_and_sharp_rows():
    g = torch.Generator().manual_seed(8)
    n = 300
    q, K, V = (values(g, (n, h, 128), torch.bfloat16).cuda() for h in (4, 2, 2))
    for scale, f in ((0.5, 1.0), (0.0, 40.0), (1e-4, 1.0)):
        qq = (q * f).to(torch.bfloat16)
        out, lse = prefill(qq, K, V, [0, n], dict(scale=scale))
        check_prefill(qq, K, V, [0, n], lambda b: (K, V), out, lse, scale=scale or None)


def test_prefill_growing_maximum():
    # keys whose logits rise by a little more than the lazy rescaling step each tile, then fall
    n, d = 900, 128
    q = torch.zeros((n, 1, d)); q[..., 0] = 8.0
    K = torch.zeros((n, 1, d)); K[:, 0, 0] = torch.linspace(0, 200, n).where(torch.arange(n) < 700, 3.0)
    V = torch.randn((n, 1, d), generator=torch.Generator().manual_seed(9))
    q, K, V = (x.to(torch.bfloat16).cuda() for x in (q, K, V))
    out, lse = prefill(q, K, V, [0, n])
    check_prefill(q, K, V, [0, n], lambda b: (K, V), out, lse)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_prefill_nan_keys_reach_the_rows_that_see_them(dtype):
    # a NaN key at every place of a tile: rows before it as without it, rows from it on NaN
    g = torch.Generator().manual_seed(21)
    n, batch = 90, 70
    q, K, V = (values(g, (n, h, 64), dtype).cuda() for h in (2, 1, 1))
    clean, _ = prefill(q, K, V, [0, n])
    bad = [1 + i for i in range(batch)]
    K2 = K.repeat(batch, 1, 1)
    for i, at in enumerate(bad):
        K2[i * n + at, 0, 5] = math.nan
    out, lse = prefill(q.repeat(batch, 1, 1), K2, V.repeat(batch, 1, 1), [n * i for i in range(batch + 1)])
    for i, at in enumerate(bad):
        rows, logs = out[i * n:(i + 1) * n], lse[i * n:(i + 1) * n]
        assert torch.equal(rows[:at], clean[:at]), at
        assert rows[at:].isnan().all() and logs[at:].isnan().all(), at


def test_prefill_masked_values_of_the_types_limit():
    # values of 2^127 that earlier rows do not see leave those rows as they were
    g = torch.Generator().manual_seed(22)
    n = 128
    q, K, V = (values(g, (n, h, 128), torch.bfloat16).cuda() for h in (4, 1, 1))
    clean, _ = prefill(q, K, V, [0, n])
    for at in (1, 17, 63, 64, 100):
        V2 = V.clone()
        V2[at:] = 2.0 ** 127
        out, _ = prefill(q, K, V2, [0, n])
        assert torch.equal(out[:at], clean[:at]), at


def test_prefill_logits_of_any_size():
    # every logit near -2^110: the largest still gives its row a finite mean
    n, d = 70, 64
    q = torch.zeros((n, 1, d), dtype=torch.bfloat16, device="cuda")
    K = torch.zeros((n, 1, d), dtype=torch.bfloat16, device="cuda")
    V = values(torch.Generator().manual_seed(23), (n, 1, d), torch.bfloat16).cuda()
    q[..., 0] = 2.0 ** 56
    K[..., 0] = -(2.0 ** 57)
    out, _ = prefill(q, K, V, [0, n])
    want = V.double().cumsum(0) / torch.arange(1, n + 1, device="cuda")[:, None, None]
    mag = V.double().abs().cumsum(0) / torch.arange(1, n + 1, device="cuda")[:, None, None]
    # equal weights of exactly 2^0: one 32-bit addition per key, one division, the output's rounding
    assert ((out.double() - want).abs() <= mag * (2 * n * 2.0 ** -23) + 2.0 ** -8 * want.abs()).all()


def test_prefill_reports_bad_offsets_and_serves_the_rest():
    g = torch.Generator().manual_seed(10)
    q, K, V = (values(g, (200, h, 128), torch.bfloat16).cuda() for h in (4, 1, 1))
    bad = rkv.STATUS_CODE["RKV_ERR_INVALID_ARG"]
    out, lse = prefill(q, K, V, [0, 100, 201], expect=bad)          # the second leaves q
    check_prefill(q, K, V, [0, 100], lambda b: (K[:100], V[:100]), out, lse)
    assert (out[100:] == 7).all()
    out, lse = prefill(q, K, V, [100, 50, 150], kv_off=[0, 50, 150], expect=bad)   # a negative length
    check_prefill(q, K, V, [50, 150], lambda b: (K[50:150], V[50:150]), out, lse)
    out, lse = prefill(q, K, V, [0, 100, 200], kv_off=[0, 100, 200], kv_len=[100, 101], expect=bad)
    check_prefill(q, K, V, [0, 100], lambda b: (K[:100], V[:100]), out, lse)
    out, lse = prefill(q, K, V, [0, 100, 200], kv_off=[-1, 99, 199], expect=bad)
    assert (out[:100] == 7).all()


def test_prefill_many_sequences_and_streams():
    g = torch.Generator().manual_seed(11)
    r = random.Random(11)
    lens = [r.randint(0, 40) for _ in range(256)]
    n = sum(lens)
    q, K, V = (values(g, (n, h, 64), torch.float16).cuda() for h in (4, 2, 2))
    off = offsets(lens)
    want, _ = prefill(q, K, V, off)
    check_prefill(q, K, V, off, lambda b: (K[off[b]:off[b + 1]], V[off[b]:off[b + 1]]), want, None)
    op = rkv.Prefill(rkv.make_prefill_config(64, 2, 4, 256, n, n, in_dtype=rkv.RKV_DTYPE_F16))
    o, outs = ints(off), [torch.zeros_like(q) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, out in zip(streams, outs):
            op.attend(q, K, V, o, out, stream=s)
    torch.cuda.synchronize()
    assert op.device_error() == 0
    assert all(torch.equal(out, want) for out in outs)


def test_prefill_captured_graph_follows_device_lengths():
    g = torch.Generator().manual_seed(12)
    q, K, V = (values(g, (300, h, 128), torch.bfloat16).cuda() for h in (8, 2, 2))
    off, out = ints([0, 100, 300]), torch.zeros((300, 8, 128), dtype=torch.bfloat16, device="cuda")
    op = rkv.Prefill(rkv.make_prefill_config(128, 2, 8, 2, 300, 300))
    op.attend(q, K, V, off, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        op.attend(q, K, V, off, out)
    for cut in (100, 257, 0, 299):
        off.copy_(ints([0, cut, 300]))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        o = [0, cut, 300]
        check_prefill(q, K, V, o, lambda b: (K[o[b]:o[b + 1]], V[o[b]:o[b + 1]]), out, None)


# --- block tables -----------------------------------------------------------------------------

def check_tables(t, want):
    assert t.lengths.tolist() == want.len
    assert int(t.n_free) == len(want.free)
    assert t.free_list[:len(want.free)].tolist() == want.free
    for b, n in enumerate(want.len):
        k = -(-n // want.block)
        assert t.table[b, :k].tolist() == want.table[b][:k]


@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("batch,most", [(1, 3000), (5, 700), (33, 90), (256, 40)])
def test_tables_follow_the_definition(block, batch, most):
    r = random.Random(block + batch)
    max_blocks, n_blocks = -(-4 * most // block) + 1, batch * (-(-4 * most // block) + 1)
    t, want = rkv.BlockTables(batch, max_blocks, block, n_blocks), ref.Tables(batch, max_blocks, block, n_blocks)
    for step in range(4):
        new = [r.choice([0, 1, r.randint(0, most)]) for _ in range(batch)]
        slots, off = want.extend(new)
        pad = r.choice([0, 1, 77])
        got = torch.full((len(slots) + pad,), 5, dtype=torch.int32, device="cuda")
        t.extend(ints(new), got)
        assert t.device_error() == 0
        assert got.tolist() == slots + [-1] * pad
        assert t.new_off.tolist() == off
        check_tables(t, want)
        ended = [int(r.random() < 0.3) for _ in range(batch)]
        t.release(ints(ended))
        want.release(ended)
        assert t.device_error() == 0
        check_tables(t, want)


def test_tables_refuse_without_taking():
    t = rkv.BlockTables(3, 4, 16, 6)
    slots = torch.zeros(100, dtype=torch.int32, device="cuda")
    t.extend(ints([16, 17, 0]), slots)                     # 3 of 6 blocks
    assert t.device_error() == 0
    before = [x.clone() for x in (t.table, t.lengths, t.n_free, t.free_list)]
    work, bad = rkv.STATUS_CODE["RKV_ERR_WORKSPACE"], rkv.STATUS_CODE["RKV_ERR_INVALID_ARG"]
    for new, size, code in (([16, 16, 33], 100, work),     # four more blocks
                            ([49, 0, 0], 100, work),       # five blocks in a row of four
                            ([8, 8, 8], 23, work),         # slot map too short
                            ([1, -1, 1], 100, bad), ([2 ** 31 - 1, 2 ** 31 - 1, 0], 100, work)):
        s = torch.full((size,), 9, dtype=torch.int32, device="cuda")
        t.extend(ints(new), s)
        assert t.device_error() == code
        assert (s == -1).all() and (t.new_off == 0).all()
        assert all(torch.equal(a, b) for a, b in zip(before, (t.table, t.lengths, t.n_free, t.free_list)))
    # giving back more than the pool holds
    t.n_free.fill_(5)
    t.release(ints([1, 1, 0]))
    assert t.device_error() == rkv.STATUS_CODE["RKV_ERR_CORRUPT"]
    assert int(t.n_free) == 5 and torch.equal(t.lengths, before[1])


@pytest.mark.parametrize("batch,new,room", [(5, 2000, 12000), (3, 10, 40), (200, 9, 2000)])
def test_tables_replayed_in_place(batch, new, room):
    # a captured call that grows its own lengths, for the one-CTA forms and the one with a second launch; two such graphs
    # replayed in turn on two table sets
    r = random.Random(batch)
    block, width = 32, 400
    sets = [(rkv.BlockTables(batch, width, block, 9000), ref.Tables(batch, width, block, 9000)) for _ in range(2)]
    counts = ints([0] * batch)
    slots = torch.zeros(room, dtype=torch.int32, device="cuda")
    graphs = []
    for t, _ in sets:
        t.extend(counts, slots)                      # nothing new: also loads the kernels
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            t.extend(counts, slots)
        graphs.append(g)
    for step in range(6):
        t, want = sets[step % 2]
        add = [r.randint(0, new) for _ in range(batch)]
        counts.copy_(ints(add))
        graphs[step % 2].replay()
        ws, _ = want.extend(add)
        assert slots.tolist() == ws + [-1] * (room - len(ws))
        check_tables(t, want)
        assert t.device_error() == 0


def test_tables_report_block_ids_outside_the_pool():
    t = rkv.BlockTables(1, 4, 16, 6)
    t.free_list[5] = 6
    slots = torch.zeros(4, dtype=torch.int32, device="cuda")
    t.extend(ints([4]), slots)
    assert t.device_error() == rkv.STATUS_CODE["RKV_ERR_CORRUPT"]
    assert (slots == -1).all()


# --- the 8-bit store --------------------------------------------------------------------------

def cache_of(code, d=128, hkv=2, hq=None, block=16, n_blocks=40, max_blocks=20, batch=4, dtype=torch.bfloat16, **kw):
    cfg = rkv.make_kv8_config(d, hkv, hq or hkv, block, n_blocks, max_blocks, batch, KV8[code], CODE[dtype], **kw)
    return rkv.KV8Cache(cfg)


def same_cache(cache, rk, rv):
    for c, s, r in ((cache.codes_K, cache.scale_K, rk), (cache.codes_V, cache.scale_V, rv)):
        assert torch.equal(s.cpu(), r.scale)
        assert torch.equal(c.cpu().view(torch.uint8), r.codes.view(torch.uint8))


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("d,block,dtype", [(128, 16, torch.bfloat16), (64, 32, torch.float16), (128, 64, torch.float16),
                                           (64, 128, torch.bfloat16), (128, 128, torch.bfloat16)])
def test_store_bit_for_bit(code, d, block, dtype):
    # whole prompts, then ragged pieces, then single tokens whose size grows and falls
    g = torch.Generator().manual_seed(d + block)
    t = ref.Tables(4, 20, block, 40)
    cache = cache_of(code, d=d, block=block, dtype=dtype)
    rk, rv = (ref.Store(40, 2, block, d, code) for _ in range(2))
    r = random.Random(3)
    for step, new in enumerate([[2 * block + 3, block, 1, 0], [5, block + 1, 0, 7], [1, 1, 1, 1], [1, 0, 1, 1],
                                [1, 1, 1, 1], [1, 1, 1, 1], [3, 2, 1, 4]]):
        slots, _ = t.extend(new)
        size = r.choice([0.01, 1.0, 5.0, 300.0])
        K, V = ((values(g, (len(slots), 2, d), dtype).float() * size).to(dtype) for _ in range(2))
        if step == 3:
            K[0] = 0
        cache.store(K.cuda(), V.cuda(), ints(slots))
        rk.put(K, slots)
        rv.put(V, slots)
        assert cache.device_error() == 0
        same_cache(cache, rk, rv)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_store_extremes(code):
    # zeros, the largest and smallest values, ties between codes, a block that starts with zeros
    d, block = 64, 16
    cache = cache_of(code, d=d, block=block, hkv=1)
    rk, rv = (ref.Store(40, 1, block, d, code) for _ in range(2))
    big = torch.finfo(torch.bfloat16).max
    rows = [torch.zeros(d), torch.full((d,), big), torch.full((d,), 1e-38), torch.full((d,), 2.0 ** -133),
            (torch.arange(d).float() - 32) / 4, torch.arange(d).float() * 127 / 64]
    x = torch.stack(rows).to(torch.bfloat16).unsqueeze(1)
    slots = [0, 16, 32, 48, 64, 80]
    for s in (slots, [v + 1 for v in slots], [v + 2 for v in reversed(slots)]):
        cache.store(x.cuda(), x.flip(0).contiguous().cuda(), ints(s))
        rk.put(x, s)
        rv.put(x.flip(0), s)
        assert cache.device_error() == 0
        same_cache(cache, rk, rv)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_store_skips_and_reports(code):
    g = torch.Generator().manual_seed(2)
    d, block = 128, 32
    cache = cache_of(code, d=d, block=block, hkv=3)
    rk, rv = (ref.Store(40, 3, block, d, code) for _ in range(2))
    K, V = (values(g, (40, 3, d), torch.bfloat16) for _ in range(2))
    slots = list(range(64, 96)) + [-1, -5, 40 * block, 2 ** 31 - 1, 5 * block, 5 * block + 1, -1, 7 * block]
    cache.store(K.cuda(), V.cuda(), ints(slots))
    rk.put(K, slots)
    rv.put(V, slots)
    assert cache.device_error() == rkv.STATUS_CODE["RKV_ERR_CORRUPT"]
    same_cache(cache, rk, rv)
    K[3, 1, 5], K[3, 1, 6], V[34, 2, 0] = math.inf, math.nan, -math.inf
    slots = list(range(256, 288)) + [-1] * 2 + [288, 289] + [-1] * 4
    cache.store(K.cuda(), V.cuda(), ints(slots))
    rk.put(K, slots)
    rv.put(V, slots)
    assert cache.device_error() == rkv.STATUS_CODE["RKV_ERR_INVALID_ARG"]
    same_cache(cache, rk, rv)


def test_store_strided_rows():
    # K and V inside one fused buffer, and heads-first rows of the compressor's layout
    g = torch.Generator().manual_seed(4)
    d, block = 128, 16
    fused = values(g, (50, 8, d), torch.bfloat16).cuda()
    for K, V in ((fused[:, 2:4], fused[:, 6:8]), (fused[:, 2:4].transpose(0, 1).contiguous().transpose(0, 1),
                                                  fused[:, 6:8].transpose(0, 1).contiguous().transpose(0, 1))):
        cache = cache_of("int8", d=d, block=block)
        rk, rv = (ref.Store(40, 2, block, d, "int8") for _ in range(2))
        slots = list(range(16, 66))
        cache.store(K, V, ints(slots))
        rk.put(K.cpu(), slots)
        rv.put(V.cpu(), slots)
        assert cache.device_error() == 0
        same_cache(cache, rk, rv)


# --- decode over the 8-bit cache ----------------------------------------------------------------

def random_cache(gen, code, lens, d, hkv, hq, block, dtype, spread=4.0, out_dtype=None):
    need = [-(-n // block) for n in lens]
    width = max(1, max(need))
    n_blocks = sum(need) + 5
    cache = cache_of(code, d=d, hkv=hkv, hq=hq, block=block, n_blocks=n_blocks, max_blocks=width, batch=len(lens),
                     dtype=dtype, out_dtype=None if out_dtype is None else CODE[out_dtype])
    ids = torch.randperm(n_blocks, generator=gen).tolist()
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    for b, k in enumerate(need):
        table[b, :k] = torch.tensor(ids[:k])
        ids = ids[k:]
    # rows behind the lengths and blocks outside the tables: the worst patterns (NaN codes, NaN scales)
    for codes, scale in ((cache.codes_K, cache.scale_K), (cache.codes_V, cache.scale_V)):
        codes.view(torch.uint8).fill_(0x7f)
        scale.fill_(math.nan)
        for b, n in enumerate(lens):
            for j in range(need[b]):
                live = min(block, n - j * block)
                x = torch.randn((hkv, live, d), generator=gen)
                x = (x * 30).round().clamp(-127, 127).to(torch.int8) if code == "int8" else (x * 100).clamp(-448, 448).to(ref.KIND[code])
                codes[table[b, j], :, :live] = x.cuda()
                scale[table[b, j]] = (torch.exp2((torch.rand(hkv, generator=gen) - 0.5) * spread) / 30).cuda()
    return cache, table


def side_rows(codes, scale, ids, n):
    v = codes.cpu().double()[ids] * scale.cpu().double()[ids][..., None, None]
    return v.transpose(1, 2).reshape(-1, v.shape[1], v.shape[3])[:n]


def check_decode(cache, table, lens, q, out):
    block = cache.c.block_size
    for b, n in enumerate(lens):
        ids = table[b, :-(-n // block)].long()
        k, v = side_rows(cache.codes_K, cache.scale_K, ids, n), side_rows(cache.codes_V, cache.scale_V, ids, n)
        want, _, mag, spread = ref.attention(q[b:b + 1].cpu(), k, v, torch.ones((1, n), dtype=torch.bool))
        floor = 2.0 ** -40 * (127.0 if cache.codes_V.dtype is torch.int8 else 448.0)
        floor *= float(cache.scale_V[ids.cuda()].max()) if n else 0.0
        tol, _ = ref.bounds(want, mag, spread, q.shape[2], n, torch.float16, out.dtype, floor)
        err = (out[b:b + 1].double().cpu() - want).abs()
        assert (err <= tol).all(), f"request {b} of {n}: {float((err / tol).max())} times the bound"


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("hq,hkv,d,block,dtype", [
    (4, 1, 128, 16, torch.bfloat16), (8, 2, 64, 32, torch.float16), (14, 2, 128, 64, torch.bfloat16),
    (2, 2, 128, 128, torch.float16), (16, 1, 128, 16, torch.bfloat16), (18, 2, 64, 16, torch.bfloat16),
    (16, 2, 128, 32, torch.bfloat16), (26, 2, 128, 64, torch.float16)])
def test_decode_lengths_and_heads(code, hq, hkv, d, block, dtype):
    g = torch.Generator().manual_seed(hq + d + block)
    lens = [0, 1, 15, 16, 17, 63, 64, 65, 200, 1000, 129]
    for odt in (dtype, torch.float32):
        cache, table = random_cache(g, code, lens, d, hkv, hq, block, dtype, out_dtype=odt)
        q = values(g, (len(lens), hq, d), dtype).cuda()
        out = torch.full((len(lens), hq, d), 7.0, dtype=odt, device="cuda")
        cache.decode(q, table.cuda(), ints(lens), out)
        assert cache.device_error() == 0
        check_decode(cache, table, lens, q, out)
        assert (out[0] == 0).all()


@pytest.mark.parametrize("n", [2048, 9999, 40000])
def test_decode_long_requests(n):
    g = torch.Generator().manual_seed(n)
    cache, table = random_cache(g, "int8", [n, 3], 128, 2, 8, 128, torch.bfloat16)
    q = values(g, (2, 8, 128), torch.bfloat16).cuda()
    out = torch.empty_like(q)
    cache.decode(q, table.cuda(), ints([n, 3]), out)
    assert cache.device_error() == 0
    check_decode(cache, table, [n, 3], q, out)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_decode_scales_far_apart(code):
    # value scales over 2^80, key scales over a few octaves; a block of zeros (scale 0)
    g = torch.Generator().manual_seed(1)
    lens = [300, 77]
    cache, table = random_cache(g, code, lens, 128, 2, 8, 16, torch.bfloat16)
    n = cache.scale_V.shape[0]
    cache.scale_V.copy_(torch.exp2(torch.linspace(-40, 40, n))[:, None].expand(-1, 2))
    cache.scale_V[int(table[0, 3])] = 0.0
    cache.codes_V[int(table[0, 3])] = torch.zeros_like(cache.codes_V[0])
    q = values(g, (2, 8, 128), torch.bfloat16).cuda()
    out = torch.empty((2, 8, 128), dtype=torch.bfloat16, device="cuda")
    cache.decode(q, table.cuda(), ints(lens), out)
    assert cache.device_error() == 0
    check_decode(cache, table, lens, q, out)


def test_decode_many_requests_and_sharp_queries():
    g = torch.Generator().manual_seed(2)
    r = random.Random(2)
    lens = [r.randint(0, 90) for _ in range(256)]
    cache, table = random_cache(g, "int8", lens, 64, 2, 8, 16, torch.bfloat16)
    q = values(g, (256, 8, 64), torch.bfloat16).cuda()
    q[::3] *= 100.0
    q[1::3] *= 2.0 ** -30
    out = torch.empty_like(q)
    cache.decode(q, table.cuda(), ints(lens), out)
    assert cache.device_error() == 0
    check_decode(cache, table, lens, q, out)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_decode_zero_scales_and_nan_queries(code):
    # a value scale of 0 makes its block's values 0 whatever the codes; a NaN in a query reaches its head alone
    g = torch.Generator().manual_seed(9)
    lens = [300, 5000]
    cache, table = random_cache(g, code, lens, 64, 2, 6, 16, torch.bfloat16)
    for b, j in ((0, 2), (0, 18), (1, 100)):
        cache.scale_V[int(table[b, j])] = 0.0
    q = values(g, (2, 6, 64), torch.bfloat16).cuda()
    out = torch.empty_like(q)
    cache.decode(q, table.cuda(), ints(lens), out)
    assert cache.device_error() == 0
    # rows behind the lengths hold NaN patterns: a reference block of zeros stands for scale 0
    for b, j in ((0, 2), (0, 18), (1, 100)):
        cache.codes_V[int(table[b, j])] = torch.zeros_like(cache.codes_V[0])
    check_decode(cache, table, lens, q, out)
    q2 = q.clone()
    q2[0, 4, 63] = math.nan
    q2[1, 0, 0] = math.nan
    out2 = torch.empty_like(q)
    cache.decode(q2, table.cuda(), ints(lens), out2)
    hit = torch.zeros((2, 6), dtype=torch.bool)
    hit[0, 4] = hit[1, 0] = True
    assert out2[hit].isnan().all() and torch.equal(out2[~hit], out[~hit])


def test_decode_logits_of_any_size():
    # every logit near -2^111: the mean of the values all the same
    cache, table = random_cache(torch.Generator().manual_seed(10), "int8", [200], 64, 1, 1, 16, torch.bfloat16, spread=0.0)
    cache.codes_K.fill_(0)
    cache.codes_K[..., 0] = -64
    cache.scale_K.fill_(2.0 ** 52)
    q = torch.zeros((1, 1, 64), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 2.0 ** 56
    out = torch.empty((1, 1, 64), dtype=torch.bfloat16, device="cuda")
    cache.decode(q, table.cuda(), ints([200]), out)
    v = side_rows(cache.codes_V, cache.scale_V, table[0, :13].long(), 200)
    want, mag = v.mean(0), v.abs().mean(0)
    # equal logits x: log2 sV is added to x, whose step hides it, so the weights are equal before the V scales, which are
    # all 2^0 / 30; a weight of 2^15, one 32-bit addition per token, the factors' roundings, the output's
    assert ((out[0].double().cpu() - want).abs() <= mag * (2 * 200 + 8) * 2.0 ** -23 + 2.0 ** -8 * want.abs()).all()


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_cache_offsets_past_32_bits(code):
    # 8.6 GB of codes a side: blocks at both ends of the pool
    g = torch.Generator().manual_seed(11)
    d, hkv, block, n_blocks = 128, 8, 128, 1 << 16
    cache = cache_of(code, d=d, hkv=hkv, hq=hkv, block=block, n_blocks=n_blocks, max_blocks=3, batch=2)
    table = torch.tensor([[n_blocks - 1, 0, n_blocks // 2 + 1], [n_blocks - 2, 1, 5]], dtype=torch.int32)
    lens = [300, 130]
    K, V = (values(g, (sum(lens), hkv, d), torch.bfloat16) for _ in range(2))
    slots = [int(table[b, p // block]) * block + p % block for b, n in enumerate(lens) for p in range(n)]
    cache.store(K.cuda(), V.cuda(), ints(slots))
    small = table.flatten().tolist()                  # the same blocks in a pool of six
    rk, rv = (ref.Store(6, hkv, block, d, code) for _ in range(2))
    moved = [small.index(s // block) * block + s % block for s in slots]
    rk.put(K, moved)
    rv.put(V, moved)
    ids = table.flatten().long().cuda()
    for c, s, r in ((cache.codes_K, cache.scale_K, rk), (cache.codes_V, cache.scale_V, rv)):
        assert torch.equal(s[ids].cpu(), r.scale)
        assert torch.equal(c[ids].cpu().view(torch.uint8), r.codes.view(torch.uint8))
    q = values(g, (2, hkv, d), torch.bfloat16).cuda()
    out, want = torch.empty_like(q), torch.empty_like(q)
    cache.decode(q, table.cuda(), ints(lens), out)
    near = rkv.KV8Cache(rkv.make_kv8_config(d, hkv, hkv, block, 6, 3, 2, KV8[code]), *(x[ids].contiguous() for x in (
        cache.codes_K, cache.codes_V, cache.scale_K, cache.scale_V)))
    near.decode(q, ints(range(6)).view(2, 3), ints(lens), want)
    assert cache.device_error() == 0 and near.device_error() == 0
    assert torch.equal(out, want)


def test_prefill_offsets_past_32_bits():
    # rows 2^24 elements apart in 10 GB: the last keys and outputs lie past 2^32 elements
    g = torch.Generator().manual_seed(12)
    n, step, d = 300, 1 << 24, 64
    store = torch.empty(n * step, dtype=torch.bfloat16, device="cuda")
    at = lambda k: torch.as_strided(store, (n, 2, d), (step, d, 1), 1024 * k)  # noqa: E731
    q, K, V = (values(g, (n, 2, d), torch.bfloat16).cuda() for _ in range(3))
    want, wlse = prefill(q, K, V, [0, 100, n])
    for k, x in enumerate((q, K, V)):
        at(k).copy_(x)
    out, lse = prefill(at(0), at(1), at(2), [0, 100, n], dict(q_strides=(step, d), kv_strides=(step, d, 0),
                                                              out_strides=(step, d)), out=at(3))
    assert torch.equal(out, want) and torch.equal(lse, wlse)


def test_prefill_without_keys():
    # no key row at all: zeros and log-sums of -inf
    q = torch.ones((5, 4, 64), dtype=torch.float16, device="cuda")
    K = torch.empty((0, 2, 64), dtype=torch.float16, device="cuda")
    out, lse = prefill(q, K, K, [0, 2, 5], kv_off=[0, 0, 0])
    assert (out == 0).all() and (lse == -math.inf).all()


def test_decode_reports_corruption():
    g = torch.Generator().manual_seed(3)
    lens = [100, 90]
    cache, table = random_cache(g, "e4m3", lens, 128, 2, 8, 16, torch.bfloat16)
    q = values(g, (2, 8, 128), torch.bfloat16).cuda()
    out, want = torch.empty_like(q), torch.empty_like(q)
    cache.decode(q, table.cuda(), ints(lens), want)
    assert cache.device_error() == 0
    corrupt = rkv.STATUS_CODE["RKV_ERR_CORRUPT"]
    bad = table.clone()
    bad[0, 2] = cache.c.n_blocks
    cache.decode(q, bad.cuda(), ints(lens), out)
    assert cache.device_error() == corrupt
    assert torch.equal(out[1], want[1]) and out[0].isfinite().all()      # block skipped, the other request untouched
    cache.decode(q, table.cuda(), ints([100, 16 * table.shape[1] + 1]), out)
    assert cache.device_error() == corrupt
    cache.decode(q, table.cuda(), ints([100, -3]), out)
    assert cache.device_error() == corrupt
    assert torch.equal(out[0], want[0]) and (out[1] == 0).all()


@pytest.mark.parametrize("code,dtype", [("int8", torch.bfloat16), ("e4m3", torch.float16)])
@pytest.mark.parametrize("hq,hkv,d,block", [(8, 1, 128, 16), (3, 3, 64, 32), (24, 2, 64, 64), (14, 2, 128, 128)])
@pytest.mark.parametrize("batch", [1, 5, 40, 256])
def test_decode_short_and_long_rows(code, dtype, hq, hkv, d, block, batch):
    # the same requests by rows of few blocks (units by clusters) and by rows that could hold 5000 tokens (workspace)
    g = torch.Generator().manual_seed(batch + hq)
    r = random.Random(batch)
    top = 500 if batch < 40 else 130
    lens = [r.choice([0, 1, 63, 64, r.randint(0, top), top]) for _ in range(batch)]
    cache, table = random_cache(g, code, lens, d, hkv, hq, block, dtype)
    q = values(g, (batch, hq, d), dtype).cuda()
    wide = torch.full((batch, -(-5000 // block)), -1, dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    shape = dict(head_dim=d, n_kv_heads=hkv, n_q_heads=hq, block_size=block, n_blocks=cache.c.n_blocks, batch=batch,
                 code_type=KV8[code], in_dtype=CODE[dtype])
    long = rkv.KV8Cache(rkv.make_kv8_config(max_blocks=wide.shape[1], **shape), cache.codes_K, cache.codes_V,
                        cache.scale_K, cache.scale_V)
    corrupt = rkv.STATUS_CODE["RKV_ERR_CORRUPT"]
    for c, t in ((cache, table), (long, wide)):
        out = torch.full_like(q, 7.0)
        c.decode(q, t.cuda(), ints(lens), out)
        assert c.device_error() == 0
        check_decode(c, t, lens, q, out)
        b = max(range(batch), key=lambda i: lens[i])
        if lens[b] == 0:
            continue
        bad, other = t.clone(), torch.full_like(q, 7.0)
        bad[b, 0] = -7
        c.decode(q, bad.cuda(), ints(lens), other)
        assert c.device_error() == corrupt
        keep = torch.arange(batch) != b
        assert torch.equal(other[keep], out[keep]) and other[b].isfinite().all()
        over = list(lens)
        over[b] = t.shape[1] * block + 1
        full = t.clone()
        full[b] = t[b, 0]                            # every block of the row is one of the pool
        whole = torch.full_like(q, 7.0)
        c.decode(q, full.cuda(), ints(over), whole)
        assert c.device_error() == corrupt
        # a longer request moves the others' cuts between CTAs in the form with the workspace: not bit for bit there
        check_decode(c, t[keep], [n for i, n in enumerate(lens) if i != b], q[keep], whole[keep])


def test_decode_graphs_that_share_a_workspace_and_blocks():
    # two captured steps of one cache (one workspace), replayed in turn; requests that share a prefix's blocks; the
    # same request twice
    g = torch.Generator().manual_seed(14)
    lens = [3000, 3000, 2999, 70]
    cache, table = random_cache(g, "e4m3", lens, 128, 2, 8, 64, torch.bfloat16)
    table[1] = table[0]
    table[2, :40] = table[0, :40]
    q = [values(g, (4, 8, 128), torch.bfloat16).cuda() for _ in range(2)]
    q[0][1] = q[0][0]
    t, n = table.cuda(), ints(lens)
    outs, graphs = [torch.empty_like(x) for x in q], []
    for x, o in zip(q, outs):
        cache.decode(x, t, n, o)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            cache.decode(x, t, n, o)
        graphs.append(graph)
    want = [o.clone() for o in outs]
    for i in (0, 1, 1, 0, 1, 0):
        outs[i].zero_()
        graphs[i].replay()
        assert torch.equal(outs[i], want[i])
    assert torch.equal(want[0][0], want[0][1])
    assert cache.device_error() == 0
    for x, o in zip(q, want):
        check_decode(cache, table, lens, x, o)


def test_decode_on_two_streams_with_their_own_workspaces():
    g = torch.Generator().manual_seed(4)
    lens = [500, 3, 800]
    a, table = random_cache(g, "int8", lens, 128, 2, 8, 32, torch.bfloat16)
    b = rkv.KV8Cache(a.c, a.codes_K, a.codes_V, a.scale_K, a.scale_V)
    qs = [values(g, (3, 8, 128), torch.bfloat16).cuda() for _ in range(2)]
    t, n = table.cuda(), ints(lens)
    want = [torch.empty_like(q) for q in qs]
    for q, w in zip(qs, want):
        a.decode(q, t, n, w)
    outs = [torch.empty_like(q) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for c, q, o, s in zip((a, b), qs, outs, streams):
            c.decode(q, t, n, o, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))


# --- together -----------------------------------------------------------------------------------

@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_serving_loop(code):
    """Prompts are attended to and stored, then tokens are generated one by one, the decode step captured once and
    replayed; requests end, give their blocks back, and others begin in them."""
    g = torch.Generator().manual_seed(13)
    hq, hkv, d, block, batch, n_blocks = 8, 2, 128, 16, 3, 30
    tables, want = rkv.BlockTables(batch, 12, block, n_blocks), ref.Tables(batch, 12, block, n_blocks)
    cache = cache_of(code, d=d, hkv=hkv, hq=hq, block=block, n_blocks=n_blocks, max_blocks=12, batch=batch)
    rk, rv = (ref.Store(n_blocks, hkv, block, d, code) for _ in range(2))
    most = 200
    op = rkv.Prefill(rkv.make_prefill_config(d, hkv, hq, batch, most, most))

    def admit(new):
        n = sum(new)
        q, K, V = (values(g, (most, h, d), torch.bfloat16).cuda() for h in (hq, hkv, hkv))
        slots = torch.empty(most, dtype=torch.int32, device="cuda")
        out = torch.zeros_like(q)
        tables.extend(ints(new), slots)
        op.attend(q, K, V, tables.new_off, out)
        cache.store(K, V, slots)
        ws, off = want.extend(new)
        rk.put(K.cpu(), ws + [-1] * (most - n))
        rv.put(V.cpu(), ws + [-1] * (most - n))
        check_prefill(q, K, V, off, lambda b: (K[off[b]:off[b + 1]], V[off[b]:off[b + 1]]), out, None)
        assert (out[n:] == 0).all()

    ones, slots = ints([1] * batch), torch.empty(batch, dtype=torch.int32, device="cuda")
    q, K, V = (torch.zeros((batch, h, d), dtype=torch.bfloat16, device="cuda") for h in (hq, hkv, hkv))
    out = torch.zeros_like(q)

    def step():
        tables.extend(ones, slots)
        cache.store(K, V, slots)
        cache.decode(q, tables.table, tables.lengths, out)

    def fresh():
        for x in (q, K, V):
            x.copy_(values(g, tuple(x.shape), torch.bfloat16))

    def verify():
        ws, _ = want.extend([1] * batch)
        rk.put(K.cpu(), ws)
        rv.put(V.cpu(), ws)
        check_tables(tables, want)
        check_decode(cache, tables.table.cpu(), want.len, q, out)

    admit([100, 40, 7])
    fresh()
    step()
    verify()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(12):
        fresh()
        graph.replay()
        verify()
    tables.release(ints([1, 0, 1]))
    want.release([1, 0, 1])
    admit([0, 3, 90])
    for _ in range(5):
        fresh()
        graph.replay()
        verify()
    assert cache.device_error() == 0 and tables.device_error() == 0 and op.device_error() == 0
    used = [i for b in range(batch) for i in want.table[b][:-(-want.len[b] // block)]]
    for c, s, r in ((cache.codes_K, cache.scale_K, rk), (cache.codes_V, cache.scale_V, rv)):
        assert torch.equal(c.cpu().view(torch.uint8)[used], r.codes.view(torch.uint8)[used])
        assert torch.equal(s.cpu()[used], r.scale[used])
