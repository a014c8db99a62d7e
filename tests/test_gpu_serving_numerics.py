"""GPU parity of the serving operators where 32-bit logits, weights of few bits and scales of any size meet: what
rounding must not turn into infinities, zeros or another mean."""
import math
import random

import pytest
import torch

import long_context_attention_rkv_b200 as rkv
import serving_ref as ref
from test_gpu_serving import cache_of, check_prefill, ints, offsets, prefill, same_cache, values

pytestmark = pytest.mark.gpu


# --- decode over the 8-bit cache ----------------------------------------------------------------

def block_cache(gen, code, form, d, hq, hkv):
    """Random codes in shuffled blocks of 16 tokens, fp32 out, in the two forms of the decode, several tiles of 64 tokens per CTA
    in both: "clusters" (150 rows of at most 512 tokens) and "workspace" (5 requests of up to 30000 tokens)."""
    lens = [512, 300, 1, 64, 65] * 30 if form == "clusters" else [30000, 17, 20000, 25001, 129]
    need = [-(-n // 16) for n in lens]
    n_blocks, width = sum(need), max(need)
    cache = cache_of(code, d=d, hkv=hkv, hq=hq, block=16, n_blocks=n_blocks, max_blocks=width, batch=len(lens),
                     out_dtype=rkv.RKV_DTYPE_F32)
    ids = torch.randperm(n_blocks, generator=gen, dtype=torch.int32)
    table = torch.zeros((len(lens), width), dtype=torch.int32)
    for b, (k, lo) in enumerate(zip(need, offsets(need))):
        table[b, :k] = ids[lo:lo + k]
    for codes, scale in ((cache.codes_K, cache.scale_K), (cache.codes_V, cache.scale_V)):
        x = torch.randn(codes.shape, generator=gen) * 30
        codes.copy_((x.round() if code == "int8" else x).clamp(-127, 127).to(codes.dtype))
        scale.copy_(torch.exp2((torch.rand(scale.shape, generator=gen) - 0.5) * 4.0) / 30)
    return cache, table, lens


def check_all(cache, table, lens, q, with_logits=True):
    """Every request against the reference.  with_logits False: logits that are exact up to one rounding that equal ones
    share, so their part of the bound is 0.

    The floor of the bound (weights below binary16's normal range) also holds where a block of scale 0 sets the running
    maximum, with the smallest scale 2^-64, and all other weights are small: the sum of the weights is 2^15 2^64 or more there, so
    steps of 2^-25 times codes move the quotient by keys 2^-104 qmax at most, and no scale but 0 is below 2^-64."""
    out = torch.full(q.shape, 7.0, device="cuda")
    cache.decode(q.cuda(), table.cuda(), ints(lens), out)
    assert cache.device_error() == 0
    got = out.double().cpu()
    assert got.isfinite().all()
    sides = [(c.cpu().float(), s.cpu().double()) for c, s in ((cache.codes_K, cache.scale_K), (cache.codes_V, cache.scale_V))]
    qmax = 127.0 if cache.codes_V.dtype is torch.int8 else 448.0
    for b, n in enumerate(lens):
        ids = table[b, :-(-n // 16)].long()
        k, v = ((c[ids].double() * s[ids][..., None, None]).transpose(1, 2).reshape(-1, c.shape[1], c.shape[3])[:n]
                for c, s in sides)
        want, _, mag, spread = ref.attention(q[b:b + 1], k, v, torch.ones((1, n), dtype=torch.bool))
        floor = 2.0 ** -40 * qmax * float(sides[1][1][ids].max())
        tol, _ = ref.bounds(want, mag, spread if with_logits else 0.0 * spread, q.shape[2], n, torch.float16, torch.float32,
                            floor)
        err = (got[b:b + 1] - want).abs()
        assert (err <= tol).all(), f"request {b} of {n}: {float((err / tol).max())} times the bound"


@pytest.mark.parametrize("form", ["clusters", "workspace"])
@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("d,hq,hkv", [(64, 4, 2), (128, 3, 1), (128, 24, 2)])
@pytest.mark.parametrize("exponent", [12, 20, 23, 24, 25, 27, 28, 40, 100])
def test_decode_far_logits(form, code, d, hq, hkv, exponent):
    """One channel carries logits near +-2^exponent with odd significands, taken from three key codes, so the tokens of
    the largest logit share the weight, whatever their value scales; the others lie at least 2^(exponent - 5) below.

    A product of two codes is exact in 32 bits, so equal codes have equal logits and the logit part of the bound is
    0.  (At 2^12 the next code's weight is 2^-128 or less.)"""
    g = torch.Generator().manual_seed(exponent + hq)
    cache, table, lens = block_cache(g, code, form, d, hq, hkv)
    pick = torch.tensor([64.0, 88.0, 104.0])[torch.randint(0, 3, tuple(cache.codes_K.shape[:3]), generator=g)]
    cache.codes_K.view(torch.uint8).zero_()
    cache.codes_K[..., 0] = pick.to(cache.codes_K.dtype).cuda()
    # the largest |logit|: scale * q * 104 * scale_K
    cache.scale_K.fill_(2.0 ** (exponent // 2) * 1.2345)
    top = 2.0 ** (exponent - exponent // 2) * math.sqrt(d) / 104 / 1.2345
    q = torch.zeros((len(lens), hq, d))
    q[..., 0] = top * (0.5 + torch.rand((len(lens), hq), generator=g)) * (torch.randint(0, 2, (len(lens), hq), generator=g) * 2 - 1)
    check_all(cache, table, lens, q.to(torch.bfloat16), with_logits=False)


@pytest.mark.parametrize("form", ["clusters", "workspace"])
@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("exponents", [[-64], [-40], [-30], [-8], [80], [-64, 80], [-40, 60, 0, -10]])
@pytest.mark.parametrize("logits", ["equal", "spread", "zeros first", "zeros last"])
def test_decode_zero_value_scales_beside_any_other(form, code, exponents, logits):
    """Blocks whose value scale is 0 (values of 0, whatever their codes) among blocks with scales near 2^exponents: their
    tokens count in the sum of the weights and nowhere else.  All logits 0, spread, or those of the zero blocks
    the largest or the smallest by 2^5."""
    g = torch.Generator().manual_seed(len(exponents) + exponents[0] + 100)
    cache, table, lens = block_cache(g, code, form, 64, 6, 2)
    n, hkv = cache.scale_V.shape
    e = torch.tensor(exponents, dtype=torch.float32)[torch.randint(0, len(exponents), (n, hkv), generator=g)]
    scale_V = torch.exp2(e) * (1 + torch.rand((n, hkv), generator=g))
    zero = torch.rand((n, hkv), generator=g) < 0.2
    zero[table[:, 0].long()] = torch.tensor([True, False])
    scale_V[zero] = 0.0
    cache.scale_V.copy_(scale_V)
    q = values(g, (len(lens), 6, 64), torch.bfloat16)
    if logits == "equal":
        cache.scale_K.zero_()
    if logits.startswith("zeros"):
        codes = cache.codes_K.float()
        codes[..., 0] = torch.where(zero, 64.0, -64.0)[..., None].cuda() * (1 if logits == "zeros first" else -1)
        cache.codes_K.copy_(codes.to(cache.codes_K.dtype))
        cache.scale_K.fill_(1 / 32)
        q = q / 64
        q[..., 0] = 64.0
    check_all(cache, table, lens, q)



def test_decode_lengths_next_to_31_bits():
    """A length that the row cannot hold is clamped to the row, here the longest there is: 2^31 - 64 tokens, 2^27 - 4 times
    the same block: their mean is that block's.

    At most 2^31 / 64 / (148 * 4) + 1 = 56680 equal terms are added one after the other, in the numerator and in
    the sum, each with an error of 2^-24 of the total, then 10 merges; weights and logits as in the other bounds."""
    d, block = 64, 16
    n_blocks, width = 3, 2 ** 27 - 4
    g = torch.Generator().manual_seed(1)
    cache = cache_of("int8", d=d, hkv=1, hq=2, block=block, n_blocks=n_blocks, max_blocks=width, batch=1,
                     out_dtype=rkv.RKV_DTYPE_F32)
    for codes, scale in ((cache.codes_K, cache.scale_K), (cache.codes_V, cache.scale_V)):
        codes.copy_((torch.randn(codes.shape, generator=g) * 30).round().clamp(-127, 127).to(torch.int8))
        scale.fill_(1 / 32)
    q, out = values(g, (1, 2, d), torch.bfloat16).cuda(), torch.empty((1, 2, d), device="cuda")
    table = torch.full((1, width), 1, dtype=torch.int32, device="cuda")
    k, v = (c[1].double().cpu().transpose(0, 1) / 32 for c in (cache.codes_K, cache.codes_V))
    want, _, mag, spread = ref.attention(q.cpu(), k, v, torch.ones((1, block), dtype=torch.bool))
    tol, _ = ref.bounds(want, mag, spread, d, block, torch.float16, torch.float32, 2.0 ** -40 * 127 / 32)
    tol = tol + mag * 2 * (56680 + 10) * 2.0 ** -24
    cache.decode(q, table, ints([2 ** 31 - 1]), out)
    assert cache.device_error() == rkv.STATUS_CODE["RKV_ERR_CORRUPT"]
    assert ((out.double().cpu() - want).abs() <= tol).all()
    cache.decode(q, table, ints([2 ** 31 - 65]), out)            # one token less in the last block
    assert cache.device_error() == 0
    assert ((out.double().cpu() - want).abs() <= tol).all()


# --- prompt attention -------------------------------------------------------------------------

FAR = [(torch.bfloat16, e) for e in (12, 15, 16, 17, 20, 22, 24, 26, 28, 31, 36, 60, 100)] + \
      [(torch.float16, e) for e in (12, 15, 16, 17, 20, 22, 24, 26, 28)]


def check_far(q, K, V, off, out, lse, spread, scale=None, kv_off=None):
    kv_off = off if kv_off is None else kv_off
    for b in range(len(off) - 1):
        rows, keys = slice(off[b], off[b + 1]), slice(kv_off[b], kv_off[b + 1])
        n, L = off[b + 1] - off[b], kv_off[b + 1] - kv_off[b]
        allowed = torch.arange(L)[None] <= (L - n + torch.arange(n))[:, None]
        want, wlse, mag, s = ref.attention(q[rows].cpu(), K[keys].cpu(), V[keys].cpu(), allowed, scale)
        floor = 2.0 ** -32 * float(V[keys].abs().max()) if q.dtype is torch.float16 else 0.0
        tol, ltol = ref.bounds(want, mag, spread + 0.0 * s, q.shape[2], L, q.dtype, out.dtype, floor)
        got = out[rows].double().cpu()
        assert got.isfinite().all(), f"sequence {b}"
        assert ((got - want).abs() <= tol).all(), f"sequence {b}: {float(((got - want).abs() / tol).max())} times the bound"
        assert ((lse[rows].double().cpu() - wlse).abs() <= ref.lse_bound(wlse, ltol)).all(), f"sequence {b}: log-sums"


@pytest.mark.parametrize("dtype,exponent", FAR)
@pytest.mark.parametrize("d,hq,hkv,new,keys", [(64, 4, 1, [300, 70], None), (128, 7, 1, [150], None),
                                               (64, 8, 1, [3], [2000])])
def test_prefill_far_logits(dtype, exponent, d, hq, hkv, new, keys):
    """One channel carries logits near +-2^exponent with odd significands, three key values: the keys of the
    largest logit share the weight, the others lie at least 2^(exponent - 5) below.  A product of two 16-bit
    inputs is exact in 32 bits, so equal keys have equal logits and the logit part of the bound is 0.  Whole prompts,
    and few rows over many keys (shared by a cluster)."""
    g = torch.Generator().manual_seed(exponent + d)
    off = offsets(new)
    kv_off = off if keys is None else offsets(keys)
    n, L = off[-1], kv_off[-1]
    q, K = torch.zeros((n, hq, d)), torch.zeros((L, hkv, d))
    half = 2.0 ** (exponent // 2)
    K[..., 0] = half * torch.tensor([1.0, 1.375, 1.625])[torch.randint(0, 3, (L, hkv), generator=g)] * 1.0859375
    top = 2.0 ** exponent * math.sqrt(d) / half / 1.765
    scale = 0.0
    if dtype is torch.float16:                     # the range of q: the scale carries the rest
        scale = top / 8.0 / math.sqrt(d)
        top = 8.0
    q[..., 0] = top * (0.5 + torch.rand((n, hq), generator=g)) * (torch.randint(0, 2, (n, hq), generator=g) * 2 - 1)
    q, K, V = q.to(dtype).cuda(), K.to(dtype).cuda(), values(g, (L, hkv, d), dtype).cuda()
    out, lse = prefill(q, K, V, off, dict(out_dtype=rkv.RKV_DTYPE_F32, scale=scale), kv_off=None if keys is None else kv_off)
    check_far(q, K, V, off, out, lse, 0.0, scale=float(torch.tensor(scale)) or None, kv_off=kv_off)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("bits", [10, 14, 17, 20, 22])
@pytest.mark.parametrize("step", [3, 9, -4])
def test_prefill_far_maximum_that_moves_slowly(dtype, sign, bits, step):
    """Logits of sign 255 251 2^(bits - 16) / 2 and a second channel that adds whole numbers: the maximum grows by less than
    2^8 from tile to tile (or falls).  All logits and their differences are exact in 32 bits (24 bits hold them), and the
    weights that count lie within 60 of the largest: the rounding of 0.5 log2(e) moves an exponent by at most
    60 2^-23, which spread = 1 covers ((d + 2) 2^-23)."""
    n, d = 1000, 64
    g = torch.Generator().manual_seed(bits)
    q, K = torch.zeros((n, 2, d)), torch.zeros((n, 1, d))
    q[..., 0], q[..., 1] = 255.0, 1.0
    K[:, 0, 0] = sign * 251.0 * 2.0 ** (bits - 16)
    K[:, 0, 1] = (torch.arange(n) // 64 * step).float()
    q, K, V = q.to(dtype).cuda(), K.to(dtype).cuda(), values(g, (n, 1, d), dtype).cuda()
    out, lse = prefill(q, K, V, [0, n], dict(out_dtype=rkv.RKV_DTYPE_F32, scale=0.5))
    check_far(q, K, V, [0, n], out, lse, 1.0, scale=0.5)


@pytest.mark.parametrize("scale", [4.0, 1e30, 1e-30])
@pytest.mark.parametrize("keys", [468, 20, 449])
def test_prefill_rows_that_see_nothing_of_their_first_tile(scale, keys):
    """40 rows over few keys, each of a cluster's CTAs with one tile of 64 of them at most (the plane could hold 2000):
    the last tile's CTA has rows that see none of it, and with 20 keys half of the rows see none at all.  With
    factors whose product with the lowest maximum overflows, and a small one."""
    g = torch.Generator().manual_seed(keys)
    q, K, V = (values(g, (n, h, 64), torch.bfloat16).cuda() for n, h in ((40, 8), (2000, 1), (2000, 1)))
    q = (q.float() * (0.1 if scale == 4.0 else 1.0 / scale)).to(torch.bfloat16)
    out, lse = prefill(q, K, V, [0, 40], dict(scale=scale), kv_off=[0, 0], kv_len=[keys])
    check_prefill(q, K, V, [0, 40], lambda b: (K[:keys], V[:keys]), out, lse, scale=float(torch.tensor(scale)))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("hq,hkv,prefix", [(2, 2, 0), (4, 2, 9), (7, 1, 0), (16, 1, 130)])
def test_prefill_infinite_values_reach_no_further_than_said(dtype, hq, hkv, prefix):
    """An infinite or NaN value at a key: rows more than 128 / G + 14 before the first that sees it, other
    sequences and other channels are as without it; the rows that see it are not finite in its channel."""
    g = torch.Generator().manual_seed(hq)
    n, d, copies = 260, 64, 24
    L, group = n + prefix, hq // hkv
    q, K, V = (values(g, (m, h, d), dtype).cuda() for m, h in ((n, hq), (L, hkv), (L, hkv)))
    off, kv_off = [n * i for i in range(copies + 1)], [L * i for i in range(copies + 1)]
    clean, _ = prefill(q, K, V, [0, n], kv_off=[0, L])
    at = [prefix + 11 * i for i in range(copies)]
    V2 = V.repeat(copies, 1, 1)
    for i, key in enumerate(at[:-1]):                                # the last sequence stays clean
        V2[i * L + key, :, 5] = (math.inf, -math.inf, math.nan)[i % 3]
    out, lse = prefill(q.repeat(copies, 1, 1), K.repeat(copies, 1, 1), V2, off, kv_off=kv_off)
    assert lse.isfinite().all()
    for i, key in enumerate(at):
        rows, first = out[n * i:n * (i + 1)], key - prefix
        others = torch.arange(d) != 5
        assert torch.equal(rows[..., others], clean[..., others])
        if i == copies - 1:
            assert torch.equal(rows, clean)
            continue
        assert not rows[first:, :, 5].isfinite().any()
        far = max(0, first - (128 // group + 14))
        assert torch.equal(rows[:far], clean[:far]), (i, key)


# --- the 8-bit store --------------------------------------------------------------------------

@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("d,hkv,block,batch,rows,dtype", [
    # sizes at which the writer's windows of rows are 16, 16, 32, 64, 64, 128 and 128 long
    (64, 8, 16, 1, 700, torch.bfloat16), (128, 8, 16, 3, 1300, torch.float16), (64, 8, 32, 2, 1300, torch.float16),
    (128, 8, 64, 1, 2500, torch.bfloat16), (64, 12, 64, 2, 1700, torch.bfloat16), (64, 8, 128, 2, 5200, torch.float16),
    (128, 16, 128, 3, 2700, torch.bfloat16)])
def test_store_windows_of_many_runs(code, d, hkv, block, batch, rows, dtype):
    """Calls of many rows, bit for bit: runs that go on in a block from its middle, whole blocks, single tokens by the dozen
    (many runs in a window), skipped rows between them, runs over a window's end; sizes that grow and fall between runs, so
    scales grow in blocks that hold codes."""
    r = random.Random(rows + block)
    g = torch.Generator().manual_seed(rows)
    n_blocks = 3 * rows // block + 400
    cfg = rkv.make_kv8_config(d, hkv, hkv, block, n_blocks, n_blocks, batch, rkv.RKV_KV8_INT8 if code == "int8" else
                              rkv.RKV_KV8_E4M3, rkv.RKV_DTYPE_BF16 if dtype is torch.bfloat16 else rkv.RKV_DTYPE_F16)
    cache = rkv.KV8Cache(cfg)
    rk, rv = (ref.Store(n_blocks, hkv, block, d, code) for _ in range(2))
    held = [0] * n_blocks
    for call in range(3):
        slots, sizes = [], []
        free = [b for b in range(n_blocks) if held[b] < block]
        r.shuffle(free)
        while len(slots) < rows:
            kind = r.choice(["gap", "whole", "whole", "whole", "some", "singles"])
            if kind == "gap":
                m = r.randint(1, 40)
                slots += [r.choice([-1, -7])] * m
                sizes += [1.0] * m
                continue
            for _ in range(r.randint(1, 24) if kind == "singles" else 1):
                b = free.pop()
                m = 1 if kind == "singles" else block - held[b] if kind == "whole" else r.randint(1, block - held[b])
                slots += range(b * block + held[b], b * block + held[b] + m)
                sizes += [r.choice([0.02, 1.0, 1.0, 30.0])] * m
                held[b] += m
        for b in range(n_blocks):                      # the last run may have passed the end: keep what the call holds
            held[b] -= sum(b * block <= s < (b + 1) * block for s in slots[rows:])
        slots, sizes = slots[:rows], torch.tensor(sizes[:rows])[:, None, None]
        K, V = ((values(g, (rows, hkv, d), torch.float32) * sizes).to(dtype) for _ in range(2))
        cache.store(K.cuda(), V.cuda(), ints(slots))
        rk.put(K, slots)
        rv.put(V, slots)
        assert cache.device_error() == 0
        same_cache(cache, rk, rv)
