"""GPU parity of the serving operators where 32-bit logits, weights of few bits and scales of any size meet: what
rounding must not turn into infinities, zeros or another mean."""
import math

import pytest
import torch

import long_context_attention_rkv_b200 as rkv
import serving_ref as ref
from test_gpu_serving import CODE, ints, random_cache, side_rows

pytestmark = pytest.mark.gpu


# --- decode over the 8-bit cache ----------------------------------------------------------------

def widened(cache, table, tokens):
    """The same cache behind table rows that could hold `tokens` tokens (the form with the workspace and the join)."""
    c = cache.c
    wide = torch.full((table.shape[0], -(-tokens // c.block_size)), -1, dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    cfg = rkv.make_kv8_config(c.head_dim, c.n_kv_heads, c.n_q_heads, c.block_size, c.n_blocks, wide.shape[1], c.batch,
                              c.code_type, c.in_dtype, c.out_dtype, c.scale)
    return rkv.KV8Cache(cfg, cache.codes_K, cache.codes_V, cache.scale_K, cache.scale_V), wide


def decode_both(cache, table, lens, q, check):
    """By both forms: `check` on the output of each."""
    odt = {v: k for k, v in CODE.items()}[cache.c.out_dtype]
    for c, t in ((cache, table), widened(cache, table, 40000)):
        out = torch.full(q.shape, 7.0, dtype=odt, device="cuda")
        c.decode(q, t.cuda(), ints(lens), out)
        assert c.device_error() == 0
        check(out)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("d,hq,hkv", [(64, 4, 2), (128, 3, 1), (128, 24, 2)])
@pytest.mark.parametrize("exponent", [12, 20, 23, 24, 25, 26, 27, 28, 30, 40, 70, 100])
def test_decode_far_logits(code, d, hq, hkv, exponent):
    """One channel carries logits near +-2^exponent with odd significands, taken from three key codes, so the tokens of
    the largest logit share the weight, whatever their value scales; the others lie at least 2^(exponent - 5) below.

    A product of two codes is exact in 32 bits, so equal codes have equal logits and the logit part of the bound is
    0: spread is 0 in it.  (At 2^12 the next code's weight is 2^-128 or less.)"""
    g = torch.Generator().manual_seed(exponent + hq)
    lens = [700, 130, 1]
    cache, table = random_cache(g, code, lens, d, hkv, hq, 16, torch.bfloat16, out_dtype=torch.float32)
    pick = torch.tensor([64.0, 88.0, 104.0])[torch.randint(0, 3, tuple(cache.codes_K.shape[:3]), generator=g)]
    cache.codes_K.view(torch.uint8).zero_()
    cache.codes_K[..., 0] = pick.to(cache.codes_K.dtype).cuda()
    # the largest |logit|: scale * q * 104 * scale_K
    cache.scale_K.fill_(2.0 ** (exponent // 2) * 1.2345)
    top = 2.0 ** (exponent - exponent // 2) * math.sqrt(d) / 104 / 1.2345
    q = torch.zeros((len(lens), hq, d))
    q[..., 0] = top * (0.5 + torch.rand((len(lens), hq), generator=g)) * (torch.randint(0, 2, (len(lens), hq), generator=g) * 2 - 1)
    q = q.to(torch.bfloat16).cuda()

    def check(out):
        assert out.isfinite().all()
        for b, n in enumerate(lens):
            ids = table[b, :-(-n // 16)].long()
            k, v = side_rows(cache.codes_K, cache.scale_K, ids, n), side_rows(cache.codes_V, cache.scale_V, ids, n)
            want, _, mag, spread = ref.attention(q[b:b + 1].cpu(), k, v, torch.ones((1, n), dtype=torch.bool))
            floor = 2.0 ** -40 * ref.QMAX[code] * float(cache.scale_V[ids.cuda()].max())
            tol, _ = ref.bounds(want, mag, 0.0 * spread, d, n, torch.float16, torch.float32, floor)
            err = (out[b:b + 1].double().cpu() - want).abs()
            assert (err <= tol).all(), f"request {b}: {float((err / tol).max())} times the bound"

    decode_both(cache, table, lens, q, check)
