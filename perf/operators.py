"""Performance cases of the prompt and 8-bit-cache operators of librkv.

Four operators, in the order in which a serving loop uses them:

* ``prompt``: causal attention of packed prompts over their keys and values (grouped heads);
* ``tables``: block tables and slot maps from request lengths (blocks taken and given back);
* ``store8``: new keys and values into an 8-bit block cache, one scale per block and head;
* ``decode8``: attention of one new token per request over that cache.

``run`` computes an operator in its plain form with elementary torch operations, or, where the
module's ``own`` is true, through the library.  Lengths are drawn from the case alone, values
from the seed.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
QMAX = {"int8": 127.0, "e4m3": 448.0}
MIN_SCALE = 2.0 ** -64


# --- cases ------------------------------------------------------------------------------

def listed():
    return [
        # chat turns that arrive together: many short prompts, tiles mostly empty, latency counts
        dict(name="prompt_short_ragged", op="prompt", batch=16, lo=1, hi=200, prefix=0, hq=32, hkv=8, d=128,
             dtype="bf16", lse=False, lens=1),
        # the Qwen-shaped head layout (7 query heads per kv-head), documents of unequal length
        dict(name="prompt_ragged_g7", op="prompt", batch=8, lo=300, hi=2500, prefix=0, hq=28, hkv=4, d=128,
             dtype="bf16", lse=False, lens=2),
        # the next chunk of long prompts over the chunks before it; its log-sums join other parts
        dict(name="prompt_chunk_d64_f16", op="prompt", batch=4, lo=512, hi=512, prefix=4096, hq=16, hkv=4, d=64,
             dtype="f16", lse=True, lens=3),
        # one long prompt in the Llama-shaped layout, the largest call
        dict(name="prompt_long", op="prompt", batch=1, lo=8192, hi=8192, prefix=0, hq=32, hkv=8, d=128,
             dtype="bf16", lse=False, lens=4),
        # a decode step: one token for each of 256 requests
        dict(name="tables_step", op="tables", what="extend", batch=256, held=4000, new=1, block=16, lens=5),
        # prompts of the ragged batch admitted at once
        dict(name="tables_prompts", op="tables", what="extend", batch=8, held=0, new=32768, block=64, lens=6),
        # half of the requests end and give their blocks back
        dict(name="tables_release", op="tables", what="release", batch=64, held=16384, new=0, block=16, lens=7),
        # one token for each of 64 requests, into blocks that are partly full
        dict(name="store8_step", op="store8", batch=64, held=1000, new=1, hkv=8, d=128, block=64, code="int8",
             dtype="bf16", lens=8),
        # a whole 32768-token prompt of the Llama-shaped layer
        dict(name="store8_prompt", op="store8", batch=1, held=0, new=32768, hkv=8, d=128, block=64, code="e4m3",
             dtype="bf16", lens=9),
        # one request, short context: latency counts
        dict(name="decode8_one", op="decode8", batch=1, lo=2049, hi=2049, hq=32, hkv=8, d=128, block=16,
             code="int8", dtype="bf16", lens=10),
        # the ragged Qwen-shaped batch
        dict(name="decode8_ragged_g7", op="decode8", batch=8, lo=16384, hi=32768, hq=28, hkv=4, d=128, block=32,
             code="e4m3", dtype="bf16", lens=11),
        # long contexts in the Llama-shaped layout, the largest call
        dict(name="decode8_long", op="decode8", batch=4, lo=131072, hi=131072, hq=32, hkv=8, d=128, block=128,
             code="int8", dtype="bf16", lens=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "tables", "store8", "decode8"])
    heads = rng.choice([(32, 8), (28, 4), (16, 4), (8, 8), (16, 1), (12, 4), (10, 2)])
    d, dtype, code = rng.choice([64, 128]), rng.choice(["bf16", "f16"]), rng.choice(["int8", "e4m3"])
    block, lens = rng.choice([16, 32, 64, 128]), rng.randrange(1 << 20)
    if op == "prompt":
        hi = _log(rng, 2, 5000)
        batch = max(1, min(64, _log(rng, 1, 64), 40_000_000 // (hi * hi) or 1))
        prefix = rng.choice([0, 0, _log(rng, 1, 2000)]) if batch * hi * (hi + 2000) < 40_000_000 else 0
        return dict(op=op, batch=batch, lo=rng.choice([1, hi]), hi=hi, prefix=prefix, hq=heads[0], hkv=heads[1], d=d,
                    dtype=dtype, lse=rng.random() < 0.5, lens=lens)
    if op == "tables":
        batch = _log(rng, 1, 256)
        what = rng.choice(["extend", "extend", "release"])
        held = _log(rng, 1, 16384) if what == "release" else rng.choice([0, _log(rng, 1, 16384)])
        new = 0 if what == "release" else rng.choice([1, _log(rng, 2, 32768 * 8 // max(8, batch))])
        return dict(op=op, what=what, batch=batch, held=held, new=new, block=block, lens=lens)
    if op == "store8":
        batch = _log(rng, 1, 128)
        new = rng.choice([1, _log(rng, 2, max(3, 30000 // batch))])
        return dict(op=op, batch=batch, held=rng.choice([0, _log(rng, 1, 1000)]), new=new, hkv=heads[1], d=d,
                    block=block, code=code, dtype=dtype, lens=lens)
    hi = _log(rng, 1, 120000)
    batch = max(1, min(128, _log(rng, 1, 128), 4_000_000 // (hi * heads[1])))
    return dict(op=op, batch=batch, lo=rng.choice([1, hi]), hi=hi, hq=heads[0], hkv=heads[1], d=d, block=block,
                code=code, dtype=dtype, lens=lens)


def _lengths(case):
    """Host lengths of a case: (tokens held before, new tokens) of each request."""
    r = random.Random(case["lens"])
    n = case["batch"]
    if case["op"] == "prompt":
        new = [r.randint(case["lo"], case["hi"]) for _ in range(n)]
        return [r.randint((case["prefix"] + 1) // 2, case["prefix"]) for _ in range(n)], new
    if case["op"] == "decode8":
        return [r.randint(case["lo"], case["hi"]) for _ in range(n)], [1] * n
    held = [r.randint((case["held"] + 1) // 2, case["held"]) for _ in range(n)]
    return held, [r.randint((case["new"] + 1) // 2, case["new"]) for _ in range(n)]


def _blocks(n, block):
    return -(-n // block)


def work(case):
    held, new = _lengths(case)
    op = case["op"]
    if op == "prompt":
        d, hq, hkv = case["d"], case["hq"], case["hkv"]
        pairs = sum(n * h + n * (n + 1) // 2 for h, n in zip(held, new))
        rows, keys = sum(new), sum(held) + sum(new)
        return {"bytes": 2 * d * (2 * rows * hq + 2 * keys * hkv) + (4 * rows * hq if case["lse"] else 0),
                "flops": 4 * d * hq * pairs}
    if op == "tables":
        bs, n = case["block"], case["batch"]
        if case["what"] == "release":
            ended = [_blocks(h, bs) for i, h in enumerate(held) if i % 2 == 0]
            return {"bytes": 4 * (2 * sum(ended) + 3 * n + 2), "flops": n}
        more = sum(_blocks(h + m, bs) - _blocks(h, bs) for h, m in zip(held, new))
        return {"bytes": 4 * (sum(new) + 2 * more + 4 * n + 2), "flops": sum(new)}
    d, hkv, bs = case["d"], case["hkv"], case["block"]
    if op == "store8":
        blocks = sum(_blocks(h + m, bs) - h // bs for h, m in zip(held, new) if m)
        rows = sum(new)
        return {"bytes": 2 * hkv * (rows * d * 3 + blocks * 8) + 4 * rows, "flops": 2 * hkv * rows * d * 3}
    keys, blocks = sum(held), sum(_blocks(h, bs) for h in held)
    return {"bytes": 2 * hkv * (keys * d + 4 * blocks) + 4 * (blocks + case["batch"]) + 4 * case["batch"] * case["hq"] * d,
            "flops": 4 * d * case["hq"] * keys}


# --- inputs -----------------------------------------------------------------------------

def _values(g, shape, dtype, channels=4):
    """Rows as attention meets them: unit normal, a few channels eight times larger."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    hot = torch.randint(0, shape[-1], (channels,), generator=g, device="cuda")
    x[..., hot] *= 8.0
    return x.to(dtype)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _offsets(v):
    o = [0]
    for n in v:
        o.append(o[-1] + n)
    return o


def _pool(case, g, blocks_each):
    """Block ids for every request out of a shuffled pool: (table, pool size, ids left over)."""
    need = sum(blocks_each)
    total = need + max(8, need // 16)
    ids = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    width = max(1, max(blocks_each))
    at = _ints(_offsets(blocks_each)[:-1])[:, None] + torch.arange(width, dtype=torch.int32, device="cuda")
    inside = torch.arange(width, device="cuda") < _ints(blocks_each)[:, None]
    table = torch.where(inside, ids[at.clamp(max=total - 1).long()], torch.full_like(at, -1))
    return table.contiguous(), total, ids[need:]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    held, new = _lengths(case)
    op = case["op"]
    st = dict(case, held_host=held, new_host=new)
    if op == "prompt":
        dt, d, rows = DTYPES[case["dtype"]], case["d"], sum(new)
        keys = [h + m for h, m in zip(held, new)]
        st["q"] = torch.randn((rows, case["hq"], d), generator=g, device="cuda").to(dt)
        st["K"] = _values(g, (sum(keys), case["hkv"], d), dt)
        st["V"] = _values(g, (sum(keys), case["hkv"], d), dt)
        st["q_off"], st["kv_off"] = _ints(_offsets(new)), _ints(_offsets(keys))
        st["out"] = torch.empty_like(st["q"])
        st["lse_out"] = torch.empty((rows, case["hq"]), device="cuda") if case["lse"] else None
        if own:
            import long_context_attention_rkv_b200 as rkv
            code = rkv.RKV_DTYPE_BF16 if case["dtype"] == "bf16" else rkv.RKV_DTYPE_F16
            st["op_"] = rkv.Prefill(rkv.make_prefill_config(
                head_dim=d, n_kv_heads=case["hkv"], n_q_heads=case["hq"], batch=case["batch"], q_rows=rows,
                kv_rows=sum(keys), in_dtype=code))
        return st
    bs = case["block"]
    if op == "tables":
        n, have = case["batch"], [_blocks(h, bs) for h in held]
        total_each = [_blocks(h + m, bs) for h, m in zip(held, new)]
        width = max(1, max(total_each))
        table, n_blocks, left = _pool(case, g, have)
        more = sum(total_each) - sum(have)
        free = torch.full((n_blocks + more,), -1, dtype=torch.int32, device="cuda")
        ids = torch.cat([left, torch.arange(n_blocks, n_blocks + more, dtype=torch.int32, device="cuda")])
        free[:len(ids)] = ids[torch.randperm(len(ids), generator=g, device="cuda")]
        st["table"] = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
        st["table"][:, :table.shape[1]] = table[:, :width]
        st["lengths"], st["new"], st["free"], st["n_free"] = _ints(held), _ints(new), free, _ints([len(ids)])
        st["ended"] = _ints([1 - i % 2 for i in range(n)])
        st["rows"] = sum(new)
        st["slots"] = torch.empty(max(1, sum(new)), dtype=torch.int32, device="cuda")
        st["off"] = torch.empty(n + 1, dtype=torch.int32, device="cuda")
        st["lengths_out"], st["n_free_out"] = torch.empty_like(st["lengths"]), torch.empty_like(st["n_free"])
        st["status"] = _ints([0])
        if own:
            import long_context_attention_rkv_b200 as rkv
            st["cfg"] = rkv.make_blocks_config(batch=n, max_blocks=width, block_size=bs, n_blocks=len(free))
        return st
    dt, d, hkv = DTYPES[case["dtype"]], case["d"], case["hkv"]
    keys = [h + m for h, m in zip(held, new)] if op == "store8" else held
    table, n_blocks, _ = _pool(case, g, [_blocks(k, bs) for k in keys])
    for side in "KV":
        # rows of the values above in 8 bits: unit normal channels against a scale that a hot channel set
        codes = torch.randn((n_blocks, hkv, bs, d), generator=g, device="cuda")
        if case["code"] == "int8":
            codes = codes.mul_(28.0).round_().clamp_(-127, 127).to(torch.int8)
        else:
            codes = codes.mul_(100.0).clamp_(-448, 448).to(torch.float8_e4m3fn)
        st["codes_" + side] = codes
        size = 4.0 * torch.exp2(torch.rand((n_blocks, hkv), generator=g, device="cuda") - 0.5)
        st["scale_" + side] = size / QMAX[case["code"]]
    st["table"], st["n_blocks"] = table, n_blocks
    if op == "store8":
        rows = sum(new)
        st["K"], st["V"] = _values(g, (rows, hkv, d), dt), _values(g, (rows, hkv, d), dt)
        seq = torch.repeat_interleave(torch.arange(case["batch"], device="cuda"), _ints(new).long(), output_size=rows)
        pos = torch.arange(rows, device="cuda") - _ints(_offsets(new))[seq] + _ints(held)[seq]
        st["slots"] = (table[seq, pos // bs] * bs + pos % bs).to(torch.int32)
        st["touched"] = torch.unique(st["slots"] // bs).long()
    else:
        st["lengths"] = _ints(held)
        st["q"] = torch.randn((case["batch"], case["hq"], d), generator=g, device="cuda").to(dt)
        st["out"] = torch.empty_like(st["q"])
    if own:
        import long_context_attention_rkv_b200 as rkv
        cfg = rkv.make_kv8_config(
            head_dim=d, n_kv_heads=hkv, n_q_heads=case.get("hq", hkv), block_size=bs, n_blocks=n_blocks,
            max_blocks=table.shape[1], batch=case["batch"],
            code_type=rkv.RKV_KV8_INT8 if case["code"] == "int8" else rkv.RKV_KV8_E4M3,
            in_dtype=rkv.RKV_DTYPE_BF16 if case["dtype"] == "bf16" else rkv.RKV_DTYPE_F16)
        st["cache"] = rkv.KV8Cache(cfg, st["codes_K"], st["codes_V"], st["scale_K"], st["scale_V"])
    return st


# --- plain forms --------------------------------------------------------------------------

def _padded(x, off, lens):
    """Packed rows [rows][heads][d] as [batch][heads][longest][d] in 32 bits, zeros behind each end."""
    at = off[:-1, None].long() + torch.arange(max(lens), device="cuda")
    inside = torch.arange(max(lens), device="cuda") < (off[1:] - off[:-1])[:, None]
    y = x[at.clamp(max=x.shape[0] - 1)].float()
    return (y * inside[..., None, None]).transpose(1, 2)


def _softmax(s):
    """Softmax weights and log-sums over the last axis; a row of -inf alone gives zeros and -inf."""
    m = s.amax(-1, keepdim=True)
    p = s.sub_(m.masked_fill(m == -math.inf, 0.0)).exp_()
    total = p.sum(-1, keepdim=True)
    return p, total, (m + total.log()).squeeze(-1)


def _plain_prompt(st):
    q_off, kv_off, g = st["q_off"], st["kv_off"], st["hq"] // st["hkv"]
    new, keys = st["new_host"], [h + m for h, m in zip(st["held_host"], st["new_host"])]
    n, mq, mk, d = st["batch"], max(new), max(keys), st["d"]
    q, k, v = _padded(st["q"], q_off, new), _padded(st["K"], kv_off, keys), _padded(st["V"], kv_off, keys)
    q = q.reshape(n, st["hkv"], g * mq, d)
    s = torch.matmul(q, k.transpose(2, 3)).mul_(1.0 / math.sqrt(d)).view(n, st["hkv"], g, mq, mk)
    nq, nk = q_off[1:] - q_off[:-1], kv_off[1:] - kv_off[:-1]
    last = (nk - nq)[:, None] + torch.arange(mq, device="cuda")          # last key that row i of a chunk sees
    s.masked_fill_((torch.arange(mk, device="cuda") > last[..., None])[:, None, None], -math.inf)
    p, total, lse = _softmax(s)
    o = torch.matmul(p.view(n, st["hkv"], g * mq, mk), v).view(n, st["hkv"], g, mq, d)
    o = torch.where(total > 0, o / total, 0.0)
    seq = torch.repeat_interleave(torch.arange(n, device="cuda"), nq.long(), output_size=sum(new))
    row = torch.arange(sum(new), device="cuda") - q_off[seq]
    out = {"out": o.permute(0, 3, 1, 2, 4)[seq, row].reshape(sum(new), st["hq"], d).to(st["q"].dtype)}
    if st["lse"]:
        out["lse"] = lse.permute(0, 3, 1, 2)[seq, row].reshape(sum(new), st["hq"])
    return out


def _plain_tables(st):
    bs, table, lengths = st["block"], st["table"], st["lengths"]
    n, width = table.shape
    have = (lengths + bs - 1) // bs
    col = torch.arange(width, device="cuda")
    if st["what"] == "release":
        given = have * st["ended"]
        first = torch.cumsum(given, 0) - given + st["n_free"]
        at = first[:, None] + col
        live = col < given[:, None]
        free = st["free"]
        free = torch.cat([free, free.new_empty(1)]).scatter(0, torch.where(live, at, len(free)).reshape(-1),
                                                           table.reshape(-1))[:-1]
        return {"free": free, "lengths": lengths * (1 - st["ended"]), "n_free": (st["n_free"] + given.sum()).int()}
    after = lengths + st["new"]
    more = (after + bs - 1) // bs - have
    first = torch.cumsum(more, 0) - more
    at = st["n_free"] - 1 - (first[:, None] + col - have[:, None])
    fresh = (col >= have[:, None]) & (col < (have + more)[:, None])
    table.copy_(torch.where(fresh, st["free"][at.clamp(0, len(st["free"]) - 1).long()], table))
    off = torch.cat([st["new"].new_zeros(1), torch.cumsum(st["new"], 0)]).int()
    seq = torch.repeat_interleave(torch.arange(n, device="cuda"), st["new"].long(), output_size=st["rows"])
    pos = torch.arange(st["rows"], device="cuda") - off[seq] + lengths[seq]
    slots = (table[seq, pos // bs] * bs + pos % bs).int()
    return {"table": table, "slots": slots, "off": off, "lengths": after, "n_free": (st["n_free"] - more.sum()).int()}


def _codes(x, code):
    """x / scale in 8 bits."""
    return x.round().clamp(-127, 127).to(torch.int8) if code == "int8" else x.clamp(-448, 448).to(torch.float8_e4m3fn)


def _plain_store(st):
    bs, code, t = st["block"], st["code"], st["touched"]
    blk, off = (st["slots"] // bs).long(), (st["slots"] % bs).long()
    out = {}
    for side in "KV":
        x, codes, scale = st[side].float(), st["codes_" + side], st["scale_" + side]
        top = torch.zeros_like(scale).scatter_reduce_(0, blk[:, None].expand(-1, st["hkv"]), x.abs().amax(-1), "amax")[t]
        start = torch.full((st["n_blocks"],), bs, device="cuda").scatter_reduce_(0, blk, off, "amin")[t]
        old = torch.where(start[:, None] == 0, 0.0, scale[t])
        need = torch.where(top > 0, (top / QMAX[code]).clamp(min=MIN_SCALE), 0.0)
        # the old scale times the smallest power of two that reaches what the new rows need
        (mo, eo), (mn, en) = torch.frexp(old), torch.frexp(need)
        up = torch.where((old > 0) & (need > old), en - eo + (mn > mo).int(), 0)
        s = torch.where(old > 0, torch.ldexp(old, up), need)
        rows = codes[t].float()
        again = _codes(torch.ldexp(rows, -up[..., None, None]), code)
        keep = torch.arange(bs, device="cuda") < start[:, None]
        flat = codes.view(torch.uint8)
        flat[t] = torch.where(keep[:, None, :, None], again.view(torch.uint8), flat[t])
        scale[t] = s
        by = scale[blk][..., None]
        flat[blk, :, off] = _codes(torch.where(by > 0, x / by, 0.0), code).view(torch.uint8)
        out["codes_" + side], out["scale_" + side] = codes, scale
    return out


def _gathered(st, side, real=torch.float32):
    """A side of the cache in request order: [batch][heads][longest][d]."""
    t = st["table"].clamp(min=0).long()
    x = st["codes_" + side].view(torch.uint8)[t].view(st["codes_" + side].dtype).to(real)
    x *= st["scale_" + side][t][..., None, None].to(real)
    n, w, h, bs, d = x.shape
    return x.transpose(1, 2).reshape(n, h, w * bs, d)


def _plain_decode(st):
    n, h, d = st["batch"], st["hkv"], st["d"]
    q = st["q"].float().view(n, h, st["hq"] // h, d)
    s = torch.matmul(q, _gathered(st, "K").transpose(2, 3)).mul_(1.0 / math.sqrt(d))
    s.masked_fill_((torch.arange(s.shape[-1], device="cuda") >= st["lengths"][:, None])[:, None, None], -math.inf)
    p, total, _ = _softmax(s)
    o = torch.matmul(p, _gathered(st, "V"))
    return torch.where(total > 0, o / total, 0.0).view(n, st["hq"], d).to(st["q"].dtype)


def run(state):
    st, op = state, state["op"]
    if not own:
        return {"prompt": _plain_prompt, "tables": _plain_tables, "store8": _plain_store, "decode8": _plain_decode}[op](st)
    if op == "prompt":
        st["op_"].attend(st["q"], st["K"], st["V"], st["q_off"], st["out"], kv_off=st["kv_off"], lse=st["lse_out"])
        return {"out": st["out"], "lse": st["lse_out"]} if st["lse"] else {"out": st["out"]}
    if op == "tables":
        import long_context_attention_rkv_b200 as rkv
        if st["what"] == "release":
            rkv.rkv_blocks_release(st["cfg"], st["lengths"], st["ended"], st["table"], st["free"], st["n_free"],
                                   st["lengths_out"], st["n_free_out"], st["status"])
            return {"free": st["free"], "lengths": st["lengths_out"], "n_free": st["n_free_out"]}
        rkv.rkv_blocks_extend(st["cfg"], st["lengths"], st["new"], st["table"], st["free"], st["n_free"], st["off"],
                              st["slots"], st["rows"], st["lengths_out"], st["n_free_out"], st["status"])
        return {"table": st["table"], "slots": st["slots"], "off": st["off"], "lengths": st["lengths_out"],
                "n_free": st["n_free_out"]}
    if op == "store8":
        st["cache"].store(st["K"], st["V"], st["slots"])
        return {k: st[k] for k in ("codes_K", "scale_K", "codes_V", "scale_V")}
    st["cache"].decode(st["q"], st["table"], st["lengths"], st["out"])
    return st["out"]


# --- the definitions in 64 bits -----------------------------------------------------------

def _attend(q, k, v, allowed):
    """One request in 64 bits: q [rows][hq][d], k and v [keys][hkv][d], allowed [rows][keys]."""
    rows, hq, d = q.shape
    out, lse = torch.zeros_like(q), torch.full((rows, hq), -math.inf, dtype=torch.float64, device="cuda")
    some = allowed.any(1)
    for h in range(hq):
        kv = h // (hq // k.shape[1])
        logit = (q[:, h] @ k[:, kv].T / math.sqrt(d)).masked_fill_(~allowed, -math.inf)
        lse[:, h] = torch.logsumexp(logit, 1)
        weight = torch.exp(logit - lse[:, h, None].masked_fill(~some[:, None], 0.0))
        out[:, h] = weight @ v[:, kv]
    return out, lse


def exact(case, seed):
    op = case["op"]
    if op == "tables":
        return None
    st = prepare(case, seed)
    held, new = st["held_host"], st["new_host"]
    if op == "prompt":
        parts, q0, k0 = [], 0, 0
        for h, m in zip(held, new):
            q, k, v = (st[x][a:b].double() for x, a, b in (("q", q0, q0 + m), ("K", k0, k0 + h + m), ("V", k0, k0 + h + m)))
            seen = torch.arange(h + m, device="cuda") <= h + torch.arange(m, device="cuda")[:, None]
            parts.append(_attend(q, k, v, seen))
            q0, k0 = q0 + m, k0 + h + m
        out = {"out": torch.cat([p[0] for p in parts])}
        if case["lse"]:
            out["lse"] = torch.cat([p[1] for p in parts])
        return out
    bs = case["block"]
    if op == "decode8":
        parts = []
        for b, n in enumerate(held):
            ids = st["table"][b, :_blocks(n, bs)].long()
            k, v = ((st["codes_" + s].view(torch.uint8)[ids].view(st["codes_" + s].dtype).double() *
                     st["scale_" + s][ids].double()[..., None, None]).transpose(1, 2).reshape(-1, case["hkv"], case["d"])[:n]
                    for s in "KV")
            parts.append(_attend(st["q"][b:b + 1].double(), k, v, torch.ones(1, n, dtype=torch.bool, device="cuda"))[0])
        return torch.cat(parts)
    # store8: the scale in 64 bits and, for codes with an exponent, the quotients before rounding
    out = {}
    for side in "KV":
        x, scale = st[side].double(), st["scale_" + side].double()
        quot = st["codes_" + side].double() if case["code"] == "e4m3" else None
        row = 0
        for b, (h, m) in enumerate(zip(held, new)):
            for first in range(h // bs, _blocks(h + m, bs)) if m else ():
                lo, hi = max(first * bs, h), min((first + 1) * bs, h + m)
                part = x[row + lo - h:row + hi - h]
                top = part.abs().amax((0, 2)) / QMAX[case["code"]]
                top = torch.where(top > 0, top.clamp(min=MIN_SCALE), top)
                ident = int(st["table"][b, first])
                was = scale[ident] if lo > first * bs else torch.zeros_like(top)
                # the border between two powers lies where the 32-bit need is compared
                steps = torch.ceil(torch.log2(top.float().double() / was)).clamp(min=0).nan_to_num(posinf=0.0)
                now = torch.where(was > 0, was * torch.exp2(steps), top)
                scale[ident] = now
                if quot is not None:
                    quot[ident, :, :lo - first * bs] *= torch.exp2(-steps)[:, None, None]
                    quot[ident, :, lo - first * bs:hi - first * bs] = (part / now[:, None].clamp(min=MIN_SCALE)).transpose(0, 1)
            row += m
        out["codes_" + side], out["scale_" + side] = quot, scale
    return out
