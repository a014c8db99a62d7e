"""64-bit references of the serving operators (prompt attention, block tables, 8-bit block cache) and
the error bounds that their GPU tests use."""
from __future__ import annotations

import math

import numpy as np
import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
FIXED_HALF_STEP = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}   # below the normal range
QMAX = {"int8": 127.0, "e4m3": 448.0}
KIND = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


def attention(q, k, v, allowed, scale=None):
    """q [rows][hq][d], k and v [keys][hkv][d] (any float type), allowed [rows][keys] bool: out, lse and
    sum p|v| / sum p in 64 bits.  Rows without a key: zeros and -inf."""
    q, k, v = q.double(), k.double(), v.double()
    rows, hq, d = q.shape
    g = hq // k.shape[1]
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    out = torch.zeros_like(q)
    mag = torch.zeros_like(q)
    spread = torch.zeros((rows, hq), dtype=torch.float64, device=q.device)
    lse = torch.full((rows, hq), -math.inf, dtype=torch.float64, device=q.device)
    if k.shape[0]:
        for h in range(hq):
            kh, vh = k[:, h // g], v[:, h // g]
            s = (q[:, h] @ kh.T * scale).masked_fill(~allowed, -math.inf)
            top = s.amax(1, keepdim=True)
            p = torch.exp(s - top.masked_fill(top == -math.inf, 0.0))
            total = p.sum(1, keepdim=True)
            ok = total > 0
            out[:, h] = torch.where(ok, p @ vh / total, 0.0)
            mag[:, h] = torch.where(ok, p @ vh.abs() / total, 0.0)
            lse[:, h] = (top + total.log()).squeeze(1)
            spread[:, h] = (q[:, h].abs() @ kh.abs().T * scale).masked_fill(~allowed, 0.0).amax(1)
    return out, lse, mag, spread


def bounds(out, mag, spread, d, keys, weight_type, out_type, floor=0.0):
    """Largest allowed |error| of each output element, and of each log-sum.

    A logit is a 32-bit sum of d products: off by at most (d + 2) 2^-23 sum |q_c k_c| scale (a step of 2^-23
    per addition covers an accumulator that truncates), which moves a weight by that factor (up and down: twice
    after the division).  Weights are rounded to weight_type (half a step), the exponential is good to 2^-21 with
    its argument's rounding (|x| <= 2^3 above the running maximum; below it the weight shrinks faster than the
    argument's step grows: x 2^-23 2^x <= 2^-23), and the two sums over the keys add 2^-23 a key each.  All of it
    is relative to sum p|v| / sum p; then the output's own half step (a fixed one where the output is below its type's
    normal range).

    floor: a binary16 weight below 2^-14 has the fixed step 2^-24 instead of a relative one, so it is off by up to
    2^-25, whatever its size.  The largest weight w of a row is kept as at least 2^k (2^15 in the decode, 2^7 in
    prompt attention), which makes that 2^-(25 + k) w per key; the weights carry the value scales in the decode,
    so w |code| <= sum p * max scale * qmax, and it adds at most keys 2^-(25 + k) max|v| to the quotient, with max|v|
    the largest scale times qmax.  floor is 2^-(25 + k) max|v|."""
    logit = (d + 2) * 2.0 ** -23 * spread
    rel = 2 * logit + 2 * HALF_STEP[weight_type] * 0.5 + 2.0 ** -20 + 2 * keys * 2.0 ** -23
    tol = mag * rel[..., None] + HALF_STEP[out_type] * out.abs() + FIXED_HALF_STEP[out_type] + keys * floor + 1e-30
    return tol, logit + 2.0 ** -20 + keys * 2.0 ** -23


def lse_bound(lse, base):
    return base + 2.0 ** -22 * lse.abs().nan_to_num(posinf=0.0, neginf=0.0)


# --- the 8-bit store ------------------------------------------------------------------------

def _round_code(t, code):
    if code == "int8":
        return torch.from_numpy(np.rint(t.numpy())).clamp(-127, 127).to(torch.int8)
    return t.clamp(-448, 448).to(torch.float8_e4m3fn)


class Store:
    """One side of a block cache on the CPU, by the definition (32-bit quotients, exact powers of two)."""

    def __init__(self, n_blocks, hkv, block, d, code):
        self.code, self.block = code, block
        self.codes = torch.zeros((n_blocks, hkv, block, d), dtype=torch.uint8).view(KIND[code])
        self.scale = torch.zeros((n_blocks, hkv), dtype=torch.float32)

    def runs(self, slots):
        i = 0
        while i < len(slots):
            if slots[i] < 0 or slots[i] >= self.codes.shape[0] * self.block:
                i += 1
                continue
            j = i + 1
            while j < len(slots) and slots[j] == slots[j - 1] + 1 and slots[j] % self.block:
                j += 1
            yield i, j
            i = j

    def put(self, x, slots):
        """x [rows][hkv][d]."""
        x = x.float()
        qmax = np.float32(QMAX[self.code])
        for i, j in self.runs(list(slots)):
            blk, off = divmod(int(slots[i]), self.block)
            for h in range(x.shape[1]):
                rows = x[i:j, h]
                rows = torch.where(rows.isnan(), 0.0, rows)
                top = np.float32(torch.where(rows.isfinite(), rows, 0.0).abs().max())
                need = max(np.float32(top * (np.float32(1) / qmax)), np.float32(2.0 ** -64)) if top > 0 else np.float32(0)
                was = np.float32(self.scale[blk, h]) if off else np.float32(0)
                up = 0
                if was > 0:
                    while np.float32(np.ldexp(was, up)) < need:
                        up += 1
                    s = np.float32(np.ldexp(was, up))
                else:
                    s = need
                if up:
                    old = self.codes[blk, h, :off].float() * float(2.0 ** -up)
                    self.codes[blk, h, :off] = _round_code(old, self.code)
                self.scale[blk, h] = float(s)
                t = rows / torch.tensor(s) if s > 0 else torch.zeros_like(rows)
                self.codes[blk, h, off:off + j - i] = _round_code(t, self.code)

    def values(self):
        return self.codes.to(torch.float64) * self.scale.double()[..., None, None]

    def rows(self, ids, n):
        """The first n rows [n][hkv][d] of a request whose blocks are ids."""
        v = self.values()[torch.as_tensor(ids, dtype=torch.long)]
        return v.transpose(1, 2).reshape(-1, v.shape[1], v.shape[3])[:n]


class Tables:
    """Block tables by the definition."""

    def __init__(self, batch, max_blocks, block, n_blocks):
        self.block, self.n_blocks, self.max_blocks = block, n_blocks, max_blocks
        self.table = [[-1] * max_blocks for _ in range(batch)]
        self.free = list(range(n_blocks - 1, -1, -1))
        self.len = [0] * batch

    def extend(self, new):
        slots, off = [], [0]
        for b, m in enumerate(new):
            for p in range(self.len[b], self.len[b] + m):
                if p % self.block == 0:
                    self.table[b][p // self.block] = self.free.pop()
                slots.append(self.table[b][p // self.block] * self.block + p % self.block)
            self.len[b] += m
            off.append(len(slots))
        return slots, off

    def release(self, ended):
        for b, e in enumerate(ended):
            if e:
                self.free += self.table[b][:-(-self.len[b] // self.block)]
                self.len[b] = 0
