"""Oracle of the 8-bit paged KV cache: its store and the attention over it, in float64
NumPy, written from the formulas of include/kv8_attention.h, token by token and row by row.
Shares no code with the CUDA path.

`mutant` plants one mistake (tests check that each is noticed): store 1: the scale of a block
that grows is not applied to its earlier codes; 2: the block's old scale is forgotten; 3: the
least power of two above, not at, the maximum. attention 1: the value scale is left out; 2: key
head i % kv_heads; 3: one position too many."""
from __future__ import annotations

import math

import numpy as np

from .prologue import bf16_to_f64, e4m3_encode, e4m3_value

LEN, TABLE_WIDTH, TABLE_ENTRY, SLOT, TABLE_ROW, POSITION = 1, 2, 4, 8, 16, 32


def values(bits, dtype):
    """float64 of bf16 / fp16 bit patterns (uint16)."""
    bits = np.asarray(bits, np.uint16)
    return bits.view(np.float16).astype(np.float64) if dtype == "fp16" else bf16_to_f64(bits)


def least_scale(a: float, mutant: int = 0) -> float:
    """The least 2^e, e >= -120, with a <= 448 * 2^e (exact in float64)."""
    e = -120
    while a > 448.0 * 2.0 ** e or (mutant == 3 and a == 448.0 * 2.0 ** e):
        e += 1
    return 2.0 ** e


def place(table, row, pos, page_size, num_slots):
    """(slot, 0) of a position, or (-1, status bit)."""
    if pos < 0:
        return -1, POSITION
    if row < 0 or row >= table.shape[0]:
        return -1, TABLE_ROW
    if pos // page_size >= table.shape[1]:
        return -1, TABLE_WIDTH
    page = int(table[row, pos // page_size])
    if page < 0:
        return -1, TABLE_ENTRY
    slot = page * page_size + pos % page_size
    return (slot, 0) if slot < num_slots else (-1, SLOT)


def store(x, positions, token_table, table, page_size, block, codes, scales, mutant=0):
    """x float64 [tokens, heads, dim]; codes uint8 [num_slots, heads, dim] and scales
    float32 [num_slots / block, heads] are changed in place. Returns the status bits."""
    status, t = 0, 0
    tokens = len(positions)
    while t < tokens:
        pos, row = int(positions[t]), int(token_table[t])
        n = 1
        while (t + n < tokens and pos >= 0 and int(positions[t + n]) == pos + n
               and int(token_table[t + n]) == row and (pos + n) % block):
            n += 1
        slot, err = place(table, row, pos, page_size, codes.shape[0])
        status |= err
        if not err:
            off, b = pos % block, slot // block
            for h in range(codes.shape[1]):
                y = x[t:t + n, h]
                mag = np.abs(y)[np.isfinite(y)]
                s = least_scale(float(mag.max()) if mag.size else 0.0, mutant)
                old = float(scales[b, h])
                if off and mutant != 2:
                    s = max(s, old)
                if off and s > old and mutant != 1:
                    was = e4m3_value(codes[slot - off:slot, h])
                    codes[slot - off:slot, h] = e4m3_encode(was * (old / s))
                # the quotient is an fp32 number before it is rounded to a code
                with np.errstate(invalid="ignore", over="ignore"):
                    r = (y.astype(np.float32) / np.float32(s)).astype(np.float64)
                codes[slot:slot + n, h] = e4m3_encode(r)
                scales[b, h] = s
        t += n
    return status


def attend(q, slots, k, v, k_scale, v_scale, block, sm_scale, mutant=0):
    """One query row, q float64 [q_heads, dim], over the given slots. Returns float64 (out
    [q_heads, dim], lse [q_heads], and what the tolerance is made of: dx [q_heads], the
    largest sm_scale * sum |q k|; a [q_heads, dim], sum w |v|; top [q_heads], the largest
    w * v_scale; c [q_heads, dim], sum |v codes|)."""
    hq, dim = q.shape
    hk = k.shape[1]
    out, lse = np.zeros((hq, dim)), np.full(hq, -math.inf)
    dx, a, top, c = np.zeros(hq), np.zeros((hq, dim)), np.zeros(hq), np.zeros((hq, dim))
    slots = np.asarray(slots, np.int64)
    if slots.size == 0:
        return out, lse, dx, a, top, c
    for i in range(hq):
        h = i % hk if mutant == 2 else i // (hq // hk)
        kk = e4m3_value(k[slots, h]) * k_scale[slots // block, h].astype(np.float64)[:, None]
        code = e4m3_value(v[slots, h])
        sv = v_scale[slots // block, h].astype(np.float64)[:, None]
        vv = code if mutant == 1 else code * sv
        x = sm_scale * (kk @ q[i])
        m = x.max()
        e = np.exp(x - m)
        w = e / e.sum()
        lse[i] = m + math.log(e.sum())
        out[i] = w @ vv
        dx[i] = abs(sm_scale) * (np.abs(kk) @ np.abs(q[i])).max()
        a[i] = w @ np.abs(vv)
        top[i] = (w * sv[:, 0]).max()
        c[i] = np.abs(code).sum(0)
    return out, lse, dx, a, top, c


def row_slots(table, row, length, max_len, page_size, num_slots, mutant=0):
    """(slots, status) of the positions [0, length) of a table row."""
    if length < 0 or length > max_len:
        return np.zeros(0, np.int64), LEN
    if row < 0 or row >= table.shape[0]:
        return np.zeros(0, np.int64), TABLE_ROW
    if -(-length // page_size) > table.shape[1]:
        return np.zeros(0, np.int64), TABLE_WIDTH
    got, status = [], 0
    for p in range(length + (mutant == 3)):
        slot, err = place(table, row, p, page_size, num_slots)
        status |= err
        if not err:
            got.append(slot)
    return np.asarray(got, np.int64), status
