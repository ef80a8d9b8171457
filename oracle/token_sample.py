"""Oracle of token sampling (include/token_sample.h): one row at a time, weights by NumPy's fp32
step by step, sums and comparisons in Python integers and fractions. Shares no code with the
CUDA path.

`mutant` plants one mistake: 1: ties go to the higher index; 2: top-p keeps the tokens whose sum
is below p (one too few); 3: top-p is taken of all tokens, not of the first k; 4: the drawn
point is compared with >= ; 5: min-p against the probability."""
from __future__ import annotations

import math
from fractions import Fraction

import numpy as np

NAN, EMPTY, PARAM, UNIFORM = 1, 2, 4, 8
C = [np.float32(float.fromhex(x)) for x in (
    "-0x1.62e42cp-1", "0x1.ebfacp-3", "-0x1.c6948ep-5", "0x1.39e3fcp-7", "-0x1.4e2aeap-10",
    "0x1.c946d2p-14")]
LOG2E = np.float32(float.fromhex("0x1.715476p0"))


def weights(x, temperature):
    """Python integers: the weights of fp32 logits x (no NaN, some above -infinity)."""
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        scale = np.minimum(LOG2E / np.float32(temperature), np.finfo(np.float32).max)
        top = x.max()
        z = np.where(x == top, np.float32(0), (top - x) * scale)
    out = []
    for v in z:
        if not v < 41:
            out.append(0)
            continue
        n = np.floor(v)
        f = np.float32(v - n)
        y = C[5]
        for c in C[4::-1]:
            y = np.float32(y * f) + c
        y = np.float32(y * f) + np.float32(1)
        out.append(int(Fraction(float(y)) * 2 ** 40 / 2 ** int(n)))
    return out


def row(x, u=None, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, mutant=0):
    """(token or None, weights kept, status) of one row of fp32 logits."""
    status = 0
    x = np.array(x, np.float32)
    if np.isnan(x).any():
        status |= NAN
        x[np.isnan(x)] = -np.inf
    if not (0 <= temperature < math.inf):
        status |= PARAM
        temperature = 1.0
    if math.isnan(top_p):
        status |= PARAM
        top_p = 1.0
    if not min_p <= 1:
        status |= PARAM
        min_p = 0.0
    if u is not None and not 0 <= u < 1:
        status |= UNIFORM
        u = float(np.nextafter(np.float32(1), np.float32(0))) if u >= 1 else 0.0
    if (x == -np.inf).all():
        return (None if u is None else -1), [0] * len(x), status | EMPTY
    if temperature == 0:
        w = [0] * len(x)
        w[int(np.argmax(x))] = 1 << 40
    else:
        every = weights(x, temperature)
        order = sorted(range(len(x)), key=lambda i: (-float(x[i]), -i if mutant == 1 else i))
        if top_k > 0 and mutant != 3:
            order = order[:top_k]
        if top_p < 1:
            total, run, n = sum(every[i] for i in order), 0, 0
            need = Fraction(float(np.float32(top_p))) * total
            while n < len(order) and (n == 0 or run < need):
                run += every[order[n]]
                n += 1
            if mutant == 2 and n > 1:
                n -= 1
            order = order[:n]
        if top_k > 0 and mutant == 3:
            order = order[:top_k]
        w = [0] * len(x)
        kept = sum(every[i] for i in order)
        for i in order:
            least = Fraction(float(np.float32(min_p))) * (kept if mutant == 5 else 1 << 40)
            if every[i] >= least:
                w[i] = every[i]
    if u is None:
        return None, w, status
    at = math.floor(Fraction(float(np.float32(u))) * sum(w))
    run = 0
    for v, a in enumerate(w):
        run += a
        if run > at or (mutant == 4 and run >= at and run):
            return v, w, status
    raise AssertionError("no token")
