"""Oracle of the drafted tokens' verification (include/draft_verify.h) in Python integers and
fractions, request by request. Shares no code with the CUDA path.

`mutant` plants one mistake: 1: a draft stands where u q <= p; 2: the draw after a refusal takes
p, not max(p - q, 0); 3: the bonus token is drawn from the last draft's row; 4: the draw takes
the least token whose running sum reaches the point (>=)."""
from __future__ import annotations

import math
from fractions import Fraction

import numpy as np

COUNT, TOKEN, PROB, EMPTY, UNIFORM = 1, 2, 4, 8, 16
ONE = 1 << 60


class _Row:
    def __init__(self):
        self.status = 0

    def prob(self, x):
        x = float(x)
        if math.isnan(x) or x < 0:
            self.status |= PROB
            return 0.0
        if x > 1:
            self.status |= PROB
            return 1.0
        return x

    def uniform(self, u):
        u = float(u)
        if math.isnan(u) or u < 0:
            self.status |= UNIFORM
            return 0.0
        if u >= 1:
            self.status |= UNIFORM
            return 1.0 - 2.0 ** -24
        return u

    def units(self, row):
        return [round(Fraction(self.prob(x)) * ONE) for x in row]


def verify(target, draft, tokens, uniforms, n_drafts=None, mutant=0):
    """target [reqs, drafts + 1, vocab], draft the same with drafts rows or None, tokens
    [reqs, drafts], uniforms [reqs, drafts + 1]. Returns (out int32, kept int32, status)."""
    reqs, rows, vocab = target.shape
    drafts = rows - 1
    out, kept, status = np.full((reqs, rows), -1, np.int32), np.zeros(reqs, np.int32), 0
    for j in range(reqs):
        n = drafts if n_drafts is None else int(n_drafts[j])
        if not 0 <= n <= drafts:
            status |= COUNT
            continue
        w = _Row()
        a = 0
        while a < n:
            d = int(tokens[j, a])
            if not 0 <= d < vocab:
                w.status |= TOKEN
                break
            p = Fraction(w.prob(target[j, a, d]))
            q = Fraction(w.prob(draft[j, a, d])) if draft is not None else Fraction(1)
            u = Fraction(w.uniform(uniforms[j, a]))
            if not (u * q < p or (mutant == 1 and u * q == p)):
                break
            a += 1
        kept[j] = a
        out[j, :a] = tokens[j, :a]
        whole = w.units(target[j, max(0, a - 1) if mutant == 3 and a == n else a])
        weights = whole
        if a < n and mutant != 2:
            if draft is not None:
                less = w.units(draft[j, a])
                weights = [max(x - y, 0) for x, y in zip(whole, less)]
            else:
                weights = [0 if v == tokens[j, a] else x for v, x in enumerate(whole)]
            if sum(weights) == 0:
                weights = whole
        total = sum(weights)
        r = w.uniform(uniforms[j, drafts])
        if total == 0:
            w.status |= EMPTY
        else:
            if total > 8 * ONE:
                w.status |= PROB
            if total >= 15 * ONE:
                status |= w.status
                continue
            at = math.floor(Fraction(r) * total)
            run = 0
            for v, x in enumerate(weights):
                run += x
                if run > at or (mutant == 4 and run == at and run > 0):
                    out[j, a] = v
                    break
        status |= w.status
    return out, kept, status
