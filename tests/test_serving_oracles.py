"""Pins of the oracles of the 8-bit cache, the page operations and the drafts' verification:
hand-worked values, invariants, distributions, and planted mistakes that must show."""
import math
from fractions import Fraction

import numpy as np
import pytest

from oracle import draft_verify as DV
from oracle import kv8 as K8
from oracle import kv_pages as KP
from oracle.prologue import e4m3_encode, e4m3_value


def test_least_scale():
    for a, s in ((448.0, 1.0), (448.0001, 2.0), (447.0, 1.0), (224.0, 0.5), (0.0, 2.0 ** -120),
                 (7.0, 2.0 ** -6), (7.5, 2.0 ** -5), (3e38, 2.0 ** 120), (1e-40, 2.0 ** -120)):
        assert K8.least_scale(a) == s, a
    assert K8.least_scale(448.0, mutant=3) != 1.0


def _fresh(block=16, pages=2, page=32, heads=2, dim=4):
    return (np.zeros((pages * page, heads, dim), np.uint8),
            np.ones((pages * page // block, heads), np.float32))


def test_store_hand_worked():
    codes, scales = _fresh()
    table = np.array([[1, 0]], np.int32)
    x = np.zeros((2, 2, 4))
    x[0, 0] = [448, 1, -2, 0]
    x[1, 0] = [0.5, 0, 0, 0]
    assert K8.store(x, [0, 1], [0, 0], table, 32, 16, codes, scales) == 0
    assert scales[2, 0] == 1.0 and scales[2, 1] == 2.0 ** -120  # page 1 holds blocks 2, 3
    assert np.array_equal(e4m3_value(codes[32, 0]), [448, 1, -2, 0])
    # a third token of magnitude 896 doubles the scale: the earlier codes halve exactly
    y = np.full((1, 2, 4), 896.0)
    assert K8.store(y, [2], [0], table, 32, 16, codes, scales) == 0
    assert scales[2, 0] == 2.0
    assert np.array_equal(e4m3_value(codes[32, 0]) * 2, [448, 1, -2, 0])
    assert np.array_equal(e4m3_value(codes[34, 0]) * 2, [896] * 4)
    # a run that starts a block forgets the scale that was there
    assert K8.store(y / 896, [0], [0], table, 32, 16, codes, scales) == 0
    assert scales[2, 0] == 2.0 ** -8


@pytest.mark.parametrize("mutant", [1, 2, 3])
def test_store_mutants_show(mutant):
    rng = np.random.default_rng(1)
    table = np.array([[0, 1]], np.int32)
    got = []
    for m in (0, mutant):
        codes, scales = _fresh()
        for start, n, mag in ((0, 5, 7.0), (5, 3, 448.0), (8, 4, 1.0)):
            x = rng.uniform(-1, 1, (n, 2, 4)) * mag
            x[0, :, 0] = mag
            K8.store(x, list(range(start, start + n)), [0] * n, table, 32, 16, codes, scales,
                     mutant=m)
        got.append((codes, scales))
        rng = np.random.default_rng(1)
    assert not all(np.array_equal(a, b) for a, b in zip(*got))


def test_store_error_is_half_a_step():
    rng = np.random.default_rng(2)
    codes, scales = _fresh(dim=64)
    x = rng.standard_normal((32, 2, 64))
    K8.store(x, list(range(32)), [0] * 32, np.array([[0]], np.int32), 32, 16, codes, scales)
    val = e4m3_value(codes[:32]) * scales[np.arange(32) // 16][..., None]
    s = scales[np.arange(32) // 16][..., None]
    assert np.all(np.abs(val - x) <= np.maximum(np.abs(x) * 2.0 ** -4, s * 2.0 ** -10) * 1.0001)


def test_attention_by_hand_and_mutants():
    rng = np.random.default_rng(3)
    k = e4m3_encode(rng.standard_normal((32, 2, 64)) * 50)
    v = e4m3_encode(rng.standard_normal((32, 2, 64)) * 50)
    ks, vs = rng.uniform(0.01, 0.1, (2, 2, 2)).astype(np.float32)
    q = rng.standard_normal((4, 64))
    out, lse = K8.attend(q, [5], k, v, ks, vs, 16, 0.125)[:2]  # one key: its value
    for i in range(4):
        assert np.allclose(out[i], e4m3_value(v[5, i // 2]) * vs[0, i // 2], atol=1e-12)
    out, lse = K8.attend(q * 0, [1, 20, 20], k, v, ks, vs, 16, 0.125)[:2]  # equal weights
    mean = sum(e4m3_value(v[s, 1]) * vs[s // 16, 1] for s in (1, 20, 20)) / 3
    assert np.allclose(out[3], mean, atol=1e-12) and np.allclose(lse, math.log(3))
    out, lse = K8.attend(q, [], k, v, ks, vs, 16, 0.125)[:2]
    assert np.all(out == 0) and np.all(lse == -math.inf)
    ref = K8.attend(q, [1, 9, 30], k, v, ks, vs, 16, 0.125)[0]
    for m in (1, 2):
        assert not np.allclose(K8.attend(q, [1, 9, 30], k, v, ks, vs, 16, 0.125, mutant=m)[0], ref)
    table = np.array([[1, 0]], np.int32)
    assert K8.row_slots(table, 0, 17, 32, 16, 32)[0].tolist() == list(range(16, 32)) + [0]
    assert len(K8.row_slots(table, 0, 17, 32, 16, 32, mutant=3)[0]) == 18
    assert K8.row_slots(table, 0, 33, 64, 16, 32)[1] == K8.TABLE_WIDTH
    assert K8.row_slots(table, 1, 3, 64, 16, 32)[1] == K8.TABLE_ROW
    assert K8.row_slots(table, 0, -1, 64, 16, 32)[1] == K8.LEN


def _state(rng, n_tables=6, width=5, pages=40, page=16):
    table = np.full((n_tables, width), -1, np.int32)
    refs = np.zeros(pages, np.int32)
    planes = [rng.integers(0, 255, (pages, 12)).astype(np.uint8), rng.random((pages, 3))]
    return table, refs, planes


def _life(mutant=0, seed=4):
    """A few sequences grow, fork, append, roll back and are compacted. After each step the
    counts are the entries' and the tokens of every sequence read back."""
    rng = np.random.default_rng(seed)
    table, refs, planes = _state(rng)
    page, ok = 16, True
    truth = {}

    def write(r, a, b):
        KP_status = KP.reserve([r], [a], [b], table, page, refs, planes, mutant=mutant)
        assert KP_status == 0
        for p in range(a, b):
            planes[1][table[r, p // page], 0] = truth.setdefault(r, {}).setdefault(p // page,
                                                                                  rng.random())

    def check():
        good = np.array_equal(refs, np.bincount(table[table >= 0], minlength=len(refs)))
        for r, pages in truth.items():
            for c, x in pages.items():
                good &= table[r, c] >= 0 and planes[1][table[r, c], 0] == x
        return good

    write(0, 0, 40)
    write(1, 0, 16)
    assert sorted(table[table >= 0].tolist()) == ([0, 1, 2, 3] if mutant != 1 else [36, 37, 38, 39])
    KP.fork([0, 0], [2, 3], [40, 30], table, page, refs, mutant=mutant)
    truth[2], truth[3] = dict(truth[0]), {c: truth[0][c] for c in (0, 1)}
    ok &= check()
    for r, a in ((2, 40), (3, 30)):  # the shared tail page is copied before it is written
        KP.reserve([r], [a], [a + 1], table, page, refs, planes, mutant=mutant)
    ok &= check() and table[2, 2] != table[0, 2] and table[3, 1] != table[0, 1]
    KP.free([0], [17], table, page, refs, mutant=mutant)
    truth[0].pop(2, None)
    ok &= check()
    KP.free([1], None, table, page, refs, mutant=mutant)
    truth.pop(1)
    st, new, (live, moved) = KP.compact(table, refs, planes, mutant=mutant)
    ok &= check() and st == 0 and (refs[:live] > 0).all() and (refs[live:] == 0).all()
    return ok


def test_pages_life():
    assert _life()


@pytest.mark.parametrize("mutant", [1, 2, 3, 4, 5])
def test_pages_mutants_show(mutant):
    try:
        good = _life(mutant)
    except (AssertionError, IndexError):
        good = False
    if mutant == 1:  # lowest first: the ids themselves, checked inside
        rng = np.random.default_rng(0)
        table, refs, planes = _state(rng)
        KP.reserve([0], [0], [1], table, 16, refs, planes, mutant=1)
        good = table[0, 0] == 0
    assert not good


def test_reserve_serves_rows_whole_and_in_order():
    rng = np.random.default_rng(5)
    table, refs, planes = _state(rng, pages=4)
    st = KP.reserve([0, 1, 2, 3], [0, 0, 0, 0], [32, 48, 1, 0], table, 16, refs, planes)
    assert st == KP.NO_PAGE
    assert (table[0] >= 0).sum() == 2 and (table[1:] < 0).all()


def test_verify_by_hand_and_mutants():
    p = np.zeros((1, 3, 4), np.float32)
    q = np.zeros((1, 2, 4), np.float32)
    p[0, 0], q[0, 0] = [0.5, 0.25, 0.25, 0], [0.25, 0.5, 0.25, 0]
    p[0, 1], q[0, 1] = [0, 0, 0.5, 0.5], [0, 0, 0.5, 0.5]
    p[0, 2] = [0.25, 0.25, 0.25, 0.25]
    tok = np.array([[1, 3]], np.int32)

    def run(u, m=0, draft=q):
        o, k, s = DV.verify(p, draft, tok, np.array([u], np.float32), mutant=m)
        return o[0].tolist(), int(k[0]), s

    assert run([0.49, 0.9, 0.3]) == ([1, 3, 1], 2, 0)     # both stand, bonus token 1
    assert run([0.5, 0.9, 0.9]) == ([0, -1, -1], 0, 0)    # refused: max(p - q, 0) is token 0 alone
    assert run([0.5, 0.9, 0.9], 1) != run([0.5, 0.9, 0.9])
    assert run([0.5, 0.9, 0.9], 2) != run([0.5, 0.9, 0.9])
    assert run([0.4, 0.9, 0.2], 3) != run([0.4, 0.9, 0.2])
    assert run([0.4, 0.9, 0.25]) == ([1, 3, 1], 2, 0)     # the running sum must pass the point
    assert run([0.4, 0.9, 0.25], 4) != run([0.4, 0.9, 0.25])
    # a point mass draft: u < p(d); refused leaves p without d
    assert run([0.24, 0.6, 0.0], draft=None) == ([1, 2, -1], 1, 0)


@pytest.mark.parametrize("point", [False, True])
def test_verify_keeps_the_targets_distribution(point):
    """The first token of each request is distributed as the target's first row."""
    rng = np.random.default_rng(6)
    n, v = 20000, 5
    p = np.tile(np.array([[0.1, 0.4, 0.2, 0.05, 0.25]], np.float32), (2, 1))
    q = np.array([0.3, 0.1, 0.3, 0.2, 0.1], np.float32)
    tok = (np.full((n, 1), 2) if point else rng.choice(v, (n, 1), p=q / q.sum())).astype(np.int32)
    u = rng.random((n, 2)).astype(np.float32)
    o, k, s = DV.verify(np.tile(p, (n, 1, 1)), None if point else np.tile(q, (n, 1, 1)), tok, u)
    freq = np.bincount(o[:, 0], minlength=v) / n
    assert s == 0 and np.all(np.abs(freq - p[0]) < 5 * np.sqrt(p[0] / n))


def test_verify_draws_at_the_floor():
    """The drawn token is the least whose running sum passes floor(r * sum), for the least r that
    draws a given one (its last bits lie far below the sums' unit)."""
    rng = np.random.default_rng(200)
    vocab, n = 5000, 40
    p = np.full((n, 1, vocab), 2.0 ** -60, np.float32)
    p[:, 0, -1] = rng.uniform(0.5, 1, n)
    want = rng.integers(1, vocab - 1, n)
    u = np.zeros((n, 1), np.float32)
    for j in range(n):
        total = vocab - 1 + int(float(p[j, 0, -1]) * 2.0 ** 60)
        u[j] = np.float32(int(want[j]) / total)
        while Fraction(float(u[j, 0])) * total < int(want[j]):
            u[j] = np.nextafter(u[j], np.float32(1))
    o, k, s = DV.verify(p, None, np.zeros((n, 0), np.int32), u)
    assert s == 0 and o[:, 0].tolist() == want.tolist()
