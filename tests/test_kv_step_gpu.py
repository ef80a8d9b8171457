"""GPU parity of kvpages_step and kvpages_shared with the oracle: whole numbers, equal."""
import numpy as np
import pytest

from oracle import kv_pages as KP

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from sparse_attention_indexer_gb300 import Kv8Cache, KvPages  # noqa: E402

I32 = lambda a: torch.tensor(np.asarray(a, np.int64), dtype=torch.int32, device="cuda")  # noqa: E731


def pool_of(rng, n_tables, width, pages, page, holes=0.0):
    table = rng.integers(0, pages, (n_tables, width)).astype(np.int32)
    table[rng.random(table.shape) < holes] = -1
    return table, KvPages(I32(table), I32(np.ones(pages)), page)


def check_step(table, pool, rows, old, new, tokens, page, pages):
    ref = KP.step(rows, old, new, table, page, pages, tokens)
    got = pool.step(I32(rows), I32(old), I32(new), tokens)
    for x, y, name in zip(got, ref, got._fields):
        assert np.array_equal(x.cpu().numpy(), y), name
    assert int(pool.status.item()) == ref[5]
    pool.status.zero_()


@pytest.mark.parametrize("page", [1, 16, 48, 64, 128])
@pytest.mark.parametrize("n,most", [(1, 1), (1, 5000), (3, 700), (64, 1), (64, 9), (300, 40), (1000, 3)])
def test_step(n, most, page):
    rng = np.random.default_rng(n * 1000 + most + page)
    width = -(-(most + 200) // page)
    table, pool = pool_of(rng, n + 2, width, 50, page)
    rows = rng.permutation(n + 2)[:n]
    old = rng.integers(0, 200, n)
    new = old + rng.integers(0, most + 1, n)
    total = int((new - old).sum())
    for tokens in (total, total + 1, total + 2000, max(0, total - 1), total // 2, 0):
        check_step(table, pool, rows, old, new, tokens, page, 50)


def test_step_many_requests():
    """More than one round of 4096 requests, and CTAs of several spans."""
    rng = np.random.default_rng(1)
    n = 9001
    table, pool = pool_of(rng, 64, 40, 90, 16)
    rows, old = rng.integers(0, 64, n), rng.integers(0, 300, n)
    new = old + rng.integers(0, 60, n)
    new[4000:4300] = old[4000:4300]
    check_step(table, pool, rows, old, new, int((new - old).sum()) + 5, 16, 90)


def test_step_one_long_prompt():
    rng = np.random.default_rng(2)
    table, pool = pool_of(rng, 3, 40000, 1000, 16)
    check_step(table, pool, [1, 2], [0, 7], [600000, 8], 600100, 16, 1000)


def test_step_refusals_and_holes():
    rng = np.random.default_rng(3)
    table, pool = pool_of(rng, 5, 10, 30, 16, holes=0.3)
    table[2, 3] = 77  # not a page
    pool.block_table.copy_(I32(table))
    rows = [0, -1, 2, 5, 1, 3, 4, 2]
    old = [0, 0, 10, 0, -1, 20, 5, 0]
    new = [100, 5, 160, 5, 5, 10, 161, 0]
    check_step(table, pool, rows, old, new, 400, 16, 30)
    check_step(table, pool, [], [], [], 10, 16, 30)
    check_step(table, pool, [], [], [], 0, 16, 30)


def check_shared(table, pool, rows, lens, starts, page, pages):
    ref, status = KP.shared(rows, lens, starts, table, page, pages)
    got = pool.shared(I32(rows), I32(lens), I32(starts))
    assert got.tolist() == ref.tolist()
    assert int(pool.status.item()) == status
    pool.status.zero_()


@pytest.mark.parametrize("width", [1, 2, 31, 512, 513, 3000])
@pytest.mark.parametrize("size", [1, 2, 3, 9, 70])
def test_shared(width, size):
    rng = np.random.default_rng(width + size)
    sets = 5
    pages = 4000
    table = np.full((sets * size, width), -1, np.int32)
    lens = []
    for s in range(sets):
        lead = rng.permutation(pages)[:width]
        for i in range(size):
            r = s * size + i
            table[r] = lead
            if s and i:  # the first set shares all
                c = int(rng.integers(0, width + 1))
                table[r, c:] = rng.permutation(pages)[:width - c]
            lens.append(int(rng.integers(max(1, 16 * width - 40), 16 * width + 1)))
    pool = KvPages(I32(table), I32(np.ones(pages)), 16)
    order = np.arange(sets * size)
    check_shared(table, pool, order, lens, list(range(0, sets * size + 1, size)), 16, pages)
    lens = [0 if rng.random() < 0.3 else n for n in lens]
    check_shared(table, pool, order, lens, list(range(0, sets * size + 1, size)), 16, pages)
    check_shared(table, pool, order, lens, [0, 0, 1, sets * size], 16, pages)


def test_shared_refusals():
    table = np.array([[3, 4, 5, -1], [3, 4, 9, 1], [3, 4, 5, 1], [3, 77, 5, 1], [3, 77, 5, 1]], np.int32)
    pool = KvPages(I32(table), I32(np.ones(10)), 16)
    for rows, lens, starts in (([0, 1, 2], [64, 64, 64], [0, 3]), ([0, 2], [64, 64], [0, 2]), ([3, 4], [64, 64], [0, 2]),
                               ([0, 5], [64, 64], [0, 2]), ([0, -1], [64, 0], [0, 2]), ([0, 2], [64, 65], [0, 2]),
                               ([0, 2], [-1, 64], [0, 2]), ([0, 2, 1, 2], [64] * 4, [0, 2, 4]),
                               ([0, 2], [64, 64], [0, 3]), ([0, 2], [64, 64], [-1, 2]), ([0, 2, 1], [64] * 3, [2, 0, 3]),
                               ([0, 2], [64, 64], [0])):
        check_shared(table, pool, rows, lens, starts, 16, 10)


def test_a_step_into_the_cache():
    """reserve, step, store and attention of ragged new tokens: what step gives is what they take."""
    rng = np.random.default_rng(4)
    cache = Kv8Cache.empty(40, 32, 2, 64)
    table = torch.full((4, 8), -1, dtype=torch.int32, device="cuda")
    pool = KvPages(table, torch.zeros(40, dtype=torch.int32, device="cuda"), 32, cache.planes())
    rows, old, new = I32([2, 0, 3]), I32([0, 0, 0]), I32([70, 1, 33])
    pool.reserve(rows, old, new)
    s = pool.step(rows, old, new, 104)
    k, v = (torch.from_numpy(rng.standard_normal((104, 2, 64)).astype(np.float32)).to("cuda", torch.bfloat16) for _ in range(2))
    cache.store(k, v, s.positions, s.token_table, table)
    q = torch.from_numpy(rng.standard_normal((104, 4, 64)).astype(np.float32)).to("cuda", torch.bfloat16)
    out, _ = cache.attention(q, s.lens, 70, table, 0.125, 1, s.token_table)
    for i, (a, b) in enumerate(zip(s.starts.tolist(), s.starts.tolist()[1:])):
        kk, vv = k[a:b].float().repeat_interleave(2, 1), v[a:b].float().repeat_interleave(2, 1)
        x = torch.einsum("qhd,khd->hqk", q[a:b].float(), kk) * 0.125
        x = x.masked_fill(torch.ones(b - a, b - a, device="cuda").triu(1).bool(), float("-inf"))
        ref = torch.einsum("hqk,khd->qhd", x.softmax(-1), vv)
        # codes of 4 significant bits: 2^-4 relative on keys and values
        assert (out[a:b].float() - ref).abs().max() < 0.35
    slot = s.slots.long()
    blocks = slot // 32
    back = cache.k[slot].view(torch.float8_e4m3fn).float() * cache.k_scale[blocks][..., None]
    # half a step of e4m3, or of its subnormals at the block's scale
    assert ((back - k.float()).abs() <= 2.0 ** -4 * k.float().abs() + 2.0 ** -10 * cache.k_scale[blocks][..., None]).all()
    assert int(pool.status.item()) == 0 and int(cache.status.item()) == 0


def test_graphs_agree():
    rng = np.random.default_rng(5)
    table, pool = pool_of(rng, 8, 30, 60, 16)
    rows, old, new = I32(rng.permutation(8)), I32([5] * 8), I32(rng.integers(5, 400, 8))
    starts = I32([0, 3, 8])
    ref, pre = pool.step(rows, old, new, 3000), pool.shared(rows, new, starts)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got, pre2 = pool.step(rows, old, new, 3000), pool.shared(rows, new, starts)
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(ref, got)) and torch.equal(pre, pre2)
