"""GPU parity of the 8-bit paged cache (kv8_store, kv8_attention, kv8_attention_selected)
against the float64 oracle (oracle/kv8.py).

Store: codes and scales are equal bit for bit (the scale comes from the input's bits, the
quotient by it is one IEEE operation, the rounding to e4m3 is to nearest even).

Attention, tolerances per output channel, from what the kernel rounds:
  - the output type: half a step, eps / 2 of the value (bf16 2^-8, fp16 2^-11);
  - each weight to fp16 relative to the row's largest weight * value scale: 2^-11 of the
    weight, so 2^-11 * a with a = sum w |v|; weights that become fp16 subnormals lose at
    most 2^-25 of that largest product, so 2^-25 * top * c with c = sum |v codes|;
  - scores in fp32: |dx| <= 2^-16 * max_p sm_scale * sum |q k| (the bound the score
    producer's tests use for the same products and sums), which moves weights by 2 |dx|
    relative, numerator and denominator;
  - fp32 sums, exponentials and the joining of parts: 2^-18 * a.
lse: |dx| + 2^-20 * (1 + |lse|).
"""
import math

import numpy as np
import pytest

from oracle import kv8 as K8

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from sparse_attention_indexer_gb300 import Kv8Cache  # noqa: E402

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def bits(t):
    return t.contiguous().cpu().view(torch.int16).numpy().view(np.uint16)


# ------------------------------------------------------------------ store
def make_cache(rng, pages, page, heads, dim, block, pow2=False):
    slots = pages * page
    codes = lambda: torch.from_numpy(rng.integers(0, 120, (slots, heads, dim)).astype(np.uint8)).to(DEV)  # noqa: E731

    def scales():
        s = rng.uniform(0.002, 0.1, (slots // block, heads))
        s = 2.0 ** np.round(np.log2(s)) if pow2 else s
        return torch.from_numpy(s.astype(np.float32)).to(DEV)
    return Kv8Cache(codes(), codes(), scales(), scales(), page, block)


def run_store(cache, k, v, positions, token_table, table, dtype):
    ref = []
    st = 0
    for x, c, s in ((k, cache.k, cache.k_scale), (v, cache.v, cache.v_scale)):
        rc, rs = c.cpu().numpy().copy(), s.cpu().numpy().copy()
        st |= K8.store(K8.values(bits(x), dtype), positions, token_table, table, cache.page_size,
                       cache.block_tokens, rc, rs)
        ref += [rc, rs]
    t = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)  # noqa: E731
    cache.store(k, v, t(positions), t(token_table), t(table))
    torch.cuda.synchronize()
    assert int(cache.status.item()) == st
    got = [x.cpu().numpy() for x in (cache.k, cache.k_scale, cache.v, cache.v_scale)]
    for name, g, r in zip(("k", "k_scale", "v", "v_scale"), got, ref):
        same = g == r
        if g.dtype == np.uint8:
            nan = ((g & 0x7F) == 0x7F) & ((r & 0x7F) == 0x7F)
            same |= nan
        assert same.all(), f"{name}: {np.argwhere(~same)[:4].tolist()}"
    return st


def runs_of(spans):
    pos = np.concatenate([np.arange(a, a + n) for _, a, n in spans]) if spans else np.zeros(0)
    row = np.concatenate([np.full(n, r) for r, _, n in spans]) if spans else np.zeros(0)
    return pos.astype(np.int32), row.astype(np.int32)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,dim,page,block,spans", [
    (1, 64, 16, 16, [(0, 0, 1)]),
    (2, 128, 64, 64, [(0, 5, 1), (1, 63, 1), (2, 64, 1), (3, 0, 1)]),
    (3, 128, 64, 32, [(0, 3, 200), (2, 31, 2), (1, 127, 66)]),
    (2, 64, 128, 128, [(1, 1, 300), (0, 127, 1)]),
    (1, 128, 256, 256, [(0, 10, 500), (1, 255, 3)]),     # rows beyond what registers hold
    (8, 128, 64, 64, [(0, 17, 1100), (1, 0, 64)]),       # chunks of tokens per CTA
    (8, 64, 32, 16, [(0, 9, 1111), (2, 40, 7)]),
    (9, 64, 48, 48, [(1, 47, 1000)]),                    # a page that is no power of two
])
def test_store(dtype, heads, dim, page, block, spans):
    rng = np.random.default_rng(len(spans) * 1000 + page)
    pos, row = runs_of(spans)
    width = -(-int(pos.max() + 1) // page)
    table = rng.permutation(4 * width).reshape(4, width).astype(np.int32)
    cache = make_cache(rng, 4 * width, page, heads, dim, block)
    x = [torch.from_numpy((rng.standard_normal((len(pos), heads, dim)) *
                           np.exp(rng.standard_normal((len(pos), heads, 1)))).astype(np.float32))
         .to(TYPES[dtype]).to(DEV) for _ in range(2)]
    assert run_store(cache, x[0], x[1], pos, row, table, dtype) == 0


def test_store_appends_token_by_token():
    """Each call one token; the magnitudes grow and shrink, so codes are rounded again."""
    rng = np.random.default_rng(7)
    cache = make_cache(rng, 2, 32, 2, 64, 16, pow2=True)
    table = np.array([[1, 0]], np.int32)
    for p in range(40):
        x = [torch.from_numpy((rng.standard_normal((1, 2, 64)) * 2.0 ** rng.integers(-12, 13))
                              .astype(np.float32)).to(torch.bfloat16).to(DEV) for _ in range(2)]
        run_store(cache, x[0], x[1], [p], [0], table, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_store_special_values(dtype):
    rng = np.random.default_rng(8)
    cache = make_cache(rng, 3, 64, 2, 128, 32)
    x = torch.zeros((100, 2, 128), dtype=TYPES[dtype])
    x[0, 0, 3] = math.inf
    x[1, 0, 4] = -math.inf
    x[2, 1, 5] = math.nan
    x[33:64] = 0.0                                        # a block with one token that is not 0
    x[40, 0, 0] = 448.0
    x[64:96, 0] = torch.finfo(TYPES[dtype]).tiny / 4      # subnormals
    x[70, 1] = torch.finfo(TYPES[dtype]).max
    x[96:] = torch.linspace(-900, 900, 4 * 2 * 128).view(4, 2, 128).to(TYPES[dtype])
    x = x.to(DEV)
    run_store(cache, x, x.flip(2).contiguous(), np.arange(100), np.zeros(100), np.array([[2, 0, 1]]),
              dtype)


def test_store_strided_and_refused_tokens():
    rng = np.random.default_rng(9)
    cache = make_cache(rng, 4, 16, 2, 64, 16)
    wide = torch.from_numpy(rng.standard_normal((9, 3 * 128)).astype(np.float32)).to(DEV)
    wide = wide.to(torch.bfloat16)
    k, v = wide[:, :128].view(9, 2, 64), wide[:, 128:256].view(9, 2, 64)
    # one token each: stored, negative position, table row, width, entry, slot, row -1, stored
    pos = [3, -1, 2, 48, 17, 33, 4, 20, 21]
    row = [0, 0, 3, 0, 0, 1, -1, 1, 1]
    table = np.array([[0, -1, 1], [2, 3, 9], [1, 1, 1]], np.int32)
    st = run_store(cache, k, v, pos, row, table, "bf16")
    assert st == K8.POSITION | K8.TABLE_ROW | K8.TABLE_WIDTH | K8.TABLE_ENTRY | K8.SLOT


def test_store_nothing():
    cache = make_cache(np.random.default_rng(1), 1, 16, 1, 64, 16)
    e = torch.empty((0, 1, 64), dtype=torch.bfloat16, device=DEV)
    i = torch.empty(0, dtype=torch.int32, device=DEV)
    before = cache.k.clone()
    cache.store(e, e, i, i, torch.zeros((1, 1), dtype=torch.int32, device=DEV))
    assert torch.equal(cache.k, before)


# ------------------------------------------------------------------ attention
def attention_cache(rng, pages, page, heads, dim, block, wide=False):
    """Codes without NaN, scales in a factor of 4 (2^24 where `wide`)."""
    slots = pages * page
    code = lambda: np.where(rng.random((slots, heads, dim)) < 0.5, 0, 128) + rng.integers(0, 119, (slots, heads, dim))  # noqa: E731,E501
    scale = lambda: np.exp2(rng.uniform(*((-20, 4) if wide else (-8, -6)), (slots // block, heads)))  # noqa: E731,E501
    return [code().astype(np.uint8), code().astype(np.uint8), scale().astype(np.float32),
            scale().astype(np.float32)]


def close(out, lse, ref, dtype, what=""):
    ro, rl, dx, a, top, c = ref
    half = torch.finfo(TYPES[dtype]).eps / 2
    dx = dx * 2.0 ** -16
    tol = (half * np.abs(ro) + (2.0 ** -11 + 2 * dx[:, None] + 2.0 ** -18) * (1 + half) * a
           + 2.0 ** -25 * top[:, None] * c + (2.0 ** -25 if dtype == "fp16" else 0.0))
    err = np.abs(out - ro)
    assert np.all(err <= tol), f"{what}: out off by {np.max(err / np.maximum(tol, 1e-300)):.3g} x"
    empty = np.isneginf(rl)
    assert np.array_equal(np.isneginf(lse), empty), what
    with np.errstate(invalid="ignore"):
        bad = np.abs(lse - rl) > dx + 2.0 ** -20 * (1 + np.abs(rl))
    assert not np.any(bad & ~empty), f"{what}: lse {lse[bad & ~empty][:3]} {rl[bad & ~empty][:3]}"


class Dense:
    def __init__(self, seed, lens, group, hq, hk, dim, page, block, dtype, wide=False, poison=True,
                 q_gain=1.0, q_pad=0):
        rng = np.random.default_rng(seed)
        self.rng, self.group, self.page, self.block, self.dtype = rng, group, page, block, dtype
        rows = len(lens)
        groups = -(-rows // group)
        self.lens = np.asarray(lens, np.int32)
        self.max_len = max(1, int(self.lens.max()))
        need = [-(-max(0, int(self.lens[g * group:(g + 1) * group].max())) // page)
                for g in range(groups)]
        width = max(1, max(need))
        pages = sum(need) + 2
        perm = rng.permutation(pages)
        self.table = np.full((groups, width), -1, np.int32)
        at = 0
        for g, n in enumerate(need):
            self.table[g, :n] = perm[at:at + n]
            at += n
        self.cache = attention_cache(rng, pages, page, hk, dim, block, wide)
        if poison:  # NaN codes and scales wherever no row attends
            used = np.zeros(pages * page, bool)
            for r, n in enumerate(self.lens):
                used[K8.row_slots(self.table, r // group, int(n), self.max_len, page,
                                  pages * page)[0]] = True
            for x in self.cache[:2]:
                x[~used] = 0x7F
            idle = ~used.reshape(-1, block).any(1)
            for x in self.cache[2:]:
                x[idle] = np.nan
        q = torch.from_numpy((rng.standard_normal((rows, hq, dim)) * q_gain).astype(np.float32))
        q = q.to(TYPES[dtype])
        buf = torch.zeros((rows, hq * dim + q_pad), dtype=TYPES[dtype], device=DEV)
        buf[:, :hq * dim] = q.view(rows, -1).to(DEV)
        self.q = buf[:, :hq * dim].unflatten(1, (hq, dim))
        self.scale = 1.0 / math.sqrt(dim)
        self.group_table = np.arange(groups, dtype=np.int32)

    def handle(self):
        t = [torch.from_numpy(x).to(DEV) for x in self.cache]
        return Kv8Cache(*t, self.page, self.block)

    def args(self, max_len=None):
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
        return (self.q, t(self.lens), max_len or self.max_len, t(self.table), self.scale, self.group,
                t(self.group_table))

    def ref(self, r, max_len=None):
        k, v, ks, vs = self.cache
        slots, st = K8.row_slots(self.table, int(self.group_table[r // self.group]),
                                 int(self.lens[r]), max_len or self.max_len, self.page, k.shape[0])
        q = K8.values(bits(self.q[r]), self.dtype)
        return K8.attend(q, slots, k, v, ks, vs, self.block, self.scale), st

    def check(self, max_len=None, rows=None):
        h = self.handle()
        out, lse = h.attention(*self.args(max_len))
        torch.cuda.synchronize()
        o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
        st = 0
        for r in range(len(self.lens)):
            ref, s = self.ref(r, max_len)
            st |= s
            if rows is None or r in rows:
                close(o[r], l[r], ref, self.dtype, f"row {r} len {self.lens[r]}")
        assert int(h.status.item()) == st
        return out, lse, st


def check_rows(d, rows):
    """Dense.check without the references of the other rows."""
    h = d.handle()
    out, lse = h.attention(*d.args())
    for r in rows:
        ref, st = d.ref(r)
        assert st == 0
        close(out[r].double().cpu().numpy(), lse[r].double().cpu().numpy(), ref, d.dtype, f"row {r}")
    assert int(h.status.item()) == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page,block", [(16, 16), (64, 64), (64, 16), (48, 16), (128, 32), (80, 80)])
def test_lengths(page, block, dim, dtype):
    lens = [0, 1, 2, 7, 8, 15, 16, 17, 31, 32, 33, 47, 48, 63, 64, 65, 79, 80, 127, 128, 129, 200]
    Dense(page + block + dim, lens, 1, 8, 2, dim, page, block, dtype).check()


@pytest.mark.parametrize("hq,hk", [(1, 1), (2, 1), (16, 1), (7, 1), (12, 4), (40, 8), (8, 8), (64, 4)])
@pytest.mark.parametrize("group", [1, 2, 3, 7, 8])
def test_heads_and_groups(hq, hk, group):
    """Groups of query rows (the last one shorter), causal lengths inside a group."""
    lens = []
    for n in (70, 5, 300):
        lens += [max(0, n - group + 1 + i) for i in range(group)]
    lens = lens[:-1] if group > 1 else lens
    Dense(hq * 10 + group, lens, group, hq, hk, 128 if hq % 2 else 64, 64, 32, "bf16").check()


# More than 32 query rows to a key head, 128 channels: (query heads, key heads, group)
WIDE = [(16, 1, 3), (56, 8, 7), (16, 1, 4), (40, 5, 8), (16, 2, 5), (16, 1, 5), (15, 1, 7), (32, 2, 8)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("hq,hk,group", WIDE)
def test_wide_groups(hq, hk, group, dtype):
    lens = []
    for n in (group + 70, group, 130 + group, 513):
        lens += [n - group + 1 + i for i in range(group)]
    Dense(hq * 10 + group, lens[:-1], group, hq, hk, 128, 64, 32, dtype).check()


@pytest.mark.parametrize("page,block", [(16, 16), (48, 48), (128, 16), (256, 256)])
def test_wide_lengths(page, block):
    """Rows of a group of any lengths, none among them, around the tiles of 128 keys."""
    for lens in ([0, 1, 127, 128, 129, 2, 0], [0] * 7, [255, 256, 257, 300, 31, 32, 33],
                 [1, 0, 0, 0, 0, 0, 0]):
        Dense(page + len(lens), lens, 7, 8, 1, 128, page, block, "bf16").check()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_wide_split_over_the_grid(dtype):
    Dense(50, [20000 + i for i in range(7)], 7, 8, 1, 128, 64, 64, dtype).check(rows={0, 3, 6})
    Dense(51, [3000, 2999, 1, 0, 700, 650, 600, 601] * 3, 4, 16, 1, 128, 64, 16, dtype).check()


def test_wide_many_groups():
    rng = np.random.default_rng(52)
    lens = rng.integers(0, 200, 4 * 650).tolist()
    Dense(53, lens, 4, 20, 2, 128, 16, 16, "bf16").check(rows=set(range(0, 2600, 37)))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_wide_scales_and_peaks(dtype):
    Dense(54, [500, 64, 100, 900], 4, 16, 1, 128, 64, 16, dtype, wide=True).check()
    Dense(55, [400, 300, 20, 1], 4, 16, 1, 128, 64, 64, dtype, q_gain=40.0).check()
    Dense(56, [400, 300, 20, 1], 4, 16, 1, 128, 64, 64, dtype, q_gain=0.0).check()


def test_wide_zero_scales_and_queries():
    d = Dense(57, [200, 40, 300, 290], 4, 16, 1, 128, 64, 16, "bf16")
    d.cache[2][:] = 0.0
    d.cache[3][::3] = 0.0
    d.check()
    d.cache[3][:] = 0.0
    d.check()
    for gain in (1e-30, 1e30):
        d = Dense(58, [90, 33, 200, 1], 4, 16, 1, 128, 16, 16, "bf16", q_gain=gain)
        d.scale = 0.125 / gain
        d.check()


def test_wide_refused_and_streams():
    d = Dense(59, [300] * 8, 4, 16, 1, 128, 16, 16, "bf16", poison=False)
    d.lens[0], d.lens[1] = -1, 301
    d.table[1, 2], d.table[1, 6] = -1, 10 ** 6
    assert d.check(max_len=300)[2] == K8.LEN | K8.TABLE_ENTRY | K8.SLOT
    d = Dense(60, [5000, 77, 0, 1300], 4, 16, 2, 128, 64, 64, "bf16")
    h, a = d.handle(), d.args()
    ref = h.attention(*a)
    for _ in range(3):
        got = h.attention(*a)
        assert torch.equal(ref[0], got[0]) and torch.equal(ref[1], got[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, lse = torch.empty_like(ref[0]), torch.empty_like(ref[1])
    with torch.cuda.stream(s):
        h.attention(*a, out=out, lse=lse)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        h.attention(*a, out=out, lse=lse)
    for _ in range(2):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(ref[0], out) and torch.equal(ref[1], lse)


def test_rows_of_a_group_differ_freely():
    Dense(3, [0, 100, 17, 64, 0, 1, 333], 7, 16, 2, 128, 64, 64, "fp16").check()
    Dense(4, [0] * 7, 7, 16, 2, 128, 64, 64, "bf16").check()


def test_long_rows_split_over_the_grid():
    Dense(5, [20011], 1, 16, 2, 128, 64, 64, "bf16").check()
    Dense(6, [9000, 8999, 3, 0, 1], 1, 8, 1, 64, 64, 32, "fp16").check()
    Dense(7, [6994 + i for i in range(7)], 7, 16, 2, 128, 64, 16, "bf16").check()


def test_many_short_rows():
    rng = np.random.default_rng(10)
    Dense(11, rng.integers(0, 90, 700).tolist(), 1, 4, 2, 64, 16, 16, "bf16").check(
        rows=set(range(0, 700, 7)))
    Dense(12, rng.integers(1, 40, 1201).tolist(), 8, 2, 1, 64, 32, 16, "fp16").check(
        rows=set(range(0, 1201, 11)))


@pytest.mark.parametrize("hq,dim,group,dtype", [(6, 64, 1, "bf16"), (16, 128, 1, "fp16"),
                                                (30, 128, 1, "bf16"), (8, 64, 4, "fp16")])
def test_a_unit_for_every_warp(hq, dim, group, dtype):
    """More units than the device has warps for them: a warp to a CTA, long rows split over
    several, empty ones among them."""
    rng = np.random.default_rng(dim + hq)
    lens = rng.integers(0, 70, 950 * group)
    lens[rng.permutation(950 * group)[:6]] = [3000, 700, 0, 1, 32, 2111]
    Dense(40 + hq, lens.tolist(), group, hq, 2, dim, 32, 16, dtype).check(
        rows=set(np.argsort(lens)[-8:].tolist()) | set(range(0, 950 * group, 41 * group)))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_scales_far_apart(dtype):
    """Block scales over 24 octaves: a heavily weighted block next to one of large values."""
    Dense(13, [500, 64, 100, 1000], 1, 8, 2, 128, 64, 16, dtype, wide=True).check()


# Variants of units of 8 and 16 rows (a warp to a CTA) and of 32, 64 and 128 (four): (query heads, key
# heads, group, dim)
UNITS = [(2, 2, 1, 64), (32, 8, 1, 128), (30, 2, 1, 128), (16, 2, 4, 64), (16, 1, 4, 128),
         (16, 1, 8, 64)]


@pytest.mark.parametrize("hq,hk,group,dim", UNITS)
def test_more_units_than_the_list_of_shared_ones(hq, hk, group, dim):
    """From 2049 (group, key head) units on, a shared unit is kept by the CTA it starts in: long
    rows that several CTAs share, beside one another and not, empty rows, the last row long."""
    groups = 2400 // hk
    rng = np.random.default_rng(hq + group)
    lens = rng.integers(0, 50, groups * group)
    long = [0, 1, 2, groups // 3, groups // 2, groups // 2 + 2, groups - 1]
    for g, n in zip(long, (9000, 4000, 3333, 700, 12000, 2500, 5000)):
        lens[g * group:(g + 1) * group] = np.maximum(0, n - np.arange(group)[::-1])
    lens[(groups // 2 + 1) * group:(groups // 2 + 2) * group] = 0
    d = Dense(100 + hq + group, lens.tolist(), group, hq, hk, dim, 32, 16, "bf16")
    check_rows(d, sorted({g * group + i for g in long + [groups // 2 + 1] for i in (0, group - 1)}
                         | set(range(0, groups * group, 61 * group))))


@pytest.mark.parametrize("groups", [2047, 2048, 2049])
@pytest.mark.parametrize("hq,group", [(4, 1), (16, 4)])
def test_units_around_the_list_of_shared_ones(groups, hq, group):
    lens = np.random.default_rng(groups).integers(0, 40, groups * group)
    long = [0, 1000, groups - 2, groups - 1]
    for g, n in zip(long, (8000, 3000, 6000, 1500)):
        lens[g * group:(g + 1) * group] = n
    d = Dense(110 + group, lens.tolist(), group, hq, 1, 64, 32, 16, "fp16")
    check_rows(d, sorted({g * group for g in long} | set(range(0, groups * group, 97 * group))
                         | {groups * group - 1}))


def test_peaked_and_flat_rows():
    Dense(14, [400, 300], 1, 8, 2, 128, 64, 64, "bf16", q_gain=40.0).check()
    Dense(15, [400, 300], 1, 8, 2, 128, 64, 64, "fp16", q_gain=0.0).check()


@pytest.mark.parametrize("scale", [-0.1, 0.0, 5.0])
@pytest.mark.parametrize("group", [1, 5])
def test_score_scales(scale, group):
    """Negative and zero softmax scales take the general tile."""
    d = Dense(16, [200, 40, 129, 64, 90], group, 16, 2, 128, 64, 64, "bf16")
    d.scale = scale
    d.check()


def test_zero_scales():
    d = Dense(16, [200, 40], 1, 8, 2, 128, 64, 16, "bf16")
    d.cache[2][:] = 0.0
    d.cache[3][::3] = 0.0
    d.check()
    d.cache[3][:] = 0.0
    d.check()


def far_scales(d, rng, exponents, zero):
    """Value scales 2^e, e alternating between two exponents from block to block (a tile has
    both), and a tile's blocks zero with probability `zero`."""
    sv = d.cache[3]
    blocks = np.arange(len(sv))
    sv[:] = np.exp2(np.asarray(exponents, np.float64)[blocks % 2])[:, None]
    sv[np.repeat(rng.random(len(sv) // 2 + 1) < zero, 2)[:len(sv)]] = 0.0


def one_table(seed, rows, length, group, hq, hk, dim, block=16):
    """Rows of one length over one table row, with value scales far apart, for launches in
    which a warp takes many tiles of a row."""
    d = Dense(seed, [length] * group, group, hq, hk, dim, 64, block, "bf16", poison=False)
    d.table[0] = np.arange(d.table.shape[1])  # consecutive pages: tiles take blocks in order
    q = torch.from_numpy(d.rng.standard_normal((rows, hq, dim)).astype(np.float32))
    d.q = q.to(torch.bfloat16).to(DEV)
    d.lens = np.full(rows, length, np.int32)
    d.group_table = np.zeros(-(-rows // group), np.int32)
    return d


# (rows, keys, group, query heads, key heads, dim) that give a warp about 100 tiles of a row: a warp
# to a CTA, four to a CTA, and units of 32, 64 and 128 rows
MANY_TILES = [(1900, 3200, 1, 1, 1, 128), (1900, 3200, 1, 16, 1, 64), (300, 12800, 1, 8, 1, 128),
              (2400, 12800, 8, 4, 1, 128), (2400, 12800, 8, 8, 1, 64), (2400, 12800, 8, 16, 1, 128)]


@pytest.mark.parametrize("rows,length,group,hq,hk,dim", MANY_TILES)
def test_keys_of_zero_scale_before_small_scales(rows, length, group, hq, hk, dim):
    """Tiles whose values have scale 0 set no reference for the tiles of 2^-28 and 2^-40 after
    them."""
    d = one_table(60 + group, rows, length, group, hq, hk, dim)
    far_scales(d, d.rng, (-28, -40), 0.5)
    check_rows(d, (0, rows // 2, rows - 1))


@pytest.mark.parametrize("rows,length,group,hq,hk,dim", MANY_TILES)
def test_scores_that_rise_while_value_scales_fall(rows, length, group, hq, hk, dim):
    """weight * value scale is about the same in all tiles: the reference of the weights' rounding
    does not rise with the row's maximum."""
    d = one_table(70 + group, rows, length, group, hq, hk, dim)
    blocks = np.arange(len(d.cache[2]))
    # 60 octaves over the row, in steps of a tile
    octave = 60.0 * (blocks // 2) / (len(blocks) // 2)
    # log2 of a weight: log2(e) / sqrt(dim) * q . k, with q . k = dim * key scale
    d.cache[0][:] = 0x38                    # 1.0
    d.q.fill_(1.0)
    d.cache[2][:] = (octave * math.log(2) / math.sqrt(dim))[:, None]
    d.cache[3][:] = np.exp2(-octave - 12.0 * (blocks % 2))[:, None]
    check_rows(d, (0, rows // 2, rows - 1))


@pytest.mark.parametrize("group", [1, 4])
@pytest.mark.parametrize("dim", [64, 128])
def test_heaviest_key_of_zero_scale(dim, group):
    """The block of the heaviest key has value scale 0: what is left are keys of 2^-20 to 2^-90 of
    its weight, and the output is theirs."""
    lens = [32] * (6 * group)
    d = Dense(80 + dim, lens, group, 4, 4, dim, 32, 16, "bf16", poison=False, q_gain=25.0)
    for g in range(6):
        d.q[g * group:(g + 1) * group] = d.q[g * group]   # the rows of a group agree on the key
        slots = K8.row_slots(d.table, g, 32, 32, 32, d.cache[0].shape[0])[0]
        q = K8.values(bits(d.q[g * group]), "bf16")
        for h in range(4):
            kk = K8.e4m3_value(d.cache[0][slots, h]) * d.cache[2][slots // 16, h][:, None]
            d.cache[3][slots[np.argmax(kk @ q[h])] // 16, h] = 0.0
    d.check()


@pytest.mark.parametrize("dim,hq", [(64, 8), (128, 8), (128, 32)])
def test_nan_seen_by_the_later_rows_alone(dim, hq):
    """NaN codes and scales in the last draft's key and value: the rows before it are as
    without them, the rows that see them are NaN where the definition says so."""
    n = hq // 2  # query heads of a key head
    d = Dense(24, [97, 98, 99, 100], 4, hq, 2, dim, 64, 16, "bf16", poison=False)
    slot = K8.row_slots(d.table, 0, 100, 100, 64, d.cache[0].shape[0])[0]
    d.cache[1][slot[99], 1, 5] = 0x7F       # a value: channel 5 of the last row, key head 1
    d.cache[1][slot[98], 0, 40] = 0xFF      # rows 2 and 3, key head 0
    d.cache[0][slot[99], 0, 7] = 0x7F       # a key: everything of the last row, key head 0
    h = d.handle()
    out, lse = h.attention(*d.args())
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for r in (0, 1):
        close(o[r], l[r], d.ref(r)[0], "bf16", f"row {r}")
    nan = np.zeros((4, hq, dim), bool)
    nan[2, :n, 40] = True
    nan[3, :n] = True
    nan[3, n:, 5] = True
    assert np.array_equal(np.isnan(o), nan)
    assert np.isnan(l[3, :n]).all() and not np.isnan(l[:3]).any() and not np.isnan(l[3, n:]).any()
    d.cache[3][slot[96] // 16] = np.nan     # the scale of a block that starts at position 96
    h = d.handle()
    d.lens[:] = [96, 96, 97, 100]
    o = h.attention(*d.args())[0].double().cpu().numpy()
    for r in (0, 1):
        close(o[r], l[r] * 0 + d.ref(r)[0][1], d.ref(r)[0], "bf16", f"row {r}")
    assert np.isnan(o[2:]).all()


@pytest.mark.parametrize("dim,hq", [(64, 8), (128, 8), (128, 32)])
def test_scales_that_are_nan_past_the_end_of_a_row(dim, hq):
    """The block after a row's last key has NaN scales, which the rows behind it see: outputs and lse
    of the rows before are as without it."""
    d = Dense(26, [96, 90, 97, 100], 4, hq, 2, dim, 64, 16, "bf16", poison=False)
    slot = K8.row_slots(d.table, 0, 100, 100, 64, d.cache[0].shape[0])[0]
    want = [d.ref(r)[0] for r in (0, 1)]
    for which in (3, 2):
        d.cache[which][slot[96] // 16] = np.nan
        out, lse = d.handle().attention(*d.args())
        o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
        for r in (0, 1):
            close(o[r], l[r], want[r], "bf16", f"row {r}")
        assert np.isnan(o[2:]).all()
        assert np.isnan(l[2:]).all() == (which == 2)


def test_nan_and_infinite_queries():
    d = Dense(25, [50, 60, 70], 3, 8, 2, 64, 16, 16, "bf16")
    ref = [d.ref(r)[0] for r in range(3)]
    d.q[1, 2] = float("nan")
    d.q[2, 7] = float("inf")
    out, lse = d.handle().attention(*d.args())
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.isnan(o[1, 2]).all() and np.isnan(l[1, 2])
    assert np.isnan(o[2, 7]).any() or not np.isfinite(l[2, 7])
    keep = np.ones((3, 8), bool)
    keep[1, 2] = keep[2, 7] = False
    for r in range(3):
        at = keep[r]
        close(o[r][at], l[r][at], [x[at] for x in ref[r]], "bf16")


def test_tiny_and_large_queries():
    for gain in (1e-30, 1e30):
        d = Dense(17, [90, 33], 1, 4, 2, 64, 16, 16, "bf16", q_gain=gain)
        d.scale = 0.125 / gain
        d.check()


def test_strided_rows_and_outputs():
    d = Dense(18, [100, 31, 0, 64], 2, 6, 3, 64, 32, 16, "bf16", q_pad=24)
    h = d.handle()
    buf = torch.full((4, 6 * 64 + 40), -7.0, dtype=torch.bfloat16, device=DEV)
    out = buf[:, :6 * 64].unflatten(1, (6, 64))
    lse = torch.empty((4, 6), device=DEV)
    h.attention(*d.args(), out=out, lse=lse)
    torch.cuda.synchronize()
    assert torch.all(buf[:, 6 * 64:] == -7.0)
    for r in range(4):
        close(out[r].double().cpu().numpy(), lse[r].double().cpu().numpy(), d.ref(r)[0], "bf16")


def test_refused_rows_and_entries():
    """Lengths, table rows and entries that the kernel turns into status bits."""
    d = Dense(19, [100, 100, 100, 100, 100, 100], 1, 4, 2, 64, 16, 16, "bf16", poison=False)
    d.lens[0] = -1
    d.lens[1] = 101
    d.group_table[2] = 6
    d.group_table[3] = -1
    d.table[4, 2] = -1
    d.table[4, 6] = 10 ** 6
    st = d.check(max_len=100)[2]
    assert st == K8.LEN | K8.TABLE_ROW | K8.TABLE_ENTRY | K8.SLOT
    d = Dense(20, [100, 30], 1, 4, 2, 64, 16, 16, "bf16", poison=False)
    d.table = np.ascontiguousarray(d.table[:, :5])
    assert d.check(max_len=100)[2] == K8.TABLE_WIDTH


def test_group_table_null_and_shared_rows():
    d = Dense(21, [60, 61, 62, 90], 2, 4, 2, 64, 16, 16, "bf16")
    h = d.handle()
    a = d.args()
    one = h.attention(*a)
    two = h.attention(*a[:6])
    assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])


def test_runs_streams_and_graphs_agree():
    """The same bits on every run, on another stream, and from a graph replayed twice."""
    d = Dense(22, [5000, 77, 0, 1300], 1, 16, 2, 128, 64, 64, "bf16")
    h, a = d.handle(), d.args()
    ref = h.attention(*a)
    for _ in range(3):
        got = h.attention(*a)
        assert torch.equal(ref[0], got[0]) and torch.equal(ref[1], got[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = h.attention(*a, stream=s)
    s.synchronize()
    assert torch.equal(ref[0], got[0])
    out, lse = torch.empty_like(ref[0]), torch.empty_like(ref[1])
    with torch.cuda.stream(s):
        h.attention(*a, out=out, lse=lse)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        h.attention(*a, out=out, lse=lse)
    for _ in range(2):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(ref[0], out) and torch.equal(ref[1], lse)


def test_graphs_of_one_capture_stream_replayed_on_two():
    """Two graphs captured on the same stream, with the same heads, share no workspace: replayed
    side by side and beside eager calls they give what each gives alone."""
    a, b = (Dense(seed, [30000 + seed], 1, 16, 2, 128, 64, 64, "bf16", poison=False)
            for seed in (90, 91))
    h = a.handle()
    hb = b.handle()
    args = [(h, a.args()), (hb, b.args())]
    other = list(a.args())
    other[0] = other[0].flip(1)
    args.append((h, other))            # the first cache again, other queries
    ref = [c.attention(*x) for c, x in args]
    outs, graphs = [], []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    for c, x in args:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs.append(c.attention(*x))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in args]
    for _ in range(50):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        eager = h.attention(*args[0][1])
        assert torch.equal(eager[0], ref[0][0]) and torch.equal(eager[1], ref[0][1])
    torch.cuda.synchronize()
    for got, want in zip(outs, ref):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_offsets_past_32_bits():
    """A cache of more than 2^32 code bytes: the pages in use lie at its end."""
    page, hk, dim, block = 64, 8, 128, 64
    pages = (1 << 32) // (page * hk * dim) + 40
    d = Dense(23, [200, 64], 1, 16, hk, dim, page, block, "bf16")
    n = d.cache[0].shape[0] // page
    k, v, ks, vs = [torch.from_numpy(x).to(DEV) for x in d.cache]
    K = torch.empty((pages * page, hk, dim), dtype=torch.uint8, device=DEV)
    V = torch.empty_like(K)
    KS = torch.full((pages * page // block, hk), float("nan"), device=DEV)
    VS = KS.clone()
    K[-n * page:], V[-n * page:] = k, v
    KS[-n * page // block:], VS[-n * page // block:] = ks, vs
    h = Kv8Cache(K, V, KS, VS, page, block)
    a = list(d.args())
    a[3] = torch.where(a[3] >= 0, a[3] + (pages - n), a[3])
    out, lse = h.attention(*a)
    for r in range(2):
        close(out[r].double().cpu().numpy(), lse[r].double().cpu().numpy(), d.ref(r)[0], "bf16")
    x = torch.randn((3, hk, dim), device=DEV).to(torch.bfloat16)
    i = lambda *z: torch.tensor(z, dtype=torch.int32, device=DEV)  # noqa: E731
    h.store(x, x, i(0, 1, 2), i(0, 0, 0), i(pages - 1).view(1, 1))
    last = h.k[(pages - 1) * page].view(torch.float8_e4m3fn).float() * h.k_scale[-1][:, None]
    assert torch.all((last - x[0].float()).abs() <= x[0].float().abs() / 16 + h.k_scale[-1][:, None] / 1024)


# ------------------------------------------------------------------ selected
def selected_case(seed, rows, k, hq, hk, dim, block, dtype, slots=None, num=640, wide=False):
    rng = np.random.default_rng(seed)
    cache = attention_cache(rng, num // block, block, hk, dim, block, wide)
    if slots is None:
        slots = np.stack([rng.permutation(num)[:k] if k <= num else rng.integers(0, num, k)
                          for _ in range(rows)]).astype(np.int32).reshape(rows, k)
    q = torch.from_numpy(rng.standard_normal((rows, hq, dim)).astype(np.float32)).to(TYPES[dtype])
    return cache, slots, q.to(DEV), block, 1.0 / math.sqrt(dim)


def check_selected(cache, slots, q, block, scale, dtype):
    h = Kv8Cache(*[torch.from_numpy(x).to(DEV) for x in cache], block, block)
    out, lse = h.attention_selected(q, torch.from_numpy(slots).to(DEV), scale)
    torch.cuda.synchronize()
    n, st = cache[0].shape[0], 0
    for r in range(q.shape[0]):
        at = slots[r][slots[r] >= 0]
        st |= K8.SLOT if (at >= n).any() else 0
        ref = K8.attend(K8.values(bits(q[r]), dtype), at[at < n], *cache, block, scale)
        close(out[r].double().cpu().numpy(), lse[r].double().cpu().numpy(), ref, dtype, f"row {r}")
    assert int(h.status.item()) == st


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("k", [1, 2, 15, 16, 31, 32, 33, 63, 64, 65, 100, 640, 2048])
def test_selected_sizes(k, dtype):
    check_selected(*selected_case(k, 5, k, 8, 2, 128, 16, dtype), dtype)


@pytest.mark.parametrize("hq,hk,dim", [(1, 1, 64), (16, 1, 128), (7, 7, 64), (28, 4, 128), (32, 2, 64)])
def test_selected_heads(hq, hk, dim):
    check_selected(*selected_case(hq, 9, 70, hq, hk, dim, 64, "bf16"), "bf16")


def test_selected_padding_anywhere():
    rng = np.random.default_rng(30)
    s = np.stack([rng.permutation(640)[:150] for _ in range(6)]).astype(np.int32)
    s[0] = -1                                 # nothing left
    s[1, 40:] = -1                            # the usual tail
    s[2, rng.random(150) < 0.5] = -1          # holes
    s[3, :149] = -5                           # the last one only
    s[4] = s[4, 0]                            # one slot many times
    s[5, 7], s[5, 90] = 640, 2 ** 31 - 1      # past the cache: skipped with a status
    c = selected_case(31, 6, 150, 8, 2, 128, 16, "bf16", slots=s)
    for x in c[0][:2]:                        # a slot that no row names holds NaN
        free = np.setdiff1d(np.arange(640), s[s >= 0])
        x[free] = 0x7F
    check_selected(*c, "bf16")


def test_selected_nothing_and_strides():
    cache, slots, q, block, scale = selected_case(32, 4, 0, 8, 2, 64, 16, "bf16",
                                                  slots=np.zeros((4, 0), np.int32))
    check_selected(cache, slots, q, block, scale, "bf16")
    cache, slots, q, block, scale = selected_case(33, 4, 40, 8, 2, 64, 16, "fp16", wide=True)
    h = Kv8Cache(*[torch.from_numpy(x).to(DEV) for x in cache], block, block)
    wide = torch.full((4, 55), 639, dtype=torch.int32, device=DEV)
    wide[:, :40] = torch.from_numpy(slots).to(DEV)
    a = h.attention_selected(q, wide[:, :40], scale)
    b = h.attention_selected(q, torch.from_numpy(slots).to(DEV), scale)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    check_selected(cache, slots, q, block, scale, "fp16")


def test_selected_rows_many():
    check_selected(*selected_case(34, 300, 33, 4, 1, 64, 32, "fp16"), "fp16")


@pytest.mark.parametrize("rows,hq,hk,dim,k", [
    (1100, 4, 2, 64, 33), (300, 32, 8, 128, 100), (2500, 16, 1, 64, 5), (2060, 1, 1, 128, 0),
    (2049, 2, 1, 128, 1), (2048, 2, 1, 128, 70), (2047, 2, 1, 64, 70)])
def test_selected_more_units_than_the_list_of_shared_ones(rows, hq, hk, dim, k):
    rng = np.random.default_rng(rows)
    cache, slots, q, block, scale = selected_case(37, rows, k, hq, hk, dim, 16, "bf16")
    slots[rng.random(slots.shape) < 0.2] = -1
    slots[::50] = -1
    h = Kv8Cache(*[torch.from_numpy(x).to(DEV) for x in cache], block, block)
    out, lse = h.attention_selected(q, torch.from_numpy(slots).to(DEV), scale)
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for r in sorted(set(range(0, rows, 23)) | {50, rows - 2, rows - 1}):
        ref = K8.attend(K8.values(bits(q[r]), "bf16"), slots[r][slots[r] >= 0], *cache, block, scale)
        close(o[r], l[r], ref, "bf16", f"row {r}")
    assert int(h.status.item()) == 0


@pytest.mark.parametrize("hq,dim", [(2, 128), (24, 64)])
def test_selected_a_unit_for_every_warp(hq, dim):
    check_selected(*selected_case(36, 950, 70, hq, 2, dim, 16, "bf16"), "bf16")


def test_selected_equals_dense():
    """The same positions as a list and as a length give results within both tolerances."""
    d = Dense(35, [777], 1, 16, 2, 128, 64, 64, "bf16")
    h = d.handle()
    slots = K8.row_slots(d.table, 0, 777, 777, 64, d.cache[0].shape[0])[0].astype(np.int32)
    out, lse = h.attention_selected(d.q, torch.from_numpy(slots[None]).to(DEV), d.scale)
    close(out[0].double().cpu().numpy(), lse[0].double().cpu().numpy(), d.ref(0)[0], "bf16")
