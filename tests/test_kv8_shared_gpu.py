"""GPU parity of attention over shared prefixes (kv8_attention_shared) with the float64 oracle.

The oracle knows nothing of prefixes: each row attends to the slots of its own table. The
tolerances are those of the attention tests (tests/test_kv8_gpu.py); the pass over a prefix holds
more of each weight (a reference 2^7 below the row's largest) and joins one part more, which the
2^-18 * a of that bound counts as it counts the others. Everything that no row attends to is NaN.
The bound on the prefixes is given as LARGE, so that short ones too are read once for all.
"""
import numpy as np
import pytest

from oracle import kv8 as K8

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from sparse_attention_indexer_gb300 import KvPages, binding as B  # noqa: E402
from tests.test_kv8_gpu import DEV, TYPES, Dense, attention_cache, close  # noqa: E402

LARGE = 1 << 30
I32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)  # noqa: E731


class Sets(Dense):
    """sets: (prefix positions, own tokens of each request; None: a row of length 0). The pages
    that lie wholly below the prefix are one request's; `group` rows of a request see all but the
    last tokens. loose: requests in no set before and behind them."""

    def __init__(self, seed, sets, group, hq, hk, dim, page, block, dtype, wide=False, q_gain=1.0,
                 loose=0, poison=True, q_pad=0):
        rng = np.random.default_rng(seed)
        self.rng, self.group, self.page, self.block, self.dtype = rng, group, page, block, dtype
        lens, who, shared, starts, self.prefix = [], [], [], [loose], []
        for _ in range(loose):
            who.append(len(lens))
            shared.append(0)
            lens.append(int(rng.integers(1, 300)) + group)
        for pre, own in sets:
            first = None
            for x in own:
                r = len(lens)
                if x is None:
                    who.append(r)
                    shared.append(0)
                    lens.append(0)
                    continue
                first = r if first is None else first
                who.append(first)
                shared.append(pre // page)
                lens.append(pre + x)
            starts.append(len(lens))
            self.prefix.append(pre // page * page)
        for _ in range(loose):
            who.append(len(lens))
            shared.append(0)
            lens.append(int(rng.integers(1, 300)) + group)
        groups = len(lens)
        self.request_lens = lens
        self.starts = starts
        self.lens = np.asarray([max(0, n - (group - 1 - i)) for n in lens for i in range(group)], np.int32)
        self.max_len = max(1, max(lens))
        need = [-(-n // page) for n in lens]
        width = max(1, max(need))
        pages = sum(n - (s if w != r else 0) for r, (n, s, w) in enumerate(zip(need, shared, who))) + 2
        perm = rng.permutation(pages)
        self.table = np.full((groups, width), -1, np.int32)
        at = 0
        for r, n in enumerate(need):
            own = shared[r] if who[r] != r else 0
            self.table[r, :own] = self.table[who[r], :own]
            self.table[r, own:n] = perm[at:at + n - own]
            at += n - own
        self.cache = attention_cache(rng, pages, page, hk, dim, block, wide)
        if poison:
            used = np.zeros(pages * page, bool)
            for r, n in enumerate(lens):
                used[K8.row_slots(self.table, r, n, self.max_len, page, pages * page)[0]] = True
            for x in self.cache[:2]:
                x[~used] = 0x7F
            for x in self.cache[2:]:
                x[~used.reshape(-1, block).any(1)] = np.nan
        rows = len(self.lens)
        q = torch.from_numpy((rng.standard_normal((rows, hq, dim)) * q_gain).astype(np.float32))
        buf = torch.zeros((rows, hq * dim + q_pad), dtype=TYPES[dtype], device=DEV)
        buf[:, :hq * dim] = q.to(TYPES[dtype]).view(rows, -1).to(DEV)
        self.q = buf[:, :hq * dim].unflatten(1, (hq, dim))
        self.scale = 1.0 / np.sqrt(dim)
        self.group_table = np.arange(groups, dtype=np.int32)

    def call(self, h, **kw):
        q, lens, max_len, table, scale, group, group_table = self.args()
        a = dict(q=q, lens=lens, max_len=max_len, block_table=table, sm_scale=float(scale),
                 set_starts=I32(self.starts), prefix_lens=I32(self.prefix),
                 max_prefix=LARGE, group_rows=group, group_table=group_table)
        a.update(kw)
        return h.attention_shared(**a)

    def check(self, rows=None, status=0, **kw):
        h = self.handle()
        out, lse = self.call(h, **kw)
        torch.cuda.synchronize()
        o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
        for r in range(len(self.lens)) if rows is None else rows:
            ref, _ = self.ref(r)
            close(o[r], l[r], ref, self.dtype, f"row {r} len {self.lens[r]}")
        assert int(h.status.item()) == status
        return out, lse


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page,block", [(16, 16), (64, 64), (64, 16), (48, 16), (128, 32), (80, 80)])
def test_pages_and_blocks(page, block, dim, dtype):
    Sets(page + dim, [(400, [3, 50, 1]), (128 + page, [10, 200])], 1, 8, 2, dim, page, block, dtype).check()


@pytest.mark.parametrize("pre", [127, 128, 129, 143, 144, 255, 256, 257, 384, 500, 1000])
def test_prefix_lengths(pre):
    """Prefixes around the tiles of 128 positions, on pages of 16."""
    Sets(pre, [(pre, [5, 17])], 1, 4, 1, 128, 16, 16, "bf16").check()


@pytest.mark.parametrize("hq,hk", [(1, 1), (2, 1), (16, 1), (7, 1), (12, 4), (40, 8), (8, 8)])
@pytest.mark.parametrize("group", [1, 2, 7, 8])
def test_heads_and_groups(hq, hk, group):
    Sets(hq * 10 + group, [(300, [group + 5, group, group + 90]), (160, [group + 1, 2 * group])], group,
         hq, hk, 128 if hq % 2 else 64, 32, 32, "bf16").check()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("requests", [2, 8, 9, 16, 17, 24, 32, 33, 50])
def test_set_sizes(requests, dim):
    """128 rows of a set fill a stream, 256 both."""
    own = [1 + 7 * i % 60 for i in range(requests)]
    Sets(requests, [(700, own)], 1, 16, 1, dim, 64, 64, "bf16").check(rows=range(0, requests, 3))


def test_padding_rows_and_loose_requests():
    sets = [(256, [None, 4, None, 30]), (300, [None, None]), (200, [9]), (0, [5, 6]), (512, [40, None, 41])]
    Sets(3, sets, 1, 8, 2, 128, 32, 16, "fp16", loose=3).check()
    Sets(4, sets, 3, 8, 2, 64, 32, 16, "bf16", loose=2).check()


def test_prefixes_longer_than_some_rows():
    """A row that ends inside the prefix: what is read for all ends there."""
    d = Sets(5, [(512, [20, 30, 40])], 1, 8, 1, 128, 64, 64, "bf16", poison=False)
    d.lens[1] = 300
    d.check()
    d.lens[2] = 100  # less than is worth a pass
    d.check()
    d.lens[:] = [532, 0, 0]  # one row alone
    d.check()


def test_prefix_inside_a_page():
    """A prefix length that is no multiple of anything, below what the rows share."""
    d = Sets(6, [(640, [20, 30, 40, 50])], 1, 16, 2, 128, 64, 32, "bf16")
    for pre in (129, 200, 333, 640):
        d.prefix = [pre]
        d.check()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_long_prefixes_split_over_the_grid(dtype):
    Sets(7, [(20000, [100, 3000, 1])], 1, 16, 2, 128, 64, 64, dtype).check()
    Sets(8, [(9000, [10] * 20), (5000, [20] * 33)], 1, 8, 1, 64, 32, 16, dtype).check(rows=[0, 19, 20, 52])


def test_more_units_than_the_grid():
    """Whole units beside split ones: 40 sets on 8 heads."""
    sets = [(160 + 32 * (i % 7), [3 + i, 5, 2]) for i in range(40)]
    d = Sets(9, sets, 1, 16, 8, 64, 32, 32, "bf16")
    d.check(rows=range(0, len(d.lens), 5))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_value_scales_far_apart(dtype):
    Sets(10, [(600, [64, 100, 9])], 1, 16, 1, 128, 64, 16, dtype, wide=True).check()
    Sets(11, [(2000, [64] * 20)], 1, 16, 1, 64, 64, 16, dtype, wide=True).check(rows=[0, 7, 19])


def test_peaked_and_flat_rows():
    for gain in (0.0, 20.0, 60.0):
        Sets(12, [(900, [64, 100, 9])], 1, 8, 1, 128, 64, 64, "bf16", q_gain=gain).check()


def test_zero_scales_and_score_scales():
    d = Sets(13, [(700, [20, 40, 60])], 1, 16, 1, 128, 64, 16, "bf16")
    d.cache[3][::3] = 0.0
    d.check()
    d.cache[2][::2] = 0.0
    d.check()
    d.cache[3][:] = 0.0
    d.check()
    for scale in (-0.1, 0.0, 5.0):
        d = Sets(14, [(700, [20, 40, 60])], 1, 16, 1, 128, 64, 16, "bf16")
        d.scale = scale
        d.check()


def test_blocks_of_the_least_scale():
    """A block of zeros has the store's least scale, 2^-120: its keys still count."""
    d = Sets(15, [(512, [20, 40])], 1, 8, 1, 128, 64, 64, "bf16")
    for page in (1, 4):
        at = d.table[0, page]
        d.cache[1][at * 64:(at + 1) * 64] = 0
        d.cache[3][at] = 2.0 ** -120
    d.check()
    at = d.table[0, 0]
    d.cache[1][at * 64:(at + 1) * 64] = 0
    d.cache[3][at] = 2.0 ** -120
    d.check()


def test_nan_codes_in_the_prefix():
    """A NaN key or value makes the rows that see it NaN, and no others."""
    d = Sets(16, [(300, [20, 40]), (300, [21, 41, None])], 1, 8, 2, 128, 16, 16, "bf16")
    slot = d.table[0, 3] * 16 + 5
    d.cache[1][slot, 1, 7] = 0x7F
    out, lse = d.check(rows=[2, 3, 4])
    o = out.float().cpu()
    assert torch.isnan(o[:2, 4:, 7]).all() and not torch.isnan(o[:2, :4]).any()
    assert not torch.isnan(lse).any()
    d.cache[0][slot, 0, 1] = 0xFF
    out, lse = d.check(rows=[2, 3, 4])
    assert torch.isnan(out[:2, :4]).all() and torch.isnan(lse[:2, :4]).all()


def test_same_table_row_for_all():
    """group_table: several groups through one table row, whose whole length is the prefix."""
    d = Sets(17, [(512, [0, 0, 0])], 1, 8, 2, 128, 64, 64, "bf16")
    d.group_table[:] = 1
    d.check()


def test_refused_entries_and_sets():
    d = Sets(18, [(512, [20, 40]), (256, [3, 4])], 1, 8, 2, 128, 64, 64, "bf16", poison=False)
    d.table[0, 2] = -1  # a page that is missing is skipped by all rows of the set
    d.table[1, 2] = -1
    d.check(status=B.KV8_STATUS_TABLE_ENTRY)
    d.table[0, 3] = d.table[1, 3] = 10 ** 6
    d.check(status=B.KV8_STATUS_TABLE_ENTRY | B.KV8_STATUS_SLOT)
    d = Sets(19, [(512, [20, 40]), (256, [3, 4])], 1, 8, 2, 128, 64, 64, "bf16")
    for starts in ([0, 3, 2], [-1, 2, 4], [0, 2, 5], [2, 0, 4]):  # read row by row, still right
        d.starts = starts
        d.check(status=B.KV8_STATUS_SETS)
    d.starts = [0, 2, 4]
    d.prefix = [LARGE, 256]  # the first set's is past the bound
    d.check(status=B.KV8_STATUS_SETS, max_prefix=LARGE - 1)
    d.prefix = [-1, 256]
    d.check(status=B.KV8_STATUS_SETS)
    d.lens[2] = 9999
    d.max_len = 600
    h = d.handle()
    out, lse = d.call(h)
    assert int(h.status.item()) == B.KV8_STATUS_SETS | B.KV8_STATUS_LEN
    assert (out[2] == 0).all() and torch.isneginf(lse[2]).all()


def test_no_sets_and_no_rows():
    d = Sets(20, [(256, [5, 9])], 1, 8, 2, 128, 64, 64, "bf16")
    d.starts, d.prefix = [0], []
    d.check()
    h = d.handle()
    none = I32([])
    out, lse = h.attention_shared(d.q[:0], none, 10, I32(d.table), 0.1, I32([0, 0]), I32([128]), 128)
    assert out.shape == (0, 8, 128) and lse.shape == (0, 8)


def test_prefixes_that_are_left_to_the_rows():
    """By the bound no time is saved: the plain attention's bits, whatever the sets say."""
    d = Sets(25, [(300, [5, 60, 7])], 1, 8, 2, 128, 64, 64, "bf16")
    out, lse = d.check(max_prefix=300)
    h = d.handle()
    ref = h.attention(*d.args())
    assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])


def test_strided_rows():
    Sets(21, [(300, [5, 60, 7])], 1, 8, 2, 128, 64, 64, "bf16", q_pad=64).check()


def test_runs_streams_and_graphs_agree():
    """Equal bit for bit: again, on another stream, by graphs that one capture stream made and
    two replay at once, and after a call of more rows has grown the workspace."""
    d = Sets(22, [(3000, [5, 60, 7]), (2000, [100, 2])], 1, 16, 2, 128, 64, 64, "bf16")
    h = d.handle()
    out, lse = d.call(h)
    more = Sets(23, [(500, [5] * 40)], 1, 16, 2, 128, 64, 64, "bf16")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o2, l2 = d.call(h, stream=s)
    s.synchronize()
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    big = more.handle()
    more.call(big)
    a = d.args()
    kw = dict(q=a[0], lens=a[1], max_len=a[2], block_table=a[3], sm_scale=float(a[4]), group_rows=a[5],
              group_table=a[6], set_starts=I32(d.starts), prefix_lens=I32(d.prefix), max_prefix=LARGE)
    graphs = []
    for _ in range(2):
        o, l = torch.zeros_like(out), torch.zeros_like(lse)
        h.attention_shared(out=o, lse=l, **kw)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            h.attention_shared(out=o, lse=l, **kw)
        graphs.append((g, o, l))
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(10):
        for (g, o, l), st in zip(graphs, streams):
            o.zero_()
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for _, o, l in graphs:
            assert torch.equal(out, o) and torch.equal(lse, l)
    assert int(h.status.item()) == 0


def test_with_the_pages_that_make_such_batches():
    """fork, reserve (copy on write), shared, attention_shared: as a serving step calls them."""
    rng = np.random.default_rng(24)
    page, hk, dim = 64, 2, 128
    pages = 64
    cache = [torch.from_numpy(x).to(DEV) for x in attention_cache(rng, pages, page, hk, dim, 64, False)]
    from sparse_attention_indexer_gb300 import Kv8Cache
    h = Kv8Cache(*cache, page, 64)
    table = torch.full((10, 12), -1, dtype=torch.int32, device=DEV)
    pool = KvPages(table, torch.zeros(pages, dtype=torch.int32, device=DEV), page, h.planes())
    pool.reserve(I32([0, 1]), I32([0, 0]), I32([500, 300]))
    rows, lens = I32([2, 3, 4, 5, 6]), I32([500, 500, 500, 300, 300])
    pool.fork(I32([0, 0, 0, 1, 1]), rows, lens)
    pool.free(I32([0, 1]))
    pool.reserve(rows, lens, lens + 1)
    starts = I32([0, 3, 5])
    prefix = pool.shared(rows, lens + 1, starts)
    assert prefix.tolist() == [448, 256]
    q = torch.randn((5, 16, dim), device=DEV).to(torch.bfloat16)
    got = h.attention_shared(q, lens + 1, 501, table, 0.09, starts, prefix, LARGE, group_table=rows)
    ref = h.attention(q, lens + 1, 501, table, 0.09, group_table=rows)
    assert torch.allclose(got[1], ref[1], rtol=0, atol=1e-3)
    assert torch.allclose(got[0].float(), ref[0].float(), rtol=2 ** -6, atol=2 ** -8)
    assert int(h.status.item()) == 0 and int(pool.status.item()) == 0


def test_offsets_past_32_bits():
    """Codes and workspace rows behind 2^32 bytes: the prefix's pages lie at the end of a large cache."""
    from sparse_attention_indexer_gb300 import Kv8Cache
    page, hk, dim, pages = 64, 8, 128, 70000  # 4.6e9 bytes of keys
    d = Sets(26, [(300, [5, 60])], 1, 16, hk, dim, page, page, "bf16", poison=False)
    small = d.handle()
    n = d.cache[0].shape[0] // page
    code = lambda: torch.full((pages * page, hk, dim), 0x7F, dtype=torch.uint8, device=DEV)  # noqa: E731
    scale = lambda: torch.full((pages, hk), float("nan"), device=DEV)  # noqa: E731
    large = Kv8Cache(code(), code(), scale(), scale(), page, page)
    for x, y in ((large.k, small.k), (large.v, small.v), (large.k_scale, small.k_scale), (large.v_scale, small.v_scale)):
        x[-y.shape[0]:] = y
    ref = d.call(small)
    got = d.call(large, block_table=I32(np.where(d.table >= 0, d.table + pages - n, -1)))
    assert torch.equal(ref[0], got[0]) and torch.equal(ref[1], got[1])
    assert int(large.status.item()) == 0
