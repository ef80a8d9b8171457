"""GPU parity of the page operations (kvpages_*) with the oracle: tables, counts, page data
and status bits, equal."""
import numpy as np
import pytest

from oracle import kv_pages as KP

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from sparse_attention_indexer_gb300 import KvPages  # noqa: E402


class Both:
    """One state on the GPU and in NumPy; every operation runs on both and is compared."""

    def __init__(self, seed, n_tables, width, pages, page, row_bytes=(64, 4, 12, 48, 40000)):
        rng = np.random.default_rng(seed)
        self.page = page
        self.table = np.full((n_tables, width), -1, np.int32)
        self.refs = np.zeros(pages, np.int32)
        self.planes = [rng.integers(0, 255, (pages, b)).astype(np.uint8) for b in row_bytes]
        self.rng = rng
        self.api = None

    def up(self, max_rows=64):
        t = lambda a: torch.from_numpy(a.copy()).cuda()  # noqa: E731
        self.g_planes = [t(x) for x in self.planes]
        self.api = KvPages(t(self.table), t(self.refs), self.page, self.g_planes, max_rows)

    def i(self, a):
        return None if a is None else torch.tensor(np.asarray(a, np.int64), dtype=torch.int32).cuda()

    def same(self, status):
        torch.cuda.synchronize()
        assert np.array_equal(self.api.block_table.cpu().numpy(), self.table)
        assert np.array_equal(self.api.refs.cpu().numpy(), self.refs)
        for j, (a, b) in enumerate(zip(self.g_planes, self.planes)):
            assert np.array_equal(a.cpu().numpy(), b), f"plane {j}"
        assert int(self.api.status.item()) == status
        self.api.status.zero_()

    def reserve(self, rows, old, new):
        if self.api is None:
            self.up()
        st = KP.reserve(rows, old, new, self.table, self.page, self.refs, self.planes)
        self.api.reserve(self.i(rows), self.i(old), self.i(new))
        self.same(st)
        return st

    def fork(self, parents, children, lens):
        st = KP.fork(parents, children, lens, self.table, self.page, self.refs)
        self.api.fork(self.i(parents), self.i(children), self.i(lens))
        self.same(st)
        return st

    def free(self, rows, keep=None):
        st = KP.free(rows, keep, self.table, self.page, self.refs)
        self.api.free(self.i(rows), self.i(keep))
        self.same(st)
        return st

    def compact(self):
        st, new, counts = KP.compact(self.table, self.refs, self.planes)
        ids, c = self.api.compact()
        self.same(st)
        assert np.array_equal(ids.cpu().numpy(), new) and tuple(c.tolist()) == counts
        return st

    def copy(self, src, dst):
        st = KP.copy(src, dst, self.planes, len(self.refs))
        self.api.copy(self.i(src), self.i(dst))
        self.same(st)
        return st


def test_fork_append_roll_back_compact():
    b = Both(1, 8, 9, 64, 16)
    assert b.reserve([0, 1], [0, 0], [100, 16]) == 0
    b.fork([0, 0, 1], [2, 3, 4], [100, 33, 16])
    b.reserve([0, 2, 3, 4], [100, 100, 33, 16], [101, 107, 40, 17])  # shared tails are copied
    b.free([2, 0], [65, 0])
    b.reserve([2, 5], [60, 0], [70, 3])                              # a shared page again
    b.compact()
    b.reserve([6], [0], [140])
    b.free([0, 1, 2, 3, 4, 5, 6])
    assert (b.refs == 0).all()
    b.compact()


@pytest.mark.parametrize("seed", range(6))
def test_random_lives(seed):
    rng = np.random.default_rng(100 + seed)
    page = int(rng.choice([1, 3, 16, 64]))
    b = Both(seed, 12, 20, int(rng.choice([33, 120, 1000])), page)
    b.up()
    lens = [0] * 12
    for _ in range(25):
        op = rng.integers(0, 5)
        pick = rng.permutation(12)[:rng.integers(1, 7)]
        if op <= 1:
            new = [min(20 * page, lens[r] + int(rng.integers(0, 5 * page))) for r in pick]
            before = b.table.copy()
            b.reserve(pick.tolist(), [lens[r] for r in pick], new)
            for r, n in zip(pick, new):
                if all(b.table[r, c] >= 0 for c in range(-(-n // page))):
                    lens[r] = n
                else:
                    assert np.array_equal(before[r], b.table[r])
        elif op == 2:
            kids = [r for r in pick if lens[r] == 0 and (b.table[r] < 0).all()]
            pars = [r for r in range(12) if lens[r] and r not in kids]
            if kids and pars:
                p = [int(rng.choice(pars)) for _ in kids]
                n = [int(rng.integers(0, lens[q] + 1)) for q in p]
                b.fork(p, [int(k) for k in kids], n)
                for k, x in zip(kids, n):
                    lens[k] = x
        elif op == 3:
            keep = [int(rng.integers(0, lens[r] + 1)) if rng.random() < 0.6 else 0 for r in pick]
            b.free(pick.tolist(), keep)
            for r, n in zip(pick, keep):
                lens[r] = n
        else:
            b.compact()
        assert np.array_equal(b.refs, np.bincount(b.table[b.table >= 0], minlength=len(b.refs)))


def test_reserve_runs_out_in_row_order():
    b = Both(2, 5, 10, 7, 8)
    assert b.reserve([3, 0, 1, 2], [0, 0, 0, 0], [32, 32, 8, 0]) == KP.NO_PAGE
    assert (b.table[3] >= 0).sum() == 4 and (b.table[:3] < 0).all()
    assert b.reserve([0], [0], [24]) == 0
    assert b.reserve([1], [0], [1]) == KP.NO_PAGE


def test_refused_arguments_on_the_device():
    b = Both(3, 4, 6, 16, 8)
    b.up()
    assert b.reserve([4, -1, 0, 1, 2], [0, 0, 5, -1, 0], [8, 8, 4, 8, 49]) == KP.ROW | KP.LEN
    assert (b.table < 0).all()
    b.reserve([0], [0], [40])
    assert b.fork([0, 0, 0, 9, 0], [1, 5, 2, 3, 0], [40, 8, 49, 8, 8]) == KP.ROW | KP.LEN | KP.CHILD
    assert b.free([1, 7, 0], [-1, 0, 40]) == KP.ROW | KP.LEN
    assert b.copy([0, -1, 3, 16, -1], [9, -1, -1, 2, 5]) == KP.PAGE
    b.table[3, 0], b.table[3, 1] = 20, 15       # past the pool; a page that nobody owns
    b.up()
    assert b.compact() == KP.PAGE | KP.REFS
    assert b.reserve([3], [0], [8]) == KP.PAGE
    assert b.fork([3], [2], [8]) == KP.PAGE
    assert b.free([3]) == KP.PAGE | KP.REFS


def test_reserve_of_pages_shared_inside_one_call():
    """Two owners of one page append in the same call: both get copies."""
    b = Both(4, 4, 4, 16, 8)
    b.reserve([0], [0], [12])
    b.fork([0], [1], [12])
    b.reserve([0, 1], [12, 12], [13, 20])
    assert b.table[0, 1] != b.table[1, 1] and b.table[0, 0] == b.table[1, 0]
    assert b.refs[1] == 0


@pytest.mark.parametrize("pages", [1, 2, 31, 16384, 16385, 40000])
def test_compact_pools(pages):
    b = Both(5, 3, -(-pages // 3) + 1, pages, 4, row_bytes=(16, 4))
    live = np.nonzero(b.rng.random(pages) < 0.45)[0]
    b.table.reshape(-1)[:len(live)] = b.rng.permutation(live)
    b.refs[live] = 1
    b.up()
    b.compact()
    b.compact()


def test_large_pool_reserve():
    b = Both(6, 40, 600, 50000, 4, row_bytes=(16,))
    b.refs[b.rng.random(50000) < 0.7] = 1
    b.up()
    b.reserve(list(range(40)), [0] * 40, [int(x) for x in b.rng.integers(0, 1600, 40)])


def test_more_rows_than_one_round_of_the_plan():
    b = Both(7, 2500, 3, 9000, 4, row_bytes=(16, 8))
    b.up(max_rows=2500)
    rows = b.rng.permutation(2500)
    b.reserve(rows.tolist(), [0] * 2500, b.rng.integers(0, 13, 2500).tolist())


@pytest.mark.parametrize("n", [1, 32, 1023, 1024, 1025])
@pytest.mark.parametrize("free", [0, 700, 5000])
def test_appends_of_one_or_two_pages(n, free):
    """Decode and verify steps of up to and over a CTA's rows, with pages enough and not, some of
    them shared, some rows refused."""
    b = Both(12, n + 3, 4, 6000, 8, row_bytes=(16, 8))
    rows = b.rng.permutation(n).astype(int)
    old = b.rng.integers(0, 17, n)
    new = np.minimum(old + b.rng.integers(0, 9, n), 32)
    own = b.rng.permutation(6000)
    at = 0
    for r, o in zip(rows, old):
        for c in range(-(-int(o) // 8)):
            b.table[r, c] = own[at % 900]       # shared by several rows once more than 900 are out
            at += 1
    b.refs[:] = np.bincount(b.table[b.table >= 0], minlength=6000)
    spare = np.nonzero(b.refs == 0)[0]
    b.refs[b.rng.permutation(spare)[:max(0, len(spare) - free)]] = 1
    if n > 40:
        old[5], new[6], rows[7] = -1, 40, n + 3
    b.up(max_rows=2000)
    b.reserve(rows.tolist(), old.tolist(), new.tolist())


def test_copy_planes_and_padding():
    b = Both(8, 1, 1, 300, 4, row_bytes=(16, 20, 16384, 16388, 50000))
    b.up()
    perm = b.rng.permutation(300)
    src, dst = perm[:100].copy(), perm[200:].copy()
    src[::7], dst[::7] = -1, -1
    b.copy(src, dst)
    b.copy([], [])


def test_no_planes_and_unaligned_planes():
    b = Both(9, 2, 4, 16, 8, row_bytes=())
    b.reserve([0], [0], [20])
    b.compact()
    b = Both(10, 2, 4, 16, 8, row_bytes=(32,))
    buf = torch.zeros(16 * 32 + 4, dtype=torch.uint8, device="cuda")
    view = buf[4:].view(16, 32)  # 4-byte alignment only
    view.copy_(torch.from_numpy(b.planes[0]))
    api = KvPages(torch.from_numpy(b.table).cuda(), torch.from_numpy(b.refs).cuda(), 8, [view])
    api.copy(b.i([1, 2]), b.i([9, 0]))
    KP.copy([1, 2], [9, 0], b.planes, 16)
    assert np.array_equal(view.cpu().numpy(), b.planes[0])


def test_captured_in_a_graph():
    b = Both(11, 6, 8, 64, 16)
    b.reserve([0], [0], [100])
    kids, par, n = b.i([1, 2, 3]), b.i([0, 0, 0]), b.i([100] * 3)
    more = n + 1
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        b.api.free(kids)
        b.api.fork(par, kids, n)
        b.api.reserve(kids, n, more)
    for _ in range(3):
        g.replay()
        KP.free([1, 2, 3], None, b.table, 16, b.refs)
        KP.fork([0] * 3, [1, 2, 3], [100] * 3, b.table, 16, b.refs)
        KP.reserve([1, 2, 3], [100] * 3, [101] * 3, b.table, 16, b.refs, b.planes)
        b.same(0)


def test_a_pool_dropped_while_another_stream_works():
    """The instance's buffers are not given out again while work of its stream is on its way."""
    b = Both(13, 6, 8, 64, 16)
    b.up()
    api, s = b.api, torch.cuda.Stream()
    buffers = {(t.numel(), t.dtype, t.data_ptr())
               for t in (api.workspace, api.new_ids, api.counts, api.status)}
    table, refs = api.block_table, api.refs
    rows, old, new = b.i([0, 1]), b.i([0, 0]), b.i([40, 100])
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(200_000_000)  # about a tenth of a second
        api.reserve(rows, old, new)
    b.api = api = None
    held = [torch.empty(n, dtype=t, device="cuda") for n, t, _ in buffers for _ in range(3)]
    working = not s.query()
    assert not working or not {t.data_ptr() for t in held} & {at for _, _, at in buffers}
    torch.cuda.synchronize()
    KP.reserve([0, 1], [0, 0], [40, 100], b.table, 16, b.refs, b.planes)
    assert np.array_equal(table.cpu().numpy(), b.table) and np.array_equal(refs.cpu().numpy(), b.refs)
