"""kv8_attention_shared for batches of a few hundred requests and the calls around the usual ones.
Behind a prefix the rows' own pass runs one warp to a CTA from about 1500 units (a request on a key
head) on, and keeps its split units by CTA in place of by unit from 2048 on. Oracle and tolerances
are those of tests/test_kv8_shared_gpu.py."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from sparse_attention_indexer_gb300 import Kv8Cache, binding as B  # noqa: E402
from tests.test_kv8_gpu import close  # noqa: E402
from tests.test_kv8_shared_gpu import I32, LARGE, Sets  # noqa: E402


def ragged(rng, n, long):
    """Own tokens of n requests: most a few, some none (None: a row of length 0), some `long`."""
    own = [int(x) for x in rng.integers(0, 60, n)]
    for i in range(0, n, 17):
        own[i] = long - i
    for i in range(5, n, 23):
        own[i] = None
    for i in range(7, n, 29):
        own[i] = 0
    return own


@pytest.mark.parametrize("ratio,dim,dtype", [(1, 128, "bf16"), (2, 64, "fp16"), (8, 128, "fp16"), (16, 64, "bf16")])
@pytest.mark.parametrize("requests", [180, 200, 230, 255, 257, 300])
def test_requests_by_units(requests, ratio, dim, dtype):
    """1440 to 2400 units on 8 key heads."""
    rng = np.random.default_rng(requests + ratio)
    cut = requests // 3
    own = ragged(rng, requests, 2000)
    d = Sets(requests, [(512, own[:cut]), (144, own[cut:])], 1, 8 * ratio, 8, dim, 16, 16, dtype)
    rows = [0, 1, 5, 7, 17, 34, 36, cut - 1, cut, cut + 1, requests // 2, requests - 3, requests - 2, requests - 1]
    d.check(rows=rows)


@pytest.mark.parametrize("requests", [120, 300])
def test_verify_steps_by_units(requests):
    """Two and three query rows to a request, 16 rows and 32 to a unit."""
    rng = np.random.default_rng(requests)
    for group, hq in ((2, 64), (3, 64)):
        own = [None if x is None else x + group for x in ragged(rng, requests, 1000)]
        d = Sets(requests + group, [(256, own)], group, hq, 8, 64, 32, 32, "bf16", loose=1)
        n = len(d.lens)
        d.check(rows=list(range(0, 9)) + [n // 2, n - 4, n - 3, n - 2, n - 1])


def test_every_row_of_a_batch():
    rng = np.random.default_rng(3)
    Sets(3, [(512, ragged(rng, 270, 1500)), (256, ragged(rng, 30, 300))], 1, 16, 8, 128, 64, 64, "bf16").check()


@pytest.mark.parametrize("group,short", [(2, 1), (7, 3), (8, 5)])
def test_last_group_is_shorter(group, short):
    d = Sets(4 + group, [(300, [40, group, 60])], group, 16, 2, 128, 32, 32, "bf16")
    d.lens = d.lens[:-short]
    d.q = d.q[:-short]
    d.check()


def test_most_sets():
    """KV8_MAX_SETS sets of a request or two, and one set more, which is refused."""
    sets = [(128 + 16 * (i % 3), [1 + i % 5] * (1 + i % 2)) for i in range(B.KV8_MAX_SETS)]
    d = Sets(5, sets, 1, 4, 1, 64, 16, 16, "fp16")
    d.check(rows=list(range(0, len(d.lens), 101)) + [len(d.lens) - 1])
    d.starts.append(d.starts[-1])
    d.prefix.append(0)
    with pytest.raises(B.Kv8Error):
        d.call(d.handle())


def test_workspace_grows_and_serves_fewer_rows_again():
    """One handle on one stream: fewer rows, more, fewer again, the same bits each time."""
    few = Sets(6, [(3000, [5, 60, 7]), (2000, [100, 2])], 1, 16, 2, 128, 64, 64, "bf16")
    h = few.handle()
    ref = few.call(h)
    held = [ws[1][1] for ws in h._workspaces.values()]
    pages = h.k.shape[0] // 64
    n = 400
    table = torch.from_numpy(few.table).cuda()[[0, 1, 2] * 100 + [0] * 100]
    assert int(table.max()) < pages
    q = torch.randn((n, 16, 128), device="cuda").to(torch.bfloat16)
    more = dict(q=q, lens=torch.full((n,), 2900, dtype=torch.int32, device="cuda"), max_len=3000, block_table=table,
                sm_scale=0.09, set_starts=I32([0, n]), prefix_lens=I32([2880]), max_prefix=LARGE)
    big = h.attention_shared(**more)
    assert [ws[1][1] for ws in h._workspaces.values()] > held  # the same entry, larger
    for _ in range(3):
        got = few.call(h)
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
        got = h.attention_shared(**more)
        assert torch.equal(got[0], big[0]) and torch.equal(got[1], big[1])
    assert int(h.status.item()) == 0


def test_workspace_rows_past_32_bits():
    """The prefix's parts of 135000 rows of 64 heads lie more than 2^32 bytes into the workspace. Every
    row is one of five requests'."""
    rows, hq, hk, dim, page = 135000, 64, 8, 128, 64
    d = Sets(7, [(192, [3, 20, 30, 40, 50])], 1, hq, hk, dim, page, page, "bf16")
    h = d.handle()
    assert rows * hq * (dim + 4) * 4 > 2 ** 32
    which = torch.arange(rows, device="cuda") % 5
    q, lens, max_len, table, scale, _, _ = d.args()
    out, lse = h.attention_shared(q[which], lens[which], max_len, table, float(scale), I32([0, rows]), I32([192]),
                                  LARGE, 1, which.to(torch.int32))
    assert int(h.status.item()) == 0
    for r in range(5):  # the least and the largest of each output over a request's rows
        ref, _ = d.ref(r)
        for end in (torch.amin, torch.amax):
            close(end(out[r::5], 0).double().cpu().numpy(), end(lse[r::5], 0).double().cpu().numpy(), ref, "bf16",
                  f"request {r}")
