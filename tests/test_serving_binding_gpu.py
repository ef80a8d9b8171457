"""The binding's functions of the serving operators give what the tensor-level front end gives,
argument by argument (workspace, status and optional arguments of the caller's own)."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from sparse_attention_indexer_gb300 import Kv8Cache, KvPages, binding as B, verify_drafts  # noqa: E402

PAGE, BLOCK, HEADS, DIM = 32, 16, 2, 64


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def rand(gen, *s):
    return torch.randn(s, generator=gen, device="cuda")


@pytest.fixture
def gen():
    return torch.Generator(device="cuda").manual_seed(5)


def stored(gen, dtype=torch.bfloat16):
    """A cache that 70 tokens were stored into, and what is needed to store them again."""
    c = Kv8Cache.empty(4, PAGE, HEADS, DIM, BLOCK)
    wide = rand(gen, 70, 3 * HEADS * DIM).to(dtype)
    k = wide[:, :HEADS * DIM].unflatten(1, (HEADS, DIM))
    v = wide[:, -HEADS * DIM:].unflatten(1, (HEADS, DIM))
    args = k, v, torch.arange(70, device="cuda", dtype=torch.int32), i32(*[0] * 70), i32(2, 0, 3).view(1, 3)
    c.store(*args)
    return c, args


def test_store(gen):
    c, (k, v, pos, row, table) = stored(gen)
    codes = [torch.zeros_like(c.k) for _ in range(2)]
    scales = [torch.ones_like(c.k_scale) for _ in range(2)]
    status = i32(0)
    assert B.kv8_store(k, v, pos, row, table, PAGE, BLOCK, *codes, *scales, status) == 0
    for got, want in zip(codes + scales, (c.k, c.v, c.k_scale, c.v_scale)):
        assert torch.equal(got, want)
    assert int(status) == 0
    B.kv8_store(k, v, pos, row + 1, table, PAGE, BLOCK, *codes, *scales, status)
    assert int(status) == B.KV8_STATUS_TABLE_ROW
    B.kv8_store(k, v, pos, row, table, PAGE, BLOCK, *codes, *scales)  # no status
    with pytest.raises(B.Kv8Error) as e:
        B.kv8_store(k, v, pos, row, table, PAGE, 24, *codes, *scales)
    assert e.value.code == B.KV8_ERR_SHAPE


def test_attention(gen):
    c, (_, _, _, _, table) = stored(gen)
    q = rand(gen, 2, 8, DIM).to(torch.bfloat16)
    lens, scale = i32(69, 70), 1 / math.sqrt(DIM)
    want = c.attention(q, lens, 70, table, scale, 2, i32(0))
    ws = torch.empty(B.kv8_attention_workspace_bytes(8, HEADS, DIM, 2), dtype=torch.uint8,
                     device="cuda")
    out, lse, status = torch.empty_like(q), torch.empty(2, 8, device="cuda"), i32(0)
    cache = c.k, c.v, c.k_scale, c.v_scale
    assert B.kv8_attention(q, scale, lens, 70, 2, i32(0), table, PAGE, BLOCK, *cache, out, lse, ws,
                           status) == 0
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1]) and int(status) == 0
    out.zero_()
    B.kv8_attention(q, scale, lens, 70, 2, None, table, PAGE, BLOCK, *cache, out, None, ws)
    assert torch.equal(out, want[0])
    with pytest.raises(B.Kv8Error) as e:
        B.kv8_attention(q, scale, lens, 70, 2, None, table, PAGE, BLOCK, *cache, out, lse, ws[:-16])
    assert e.value.code == B.KV8_ERR_WORKSPACE
    slots = torch.cat([torch.arange(64, 96), torch.arange(7), torch.full((3,), -1)]).int().cuda()
    slots = slots.repeat(2, 1).contiguous()
    want = c.attention_selected(q, slots, scale)
    ws = torch.empty(B.kv8_attention_workspace_bytes(8, HEADS, DIM, 1), dtype=torch.uint8,
                     device="cuda")
    B.kv8_attention_selected(q, scale, slots, BLOCK, *cache, out, lse, ws, status)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1]) and int(status) == 0


def test_a_captured_call_with_a_workspace_of_its_own(gen):
    """What a capture without torch's pool of memory uses: every pointer is the caller's."""
    c, (_, _, _, _, table) = stored(gen)
    q = rand(gen, 1, 4, DIM).to(torch.float16)
    lens = i32(70)
    want = c.attention(q, lens, 70, table, 0.1)
    ws = torch.empty(B.kv8_attention_workspace_bytes(4, HEADS, DIM, 1), dtype=torch.uint8,
                     device="cuda")
    out, lse = torch.empty_like(q), torch.empty(1, 4, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        B.kv8_attention(q, 0.1, lens, 70, 1, None, table, PAGE, BLOCK, c.k, c.v, c.k_scale, c.v_scale,
                        out, lse, ws)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def state(gen):
    table = torch.full((5, 6), -1, dtype=torch.int32, device="cuda")
    refs = torch.zeros(16, dtype=torch.int32, device="cuda")
    planes = [torch.randint(0, 255, (16, n), generator=gen, device="cuda", dtype=torch.uint8)
              for n in (64, 4000)]
    return table, refs, planes


def test_pages(gen):
    a = state(gen)
    b = tuple(x.clone() for x in a[:2]) + ([p.clone() for p in a[2]],)
    pool = KvPages(a[0], a[1], 8, a[2])
    table, refs, planes = b
    arr = B.kvpages_planes(planes, 16)
    ws = torch.empty(B.kvpages_workspace_bytes(4, 16), dtype=torch.uint8, device="cuda")
    ids, counts, status = i32(*[0] * 16), i32(0, 0), i32(0)

    def same():
        assert torch.equal(a[0], table) and torch.equal(a[1], refs)
        assert all(torch.equal(x, y) for x, y in zip(a[2], planes))

    pool.reserve(i32(0), i32(0), i32(20))
    B.kvpages_reserve(i32(0), i32(0), i32(20), table, 8, refs, arr, 2, ws, status)
    same()
    pool.fork(i32(0, 0), i32(1, 2), i32(20, 9))
    B.kvpages_fork(i32(0, 0), i32(1, 2), i32(20, 9), table, 8, refs, status)
    same()
    pool.reserve(i32(1, 2), i32(20, 9), i32(21, 30))
    B.kvpages_reserve(i32(1, 2), i32(20, 9), i32(21, 30), table, 8, refs, arr, 2, ws, status)
    same()
    pool.free(i32(0, 2), i32(0, 8))
    B.kvpages_free(i32(0, 2), i32(0, 8), table, 8, refs, status)
    same()
    pool.copy(i32(1, -1), i32(15, -1))
    B.kvpages_copy(i32(1, -1), i32(15, -1), 16, arr, 2, status)
    same()
    want = pool.compact()
    B.kvpages_compact(table, refs, arr, 2, ids, counts, ws, status)
    same()
    assert torch.equal(want[0], ids) and torch.equal(want[1], counts)
    pool.free(i32(1))
    B.kvpages_free(i32(1), None, table, 8, refs)
    same()
    assert int(status) == 0 == int(pool.status)
    with pytest.raises(B.KvPagesError) as e:
        B.kvpages_reserve(i32(0), i32(0), i32(20), table, 0, refs, arr, 2, ws)
    assert e.value.code == B.KVPAGES_ERR_SHAPE


@pytest.mark.parametrize("point", [False, True])
def test_verify(gen, point):
    p = torch.softmax(2 * rand(gen, 3, 4, 501), -1)
    q = None if point else torch.softmax(2 * rand(gen, 3, 3, 501), -1)
    tokens = torch.randint(0, 501, (3, 3), generator=gen, device="cuda", dtype=torch.int32)
    u = torch.rand((3, 4), generator=gen, device="cuda")
    n = i32(3, 1, 2)
    want = verify_drafts(p, q, tokens, u, n)
    out, kept, status = torch.zeros(3, 4, dtype=torch.int32, device="cuda"), i32(9, 9, 9), i32(0)
    B.draft_verify(p, q, tokens, u, out, kept, n, status)
    assert torch.equal(out, want[0]) and torch.equal(kept, want[1]) and int(status) == 0
    with pytest.raises(B.VerifyError) as e:
        B.draft_verify(p, q, tokens, u[:, 1:].new_empty(0), out, kept)
    assert e.value.code == B.VERIFY_ERR_NULL
