"""A step of fewer tokens than places, as a captured graph runs it: what KvPages.step writes behind the
last token goes through the store and both forms of the attention."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from sparse_attention_indexer_gb300 import Kv8Cache, KvPages, binding as B  # noqa: E402

I32 = lambda a: torch.tensor(np.asarray(a, np.int64), dtype=torch.int32, device="cuda")  # noqa: E731


@pytest.mark.parametrize("spare", [0, 1, 70])
def test_places_behind_the_last_token(spare):
    torch.manual_seed(spare)
    page, heads, dim = 32, 2, 64
    cache = Kv8Cache.empty(80, page, heads, dim)
    for x in (cache.k, cache.v):
        x.copy_(torch.randint(0, 120, x.shape, dtype=torch.uint8, device="cuda"))
    table = torch.full((6, 10), -1, dtype=torch.int32, device="cuda")
    pool = KvPages(table, torch.zeros(80, dtype=torch.int32, device="cuda"), page, cache.planes())
    rows, old, new = I32([4, 0, 3]), I32([0, 0, 0]), I32([200, 1, 150])
    pool.reserve(rows, old, new)
    before = [x.clone() for x in (cache.k, cache.v)]
    n = 351 + spare
    s = pool.step(rows, old, new, n)
    k, v, q = (torch.randn((n, h, dim), device="cuda").to(torch.bfloat16) for h in (heads, heads, 4))
    k[351:] = float("nan")
    v[351:] = float("nan")
    q[351:] = float("nan")
    cache.store(k, v, s.positions, s.token_table, table)
    bits = B.KV8_STATUS_TABLE_ROW | B.KV8_STATUS_POSITION if spare else 0
    assert int(cache.status.item()) & ~bits == 0 and (int(cache.status.item()) != 0) == (spare > 0)
    idle = torch.ones(cache.k.shape[0], dtype=torch.bool, device="cuda")
    idle[s.slots[:351].long()] = False
    for x, y in zip((cache.k, cache.v), before):
        assert torch.equal(x[idle], y[idle])
    cache.status.zero_()
    out, lse = cache.attention(q, s.lens, 200, table, 0.125, 1, s.token_table)
    assert int(cache.status.item()) == (B.KV8_STATUS_TABLE_ROW if spare else 0)
    assert (out[351:] == 0).all() and torch.isneginf(lse[351:]).all()
    assert torch.isfinite(out[:351]).all() and torch.isfinite(lse[:351]).all()
    # causal rows of a prompt share its beginning: those behind the 128th position of the two long ones
    sets, prefix = I32([127, 200, 328, n]), I32([128, 0, 128])
    both, ls = cache.attention_shared(q, s.lens, 200, table, 0.125, sets, prefix, 1 << 30, 1, s.token_table)
    assert int(cache.status.item()) == (B.KV8_STATUS_TABLE_ROW if spare else 0)
    assert (both[351:] == 0).all() and torch.isneginf(ls[351:]).all()
    # two roundings to bf16 (2^-8 of the largest together), weights to fp16 (2^-10), sums in fp32
    assert (both[:351].float() - out[:351].float()).abs().max() <= 2 ** -7 * out[:351].float().abs().max()
    assert (ls[:351] - lse[:351]).abs().max() <= 2 ** -9
