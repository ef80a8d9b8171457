"""The binding's functions of shared prefixes, step maps and sampling give what the front end does."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from sparse_attention_indexer_gb300 import KvPages, binding as B, sample_tokens, token_probs  # noqa: E402
from tests.test_kv8_shared_gpu import I32, LARGE, Sets  # noqa: E402


def test_attention_shared():
    d = Sets(1, [(300, [5, 60, 7])], 1, 8, 2, 128, 64, 64, "bf16")
    h = d.handle()
    out, lse = d.call(h)
    q, lens, max_len, table, scale, group, group_table = d.args()
    ws = torch.empty(B.kv8_attention_shared_workspace_bytes(3, 8, 2, 128, 1), dtype=torch.uint8, device="cuda")
    o, l = torch.zeros_like(out), torch.zeros_like(lse)
    status = I32([0])
    B.kv8_attention_shared(q, float(scale), lens, max_len, group, group_table, I32(d.starts), I32(d.prefix), LARGE, table, 64, 64,
                           h.k, h.v, h.k_scale, h.v_scale, o, l, ws, status)
    assert torch.equal(o, out) and torch.equal(l, lse) and int(status) == 0
    with pytest.raises(B.Kv8Error):
        B.kv8_attention_shared(q, float(scale), lens, max_len, group, group_table, I32(d.starts), I32(d.prefix), LARGE, table, 64,
                               64, h.k, h.v, h.k_scale, h.v_scale, o, l, ws[:1024], status)


def test_maps():
    table = I32([[3, 1, 4], [2, 0, 5], [3, 1, 6]])
    pool = KvPages(table, I32([1] * 8), 16)
    rows, old, new = I32([2, 0]), I32([3, 30]), I32([9, 33])
    ref = pool.step(rows, old, new, 12)
    got = [torch.zeros(12, dtype=torch.int32, device="cuda") for _ in range(4)] + [I32([0] * 3)]
    assert B.kvpages_step(rows, old, new, table, 16, 8, *got) == 0
    assert all(torch.equal(x, y) for x, y in zip(ref, got))
    lens, starts, prefix = I32([40, 33]), I32([0, 2]), I32([0])
    assert B.kvpages_shared(rows, lens, starts, table, 16, 8, prefix) == 0
    assert prefix.tolist() == pool.shared(rows, lens, starts).tolist() == [32]


def test_sample():
    x = torch.randn((3, 5000), device="cuda")
    u, p, k = torch.rand(3, device="cuda"), torch.full((3,), 0.9, device="cuda"), I32([0, 7, 500])
    tokens, probs = I32([0] * 3), torch.zeros_like(x)
    assert B.token_sample(x, u, tokens, probs, top_k=k, top_p=p) == 0
    ref = sample_tokens(x, u, top_k=k, top_p=p, with_probs=True)
    assert torch.equal(tokens, ref[0]) and torch.equal(probs, ref[1])
    assert B.token_sample(x, probs=probs, top_p=p) == 0
    assert torch.equal(probs, token_probs(x, top_p=p))
    with pytest.raises(B.SampleError):
        B.token_sample(x, None, tokens)
