"""The example that runs the serving operators together (examples/speculative_step.py)."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "speculative_step.py")


def example():
    spec = importlib.util.spec_from_file_location("speculative_step", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("k", [2048, 128])
def test_verify_steps(k):
    """Pages and counts agree after every kind of step; a sample only ever grows by what was
    kept and one token; the same seed gives the same text."""
    m = example()
    r = m.main(steps=5, k=k)
    assert r["status"] == 0 and r["owners_match"] and r["shared"] > 0
    grown = [n - p for n, p in zip(r["lens"], (300, 300, 339, 339))]
    kept = [0] * 4
    for tokens in r["texts"][1:]:
        for s, row in enumerate(tokens):
            n = sum(t >= 0 for t in row)
            assert 1 <= n <= 4 and all(t < 0 for t in row[n:])
            kept[s] += n
    assert grown == kept
    again = m.main(steps=5, k=k)
    assert again["texts"] == r["texts"] and again["lens"] == r["lens"]


def test_samples_read_their_prompts_through_shared_pages():
    """After the compaction every sample attends to the same prompt keys as its sibling: the
    dense attention of one query over the prompt alone is equal in both."""
    m = example()
    r = m.main(steps=3)
    layer = r["layer"]
    q = torch.randn((4, m.Q_HEADS, m.DIM), device="cuda").to(torch.bfloat16)
    q[1], q[3] = q[0], q[2]
    lens = m.i32([300, 300, 339, 339])
    out, lse = layer.cache.attention(q, lens, 339, layer.table, 0.1, 1, m.i32([2, 3, 4, 5]))
    assert torch.equal(lse[0], lse[1]) or torch.allclose(lse[0], lse[1], rtol=1e-5)
    assert torch.allclose(out[0].float(), out[1].float(), rtol=1e-2, atol=1e-3)
    assert torch.allclose(out[2].float(), out[3].float(), rtol=1e-2, atol=1e-3)
