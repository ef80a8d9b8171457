"""kv8_attention_shared at the largest length: 2^31 - 1 positions, a table row that names one page again
and again. The length's last tile ends past 2^31."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from sparse_attention_indexer_gb300 import Kv8Cache  # noqa: E402


def test_longest_prefix():
    """Queries of 0 weigh all positions alike: out is the values' mean, here one value in all positions,
    and lse the length's logarithm. A CTA adds up to 2^31 / 128 / 152 / 2 < 2^16 tiles of a stream, 8
    products each: sums of weights lose at most 2^16 half steps, 2^-8, and sums of values at most
    2^19 steps of 2^-23, 2^-4."""
    page, n = 1 << 16, (1 << 31) - 1
    cache = Kv8Cache.empty(1, page, 1, 64, 64)
    cache.k.copy_(torch.randint(0, 120, cache.k.shape, dtype=torch.uint8, device="cuda"))
    value = torch.linspace(-3, 3, 64, device="cuda").to(torch.float8_e4m3fn)
    cache.v.copy_(value.view(torch.uint8).expand(cache.v.shape))
    table = torch.zeros((1, 1 << 15), dtype=torch.int32, device="cuda")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    q = torch.zeros((2, 2, 64), dtype=torch.bfloat16, device="cuda")
    out, lse = cache.attention_shared(q, i32(n, n), n, table, 0.125, i32(0, 2), i32(n), n, group_table=i32(0, 0))
    assert int(cache.status.item()) == 0
    assert (lse - math.log(n)).abs().max() <= 2 ** -7
    assert ((out.float() - value.float()).abs() <= (2 ** -3) * value.float().abs() + 2 ** -8).all()
