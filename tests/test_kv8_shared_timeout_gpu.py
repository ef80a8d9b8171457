"""A wait of kv8_attention_shared that runs out shows in the results, not in the status alone: what
the CTA was to give is NaN, never what an earlier call left in the workspace. The wait runs out
because the keys and values of one CTA never come (kv8_attention_shared_test); no GPU fault."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from sparse_attention_indexer_gb300 import binding as B  # noqa: E402
from tests.test_kv8_shared_gpu import I32, LARGE, Sets  # noqa: E402

CASES = {
    # a unit of two pairs of streams split over the grid, one of streams that take keys in turn
    "split": ([(9000, [10] * 20), (5000, [20] * 40)], 1, 8, 1, 64),
    # several whole units to a CTA: those behind the one that waits are not begun
    "whole": ([(160 + 32 * (i % 7), [3 + i, 5, 2, None]) for i in range(40)], 1, 16, 8, 128),
    # verify steps
    "groups": ([(3000, [20] * 9)], 7, 16, 2, 128),
}


@pytest.mark.parametrize("cta", [0, 20])
@pytest.mark.parametrize("name", list(CASES))
def test_rows_of_a_wait_that_ran_out_are_nan(name, cta):
    sets, group, hq, hk, dim = CASES[name]
    d = Sets(40, sets, group, hq, hk, dim, 32, 32, "bf16", loose=2)
    h = d.handle()
    q, lens, max_len, table, scale, group, group_table = d.args()
    ws = torch.empty(B.kv8_attention_shared_workspace_bytes(q.shape[0], hq, hk, dim, group),
                     dtype=torch.uint8, device="cuda")

    def call(skip):
        out, lse, status = torch.zeros_like(q).contiguous(), torch.zeros(q.shape[:2], device="cuda"), I32([0])
        B.kv8_attention_shared(q, float(scale), lens, max_len, group, group_table, I32(d.starts), I32(d.prefix),
                               LARGE, table, d.page, d.block, h.k, h.v, h.k_scale, h.v_scale, out, lse, ws,
                               status, skip_cta=skip)
        return out, lse, int(status.item())

    out, lse, status = call(-1)
    assert status == 0 and not torch.isnan(out).any() and not torch.isnan(lse).any()
    o, l, status = call(cta)
    assert status == B.KV8_STATUS_TIMEOUT
    void = torch.isnan(l)
    assert void.any() and not void.all()
    assert torch.isnan(o[void]).all()
    assert torch.equal(o[~void], out[~void]) and torch.equal(l[~void], lse[~void])
    assert not void[lens == 0].any()
    first, last = d.starts[0] * group, d.starts[-1] * group
    assert not void[:first].any() and not void[last:].any()  # requests of no set
    o, l, status = call(-1)  # the workspace serves the next call
    assert status == 0 and torch.equal(o, out) and torch.equal(l, lse)
