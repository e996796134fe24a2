"""The 8-bit verify at the ends of its settings."""
import pytest
import torch

import mla_tree_verify_gb300 as mtv
from q8_util import Batch, SM_SCALE

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("limit", [10 ** 9, (1 << 63) - 1, 1 << 63, (1 << 63) + 1, (1 << 64) - 1])
def test_long_wait_limits(limit):
    """Twice 2^63 ns, the limit in clocks, is 0 in 64 bits."""
    b = Batch([3000, 700], [16, 8], 64, seed=41)
    want = b.run()
    out, lse = b.out()
    mtv.mla_tree_verify_q8_debug_ex(b.q, b.kv, b.scales, b.kv_indices, b.kv_indptr, b.out_cache_loc, b.mask,
                                    b.mask_indptr, b.qo_indptr, SM_SCALE, out, lse, b.ws, 16, wait_limit_ns=limit)
    assert b.flags() == 0
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
