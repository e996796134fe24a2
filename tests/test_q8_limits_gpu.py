"""The 8-bit verify at the ends of its settings."""
import pytest
import torch

import mla_tree_verify_gb300 as mtv
from mla_tree_verify_gb300 import binding
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


@pytest.mark.parametrize("bs,max_q,heads,fits", [(4095, 4096, 64, True), (4096, 4096, 64, False),
                                                 (1 << 20, 4096, 64, False), (32767, 4096, 8, True),
                                                 (32768, 4096, 8, False), ((1 << 31) - 1, 4096, 64, False)])
def test_workspace_query_refuses_what_the_call_refuses(bs, max_q, heads, fits):
    lib = binding.load()
    size = lib.mla_tree_verify_q8_workspace_bytes(bs, max_q, heads)
    assert (size > 0) == fits
    if not fits:
        with pytest.raises(mtv.MlaTreeVerifyError):
            mtv.workspace_bytes_q8(bs, max_q, heads)
    # host checks alone: the workspace is too small (-5) where the shape is not refused (-3)
    a = dict(q=16, kv=16, sc=16, kvi=16, kvp=16, ocl=16, mask=16, mip=16, qop=16, scale=0.1, out=16, lse=16, ws=256,
             wsb=1, bs=bs, mq=max_q, heads=heads, slots=10, total_q=4, nkvi=3, mlen=28, block=1)
    assert lib.mla_tree_verify_q8(*a.values(), None) == (-5 if fits else -3)
