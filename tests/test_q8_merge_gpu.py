"""Who merges a token's pieces in the 8-bit verify: the paths are taken one by one, and the output has
the same bits with all of them."""
import pytest
import torch

import mla_tree_verify_gb300 as mtv
import q8_tight
from q8_util import Batch, SM_SCALE

pytestmark = pytest.mark.gpu

BATCHES = {
    "one long request": lambda: Batch([40000], [16], 8, seed=51),
    "pieces by the dozen": lambda: Batch([30000], [1], 64, seed=52),
    "trees": lambda: Batch([6000, 900, 30], [8, 3, 1], 64, seed=53),
    "decoding": lambda: Batch([500 + 470 * i for i in range(40)], [1] * 40, 64, seed=54),
}


def _run(b, mode, limit):
    out, lse = b.out()
    if getattr(b, "ws", None) is None:
        b.ws = torch.empty(mtv.workspace_bytes_q8(len(b.P), b.max_q, b.heads), dtype=torch.uint8, device="cuda")
    mtv.mla_tree_verify_q8_debug_merge(b.q, b.kv, b.scales, b.kv_indices, b.kv_indptr, b.out_cache_loc, b.mask,
                                       b.mask_indptr, b.qo_indptr, SM_SCALE, out, lse, b.ws, b.max_q,
                                       scale_block=b.block, merge_mode=mode, help_limit_ns=limit)
    head = mtv.plan_header(b.ws)
    assert head["error_flags"] == 0
    return out, lse, head


@pytest.mark.parametrize("batch", BATCHES)
def test_same_bits_whoever_merges(batch):
    b = BATCHES[batch]()
    out, lse, head = _run(b, mtv.Q8_MERGE_ALONE, 0)
    q8_tight.check(b, out, lse)
    split = head["merges_ws"]
    assert split > 0 and head["merges_tmem"] == head["helps"] == head["helps_left"] == 0
    settings = [(mtv.Q8_MERGE_AUTO, 0), (mtv.Q8_MERGE_NO_TMEM, 0), (mtv.Q8_MERGE_ALONE, 0),
                (mtv.Q8_MERGE_AUTO, 1), (mtv.Q8_MERGE_AUTO, 10 ** 9), (mtv.Q8_MERGE_NO_TMEM, 10 ** 9)]
    settings += [(mtv.Q8_MERGE_NO_TMEM, limit) for limit in (1, 300, 1000, 2000, 4000, 8000)]   # give up at any moment
    for mode, limit in settings * 3:
        o, l, h = _run(b, mode, limit)
        what = f"mode {mode}, limit {limit}: {h}"
        assert torch.equal(o, out) and torch.equal(l, lse), what
        assert h["merges_tmem"] + h["merges_ws"] == split, what
        if mode != mtv.Q8_MERGE_AUTO:
            assert h["merges_tmem"] == 0, what
        if mode == mtv.Q8_MERGE_ALONE:
            assert h["helps"] == h["helps_left"] == 0, what
        if (mode, limit) == (mtv.Q8_MERGE_NO_TMEM, 1):
            assert h["helps_left"] > 0, what
        if (mode, limit) == (mtv.Q8_MERGE_NO_TMEM, 10 ** 9):
            assert h["helps"] > 0 and h["helps_left"] == 0, what


def test_merges_from_tmem_are_taken():
    """Many short requests, most pieces of which end while their CTAs have more to do."""
    b = Batch([1000 + 13 * i for i in range(200)], [1] * 200, 64, seed=55)
    out, lse, _ = _run(b, mtv.Q8_MERGE_ALONE, 0)
    taken = 0
    for _ in range(10):
        o, l, h = _run(b, mtv.Q8_MERGE_AUTO, 0)
        assert torch.equal(o, out) and torch.equal(l, lse)
        taken += h["merges_tmem"]
    assert taken > 0
