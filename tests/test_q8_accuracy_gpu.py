"""The 8-bit verify against 64 bits with the tolerances of q8_tight: what small weights multiply,
whatever its order, counts."""
import math

import pytest
import torch

import mla_tree_verify_gb300 as mtv
import q8_tight
from q8_util import Batch, LATENT, ROW, codes

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("P,T,heads", [([300, 7, 0], [4, 1, 9], 64), ([20011], [1], 64), ([30000], [1], 8),
                                       ([9000, 14000], [3, 1], 64), ([40000], [16], 8), ([1500] * 40, [2] * 40, 64)])
def test_random_batches_within_tight_tolerances(P, T, heads):
    b = Batch(P, T, heads, seed=31)
    out, lse = b.run()
    q8_tight.check(b, out, lse)
    assert b.flags() == 0


@pytest.mark.parametrize("scale", [0.02, 0.2, 0.5])
def test_flat_and_steep_scores(scale):
    b = Batch([30000, 700], [1, 2], 64, seed=32)
    out, lse = b.run(sm_scale=scale)
    q8_tight.check(b, out, lse, sm_scale=scale, alike=scale < 0.1)


def _dominant(n, gap, period_of, batch):
    """`batch` requests over the same n keys of scale 1: key 0's score is `gap` binary orders above
    the others', which are all the same; values are 1 for key 0 and +-1 with dim d's period for
    the others.  The softmax scale that makes it so, and the values [n + 1, 512]."""
    g = torch.Generator().manual_seed(n)
    rows = torch.zeros((n + 1, ROW))
    for d in range(2, LATENT):
        p = period_of(d)
        sign = torch.randint(0, 2, (p,), generator=g) * 2.0 - 1
        sign[0], sign[p // 2] = 1, -1
        rows[:, d] = sign[torch.arange(n + 1) % p]
    rows[0, :LATENT] = 1
    rows[0, 1] = 8
    b = Batch([n], [1], 64, block=1 << 30, seed=33)
    b.scales[:] = 1.0
    b.kv[torch.cat([b.kv_indices.long(), b.out_cache_loc])] = codes(rows).cuda()
    b.q.zero_()
    b.q[..., 1] = 1
    b.P, b.T = [n] * batch, [1] * batch
    b.kv_indices, b.out_cache_loc, b.q = b.kv_indices.repeat(batch), b.out_cache_loc.repeat(batch), b.q.repeat(batch, 1, 1)
    b.mask = torch.ones(batch * (n + 1), dtype=torch.uint8, device="cuda")
    at = torch.arange(batch + 1, device="cuda")
    b.kv_indptr, b.qo_indptr, b.mask_indptr = (at * n).to(torch.int32), at, at * (n + 1)
    return b, gap * math.log(2.0) / 8, rows[:, :LATENT].double().cuda()


@pytest.mark.parametrize("gap", [10.3, 11.3, 13.6, 15.2, 16.7])
@pytest.mark.parametrize("n", [2000, 8000, 32000])
def test_values_that_repeat_under_a_dominant_key(n, gap):
    """Weights 2^-gap of the largest, all alike, whose values repeat with periods 2, 8, 64 and 7,
    each request walked whole by one CTA.  Tolerance: q8_tight's, and that of the 16-bit path."""
    b, scale, v = _dominant(n, gap, lambda d: (2, 8, 64, 7)[d % 4], mtv.split_grid())
    out, lse = b.run(sm_scale=scale)
    head = mtv.plan_header(b.ws)
    assert head["merges_tmem"] == head["merges_ws"] == 0
    assert torch.equal(out, out[:1].expand_as(out)) and torch.equal(lse, lse[:1].expand_as(lse))
    w = torch.full((n + 1,), 2.0 ** -gap, dtype=torch.float64, device="cuda")
    w[0] = 1
    total = float(w.sum())
    want = (w @ v / total).expand(64, LATENT)
    assert float((lse[0].double() - (gap * math.log(2.0) + math.log(total))).abs().max()) <= 1e-4
    err = (out[0].double() - want).abs()
    assert float((err / (1e-2 * (1 + want.abs()))).max()) <= 1
    q8_tight.check(b, out, lse, rows=[0, len(b.P) - 1], sm_scale=scale, alike=True)


def test_scores_that_rise_under_the_reference():
    """Keys 3.9 binary orders above the first tile's largest: the weights reach the top of their
    range (2^12) without a new reference, then 0.2 more, which needs one."""
    b, scale, v = _dominant(1000, 6.0, lambda d: 5, 1)
    at = b.kv_indices.long()
    rows = torch.zeros((3, ROW), device="cuda")
    for i, up in enumerate((0.0, 3.9, 4.1)):
        rows[i, 1] = 8 + 8 * up / 6
        rows[i, 2 + i] = 3.0
    b.scales = b.scales.expand(b.kv.shape[0]).contiguous()
    b.block = 1
    for i, k in enumerate((0, 200, 700)):
        b.scales[at[k]] = float(rows[i, 1]) / 8
        rows[i, 2:] /= float(rows[i, 1]) / 8
        rows[i, 1] = 8
        b.kv[at[k]] = codes(rows[i])
    out, lse = b.run(sm_scale=scale)
    q8_tight.check(b, out, lse, sm_scale=scale, alike=True)


@pytest.mark.parametrize("heads", [64, 8])
@pytest.mark.parametrize("amplitude", [1.0, 1e-2, 1e-4, 1e-6])
@pytest.mark.parametrize("kind", ["zeros", "half", "rope"])
def test_rows_without_values_among_small_ones(kind, amplitude, heads):
    """A visible row whose latent codes are all zero and whose scale is 1 (what kv_append stores for
    a row of zeros; with rope values too) adds nothing to the output, and takes no precision
    from keys whose scales are far smaller."""
    b = Batch([301, 40], [3, 1], heads, seed=34)
    b.scales *= amplitude
    at = b.kv_indices.long()
    at = at[::2] if kind == "half" else at[[7, 150, 310]]
    b.kv[at] = 0
    b.scales[at] = 1.0
    b.kv[at[::2], :LATENT] = 0x80            # minus zero
    if kind == "rope":
        b.kv[at, LATENT:] = codes(4 * torch.randn((at.numel(), ROW - LATENT), device="cuda"))
    out, lse = b.run()
    q8_tight.check(b, out, lse)
    assert b.flags() == 0


@pytest.mark.parametrize("first", [True, False])
def test_a_row_without_values_that_outweighs_the_others(first):
    """Scores of -30 for the keys with values, 0 for the one without: outputs of about e^-30, and
    in the other order of tiles."""
    b = Batch([600], [2], 64, seed=35)
    at = torch.cat([b.kv_indices.long(), b.out_cache_loc])
    b.kv[at, 0] = 0x77                        # 240
    b.q[..., 0] = -1
    b.scales[:] = 1 / 240
    empty = at[3 if first else 500]
    b.kv[empty] = 0
    b.scales[empty] = 2.0 ** 20
    out, lse = b.run(sm_scale=30.0)
    q8_tight.check(b, out, lse, sm_scale=30.0)
    only = Batch([200], [1], 64, seed=36)     # nothing but rows without values
    at = torch.cat([only.kv_indices.long(), only.out_cache_loc])
    only.kv[at] = 0
    out, lse = only.run()
    assert not out.any() and float((lse - math.log(201)).abs().max()) < 1e-5


@pytest.mark.parametrize("heads", [64, 8])
@pytest.mark.parametrize("order", [6, 9, 12, 15])
def test_queries_with_one_large_value(order, heads):
    """A query value 2^order times the row's others, in a dim that no key uses: the others are exact
    down to 2^-9 of it, and within 2^-17 of it below."""
    b = Batch([500, 130], [2, 1], heads, seed=37)
    b.q[..., 5] = 2.0 ** order
    b.kv[torch.cat([b.kv_indices.long(), b.out_cache_loc]), 5] = 0
    out, lse = b.run()
    q8_tight.check(b, out, lse)


@pytest.mark.parametrize("seed", range(16))
def test_random_batches_of_every_kind_within_tight_tolerances(seed):
    """Steep and flat softmaxes, a first key that outweighs the rest (0 to 24 binary orders), scales over 12
    binary orders, rows without values, masks that are no trees."""
    g = torch.Generator().manual_seed(2000 + seed)
    ri = lambda lo, hi: int(torch.randint(lo, hi + 1, (1,), generator=g))
    top = [60, 700, 6000, 25000][seed % 4]
    n = ri(1, 5)
    P, T = [ri(1, top) for _ in range(n)], [ri(1, [3, 12][seed % 2]) for _ in range(n)]
    b = Batch(P, T, 64 if seed % 3 else 8, [1, 1, 64][ri(0, 2)], seed=60 + seed)
    b.mask &= (torch.rand(b.mask.shape, generator=g).cuda() < [1.1, 0.5][ri(0, 1)]).to(torch.uint8)
    b.scales *= torch.exp2(torch.randint(-6, 7, b.scales.shape, generator=g).float()).cuda()
    at = b.kv_indices.long()
    b.kv[at[torch.rand(at.shape, generator=g).cuda() < 0.05], :LATENT] = 0
    q_small = 2.0 ** -ri(0, 6)
    b.q *= q_small
    if ri(0, 2):
        first = b.kv_indptr[:-1].long()
        b.kv[at[first]] = 0
        b.kv[at[first], :LATENT] = torch.randint(0x30, 0x38, (n, LATENT), generator=g, dtype=torch.uint8).cuda()
        b.kv[at, 3] = 0
        b.kv[at[first], 3] = 0x70                       # 128
        b.scales[at[first] // b.block] = 0.01
        b.q[..., 3] = ri(0, 24) * math.log(2.0) / (1.28 / math.sqrt(192.0))
    out, lse = b.run()
    q8_tight.check(b, out, lse)
    assert b.flags() == 0
