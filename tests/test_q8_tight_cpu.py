"""The tolerances of q8_tight see faults of the size that matters, and the way the 8-bit verify
holds its weights is as exact as its comments say (restated here)."""
import pytest
import torch

import q8_tight
from q8_util import Batch


@pytest.fixture(scope="module")
def long_request():
    b = Batch([40000], [1], 8, seed=5, device="cpu")
    (_, out, lse, tol, _), = q8_tight.reference(b)
    return b, out, lse, tol


def test_the_exact_output_passes(long_request):
    b, out, lse, tol = long_request
    worst = q8_tight.check(b, out[None].to(torch.bfloat16), lse[None].float())
    assert worst <= 1


@pytest.mark.parametrize("tile", [0, 7, 100, 200, 311])
def test_a_tile_left_out_is_seen(long_request, tile):
    b, out, lse, tol = long_request
    keep = torch.ones(40001)
    keep[128 * tile:128 * (tile + 1)] = 0
    (_, wrong, _, _, _), = q8_tight.reference(b, keep=keep)
    with pytest.raises(AssertionError, match="tolerances"):
        q8_tight.check(b, wrong[None].to(torch.bfloat16), lse[None].float())


@pytest.mark.parametrize("factor", [0.0, 0.9, 0.97, 1.03])
def test_a_scaled_output_is_seen(long_request, factor):
    b, out, lse, tol = long_request
    with pytest.raises(AssertionError, match="tolerances"):
        q8_tight.check(b, factor * out[None], lse[None].float())


@pytest.mark.parametrize("order", range(-6, 12))
def test_weights_are_held_like_bf16(order):
    """From 2^-6 to 2^12: off by at most 2^-8, and 2^-11 by their f16."""
    g = torch.Generator().manual_seed(order + 50)
    P = torch.exp2(order + torch.rand(200000, generator=g, dtype=torch.float64))
    got = q8_tight.held(P, torch.arange(P.numel()))
    assert float(((got - P) / P).abs().max()) <= q8_tight.REGULAR


@pytest.mark.parametrize("order", range(-20, -6))
def test_small_weights_are_right_on_average(order):
    """Below: within a step of e5m2 (at most half of the weight's binary order, 2^-16 at the least)
    and half a step of f16, 2^-25; weights that are alike to the right mean, also over the keys
    of any period.  The offsets are bytes: a mean may be off by 2^-9 of a step, and six
    deviations (of half a step at most) of the mean of n random ones."""
    n = 1 << 17
    column = torch.arange(n)
    for k in range(8):
        P = torch.full((n,), 2.0 ** (order + k / 8 + 0.03), dtype=torch.float64)
        got = q8_tight.held(P, column)
        step = max(2.0 ** (order - 1), 2.0 ** -16)
        assert float((got - P).abs().max()) <= step + 2.0 ** -25
        for period in (1, 2, 3, 8, 64, 128, 233, 1000):
            for phase in (0, period // 2):
                part = got[phase::period]
                off = abs(float(part.mean()) - float(P[0]))
                assert off <= step * (2.0 ** -9 + 3.0 / part.numel() ** 0.5) + 2.0 ** -25


def test_no_weight_stays_none():
    P = torch.zeros(256, dtype=torch.float64)
    assert not q8_tight.held(P, torch.arange(256)).any()
