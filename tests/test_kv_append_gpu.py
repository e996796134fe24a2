"""Appending cache rows with the position rotation against its 64-bit form."""
import math

import pytest
import torch

import mla_tree_verify_gb300 as mtv
from q8_util import LATENT, ROPE, ROW, Batch, values

pytestmark = pytest.mark.gpu


def table(n=4096):
    f = 10000.0 ** (-torch.arange(0, ROPE, 2, dtype=torch.float64) / ROPE)
    a = torch.arange(n, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float().cuda()


def rot(x, cs, interleaved):
    """x [..., 64] float64, cs [..., 64]."""
    c, s = cs[..., :32], cs[..., 32:]
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :32], x[..., 32:])
    y, z = a * c - b * s, b * c + a * s
    return torch.stack([y, z], -1).flatten(-2) if interleaved else torch.cat([y, z], -1)


class Case:
    def __init__(self, n, heads, e4m3=True, block=1, inter=True, seed=0, pool=None, mul=1.0, wide=ROW):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.n, self.heads, self.e4m3, self.block, self.inter = n, heads, e4m3, block, inter
        pool = pool or n + 20
        proj = (torch.randn((n, wide), generator=g, device="cuda") * mul).to(torch.bfloat16)
        self.latent, self.k_pe = proj[:, :LATENT], proj[:, wide - ROPE:]
        self.slots = torch.randperm(pool, generator=g, device="cuda")[:n]
        self.pos = torch.randint(0, 4096, (n,), generator=g, device="cuda")
        self.cs = table()
        self.scales = None
        if e4m3:
            self.kv = torch.randint(0, 127, (pool, ROW), generator=g, device="cuda", dtype=torch.uint8)
            self.scales = torch.rand(-(-pool // block), generator=g, device="cuda") * 0.01 * mul + 0.004 * mul
        else:
            self.kv = torch.randn((pool, ROW), generator=g, device="cuda").to(torch.bfloat16)
        self.q_pe = self.q = None
        if heads:
            self.q_pe = torch.randn((n, heads, 192), generator=g, device="cuda").to(torch.bfloat16)[..., 128:]
            self.q = torch.randn((n, heads, ROW), generator=g, device="cuda").to(torch.bfloat16)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(self, given=None, stream=None):
        self.before = (self.kv.clone(), None if self.scales is None else self.scales.clone(),
                       None if self.q is None else self.q.clone())
        given = self.block > 1 if given is None else given
        mtv.kv_append(self.latent, self.k_pe, self.pos, self.cs, self.slots, self.kv, self.status,
                      scales=self.scales, scale_block=self.block, given_scales=given,
                      q_pe=self.q_pe, q_out=None if self.q is None else self.q[..., LATENT:],
                      interleaved=self.inter, stream=stream)
        torch.cuda.synchronize()
        return given

    def check(self, given, skip=()):
        """fp32 products and sums of the rotation are allowed 2^-22 of |a| + |b|; then one
        rounding: bf16 2^-8, e4m3 2^-4 of the value or half the smallest step, 2^-10; a computed
        scale 2^-22."""
        live = torch.ones(self.n, dtype=torch.bool, device="cuda")
        for i in skip:
            live[i] = False
        at, cs = self.slots[live], self.cs[self.pos.clamp(0, 4095)[live]].double()
        pe = self.k_pe[live].double()
        row = torch.cat([self.latent[live].double(), rot(pe, cs, self.inter)], 1)
        slack = torch.zeros_like(row)
        slack[:, LATENT:] = 2.0 ** -22 * 2 * pe.abs().amax(1, keepdim=True)
        kv0, sc0, q0 = self.before
        if not self.e4m3:
            err = (self.kv[at].double() - row).abs()
            assert bool((err <= 2.0 ** -8 * row.abs() + slack).all())
        else:
            g = self.scales.double()[at // self.block]
            if not given:
                amax = row.abs().amax(1)
                want = torch.where(amax > 0, (amax / 448).clamp(min=2.0 ** -40), 1.0)
                assert bool(((g - want).abs() <= 2.0 ** -22 * want + 2.0 ** -22 * slack.amax(1)).all())
            x = (row / g[:, None]).clamp(-448, 448)
            err = (values(self.kv[at]) - x).abs()
            assert bool((err <= 2.0 ** -4 * x.abs() + 2.0 ** -10 + slack / g[:, None]).all())
            if given:
                assert torch.equal(self.scales, sc0)
            else:
                keep = torch.ones(self.scales.numel(), dtype=torch.bool, device="cuda")
                keep[at] = False
                assert torch.equal(self.scales[keep], sc0[keep])
        keep = torch.ones(self.kv.shape[0], dtype=torch.bool, device="cuda")
        keep[at] = False
        assert torch.equal(self.kv[keep], kv0[keep])
        if self.q is not None:
            x = self.q_pe[live].double()
            want = rot(x, cs[:, None], self.inter)
            err = (self.q[live][..., LATENT:].double() - want).abs()
            assert bool((err <= 2.0 ** -8 * want.abs() + 2.0 ** -21 * x.abs().amax(-1, keepdim=True)).all())
            assert torch.equal(self.q[..., :LATENT], q0[..., :LATENT])
            assert torch.equal(self.q[~live], q0[~live])


@pytest.mark.parametrize("inter", [True, False])
@pytest.mark.parametrize("n,heads", [(1, 0), (1, 64), (3, 1), (7, 5), (64, 8), (130, 17), (333, 128), (2000, 64)])
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "given"])
def test_rows(n, heads, kind, inter):
    c = Case(n, heads, kind != "bf16", 64 if kind == "given" else 1, inter, seed=n + heads)
    c.check(c.run())
    assert int(c.status) == 0


def test_wider_projection_and_separate_strides():
    c = Case(50, 8, seed=2, wide=2112)      # k_pe far from the latent
    c.check(c.run())
    c = Case(50, 8, seed=3)
    c.k_pe = torch.cat([c.k_pe.reshape(-1).new_zeros(1), c.k_pe.reshape(-1)])[1:].view(50, 64)  # 2-byte aligned
    c.q_pe = c.q_pe.transpose(0, 1).contiguous().transpose(0, 1)                                 # heads outermost
    c.check(c.run())
    assert int(c.status) == 0


def test_one_token_with_meaningless_strides_and_expanded_views():
    c = Case(1, 1, seed=3)
    c.latent = c.latent.t().contiguous().t()           # [1, 512] with stride (1, 1)
    c.q_pe = c.q_pe.as_strided((1, 1, 64), (3, 5, 1))
    c.check(c.run())
    c = Case(9, 4, seed=4)
    c.latent = c.latent[:1].expand(9, 512)             # the same latent for every token
    c.check(c.run())
    with pytest.raises(mtv.MlaTreeVerifyError, match="expanded"):
        mtv.kv_append(c.latent, c.k_pe, c.pos, c.cs, c.slots, c.kv, c.status, scales=c.scales,
                      q_pe=c.q_pe, q_out=c.q[:, :1, LATENT:].expand(9, 4, 64))


def test_given_scales_for_every_row():
    c = Case(90, 0, block=1, seed=4)
    c.check(c.run(given=True))


@pytest.mark.parametrize("mul", [2.0 ** -60, 2.0 ** -30, 1e-4, 1e4, 2.0 ** 44])
def test_magnitudes(mul):
    c = Case(40, 0, mul=mul, seed=5)
    c.latent[3] = 0
    c.k_pe[3] = 0
    c.latent[4, 1:] = 0
    c.run()
    c.check(False)
    assert int(c.status) == 0 and float(c.scales[c.slots[3]]) == 1.0


def test_padding_and_bad_tokens_are_skipped():
    c = Case(40, 8, seed=6)
    c.slots[2] = c.slots[39] = -1
    given = c.run()
    c.check(given, skip=[2, 39])
    assert int(c.status) == 0
    c = Case(40, 8, seed=7)
    c.slots[5], c.slots[6], c.pos[8], c.pos[9] = -2, c.kv.shape[0], -1, 4096
    given = c.run()
    c.check(given, skip=[5, 6, 8, 9])
    assert int(c.status) == mtv.APPEND_BAD_SLOT | mtv.APPEND_BAD_POS


def test_bad_given_scales_are_skipped():
    c = Case(300, 0, block=16, seed=8)
    bad = [0.0, math.nan, 2.0 ** -41, math.inf, -1.0]
    blocks = c.slots[:5] // 16
    for i, v in enumerate(bad):
        c.scales[blocks[i]] = v
    hit = torch.isin(c.slots // 16, blocks).nonzero()[:, 0].tolist()
    before = c.scales.clone()
    c.run()
    c.before = (c.before[0], c.scales.clone(), None)   # (NaN is not equal to itself)
    assert torch.equal(before.nan_to_num(5), c.scales.nan_to_num(5))
    c.scales = c.scales.nan_to_num(1.0)
    c.before = (c.before[0], c.scales.clone(), None)
    c.check(True, skip=hit)
    assert int(c.status) == mtv.APPEND_BAD_SCALE


@pytest.mark.parametrize("heads", [1, 8, 64])
@pytest.mark.parametrize("inter", [True, False])
def test_queries_of_tokens_with_bad_given_scales_are_left_alone(heads, inter):
    c = Case(100, heads, block=16, inter=inter, seed=15)
    bad = (c.slots[3] // 16).item()
    c.scales[bad] = 2.0 ** 41
    c.run()
    c.check(True, skip=(c.slots // 16 == bad).nonzero()[:, 0].tolist())
    assert int(c.status) == mtv.APPEND_BAD_SCALE


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dim", [0, 511, 520])
def test_nonfinite_rows(value, dim):
    c = Case(10, 0, seed=9)
    (c.latent if dim < LATENT else c.k_pe)[4, dim if dim < LATENT else dim - LATENT] = value
    c.run()
    assert int(c.status) == mtv.APPEND_BAD_VALUE
    row = c.kv[c.slots[4]]
    assert bool(((row & 127) == 127).all()) and float(c.scales[c.slots[4]]) == 1.0
    others = [i for i in range(10) if i != 4]
    c.slots, c.pos, c.latent, c.k_pe, c.n = c.slots[others], c.pos[others], c.latent[others], c.k_pe[others], 9
    g = c.scales.double()[c.slots]
    x = c.latent.double() / g[:, None]
    assert bool(((values(c.kv[c.slots])[:, :LATENT] - x).abs() <= 2.0 ** -4 * x.abs() + 2.0 ** -10).all())


@pytest.mark.parametrize("heads", [0, 8, 64])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dim", [0, 1, 255, 256, 511, 512, 520, 575])
def test_nonfinite_rows_of_a_bf16_cache(value, dim, heads):
    """Flagged, and written as they are; the other rows and the queries as ever."""
    c = Case(10, heads, e4m3=False, seed=9)
    (c.latent if dim < LATENT else c.k_pe)[4, dim if dim < LATENT else dim - LATENT] = value
    c.run()
    assert int(c.status) == mtv.APPEND_BAD_VALUE
    row = c.kv[c.slots[4]]
    assert torch.equal(row[:LATENT].view(torch.int16), c.latent[4].view(torch.int16))
    assert bool(row[LATENT:].isfinite().all()) == (dim < LATENT)
    c.kv[c.slots[4]] = c.latent[4] = c.k_pe[4] = 0
    c.check(False)


def test_largest_values_of_a_bf16_cache_are_not_flagged():
    c = Case(5, 0, e4m3=False, seed=12)
    big = torch.finfo(torch.bfloat16).max
    c.latent[0], c.latent[1, ::2], c.k_pe[:] = big, -big, 0
    c.run()
    c.check(False)
    assert int(c.status) == 0
    c.k_pe[3] = big                # rotated by an angle whose cosine and sine add up to more than 1
    c.cs[c.pos[3]] = 0.75
    c.status.zero_()
    c.run()
    assert int(c.status) == mtv.APPEND_BAD_VALUE and bool(c.kv[c.slots[3], LATENT:].isinf().any())


@pytest.mark.parametrize("block", [1, 16])
@pytest.mark.parametrize("heads", [0, 64])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dim", [0, 300, 511, 512, 520, 575])
def test_nonfinite_rows_with_given_scales(value, dim, heads, block):
    """Flagged; what is not finite becomes a NaN code, so that attention that sees the row gives NaN,
    and the row's other values are stored as ever."""
    c = Case(10, heads, block=block, seed=13)
    (c.latent if dim < LATENT else c.k_pe)[4, dim if dim < LATENT else dim - LATENT] = value
    c.run(given=True)
    assert int(c.status) == mtv.APPEND_BAD_VALUE
    s = c.slots[4]
    nan = values(c.kv[s]).isnan()
    if dim < LATENT:
        want = torch.zeros(ROW, dtype=torch.bool, device="cuda")
        want[dim] = True
    else:       # the pair that holds it, both of whose values are sums with it
        want = torch.zeros(ROW, dtype=torch.bool, device="cuda")
        k = (dim - LATENT) // 2 * 2 + LATENT
        want[k:k + 2] = True
    assert torch.equal(nan, want)
    c.kv[s] = torch.where(nan, 0, c.kv[s])
    row = values(c.kv[s])
    x = torch.cat([c.latent[4].double(), rot(c.k_pe[4].double(), c.cs[c.pos[4]].double(), True)])
    x = (x / c.scales.double()[s // block]).clamp(-448, 448)
    near = (row - x).abs() <= 2.0 ** -4 * x.abs() + 2.0 ** -10 + 2.0 ** -20 / float(c.scales[s // block])
    assert bool(near[~want].all())
    c.kv[s] = c.latent[4] = c.k_pe[4] = 0
    c.check(True)


def test_large_values_with_given_scales_are_saturated_and_not_flagged():
    c = Case(6, 0, block=16, seed=14)
    c.latent[2] = torch.finfo(torch.bfloat16).max
    c.scales[:] = 2.0 ** -40
    c.run()
    c.check(True)
    assert int(c.status) == 0


def test_rotation_in_place_and_on_another_stream():
    c = Case(60, 16, seed=10)
    c.q[..., LATENT:].copy_(c.q_pe)
    keep = c.q[..., LATENT:].clone()
    c.q_pe = c.q[..., LATENT:]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    c.run(stream=s)
    c.q_pe = keep
    c.check(False)


def test_capture_and_replay():
    c = Case(33, 8, seed=11)
    c.run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mtv.kv_append(c.latent, c.k_pe, c.pos, c.cs, c.slots, c.kv, c.status, scales=c.scales,
                      q_pe=c.q_pe, q_out=c.q[..., LATENT:])
    c.latent.mul_(2)
    c.slots.copy_(c.slots.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    c.check(False)


def test_append_then_verify_then_gather():
    """The three operators as a server runs them: two requests' prompts are appended, then a
    draft chain of each with its queries rotated on the way; verify; defragment; verify again."""
    H, P, T = 64, [300, 77], [4, 4]
    b = Batch(P, T, H, seed=12)
    g = torch.Generator(device="cuda").manual_seed(3)
    cs, st = table(), torch.zeros(1, dtype=torch.int32, device="cuda")
    pos = torch.cat([torch.arange(p) for p in P] + [p + torch.arange(t) for p, t in zip(P, T)]).cuda()
    slots = torch.cat([b.kv_indices.long(), b.out_cache_loc])
    rows = torch.randn((slots.numel(), ROW), generator=g, device="cuda").to(torch.bfloat16)
    q_pe = torch.randn((8, H, ROPE), generator=g, device="cuda").to(torch.bfloat16)
    b.kv.fill_(0x7F)
    n = sum(P)
    mtv.kv_append(rows[:n, :LATENT], rows[:n, LATENT:], pos[:n], cs, slots[:n], b.kv, st, scales=b.scales)
    mtv.kv_append(rows[n:, :LATENT], rows[n:, LATENT:], pos[n:], cs, slots[n:], b.kv, st, scales=b.scales,
                  q_pe=q_pe, q_out=b.q[..., LATENT:])
    out, lse = b.run()
    b.check(out, lse)          # against the codes as stored
    # against attention over the unquantised rows: a code is off by 2^-4 of its value at most
    full = rows.double()
    full[:, LATENT:] = rot(full[:, LATENT:], cs[pos].double(), True)
    want = rot(q_pe.double(), cs[pos[n:]].double()[:, None], True)
    assert bool((b.q[..., LATENT:].double() - want).abs().max() <= 2.0 ** -8 * want.abs().max() + 1e-5)
    stored = values(b.kv[slots]) * b.scales.double()[slots][:, None]
    step = b.scales.double()[slots][:, None] * 2.0 ** -10
    assert bool(((stored - full).abs() <= 2.0 ** -4 * full.abs() + step + 1e-6).all())
    dst, dsc = torch.empty((n, ROW), dtype=torch.uint8, device="cuda"), torch.empty(n, device="cuda")
    new = torch.zeros_like(b.kv_indices)
    mtv.kv_gather_q8(b.kv, b.scales, b.kv_indices, b.kv_indptr, dst, dsc, b.kv.shape[0], new, st)
    b.kv, b.scales, b.kv_indices = torch.cat([b.kv, dst]), torch.cat([b.scales, dsc]), new
    o, l = b.run()
    assert torch.equal(o, out) and torch.equal(l, lse) and int(st) == 0


@pytest.mark.parametrize("inter", [True, False])
@pytest.mark.parametrize("heads", [0, 1, 2, 3, 6, 7, 8, 9, 16])
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "given"])
def test_few_heads_with_skipped_tokens_among_them(heads, kind, inter):
    """Several tokens share a warp here: ragged ends, padding and bad tokens between good ones."""
    for n in (1, 2, 5, 16, 33):
        c = Case(n, heads, kind != "bf16", 64 if kind == "given" else 1, inter, seed=100 * heads + n)
        skip = [i for i in (1, 4, 11, 31) if i < n]
        for i, bad in zip(skip, [(-1, None), (None, -1), (c.kv.shape[0], None), (None, 4096)]):
            if bad[0] is not None:
                c.slots[i] = bad[0]
            else:
                c.pos[i] = bad[1]
        c.check(c.run(), skip=skip)
        want = (mtv.APPEND_BAD_POS if n > 4 else 0) | (mtv.APPEND_BAD_SLOT if n > 11 else 0)
        assert int(c.status) == want


@pytest.mark.parametrize("heads", [3, 8])
def test_few_heads_rotated_in_place(heads):
    c = Case(37, heads, inter=False, seed=9)
    c.q_pe = c.q[..., LATENT:]
    x = c.q_pe.clone()
    given = c.run()
    c.q_pe = x
    c.check(given)
