"""Tolerances of the 8-bit verify that see what a rounding may do and no more, and a restatement
of how it holds its weights.

q8_util.Batch.reference() allows every key's weight a whole step of e4m3 in one direction, which on
long requests is as much as the output; here the errors of different keys' roundings are taken as
independent, and the bounds are those of weights held as e4m3 + e5m2.
"""
import math

import torch

from q8_util import LATENT, SM_SCALE, values

# Of a weight P from 2^-6 up: half a step of its finer 8-bit part, and of the f16 it is taken from.
REGULAR = 2.0 ** -8 + 2.0 ** -11
# A largest weight of at least 2^7 keeps weights to 13 binary orders below it from 2^-6 up.
SMALL = 2.0 ** -13
# Six times the root of the sum of squares of errors that are at most so large, independent and of
# mean 0, is passed with a probability of at most 2 e^-18 (Hoeffding).
SIGMAS = 6.0


def reference(b, rows=None, sm_scale=SM_SCALE, alike=False, keep=None):
    """Yields (row, out [H, 512], lse [H], tol_out, tol_lse) in float64 for the token rows of Batch
    b (all, or those in `rows`).  alike: weights may be alike, so that roundings to nearest may
    all go one way (those of small weights are random).  keep: False for key columns to leave
    out, all other things being as they are.

    With u = w g and M its maximum over the keys that hold any value: P is u up to a factor, and
    2^7 or more at M.  A weight is off by REGULAR of itself, or below SMALL M by at most 2^-2 of
    itself, or one step of e5m2 (2^-16 of P), at random.  Scores are exact products summed in
    fp32 (2^-20 of the sum of magnitudes) of queries held exactly down to 2^-9 of the row's largest
    value and within 2^-17 of that below; out is rounded to bf16; exponentials and sums in
    fp32 are allowed 2^-18."""
    kvp, qo, mp = (v.tolist() for v in (b.kv_indptr, b.qo_indptr, b.mask_indptr))
    pool = b.kv.shape[0]
    for i in range(len(kvp) - 1):
        P, T = kvp[i + 1] - kvp[i], qo[i + 1] - qo[i]
        slot = torch.cat([b.kv_indices[kvp[i]:kvp[i + 1]].long(), b.out_cache_loc[qo[i]:qo[i + 1]]])
        good = (slot >= 0) & (slot < pool)
        slot = slot.clamp(0, pool - 1)
        g = b.scales.double()[slot // b.block]
        good &= (g >= 2.0 ** -40) & (g <= 2.0 ** 40)
        code = values(b.kv[slot])
        vis = b.mask[mp[i]:mp[i + 1]].view(T, P + T) != 0
        vis[:, :P] = True
        for t in range(T):
            r = qo[i] + t
            if rows is not None and r not in rows:
                continue
            on = (vis[t] & good).nonzero()[:, 0]
            x, gx, q = code[on], g[on], b.q[r].double()
            s = (q @ x.T) * gx * sm_scale
            lse = torch.logsumexp(s, 1)
            w = (s - lse[:, None]).exp()
            v = x[:, :LATENT] * gx[:, None]
            if keep is None:
                out = w @ v
            else:
                out = (w * keep[on]) @ v
            top = q.abs().amax(1, keepdim=True)
            tiny = (q.abs() < top * 2.0 ** -9).double() * top * 2.0 ** -17
            eps = ((2.0 ** -20 * q.abs() + tiny) @ x.abs().T * gx * abs(sm_scale)).amax(1)
            u = w * gx
            M = torch.where(x[:, :LATENT].any(1), u, 0.0).amax(1)[:, None]
            small = u < SMALL * M
            wv = w @ v.abs()
            var = (w * w * torch.where(small, 2.0 ** -4, 0.0 if alike else REGULAR ** 2)) @ (v * v)
            var += 2.0 ** -46 * M * M * (small.double() @ x[:, :LATENT] ** 2)
            tol = 2.0 ** -8 * out.abs() + SIGMAS * var.sqrt() + (2.0 ** -18 + 2 * eps[:, None]) * wv
            if alike:
                tol += REGULAR * ((w * ~small) @ v.abs())
            yield r, out, lse, tol, eps + 2.0 ** -18 * (1 + lse.abs())


def check(b, out, lse, **kw):
    """The largest error of out and lse in tolerances; raises if it is over 1."""
    worst = 0.0
    for r, o, l, to, tl in reference(b, **kw):
        e = float(((out[r].double() - o).abs() / (to + 1e-300)).max())
        el = float(((lse[r].double() - l).abs() / tl).max())
        assert math.isfinite(e) and e <= 1, f"row {r}: output off by {e:.2f} tolerances"
        assert math.isfinite(el) and el <= 1, f"row {r}: lse off by {el:.2f} tolerances"
        worst = max(worst, e, el)
    return worst


def dither(column):
    """The random byte of a key column (int64 tensor), of the even columns of a weight pair."""
    x = (column * 0x9E3779B1) & 0xFFFFFFFF
    x ^= x >> 16
    x = (x * 0x9E3779B1) & 0xFFFFFFFF
    return x >> 24


def held(P, column):
    """Weights P (float64, at most 2^12) as the kernel holds them, restated: an e4m3 and an e5m2 value."""
    y = P.to(torch.float16)
    bits = y.view(torch.int16).int()
    coarse = torch.where(y >= 1, (bits + 0x80) & 0xFF00, 0).to(torch.int16).view(torch.float16)
    hi = (y - coarse).float().clamp(-448, 448).to(torch.float8_e4m3fn).to(torch.float16)
    left = (y - hi).view(torch.int16).int() & 0xFFFF
    off = torch.where(y < 2.0 ** -6, dither(column).int(), 0x80)
    lo = ((left + off) & 0xFF00).to(torch.int16).view(torch.float16)
    return hi.double() + lo.double()
