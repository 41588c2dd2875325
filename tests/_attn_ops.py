"""Plain float64 forms of the query/key rotation, the cache append and the cached decode, and their tolerances.

Written from the formulas, in numpy on the CPU.

Tolerances (derived, per element; u = 2^-24 is half a float32 step, h the half step of the stored type relative to
the value: 2^-24 f32, 2^-8 bf16, 2^-4 E4M3):

* rotated rows: |err| <= h |z| + 2^-19 (|y1| + |y2|), y1, y2 the pair before the rotation.  The angle's phase is
  cut to 32 bits and rounded to 24 (at most 2^-25 half turns = 2^-23.3 rad), sine and cosine are within 2^-23, the
  two products and the sum round three times (3 u each part), and the norm's factor is off by rsqrtf's 2 ulp
  (2^-22) plus half the relative error of a 256-term sum taken 16 at a time (20 u / 2) and two products (2 u):
  together below 2^-20 (|y1| + |y2|), doubled.
* dx with norm weights: |err| <= h |dx| + 2^-17 r (max|w g| + |xh| mean|w g xh| scale): see ``rope_bwd_tol``.
* weight gradients: sums of n terms t_i = g xh, added in float32 in chains below 2^10 and trees: |err| <= 2^-13
  sqrt(sum t^2) + 2^-18 max|t| would hold for random signs; the bound used is the certain one, 2^-19 * 2^3 sum|t|
  for the terms' own errors (2^-19 relative to their parts, as above) plus chain rounding (2^10 u) sum|t|.
* decode: see ``decode_tol``.
"""
import math

import numpy as np

HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "e4m3": 2.0 ** -4}


def inv_freq(rot, theta=10000.0):
    return np.array([theta ** (-2.0 * i / rot) for i in range(rot // 2)])


def rotate(h, pos, freq, rot, interleaved, sign=1.0):
    """h [rows, heads, d] float64, pos [rows]; rotation by sign * pos * freq."""
    out = h.copy()
    if rot == 0:
        return out
    # angles reduced in exact integer-free float64: |pos| < 2^31 and 53 bits leave 2^-22 rad at worst, so far
    # positions are reduced with extended precision first
    a = np.remainder(pos.astype(np.longdouble)[:, None] * freq.astype(np.longdouble)[None, :], 2 * PI_L)
    a = sign * a.astype(np.float64)
    c, s = np.cos(a)[:, None, :], np.sin(a)[:, None, :]
    i1 = np.arange(0, rot, 2) if interleaved else np.arange(rot // 2)
    i2 = i1 + (1 if interleaved else rot // 2)
    x, y = h[:, :, i1], h[:, :, i2]
    out[:, :, i1] = x * c - y * s
    out[:, :, i2] = y * c + x * s
    return out


PI_L = np.longdouble(math.pi) + np.longdouble(1.2246467991473532e-16)


def pair_mass(h, rot, interleaved):
    """|y1| + |y2| at both places of each pair (the value itself behind rot)."""
    m = np.abs(h)
    if rot == 0:
        return m
    i1 = np.arange(0, rot, 2) if interleaved else np.arange(rot // 2)
    i2 = i1 + (1 if interleaved else rot // 2)
    t = m[:, :, i1] + m[:, :, i2]
    m[:, :, i1] = t
    m[:, :, i2] = t
    return m


def norm(h, w, eps):
    if w is None:
        return h
    return h / np.sqrt(np.mean(h * h, -1, keepdims=True) + eps) * w


def rope(x, nq, nkv, d, pos, rot, interleaved, qw, kw, eps, kind):
    """(out, tolerance) [rows, (nq + nkv) d] of the forward rows stored as `kind`."""
    rows = x.shape[0]
    h = x[:, : (nq + nkv) * d].reshape(rows, nq + nkv, d)
    y = np.concatenate([norm(h[:, :nq], qw, eps), norm(h[:, nq:], kw, eps)], 1)
    z = rotate(y, pos, inv_freq(rot), rot, interleaved)
    tol = HALF[kind] * np.abs(z) + 2.0 ** -19 * pair_mass(y, rot, interleaved) + 1e-37
    return z.reshape(rows, -1), tol.reshape(rows, -1)


def rope_bwd(x, dout, nq, nkv, d, pos, rot, interleaved, qw, kw, eps, kind):
    """((dx, tol), (dqw, tol), (dkw, tol)); the weight entries None without the weight."""
    rows = dout.shape[0]
    dz = dout.reshape(rows, nq + nkv, d)
    g = rotate(dz, pos, inv_freq(rot), rot, interleaved, -1.0)
    gerr = 2.0 ** -19 * pair_mass(dz, rot, interleaved)
    dx, tol, dws = g.copy(), HALF[kind] * np.abs(g) + gerr + 1e-37, []
    for lo, n, w in ((0, nq, qw), (nq, nkv, kw)):
        if w is None:
            dws.append(None)
            continue
        sl = slice(lo, lo + n)
        h, gg, ge = x[:, : (nq + nkv) * d].reshape(rows, nq + nkv, d)[:, sl], g[:, sl], gerr[:, sl]
        r = 1.0 / np.sqrt(np.mean(h * h, -1, keepdims=True) + eps)
        xh = h * r
        m = np.mean(w * gg * xh, -1, keepdims=True)
        v = r * (w * gg - xh * m)
        # every factor is within 2^-19 of its size (the gradient within ge); the mean of d terms as well
        mass = np.abs(w) * ge + 2.0 ** -19 * np.abs(w * gg) + np.abs(xh) * np.mean(
            np.abs(w * xh) * ge + 2.0 ** -18 * np.abs(w * gg * xh), -1, keepdims=True)
        dx[:, sl] = v
        tol[:, sl] = HALF[kind] * np.abs(v) + 2.0 * r * mass + 1e-37
        t = gg * xh
        dws.append((t.sum((0, 1)), (np.abs(xh) * ge).sum((0, 1)) * 2 + (2.0 ** -18 + 2.0 ** -14) * np.abs(t).sum((0, 1)) + 1e-37))
    return (dx.reshape(rows, -1), tol.reshape(rows, -1)), dws[0], dws[1]


def decode(q, k, v, scale, kind):
    """One sequence: q [nq, d], k, v [tokens, nkv, d] (visible ones): out, its tolerance, lse, its tolerance.

    Tolerance of the output, per element: its own rounding 2^-8 |out|, plus an error of each probability and value:
    a score off by e = (d + 4) u sum|q k| scale (float32 accumulation) shifts a weight by e relative; the exponential
    instruction adds 2^-22, the score's scaling 2 u |s|, P's split into two bf16 values 2^-17 (f16 with E4M3: 2^-11,
    and 2^-25 of the largest weight below f16's normal range), the sums (tokens / 64 tiles of one lane, trees and up
    to 600 partials) 2^-14 at most for the lengths here; each applies to sum p |v|, twice (numerator, denominator)."""
    nq, d = q.shape
    nkv = k.shape[1]
    if k.shape[0] == 0:
        return np.zeros((nq, d)), np.zeros((nq, d)), np.full(nq, -np.inf), np.zeros(nq)
    qg = q.reshape(nkv, nq // nkv, d)
    s = np.einsum("ghd,tgd->ght", qg, k) * scale
    mass = np.einsum("ghd,tgd->ght", np.abs(qg), np.abs(k)) * abs(scale)
    e = ((d + 4) * 2.0 ** -24 * mass + 2.0 ** -23 * np.abs(s)).max(-1) + 2.0 ** -22
    top = s.max(-1, keepdims=True)
    p = np.exp(s - top)
    tot = p.sum(-1, keepdims=True)
    p /= tot
    out = np.einsum("ght,tgd->ghd", p, v)
    absout = np.einsum("ght,tgd->ghd", p, np.abs(v))
    rel = 2 * e + 2.0 ** -14 + (2.0 ** -17 if kind == "bf16" else 2.0 ** -11)
    tol = 2.0 ** -8 * np.abs(out) + rel[..., None] * absout
    if kind == "e4m3":  # weights below f16's normal range; q below 2^-14 of its largest value
        tol += 2.0 ** -24 * k.shape[0] / tot * np.abs(v).max(0)[:, None, :]
        tol += 2.0 ** -12 * absout
    lse = (top + np.log(tot))[..., 0]
    ltol = e + 2.0 ** -14 + 2.0 ** -22 * np.abs(lse) + (2.0 ** -12 if kind == "e4m3" else 0.0)
    return out.reshape(nq, d), tol.reshape(nq, d) + 1e-37, lse.reshape(nq), ltol.reshape(nq)


def within(name, got, want, tol):
    got = np.asarray(got, dtype=np.float64)
    assert got.shape == want.shape, (name, got.shape, want.shape)
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf]), f"{name}: infinities differ"
    assert np.isfinite(got[~inf]).all(), f"{name}: not finite"
    over = np.abs(got[~inf] - want[~inf]) - np.broadcast_to(tol, want.shape)[~inf]
    assert over.size == 0 or over.max() <= 0, (
        f"{name}: {int((over > 0).sum())} of {over.size} beyond the tolerance, worst by {over.max():.3g}")
