"""Bounds of the 8-bit paged attention, row by row, for the tests beside it (no GPU needed here).

For one output element of a row, with p_j the weights, A = sum_j p_j |v_j|, R = the row's largest
scale * sum_d |q_d k_jd| times log2(e), and n the tokens cached for its request:
  - the output is rounded to its type once: half a step, 2^-8 (bf16) or 2^-24 (fp32) of the value;
  - a weight is kept in fp16, 2^-11 of itself (fp32: two fp16, 2^-22), down to 2^-14 (2^-26) of the row's largest weight
    times page scale; below that it is off by at most 2^-25 (2^-37) of that product P = max_j p_j 2^e_j, which
    the codes multiply: 2^-25 P sum_j |code_j|;
  - the products add up in fp32, each addition off by at most 2^-22 of what it holds (the tensor core truncates): at most
    n / 16 + 8 additions (fp32: twice the products, 2 n / 16 + 16), of A each;
  - a score: its products in fp32 over at most 16 additions, 2^-18 R; queries in two fp16 for fp32, 2^-22 R; its own
    steps and the base-2 exponential, 2^-21 R + 2 * 2^-22 R + 2^-21; it is kept with its page's value exponent, at most E in
    size, added, one rounding: 2^-24 (R + E).  A score that is off by d changes a weight by d ln2 of itself and the
    sum of weights likewise: 2 ln2 d A;
  - lse is the reference m, the largest score with its exponent less 12 at most, plus the logarithm of the sum: a score's
    error, and three roundings of numbers up to R + E + 12 (the score, m, their sum): 3 ln2 2^-24 (R + E + 12);
  - a cap: up to 256 as cap - 2 cap / (1 + e), e = 2^(2 log2(e) s / cap): the division is off by 2^-22 of up to twice the
    cap, the exponential's 2^-22 comes through e / (1 + e)^2 <= 1/4 of that, the sums beside them add 3 * 2^-24 of the
    cap: below 2^-20 cap log2(e).  Above 256 (fp32: always) as cap * tanh(s / cap), whose division, tanh and product are off
    by 2^-22, 2^-22 and 2^-24 of the score: below 2^-20 R, whatever the cap.
"""
import math

import numpy as np
import torch

from oracle import attn as A

F32 = torch.float32


def bounds(c, scale=0.0, cap=0.0, window=0, slopes=None, prefix=None, parents=None):
    """(out, lse, bound of out, bound of lse) of a case, from the 64-bit definition."""
    f32 = c.dtype == F32
    out, lse, spread, reach, faint = A.attend(c.np, c.q.double().numpy(), c.lens, c.kv, c.table, c.ps, scale, cap, window,
                                              slopes, prefix, parents, faint=True)
    n = np.repeat(np.maximum(c.kv, 1), c.lens).astype(np.float64)[:, None]
    R = reach * math.log2(math.e)
    E = float(np.abs(c.np["v_exp"].astype(int)).max())
    d = R * (2.0 ** -18 + 2.0 ** -21 + 3 * 2.0 ** -22) + 2.0 ** -21 + 2.0 ** -24 * (R + E)
    if cap:
        d = d + (R * 2.0 ** -20 if f32 or cap > 256.0 else cap * math.log2(math.e) * 2.0 ** -20)
    if slopes is not None:  # the bias is a product and a sum in fp32, of values up to n * slope
        d = d + 2.0 ** -23 * n * max(slopes) * math.log2(math.e)
    sums = (n / 16 + 8) * 2.0 ** -22 * (2 if f32 else 1)
    rel = (2.0 ** -22 if f32 else 2.0 ** -11) + 2 * math.log(2) * d + sums
    tol = (2.0 ** -24 if f32 else 2.0 ** -8) * np.abs(out) + spread * rel[..., None] \
        + faint * 2.0 ** (-37 if f32 else -25) + 1e-30
    some = np.isfinite(lse)
    ltol = np.where(some, math.log(2) * (d + 3 * 2.0 ** -24 * (R + E + 12)) + 2.0 ** -21 * (1 + np.abs(np.where(some, lse, 0.0))),
                    0.0)
    return out, lse, tol, ltol


def check_rows(c, got, **kw):
    """The outputs and lse of a call against the definition, each row within its own bound."""
    out, lse = (x.double().numpy() for x in got)
    ref, rlse, tol, ltol = bounds(c, **kw)
    assert np.isfinite(out).all()
    worst = float(np.max(np.abs(out - ref) / tol)) if out.size else 0.0
    assert worst <= 1.0, f"error {worst:.2f} of its bound"
    none = np.isneginf(rlse)
    assert np.array_equal(np.isneginf(lse), none) and not out[none].any()
    assert np.all(np.abs(lse[~none] - rlse[~none]) <= ltol[~none])


def extreme_case(make, lens, dtype, hq=4, hkv=2):
    """Exponents far apart, queries of 1e4 and of 1e-20, pages of zeros; make: the class of the cases.  Only request
    0 has the page of large values, so that request 1 shows what the other pages alone do."""
    c = make(lens, [200, 150], hq, hkv, 128, 16, dtype, seed=9, elo=-12, ehi=-4)
    c.np["v_exp"][c.table[0, 2]] = 20
    c.np["v_exp"][c.table[0, 3]] = -32
    c.np["v"][c.table[0, 3]] = 0
    c.np["k_exp"][c.table[1, 1]] = -30
    c.np["k"][c.table[1, 2]] = 0
    c.q[0, 0] *= 1e4
    c.q[0, 1] *= 1e-20
    c.q[-1, 2] = 0.0
    return c
