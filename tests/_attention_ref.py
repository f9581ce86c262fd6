"""Rotary positions, the key-value cache and attention by their definitions in 64
bits, and how far 32-bit arithmetic may be from them.

Tolerances (u = 2^-24, the fp32 unit roundoff), derived from the operations:

* rotary: the angle's fraction of a turn is rounded to fp32 (below pi u of angle) and
  its sine and cosine are within 2 ulp (4 u): below 2^-21 with the angle's part; the two
  products and the sum take 3 u of |a| + |b|: (2^-20 + |angle| 2^-51)(|a| + |b|), the
  last for the frequency's and the reference's own 53 bits.
* a score is a sum of D products: 16 at a time join with a truncation of at most 2^-23
  of the running magnitude, so within (D/16 + 4) 2^-23 S, S = scale * sum |q||k|; scales,
  the change to base 2, the cap's and the slope's steps add 16 roundings of values below
  S + |slope| distance (or below the cap), the approximate exponential and logarithm
  2^-20 in the exponent: a weight's relative error is below
      e = 1.05 ((D/16 + 4) 2^-23 S + 2^-20 (S + cap + |slope| distance) + 2^-19).
* the maximum that weights are taken relative to cancels. Weights are rounded to 16 bits
  for their product with the values: half a step, 2^-11 (fp16 weights) or 2^-8 (bf16),
  relative, and 2^-25 absolute for the fp16's subnormals, relative to the largest
  weight (times scale).
* with A = sum p|v| / sum p the result is within A (2 e + half a step + (n/16 + 32) 2^-22)
  (the numerator's and the sum's errors, one product's truncation and one rescaling for
  each 16 tokens), then rounded once.
"""
import math

import torch

from _token_ref import check_rounded

HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
QMAX = {torch.int8: 127.0, torch.float8_e4m3fn: 448.0}


def ladder64(sections, base=10000.0, ladder="axis", scales=None):
    """(axis of each pair, radians per position)"""
    axis = [a for a, s in enumerate(sections) for _ in range(s)]
    n = len(axis)
    freq = ([base ** (-i / s) for s in sections for i in range(s)] if ladder == "axis"
            else [base ** (-i / n) for i in range(n)])
    return axis, [f * (1 if scales is None else scales[a]) for f, a in zip(freq, axis)]


def rotary64(x, positions, axis, freq, interleaved=False, inverse=False):
    """(reference, tolerance before the output's rounding) of [tokens, heads, width]."""
    n = len(axis)
    angle = positions.reshape(x.shape[0], -1).double()[:, axis] * torch.tensor(
        freq, dtype=torch.float64, device=x.device)
    c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    if inverse:
        s = -s
    y, tol = x.double().clone(), torch.zeros_like(x, dtype=torch.float64)
    ia = torch.arange(n, device=x.device) * (2 if interleaved else 1)
    ib = ia + (1 if interleaved else n)
    a, b = x.double()[..., ia], x.double()[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    t = (2.0 ** -20 + angle.abs()[:, None] * 2.0 ** -51) * (a.abs() + b.abs())
    tol[..., ia] = tol[..., ib] = t
    return y, tol


def seen(nq, nk, causal, window, prefix, device):
    i = torch.arange(nk - nq, nk, device=device)[:, None]
    j = torch.arange(nk, device=device)[None]
    m = torch.ones(nq, nk, dtype=torch.bool, device=device)
    if window:
        m &= (i - j).abs() < window
    if causal:
        m &= j <= i
    return m | (j < prefix), (i - j).abs()


def attention64(q, k, v, causal=True, window=0, prefix=0, scale=None, cap=0.0, slopes=None,
                weights=None, coarse=None):
    """One sequence: q [nq, heads, D], k, v [nk, kv_heads, D] in 64 bits -> (reference,
    tolerance before the output's rounding) [nq, heads, D].  weights: the type the kernel
    rounds weights to; coarse: the largest scale of v's rows times its largest code."""
    nq, heads, d = q.shape
    nk, kv, _ = k.shape
    scale = d ** -0.5 if scale is None else scale
    out = torch.zeros(nq, heads, d, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    mask, far = seen(nq, nk, causal, window, prefix, q.device)
    for h in range(heads if nk else 0):
        kk, vv = k[:, h * kv // heads].double(), v[:, h * kv // heads].double()
        used = mask.any(0)
        kk = torch.where(used[:, None], kk, torch.zeros_like(kk))
        vv = torch.where(used[:, None], vv, torch.zeros_like(vv))
        s = q[:, h].double() @ kk.t() * scale
        size = (q[:, h].double().abs() @ kk.abs().t() * abs(scale))
        if cap:
            s = cap * torch.tanh(s / cap)
        bias = 0.0
        if slopes is not None:
            bias = float(slopes[h]) * far.double()
            s = s - bias
            bias = abs(bias)
        s = s.masked_fill(~mask, -math.inf)
        top = s.amax(1, keepdim=True)
        p = torch.exp(s - torch.where(top == -math.inf, torch.zeros_like(top), top))
        total = p.sum(1, keepdim=True)
        total = torch.where(total == 0, torch.ones_like(total), total)
        p = p / total
        out[:, h] = p @ vv
        a = p @ vv.abs()
        e = 1.05 * ((d / 16 + 4) * 2.0 ** -23 * size + 2.0 ** -20 * (size + cap + bias) + 2.0 ** -19)
        e = torch.where(mask, e, torch.zeros_like(e)).amax(1, keepdim=True)
        step = HALF_STEP[weights]
        t = a * (2 * e + step + (nk / 16 + 32) * 2.0 ** -22)
        if weights is torch.float16:   # subnormal weights, next to the largest (1 / total at most)
            largest = vv.abs().amax() if coarse is None else coarse
            t = t + 2.0 ** -25 * mask.sum(1, keepdim=True) * float(largest) / total
        tol[:, h] = t
    return out, tol


def check(got, ref, tol):
    assert got.shape == ref.shape
    check_rounded(got, ref, tol)
