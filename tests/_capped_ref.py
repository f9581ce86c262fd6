"""Attention with a cap on its scores by its definition in 64 bits, and how far 32-bit
arithmetic may be from it when a cap costs a score no more than its own relative
accuracy, however large the cap is.

Tolerance (``_attention_ref``'s, with another term for the cap): cap * tanh(s / cap) is
at most min(|s|, cap), and is within 2^-20 of itself: below 0.6 caps a polynomial times s
(1.3e-7, and the roundings of s / cap, its square and the product, 4 of 2^-24, below
2^-21 together), above it 1 - 2 / (1 + e^2x) with 2^-22 for the exponential, x 2^-22 in its
argument and 2^-23 for the reciprocal: within 2.5e-7 where tanh is 0.537 or more."""
import math

import torch

import _attention_ref as ref


def capped64(q, k, v, cap, weights, causal=True, scale=None, coarse=None):
    """q [nq, heads, D], k, v [nk, kv_heads, D] -> (reference, tolerance before the output's rounding)."""
    nq, heads, d = q.shape
    nk, kv, _ = k.shape
    scale = d ** -0.5 if scale is None else scale
    want, tol = (torch.zeros(nq, heads, d, dtype=torch.float64, device=q.device) for _ in range(2))
    mask, _ = ref.seen(nq, nk, causal, 0, 0, q.device)
    for h in range(heads):
        kk, vv = k[:, h * kv // heads].double(), v[:, h * kv // heads].double()
        s = q[:, h].double() @ kk.t() * scale
        size = q[:, h].double().abs() @ kk.abs().t() * abs(scale)
        x = s / cap
        s = cap * torch.where(x.abs() < 1e-5, x, torch.tanh(x))   # (a third of x^3: 3e-11 of x)
        s = s.masked_fill(~mask, -math.inf)
        p = torch.exp(s - s.amax(1, keepdim=True))
        total = p.sum(1, keepdim=True)
        p = p / total
        want[:, h] = p @ vv
        a = p @ vv.abs()
        e = 1.05 * ((d / 16 + 4) * 2.0 ** -23 * size + 2.0 ** -20 * (size + size.clamp(max=cap)) + 2.0 ** -19)
        e = torch.where(mask, e, torch.zeros_like(e)).amax(1, keepdim=True)
        t = a * (2 * e + ref.HALF_STEP[weights] + (nk / 16 + 32) * 2.0 ** -22)
        if weights is torch.float16:
            largest = vv.abs().amax() if coarse is None else coarse
            t = t + 2.0 ** -25 * mask.sum(1, keepdim=True) * float(largest) / total
        tol[:, h] = t
    return want, tol
