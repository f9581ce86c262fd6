"""The token operators' definitions in 64 bits, and how far 32-bit arithmetic
may be from them.

Tolerances (u = 2^-24, the fp32 unit roundoff), derived from the operations:

* a row's sum of n squares: no term passes through more than n/32 + 32
  additions in any of the reductions (32 or more lanes a row, then a tree), so
  its relative error is below (n/32 + 32) u; the norm takes half of that
  through the square root, and a handful of further roundings follow: the
  relative error of v is below t = (n/32 + 64) u, for activations t = 2^-19
  (the exponential's and the complementary error function's few units, times
  their condition over the inputs used here).
* the scale is max|v| / qmax: within t.  A code is the nearest to v / scale:
  within half a step plus 2 t times the quotient.
* the product: every partial sum is below S = sum |x| |w|, and 16 products at
  a time join the sum with a truncation of at most 2^-23 of the running
  magnitude: (K/16 + 4) 2^-23 S; scales and bias add 4 roundings of values
  below |y| + |bias|.  The activations' slopes are below 1.13.
* a store rounds once, and rounding is monotonic: a result lies between the
  roundings of (reference - tolerance) and (reference + tolerance).
"""
import torch

QMAX = {torch.int8: 127.0, torch.float8_e4m3fn: 448.0}
def act64(v, act):
    if act == "relu":
        return v.clamp(min=0)
    if act == "silu":
        return v / (1 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * torch.special.erfc(-v / 2 ** 0.5)
    return v


def norm64(x, weight, eps, residual):
    h = x.double() if residual is None else x.double() + residual.double()
    v = h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps)
    return h, v if weight is None else v * weight.double()


def check_quant(v, codes, scale, t):
    """codes and scale against the exact rows v (64 bits, [..., width])."""
    qmax = QMAX[codes.dtype]
    amax = v.abs().amax(-1)
    s = torch.where(amax > 0, amax / qmax, torch.ones_like(amax))
    assert scale.dtype == torch.float32 and scale.shape == v.shape[:-1]
    assert codes.shape == v.shape
    bad = (scale.double() - s).abs() > t * s
    assert not bad.any(), (int(bad.sum()), scale[bad][:4], s[bad][:4])
    c = v / s[..., None]
    got = codes.double()
    if codes.dtype == torch.int8:
        half = torch.full_like(c, 0.5)
        assert int(codes.min()) >= -127
    else:
        _, e = torch.frexp(c.abs() * (1 + 2 * t))
        half = torch.ldexp(torch.ones_like(c), (e - 1).clamp(min=-6) - 4)
    bad = (got - c).abs() > half * (1 + 1e-9) + 2 * t * c.abs()
    assert not bad.any(), (int(bad.sum()), got[bad][:4], c[bad][:4])
    # the largest element of a row takes the largest code
    top = got.abs().amax(-1)
    assert torch.equal(top, torch.where(amax > 0, torch.full_like(top, qmax),
                                        torch.zeros_like(top)))


def check_rounded(got, ref, tol):
    """got is a value within tol of ref, rounded once to got's type (2^-23 |ref|
    more: the bounds here go to 16 bits through fp32)."""
    tol = tol + 2.0 ** -23 * ref.abs()
    lo, hi = (ref - tol).to(got.dtype).double(), (ref + tol).to(got.dtype).double()
    bad = ~((got.double() >= lo) & (got.double() <= hi))
    assert not bad.any(), (int(bad.sum()), got[bad][:4], ref[bad][:4])


def linear64(x, w, sx=None, sw=None, bias=None, act="none"):
    """(reference, tolerance before the output's rounding)."""
    xd, wd = x.double(), w.double()
    k = x.shape[-1]
    y, s = xd @ wd.t(), xd.abs() @ wd.abs().t()
    f = torch.ones_like(y)
    if sx is not None:
        f = f * sx.double()[..., None]
    if sw is not None:
        f = f * sw.double()
    y, s = y * f, s * f.abs()
    tol = (k / 16 + 4) * 2.0 ** -23 * s + 4 * 2.0 ** -24 * y.abs()
    if bias is not None:
        y = y + bias.double()
        tol = tol + 2.0 ** -24 * (y.abs() + bias.double().abs())
    return act64(y, act), 1.13 * tol, y


def check_linear(got, x, w, sx=None, sw=None, bias=None, act="none"):
    ref, tol, y = linear64(x, w, sx, sw, bias, act)
    assert got.shape == ref.shape
    if act in ("silu", "gelu"):
        if got.dtype == torch.float32:   # a few roundings, times the tail's condition
            tol = tol + ref.abs() * (4 + y * y) * 2.0 ** -22
        else:                            # the convolutions' epilogue forms: 1.5e-7 in erf,
            tol = tol + y.abs() * 2.0 ** -20 + ref.abs() * (2 + y.abs()) * 2.0 ** -21
    assert torch.isfinite(got.double()).all()
    check_rounded(got, ref, tol)
