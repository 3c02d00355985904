"""64-bit definitions of the RMSNorm and the gated feed-forward block, and the bounds their kernels are held to.

Rounding to bf16 is off by at most U = 2^-8 of the value; over many values its relative error is uniform-like with a
root mean square of at most U / sqrt(3).
"""
import math

import torch

U = 2.0 ** -8
RMS_U = U / math.sqrt(3.0)
F32 = 2.0 ** -24


# ------------------------------------------------------------------ RMSNorm

def norm_fwd(x, residual, weight, eps):
    h = x.double() if residual is None else x.double() + residual.double()
    rstd = 1.0 / torch.sqrt(h.pow(2).mean(-1) + eps)
    return h, rstd, h * rstd[:, None] * weight.double()


def norm_bwd(dy, h, weight, rstd, dh):
    xhat = h.double() * rstd.double()[:, None]
    g = dy.double() * weight.double()
    dx = rstd.double()[:, None] * (g - xhat * (g * xhat).mean(-1, keepdim=True))
    if dh is not None:
        dx = dx + dh.double()
    return dx, (dy.double() * xhat).sum(0)


# ------------------------------------------------------------------ MXFP8

def mx_scale_exp(amax):
    """floor(log2 amax) - 8, the exponent of a block's scale; -127 for a block of zeros."""
    m, e = torch.frexp(amax.double())
    return torch.where(amax > 0, (e - 1 - 8).clamp(-127, 127), torch.full_like(e, -127))


def e4m3(v):
    """Nearest e4m3 value (even on ties), saturated at 448, of 64-bit values."""
    a = v.abs().clamp_min(2.0 ** -6)
    step = torch.ldexp(torch.ones_like(a), torch.frexp(a)[1] - 4)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def mx_quant(v):
    """Values of the MXFP8 quantisation of 64-bit v in 1x32 blocks, and the scales' exponents."""
    b = v.double().reshape(v.shape[:-1] + (-1, 32))
    k = mx_scale_exp(b.abs().amax(-1))
    s = torch.ldexp(torch.ones_like(b[..., :1]), k[..., None])
    return (e4m3(b / s) * s).reshape(v.shape), k


def mx_values(codes, sf):
    """Values of codes (uint8) and scale bytes, in 64 bits."""
    q = codes.view(torch.float8_e4m3fn).float().double()
    s = torch.ldexp(torch.ones(sf.shape, dtype=torch.float64), sf.to(torch.int32) - 127)
    return (q.reshape(sf.shape + (32,)) * s[..., None]).reshape(codes.shape)


def check_mx(codes, sf, v, rel):
    """codes, sf must be the quantisation of values within `rel` of v: the scale that of a block maximum within rel
    of v's, every element between the roundings of v (1 - rel) and v (1 + rel) at the scale that was taken."""
    codes, sf, v = codes.cpu(), sf.cpu(), v.double().cpu()
    b = v.reshape(v.shape[:-1] + (-1, 32))
    amax = b.abs().amax(-1)
    k = sf.to(torch.int32) - 127
    assert bool(((k >= mx_scale_exp(amax * (1 - rel))) & (k <= mx_scale_exp(amax * (1 + rel)))).all())
    s = torch.ldexp(torch.ones_like(amax), k)[..., None]
    q = codes.view(torch.float8_e4m3fn).float().double().reshape(b.shape)
    lo, hi = e4m3(b * (1 - rel) / s), e4m3(b * (1 + rel) / s)
    lo, hi = torch.minimum(lo, hi), torch.maximum(lo, hi)
    assert bool(((q >= lo) & (q <= hi)).all())


# ------------------------------------------------------------------ gated feed-forward block

def ffn_fwd(x, W_g, W_u, W_d):
    g, u = x.double() @ W_g.double().T, x.double() @ W_u.double().T
    a = g * torch.sigmoid(g) * u
    return g, u, a, a @ W_d.double().T


def ffn_bwd(dy, x, W_g, W_u, W_d):
    g, u, a, _ = ffn_fwd(x, W_g, W_u, W_d)
    s = torch.sigmoid(g)
    v = dy.double() @ W_d.double()
    dg, du = v * u * s * (1 + g * (1 - s)), v * g * s
    return {"dX": dg @ W_g.double() + du @ W_u.double(), "dW_g": dg.T @ x.double(), "dW_u": du.T @ x.double(),
            "dW_d": dy.double().T @ a, "dg": dg, "du": du, "a": a}


def check_sum(got, ref, sigma, rel, K, jump=None):
    """A bf16 result of a K-term sum whose terms carry independent errors of root mean square `rel` (relative), with
    sigma = sqrt(sum of the terms' squares). Allowed: its own rounding; eight standard deviations of the terms' errors
    (an error is at most sqrt(3) rel of its term, so up to 21 terms this covers the worst case, sqrt(3 K) <= 8; with
    more, a sum of bounded independent errors passes 8 deviations with a probability below 2 exp(-32 / 3), and only if
    all its errors are at their bounds); and the fp32 additions, each off by at most 2^-23 (the tensor core truncates)
    of a partial sum of the order of sigma. jump(i, j), where given, is what one term's rare and larger error may add to
    the elements (i, j): one in 10^5 of them at most may need it."""
    got, ref, sigma = got.double().cpu(), ref.double().cpu(), sigma.double().cpu()
    assert got.shape == ref.shape
    tol = U * ref.abs() + (8 * rel + 2 * F32 * K) * sigma + 1e-30
    d = (got - ref).abs()
    assert bool(torch.isfinite(got).all())
    if jump is not None:
        i, j = (d > tol).nonzero(as_tuple=True)
        assert len(i) <= max(1, d.numel() // 10 ** 5)
        if len(i):
            tol[i, j] += jump(i, j).cpu()
    worst = float((d / tol).max())
    assert worst <= 1.0, f"off by {worst:.2f} of the tolerance at {int((d / tol).argmax())} of {d.numel()}"
    return worst
