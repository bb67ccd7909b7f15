"""References in 64 bits of the norm, the 8-bit product and the gated block, from their definitions,
and the error bounds of their tests."""
import math

import torch

EPS = 1e-6
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}   # a rounding to the type is within this of its value


def rounded(got, ref, slack, what):
    """|got - ref| within one rounding to got's type and `slack` (of fp32 arithmetic) more.  What is not
    finite in the reference is so here, the same infinity or a NaN, and nothing else is."""
    got, ref = got.detach().cpu(), ref.double()
    h, got = HALF[got.dtype], got.double()
    fine = torch.isfinite(ref)
    assert bool((torch.isfinite(got) == fine).all()), f"{what}: finite on one side only"
    assert bool((torch.isnan(got) == torch.isnan(ref)).all()), f"{what}: NaN on one side only"
    inf = torch.isinf(ref)
    assert bool((got[inf] == ref[inf]).all()), f"{what}: other infinities"
    err = torch.where(fine, (got - ref).abs(), 0.0)
    bound = torch.where(fine, h * ref.abs() + (1 + h) * torch.as_tensor(slack).double() + 1e-44, 0.0)
    over = err > bound
    if bool(over.any()):
        at = tuple(int(v) for v in torch.nonzero(over)[0])
        raise AssertionError(f"{what}: {int(over.sum())} of {got.numel()} outside the bound, first {at}: got "
                             f"{float(got[at])!r}, reference {float(ref[at])!r}, bound {float(bound[at]):.3e}")


# ------------------------------------------------------------------ norm
def stream_of(X, R):
    """V, in the tensors' type: one fp32 addition, rounded."""
    return X if R is None else (X.float() + R.float()).to(X.dtype)


def rstd_of(V, eps):
    V = V.double()
    return 1.0 / torch.sqrt((V * V).sum(1, keepdim=True) / max(1, V.shape[1]) + eps)


def norm_reference(V, w, eps):
    return V.double() * rstd_of(V, eps) * w.double()


def rows8_reference(p):
    """(q, scale, finite) of the rows of p in 64 bits: q = rint(127 p / max|p|)."""
    p = p.double()
    top = p.abs().amax(1) if p.shape[1] else torch.zeros(p.shape[0]).double()
    fine = torch.isfinite(p).all(1)
    keep = fine & (top > 0)
    q = torch.where(keep.unsqueeze(1), torch.round(127.0 * p / torch.where(keep, top, 1.0).unsqueeze(1)), 0.0)
    return q.to(torch.int8), torch.where(fine, top / 127.0, float("nan"))


def norm_slack(V, y):
    """Of y in fp32: the sum of squares of K positive terms, added up in runs and a tree, is off by at most
    (K / 32 + 40) 2^-24 of itself (a thread adds up to 32 terms of a segment of a row, one segment in 16384
    columns, then 5 + 32 more), rstd by half of that and 4 roundings (mean, eps, root, reciprocal), y by two more."""
    return (0.5 * (V.shape[1] / 512 + 32 + 40) + 6) * 2.0 ** -24 * y.abs()


def norm_backward_reference(dY, V, w, dS, eps):
    """(dX, dw) in 64 bits and the magnitudes that their fp32 errors go by."""
    dY, V, w = dY.double(), V.double(), w.double()
    K, rstd = V.shape[1], rstd_of(V, eps)
    n, g = V * rstd, dY * w
    mean, mag = (g * n).sum(1, keepdim=True) / K, (g * n).abs().sum(1, keepdim=True) / K
    dX = rstd * (g - n * mean)
    dmag = rstd * (g.abs() + n.abs() * mag)
    if dS is not None:
        dX, dmag = dX + dS.double(), dmag + dS.double().abs()
    return dX, (dY * n).sum(0), dmag, (dY * n).abs().sum(0)


# ------------------------------------------------------------------ 8-bit product
def linear8_reference(q, scale, W, wscale, bias):
    """(y, magnitude) in 64 bits; the integer sums are exact there too."""
    v = (q.double() @ W.double()) * scale.double().unsqueeze(1) * wscale.double()
    mag = v.abs()
    return (v, mag) if bias is None else (v + bias.double(), mag + bias.double().abs())


# ------------------------------------------------------------------ gated block
def act_reference(z, act):
    """(act, act') in 64 bits."""
    z = z.double()
    if act == "none":
        return z, torch.where(z == z, 1.0, z)
    if act == "relu":
        return torch.where(z < 0, 0.0, z), torch.where(z > 0, 1.0, torch.where(z <= 0, 0.0, z))
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return z * s, s + z * s * (1 / (1 + torch.exp(z)))
    cdf = 0.5 * torch.erfc(-z / math.sqrt(2.0))
    return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)


def act_slack(z, act):
    """What fp32 makes of (act(z), act'(z)): SILU by an exponential (2 units in the last place of float32; by an
    argument rounded at |z| in bfloat16), a quotient and products; GELU by a tail whose error is up to 1.5e-7 for
    bfloat16, and the bell of the derivative by an exponential of z^2 / 2 as the checkpoints' gradient."""
    z = z.double()
    value, slope = act_reference(z, act)
    if act in ("none", "relu"):
        return torch.zeros_like(z), torch.zeros_like(z)
    if act == "silu":
        rel = (z.abs() + 16) * 2.0 ** -23
        return rel * value.abs(), rel * (1 + value.abs())
    return 2e-7 * z.abs() + 16 * 2.0 ** -24 * value.abs(), 3e-7 * (1 + z.abs()) + 16 * 2.0 ** -24 * slope.abs()


def gated_reference(X, Wg, Wu, act):
    """(H, G, U) in 64 bits and the fp32 errors that they may have: sums of K products, each of whose additions,
    products and splittings is off by at most 2^-23 of the sum of magnitudes; H by those of G and U, the
    slope of an activation being at most 1.13."""
    X, Wg, Wu = X.double(), Wg.double(), Wu.double()
    G, U = X @ Wg, X @ Wu
    unit = (X.shape[1] + 16) * 2.0 ** -23
    dg, du = unit * (X.abs() @ Wg.abs()), unit * (X.abs() @ Wu.abs())
    value, _ = act_reference(G, act)
    slack = 1.13 * dg * (U.abs() + du) + value.abs() * du + act_slack(G, act)[0] * U.abs() + 2.0 ** -23 * (value * U).abs()
    return value * U, G, U, slack, dg, du


def gated_backward_reference(dH, X, Wg, Wu, G, U, act):
    """(dX, dWg, dWu) in 64 bits and the errors that they may have: those of dG and dU (in bfloat16 a rounding, 2^-8 of
    the value at most, more than all fp32 ones) through sums of magnitudes, and the sums' own."""
    half = 2.0 ** -8 if dH.dtype == torch.bfloat16 else 2.0 ** -23
    dH, X, Wg, Wu, G, U = (t.double() for t in (dH, X, Wg, Wu, G, U))
    (value, slope), (vs, ss) = act_reference(G, act), act_slack(G, act)
    dG, dU = dH * U * slope, dH * value
    eg = (half + 2.0 ** -22) * dG.abs() + ss * (dH * U).abs()
    eu = (half + 2.0 ** -22) * dU.abs() + vs * dH.abs()
    un, um = (2 * G.shape[1] + 32) * 2.0 ** -23, (G.shape[0] + 16) * 2.0 ** -23
    dX = dG @ Wg.t() + dU @ Wu.t()
    sX = (eg + un * dG.abs()) @ Wg.abs().t() + (eu + un * dU.abs()) @ Wu.abs().t()
    sg, su = X.abs().t() @ (eg + um * dG.abs()), X.abs().t() @ (eu + um * dU.abs())
    return dX, X.t() @ dG, X.t() @ dU, sX, sg, su


def norm_close(got, ref, what, least=256):
    """The 2-norm of the difference: the errors of many terms do not all lie on one side.  float32 2e-6 (sums of up to
    512 terms that truncate, 2^-23 each, then fp32); bfloat16 the rms of two roundings, of the terms and of
    the result, each at most 2^-8 / sqrt 3."""
    if ref.numel() < least or float(ref.norm()) == 0:
        return
    rel = float((got.detach().cpu().double() - ref.cpu()).norm() / ref.norm())
    assert rel <= (2.0 ** -8 * math.sqrt(2 / 3) if got.dtype == torch.bfloat16 else 2e-6), f"{what}: relative error {rel:.3e}"
