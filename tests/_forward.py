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
