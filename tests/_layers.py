"""References in 64 bits of the adapter layer and of the 8-bit checkpoints, from their
definitions, and the inputs and error bounds of their tests."""
import numpy as np
import torch

U32 = 2.0 ** -23     # a truncated fp32 addition or product is within this of its value
U16 = 2.0 ** -7      # bfloat16 keeps 8 bits: its spacing is up to this of the value, a rounding half of it


def device_matrix(x, pad=0, offset=0, fill=float("nan")):
    """x on the GPU as a view with `pad` more elements per row and its first element
    `offset` elements into the allocation; everything around it holds `fill`."""
    rows, cols = x.shape
    flat = torch.full((rows * (cols + pad) + offset + 8,), fill, dtype=torch.float64)
    view = flat[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    view.copy_(x.double())
    out = flat.to(x.dtype).cuda()
    return out[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]


def device_stack(x, pad=0, offset=0):
    count, rows, cols = x.shape
    m = device_matrix(x.reshape(count * rows, cols), pad, offset)
    return torch.as_strided(m, (count, rows, cols), (rows * (cols + pad), cols + pad, 1),
                            m.storage_offset())


def row_ids(M, L, mode, seed):
    """Adapter of each row: "runs" of rows of one request, "mixed" (row by row), one
    "single" adapter, "none", or "outside" (row by row, with ids past the stack)."""
    rng = np.random.default_rng(seed)
    if mode == "none" or L == 0:
        return torch.full((M,), -1, dtype=torch.int32)
    if mode == "single":
        return torch.full((M,), L - 1, dtype=torch.int32)
    if mode == "mixed":
        return torch.from_numpy(rng.integers(-1, L, M).astype(np.int32))
    if mode == "outside":
        return torch.from_numpy(rng.integers(-3, L + 4, M).astype(np.int32))
    cuts = np.sort(rng.integers(0, M + 1, 2 * L))
    ids = rng.integers(-1, L, 2 * L + 1).astype(np.int32)
    return torch.from_numpy(ids[np.searchsorted(cuts, np.arange(M), side="right")])


def rank_of(ranks, a, R):
    return R if ranks is None else min(max(int(ranks[a]), 0), R)


def rows_of(ids, L):
    return [(a, torch.nonzero(ids == a).flatten()) for a in range(L)]


def lora_reference(X, W, A, B, ids, scale, ranks, bias):
    """(Y, H) in 64 bits and the sums of magnitudes of Y's and H's terms."""
    X, W, A, B = (t.double() for t in (X, W, A, B))
    L, R = A.shape[0], A.shape[2]
    Y, mag = X @ W, X.abs() @ W.abs()
    H, hmag = torch.zeros(X.shape[0], R).double(), torch.zeros(X.shape[0], R).double()
    if bias is not None:
        Y, mag = Y + bias.double(), mag + bias.double().abs()
    for a, rows in rows_of(ids, L):
        r, f = rank_of(ranks, a, R), 1.0 if scale is None else float(scale[a])
        if len(rows) == 0 or r == 0:
            continue
        Aa, Ba = A[a, :, :r], B[a, :r]
        H[rows, :r] = X[rows] @ Aa
        hmag[rows, :r] = X[rows].abs() @ Aa.abs()
        Y[rows] += f * (H[rows, :r] @ Ba)
        mag[rows] += abs(f) * (hmag[rows, :r] @ Ba.abs())
    return Y, H, mag, hmag


def lora_backward_reference(dY, X, W, A, B, ids, H, scale, ranks):
    dY, X, W, A, B, H = (t.double() for t in (dY, X, W, A, B, H))
    L, R = A.shape[0], A.shape[2]
    dX, mag = dY @ W.t(), dY.abs() @ W.abs().t()
    dA, dB = torch.zeros_like(A), torch.zeros_like(B)
    amag, bmag = torch.zeros_like(A), torch.zeros_like(B)
    for a, rows in rows_of(ids, L):
        r, f = rank_of(ranks, a, R), 1.0 if scale is None else float(scale[a])
        if len(rows) == 0 or r == 0:
            continue
        Aa, Ba = A[a, :, :r], B[a, :r]
        G, gmag = f * (dY[rows] @ Ba.t()), abs(f) * (dY[rows].abs() @ Ba.abs().t())
        dX[rows] += G @ Aa.t()
        mag[rows] += gmag @ Aa.abs().t()
        dA[a, :, :r], amag[a, :, :r] = X[rows].t() @ G, X[rows].abs().t() @ gmag
        dB[a, :r] = f * (H[rows, :r].t() @ dY[rows])
        bmag[a, :r] = abs(f) * (H[rows, :r].abs().t() @ dY[rows].abs())
    return dX, dA, dB, mag, amag, bmag


def assert_close(got, ref, mag, terms, what, norm=True):
    """|got - ref| within the rounding of a sum of `terms` products in fp32: each of the
    at most `terms` + 16 additions, products and splittings on the way is off by at most
    2^-23 of the sum of magnitudes `mag`, and a bfloat16 result by half a spacing more.
    Over a whole matrix of many terms the errors do not all lie on one side: its norm is
    held to 4e-6 (sums over up to 32 steps that truncate, 2^-23 each, then fp32), or to
    2^-8.5 for bfloat16 (the rms of a rounding is under half a spacing).  What is not
    finite in the reference has to be non-finite here, and nothing else may be."""
    bf = got.dtype == torch.bfloat16
    got, ref = got.detach().cpu().double(), ref.double()
    fine = torch.isfinite(ref) & torch.isfinite(mag)
    bad = torch.isfinite(got) != fine
    assert not bad.any(), f"{what}: {int(bad.sum())} values finite on one side only"
    err = torch.where(fine, (got - ref).abs(), 0.0)
    bound = (terms + 16) * U32 * torch.where(fine, mag, 0.0)
    if bf:
        bound = bound + 0.5 * U16 * (torch.where(fine, ref.abs(), 0.0) + bound) + 1e-38
    over = err > bound
    if over.any():
        at = tuple(int(v) for v in torch.nonzero(over)[0])
        raise AssertionError(f"{what}: {int(over.sum())} of {got.numel()} outside the bound, first "
                             f"{at}: got {float(got[at])!r}, reference {float(ref[at])!r}, "
                             f"bound {float(bound[at]):.3e}")
    if norm and fine.all() and float(ref.norm()) > 0 and ref.numel() >= 256:
        rel = float(err.norm() / ref.norm())
        # cancellation: relative to the terms where the sum is much smaller than they are
        slack = max(1.0, float(mag.norm() / ref.norm()) / (4.0 * max(terms, 1) ** 0.5))
        assert rel <= (2.0 ** -8.5 if bf else 4e-6) * slack, f"{what}: relative error {rel:.3e}"


def quantise(x):
    """(q, e) of the 8-bit form in 64 bits, by its definition: the least exponent is
    found by trying them."""
    x = x.double().numpy()
    M, K = x.shape
    blocks = -(-K // 32)
    q, e = np.zeros((M, K), np.int8), np.zeros((M, blocks), np.int8)
    for i in range(M):
        for b in range(blocks):
            v = x[i, 32 * b:32 * b + 32]
            if not np.isfinite(v).all():
                e[i, b] = -128
                continue
            t, p = np.abs(v).max(initial=0.0), -126
            while p < 121 and t > 127.0 * 2.0 ** p:
                p += 1
            e[i, b] = p
            q[i, 32 * b:32 * b + 32] = np.clip(np.rint(v / 2.0 ** p), -127, 127)
    return torch.from_numpy(q), torch.from_numpy(e)


def values(q, e):
    """What a checkpoint stands for, in 64 bits."""
    step = torch.where(e == -128, float("nan"), torch.pow(torch.tensor(2.0).double(), e.double()))
    return q.double() * step.repeat_interleave(32, dim=1)[:, :q.shape[1]]
