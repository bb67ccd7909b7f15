"""The root-mean-square norm, its 8-bit rows and its backward pass against 64 bits."""
import pytest
import torch

from _forward import (EPS, norm_backward_reference, norm_reference, norm_slack, rounded, rows8_reference, rstd_of,
                      stream_of)
from _layers import device_matrix

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16]


@pytest.fixture(scope="module", autouse=True)
def _gpu(cuda_device):
    yield


def binding():
    from dense_fp32_gemm_02_gb300 import binding
    return binding


def normal(rows, cols, dtype, seed, scale=1.0):
    g = torch.Generator()
    g.manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * scale
    x[:, torch.rand(cols, generator=g) < 0.01] *= 20.0
    return x.to(dtype)


def weight(K, dtype, seed=9):
    g = torch.Generator()
    g.manual_seed(seed)
    return (1.0 + 0.3 * torch.randn(K, generator=g)).to(dtype)


def check_rows8(q, scale, V, w, rstd, what):
    ref_q, _ = rows8_reference(V.double() * w.double())
    _, ref_scale = rows8_reference(V.double() * rstd * w.double())
    assert torch.equal(q.cpu(), ref_q), f"{what}: {int((q.cpu() != ref_q).sum())} of {q.numel()} q differ"
    # max|p| (1 rounding), times rstd (norm_slack's), over 127: two more
    rounded(scale, ref_scale, norm_slack(V, ref_scale) + 3 * 2.0 ** -24 * ref_scale.abs(), what + " scale")


SHAPES = [(1, 1), (1, 7), (3, 8), (5, 64), (2, 256), (9, 257), (70, 1000), (33, 1024), (4, 1032), (200, 2048),
          (155, 4096), (3, 4100), (301, 8192), (2, 8200), (5, 16384), (160, 9001), (2, 16392), (3, 40001)]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("M,K", SHAPES)
def test_forward(M, K, dtype):
    """Every output, alone and together, with and without a residual."""
    b = binding()
    X, R, w = normal(M, K, dtype, 1), normal(M, K, dtype, 2), weight(K, dtype)
    dX, dR, dw = X.cuda(), R.cuda(), w.cuda()
    for residual in (False, True):
        V = stream_of(X, R if residual else None)
        y = norm_reference(V, w, EPS)
        S, Y = torch.full_like(dX, 77), torch.full_like(dX, 77)
        q, scale = torch.full((M, K), 77, dtype=torch.int8, device="cuda"), torch.full((M,), 77.0, device="cuda")
        r = dR if residual else None
        out = b.rmsnorm_into(dX, dw, Y=Y, q=q, scale=scale, R=r, S=S)
        assert out[0] is S and out[1] is Y and out[2] is q and out[3] is scale
        assert torch.equal(S.cpu(), V)
        rounded(Y, y, norm_slack(V, y), "Y")
        check_rows8(q, scale, V, w, rstd_of(V, EPS), "together")
        Y2, q2, s2 = torch.empty_like(Y), torch.empty_like(q), torch.empty_like(scale)
        b.rmsnorm_into(dX, dw, Y=Y2, R=r)
        b.rmsnorm_into(dX, dw, q=q2, scale=s2, R=r)
        assert torch.equal(Y2, Y) and torch.equal(q2, q) and torch.equal(s2, scale)
    assert b.device_status() == 0


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("pad,offset", [(0, 1), (3, 0), (8, 8), (5, 3)])
@pytest.mark.parametrize("M,K", [(6, 64), (5, 1000), (7, 4096), (3, 16400)])
def test_views(M, K, pad, offset, dtype):
    """Any pitch and alignment; what lies between the rows is left as it was."""
    b = binding()
    X, R, w = normal(M, K, dtype, 3), normal(M, K, dtype, 4), weight(K, dtype)
    dX, dR = device_matrix(X, pad, offset), device_matrix(R, pad + 1, offset)
    V = stream_of(X, R)
    outs = {}
    for name, p in (("S", pad), ("Y", pad + 2)):
        flat = torch.full((M, K + p + 3), 5.0, dtype=dtype, device="cuda")
        outs[name] = (flat, flat[:, 1:1 + K])
    qflat = torch.full((M, K + pad), 55, dtype=torch.int8, device="cuda")
    wflat = torch.zeros(K + 3, dtype=dtype, device="cuda")
    wflat[1:1 + K] = w.cuda()
    scale = torch.empty(M, device="cuda")
    b.rmsnorm_into(dX, wflat[1:1 + K], Y=outs["Y"][1], q=qflat[:, :K], scale=scale, R=dR, S=outs["S"][1])
    y = norm_reference(V, w, EPS)
    assert torch.equal(outs["S"][1].cpu(), V)
    rounded(outs["Y"][1], y, norm_slack(V, y), "Y")
    check_rows8(qflat[:, :K], scale, V, w, rstd_of(V, EPS), "views")
    assert bool((qflat[:, K:] == 55).all())
    for flat, _ in outs.values():
        assert bool((flat[:, 0] == 5).all()) and bool((flat[:, 1 + K:] == 5).all())


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("M,K", [(4, 100), (3, 3000), (2, 33000)])
def test_in_place(M, K, dtype):
    b = binding()
    X, R, w = normal(M, K, dtype, 5).cuda(), normal(M, K, dtype, 6).cuda(), weight(K, dtype).cuda()

    def fresh():
        return (torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda"))
    S, Y, (q, scale) = torch.empty_like(X), torch.empty_like(X), fresh()
    b.rmsnorm_into(X, w, Y=Y, q=q, scale=scale, R=R, S=S)
    for s_of, y_of in (("X", None), ("R", None), (None, "X"), (None, "R"), ("X", "R"), ("R", "X")):
        x, r, (q2, s2) = X.clone(), R.clone(), fresh()
        s = {"X": x, "R": r, None: None}[s_of]
        y = {"X": x, "R": r, None: torch.empty_like(Y)}[y_of]
        b.rmsnorm_into(x, w, Y=y, q=q2, scale=s2, R=r, S=s)
        assert s is None or torch.equal(s, S)
        assert torch.equal(y, Y) and torch.equal(q2, q) and torch.equal(s2, scale)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("K", [40, 900, 5000, 20000])
def test_values_out_of_range(K, dtype):
    """Magnitudes whose squares or products leave fp32's range, zeros, infinities and NaNs: what the
    formulas give."""
    b = binding()
    base = normal(9, K, dtype, 7).float()
    X = torch.stack([base[0] * 1e30, base[1] * 1e-30, torch.zeros(K), base[3], base[4], base[5] * 2.0 ** -120, base[6],
                     base[7] * 1e36, base[8] * 1e-3]).to(dtype)
    X[3, K // 2] = float("inf")
    X[4, K - 1] = float("nan")
    X[6, 0] = float("-inf")
    w = weight(K, dtype)
    q = torch.empty(9, K, dtype=torch.int8, device="cuda")
    scale, Y = torch.empty(9, device="cuda"), torch.empty(9, K, dtype=dtype, device="cuda")
    for eps in (EPS, 0.0):
        b.rmsnorm_into(X.cuda(), w.cuda(), Y=Y, q=q, scale=scale, eps=eps)
        y = norm_reference(X, w, eps)
        rounded(Y, y, norm_slack(X, y), "Y")
        ref_q, _ = rows8_reference(X.double() * w.double())
        rows = [0, 1, 3, 4, 5, 6, 7, 8] if eps == 0.0 else list(range(9))    # (a row of zeros is 0 / 0 there)
        assert torch.equal(q.cpu()[rows], ref_q[rows])
        ref = X.double().mul(w.double()).abs().amax(1) * rstd_of(X, eps).squeeze(1) / 127.0
        bad = ~torch.isfinite(X).all(1)
        assert bool(torch.isnan(scale.cpu()[bad]).all())
        good = [i for i in rows if not bool(bad[i])]
        rounded(scale[good], ref[good], norm_slack(X, ref[good]) + 3 * 2.0 ** -24 * ref[good], "scale")
    big = torch.full((2, K), 1e-25, dtype=dtype)
    big[1] = 1e25
    small = torch.full((K,), 1e-25, dtype=dtype)
    b.rmsnorm_into(big.cuda(), small.cuda(), q=q[:2], scale=scale[:2], eps=0.0)
    assert bool((q[:2] == 127).all())
    assert b.device_status() == 0


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("K", [200, 900, 3000, 17000])
def test_values_out_of_range_in_place(K, dtype):
    """The rows that are read again, with the outputs in the inputs' place."""
    b = binding()
    X, R, w = normal(40, K, dtype, 8) * 1e30, normal(40, K, dtype, 9) * 1e30, weight(K, dtype) * 1e-25
    X, R, w = X.cuda(), R.cuda(), w.cuda()
    S, Y, q, scale = torch.empty_like(X), torch.empty_like(X), torch.empty(40, K, dtype=torch.int8, device="cuda"), torch.empty(40, device="cuda")
    b.rmsnorm_into(X, w, Y=Y, q=q, scale=scale, R=R, S=S, eps=0.0)
    for s_of, y_of in (("X", "R"), ("R", "X"), (None, "X"), (None, "R")):
        x, r, q2, s2 = X.clone(), R.clone(), torch.empty_like(q), torch.empty_like(scale)
        at = {"X": x, "R": r, None: None}
        b.rmsnorm_into(x, w, Y=at[y_of], q=q2, scale=s2, R=r, S=at[s_of], eps=0.0)
        assert torch.equal(at[y_of], Y) and torch.equal(q2, q) and torch.equal(s2, scale)
    dY, dS = normal(40, K, dtype, 10).cuda(), normal(40, K, dtype, 11).cuda()
    dX = b.rmsnorm_backward_into(dY, S, w, torch.empty_like(S), dS=dS, eps=0.0)[0]
    for into in range(3):
        given = [dY.clone(), S.clone(), dS.clone()]
        assert torch.equal(b.rmsnorm_backward_into(given[0], given[1], w, given[into], dS=given[2], eps=0.0)[0], dX)


def test_ties_are_rounded_to_even():
    """Rows whose quotients lie on and next to the ties."""
    b = binding()
    half = torch.arange(-126, 127).float() + 0.5
    x = torch.cat([torch.tensor([127.0]), half, torch.nextafter(half, torch.tensor(1e9)), torch.nextafter(half, torch.tensor(-1e9))])
    rows = torch.stack([x * s for s in (1.0, 2.0 ** -20, 2.0 ** 30)])
    q, scale = torch.empty(rows.shape, dtype=torch.int8, device="cuda"), torch.empty(3, device="cuda")
    b.rmsnorm_into(rows.cuda(), torch.ones(x.numel(), device="cuda"), q=q, scale=scale)
    assert torch.equal(q.cpu(), rows8_reference(rows)[0])
    # products whose fp32 values tie with others that are larger in their last bits
    g = torch.Generator()
    g.manual_seed(3)
    v = 1.0 + torch.rand(40, 3000, generator=g) * 2.0 ** -9
    w = 1.0 + torch.rand(3000, generator=g) * 2.0 ** -10
    v[:, ::3] *= 0.5 / 127 * torch.randint(1, 250, (1000,), generator=g)
    q, scale = torch.empty(v.shape, dtype=torch.int8, device="cuda"), torch.empty(40, device="cuda")
    b.rmsnorm_into(v.cuda(), w.cuda(), q=q, scale=scale)
    assert torch.equal(q.cpu(), rows8_reference(v.double() * w.double())[0])


# ------------------------------------------------------------------ backward
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("M,K", SHAPES + [(3000, 200), (5000, 1023)])
def test_backward(M, K, dtype):
    b = binding()
    V, dY, w, dS = normal(M, K, dtype, 11), normal(M, K, dtype, 12), weight(K, dtype), normal(M, K, dtype, 13)
    for stream in (True, False):
        dX, dw = torch.full((M, K), 77, dtype=dtype, device="cuda"), torch.full((K,), 77, dtype=dtype, device="cuda")
        b.rmsnorm_backward_into(dY.cuda(), V.cuda(), w.cuda(), dX, dw=dw, dS=dS.cuda() if stream else None)
        ref, ref_w, mag, mag_w = norm_backward_reference(dY, V, w, dS if stream else None, EPS)
        # rstd and n as in norm_slack, mean(g n) a sum of as many terms again
        terms = 2 * (K / 512 + 32 + 40) + 16
        rounded(dX, ref, terms * 2.0 ** -24 * mag, "dX")
        # dw: a block's rows one after the other, 8 warps, then the blocks
        terms_w = 0.5 * (K / 512 + 72) + 6 + M / 152 + 8 + 152 * 8 / 8 + 8
        rounded(dw, ref_w, min(terms_w, M + 0.5 * (K / 512 + 72) + 16) * 2.0 ** -24 * mag_w, "dw")
        alone = torch.empty_like(dX)
        assert b.rmsnorm_backward_into(dY.cuda(), V.cuda(), w.cuda(), alone, dS=dS.cuda() if stream else None)[1] is None
        assert torch.equal(alone, dX)
    assert b.device_status() == 0


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("M,K,pad,offset", [(6, 64, 3, 1), (5, 1000, 8, 8), (7, 4097, 0, 1), (3, 16400, 8, 0)])
def test_backward_views_and_in_place(M, K, pad, offset, dtype):
    b = binding()
    V, dY, w, dS = normal(M, K, dtype, 14), normal(M, K, dtype, 15), weight(K, dtype), normal(M, K, dtype, 16)
    ref, _, mag, _ = norm_backward_reference(dY, V, w, dS, EPS)
    slack = (2 * (K / 512 + 72) + 16) * 2.0 ** -24 * mag
    for into in ("other", "dY", "dS", "V"):
        given = dict(dY=device_matrix(dY, pad, offset), V=device_matrix(V, pad, offset), dS=device_matrix(dS, pad, offset))
        dw = torch.empty(K, dtype=dtype, device="cuda")
        flat = torch.full((M, K + pad + 1), 5.0, dtype=dtype, device="cuda")
        dX = given.get(into, flat[:, :K])
        b.rmsnorm_backward_into(given["dY"], given["V"], w.cuda(), dX, dw=dw, dS=given["dS"])
        rounded(dX, ref, slack, into)
        assert bool((flat[:, K:] == 5).all())


@pytest.mark.parametrize("K", [48, 2000, 17000])
def test_backward_out_of_range(K):
    b = binding()
    V, dY, w = normal(4, K, torch.float32, 17), normal(4, K, torch.float32, 18), weight(K, torch.float32)
    V[0] *= 1e25
    V[1] *= 1e-25
    dX, dw = torch.empty(4, K, device="cuda"), torch.empty(K, device="cuda")
    b.rmsnorm_backward_into(dY.cuda(), V.cuda(), w.cuda(), dX, dw=dw, eps=0.0)
    ref, ref_w, mag, mag_w = norm_backward_reference(dY, V, w, None, 0.0)
    rounded(dX, ref, (2 * (K / 512 + 72) + 16) * 2.0 ** -24 * mag, "dX")
    rounded(dw, ref_w, (0.5 * (K / 512 + 72) + 20) * 2.0 ** -24 * mag_w, "dw")
    V[2, 3] = float("nan")
    b.rmsnorm_backward_into(dY.cuda(), V.cuda(), w.cuda(), dX, dw=dw)
    assert bool(torch.isnan(dX[2]).all()) and bool(torch.isfinite(dX[[0, 1, 3]]).all())


def test_backward_against_differences():
    """The gradients against central differences of the forward pass in 64 bits."""
    b = binding()
    V, dY, w = (t.double() for t in (normal(2, 24, torch.float32, 20), normal(2, 24, torch.float32, 21), weight(24, torch.float32)))
    dX, dw = torch.empty(2, 24, device="cuda"), torch.empty(24, device="cuda")
    b.rmsnorm_backward_into(dY.float().cuda(), V.float().cuda(), w.float().cuda(), dX, dw=dw)
    step = 1e-5

    def loss(v, u):
        return float((norm_reference(v, u, EPS) * dY).sum())
    for i in range(2):
        for j in range(24):
            d = torch.zeros_like(V)
            d[i, j] = step
            # the difference's own error: step^2 times the third derivative, and 1e-16 / step
            assert abs((loss(V + d, w) - loss(V - d, w)) / (2 * step) - float(dX[i, j])) < 2e-5
    for j in range(24):
        d = torch.zeros_like(w)
        d[j] = step
        assert abs((loss(V, w + d) - loss(V, w - d)) / (2 * step) - float(dw[j])) < 2e-5


def test_no_rows_and_no_columns():
    b = binding()
    w, dw = torch.ones(40, device="cuda"), torch.full((40,), 7.0, device="cuda")
    none = torch.empty(0, 40, device="cuda")
    b.rmsnorm_into(none, w, Y=none.clone())
    b.rmsnorm_backward_into(none, none, w, none.clone(), dw=dw)
    assert bool((dw == 0).all())
    flat = torch.empty(3, 0, device="cuda")
    b.rmsnorm_into(flat, torch.empty(0, device="cuda"), Y=flat.clone())
    b.rmsnorm_backward_into(flat, flat, torch.empty(0, device="cuda"), flat.clone(), dw=torch.empty(0, device="cuda"))
    assert b.device_status() == 0


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_bitwise_the_same_from_call_to_call(dtype):
    b = binding()
    V, dY, w = (t.cuda() for t in (normal(3000, 2048, dtype, 22), normal(3000, 2048, dtype, 23), weight(2048, dtype)))
    first = b.rmsnorm_backward_into(dY, V, w, torch.empty_like(V), dw=torch.empty_like(w))
    for _ in range(5):
        again = b.rmsnorm_backward_into(dY, V, w, torch.empty_like(V), dw=torch.empty_like(w))
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_many_rows():
    """Rows past 2^31 elements into the matrices."""
    b = binding()
    M, K = 600001, 4096
    X = torch.ones(M, K, dtype=torch.bfloat16, device="cuda")
    X[-2:] = normal(2, K, torch.bfloat16, 24).cuda()
    w = weight(K, torch.bfloat16)
    q, scale = torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    b.rmsnorm_into(X, w.cuda(), q=q, scale=scale)
    check_rows8(q[-2:], scale[-2:], X[-2:].cpu(), w, rstd_of(X[-2:].cpu(), EPS), "last rows")
    dX, dw = torch.empty_like(X), torch.empty(K, dtype=torch.bfloat16, device="cuda")
    b.rmsnorm_backward_into(X, X, w.cuda(), dX, dw=dw)
    ref, _, mag, _ = norm_backward_reference(X[-2:].cpu(), X[-2:].cpu(), w, None, EPS)
    rounded(dX[-2:], ref, 200 * 2.0 ** -24 * mag, "dX")
    assert b.device_status() == 0
