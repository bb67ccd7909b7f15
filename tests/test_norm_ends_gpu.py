"""The norm, its 8-bit rows and its backward pass where their arithmetic is at its limits: products a hair beside a
tie, rows at the ends of float32's range."""
import pytest
import torch

from _forward import norm_backward_reference, norm_reference, norm_slack, rounded, rows8_reference

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16]


@pytest.fixture(scope="module", autouse=True)
def _gpu(cuda_device):
    yield


def binding():
    from dense_fp32_gemm_02_gb300 import binding
    return binding


def normal(rows, cols, seed, scale=1.0):
    g = torch.Generator()
    g.manual_seed(seed)
    return torch.randn(rows, cols, generator=g) * scale


# ------------------------------------------------------------------ ties
# (a, b, c, d): of rows whose largest product is a b, what 127 c d / (a b) rounds to is decided by its last bits: up to
# 10 units of a 55-bit number on either side of a tie, or on it.
PAIRS = [
    (13046243, 12585762, 12569875, 13011304), (15092289, 11806318, 14410165, 12219140), (10776125, 14107167, 4608454, 10259839),
    (15632765, 10246435, 12343171, 6182064), (10614406, 10566517, 4722157, 12810733), (11726969, 14704145, 7430094, 16172263),
    (13936833, 11529875, 6102269, 11092959), (14276835, 9448266, 4724133, 14276835), (9581769, 12474698, 6563889, 16131075),
    (12438133, 15827735, 11047459, 11997036), (10549552, 12318531, 9408775, 10603781), (9645777, 13871550, 5242365, 16379055),
    (13949872, 10478049, 242825, 11849323), (12687913, 15024778, 5031318, 16259578), (10399466, 15965043, 5070263, 16372713),
    (11465179, 10540808, 1496748, 16212221), (13649414, 10106707, 1147378, 14673886), (16252236, 15794736, 6332040, 16758588),
    (15178822, 9961400, 4980700, 15178822), (14079632, 14634752, 6332481, 13707329), (11512693, 16639090, 7559381, 15264338),
    (10174054, 12550013, 5087027, 16107497), (14095111, 16748760, 7122668, 16572135), (8925179, 16029892, 2694830, 15676305),
    (14667992, 14509030, 6352280, 15959933), (12248134, 10790721, 6220509, 12463701), (14877817, 9984873, 412399, 9927239),
    (15091059, 11221450, 5161867, 16403325)]


def nearest(p, top):
    """127 p / top to the nearest integer, ties to even, in integers."""
    n, rest = divmod(127 * p, top)
    return n + (2 * rest > top or (2 * rest == top and n % 2 == 1))


@pytest.mark.parametrize("K", [2, 300, 1024, 5000, 20000])
@pytest.mark.parametrize("v_scale,w_scale", [(1.0, 1.0), (2.0 ** -40, 2.0 ** 10), (2.0 ** 60, 2.0 ** 70), (2.0 ** -90, 2.0 ** -80)])
def test_products_beside_a_tie(v_scale, w_scale, K):
    """Products of float32 values, of 48 bits, whose quotient is as good as a tie: q is that of the exact quotient, in
    fp32's range and outside it (the last two scales)."""
    b = binding()
    q, scale = torch.empty(2, K, dtype=torch.int8, device="cuda"), torch.empty(2, device="cuda")
    got, want = [], []
    for a, x, c, d in PAIRS:
        V, w = torch.zeros(2, K), torch.zeros(K)
        V[0, 0], V[0, K - 1], w[0], w[K - 1] = a * v_scale, -c * v_scale, x * w_scale, d * w_scale
        V[1] = -V[0]
        b.rmsnorm_into(V.cuda(), w.cuda(), q=q, scale=scale)
        got += q[:, [0, K - 1]].flatten().tolist()
        n = nearest(c * d, a * x)
        want += [127, -n, -127, n]
    assert got == want


# ------------------------------------------------------------------ the ends of float32's range
ENDS = [1e-44, 1e-41, 1e-39, 3e-38, 1e37, 8e37]


def rows_at_the_ends(K, dtype):
    """A row for each of ENDS; values of order 1 (none above 4) times it, as the type holds them."""
    x = normal(len(ENDS), K, 5).clamp(-4, 4)
    x[:, 0] = 2.0
    return (x.double() * torch.tensor(ENDS).double().unsqueeze(1)).to(dtype)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("K", [40, 257, 1000, 2048, 5000, 16384, 16390, 40000])
def test_rows_at_the_ends_of_the_range(K, dtype):
    """eps = 0: y is of order 1 whatever the row's size, down to the smallest values that the types hold."""
    b = binding()
    X, w = rows_at_the_ends(K, dtype), (1.0 + 0.3 * normal(1, K, 6)[0]).to(dtype)
    M = len(ENDS)
    Y, q, scale = torch.empty(M, K, dtype=dtype, device="cuda"), torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    S = torch.empty_like(Y)
    b.rmsnorm_into(X.cuda(), w.cuda(), Y=Y, q=q, scale=scale, S=S, eps=0.0)
    y = norm_reference(X, w, 0.0)
    assert torch.equal(S.cpu(), X)
    some = (X != 0).any(1)            # (1e-44 is 0 in bfloat16, whose norm is 0 / 0)
    rounded(Y[some.cuda()], y[some], norm_slack(X, y)[some], "Y")
    assert torch.equal(q.cpu()[some], rows8_reference(X.double() * w.double())[0][some])
    ref = y.abs().amax(1) / 127.0
    rounded(scale[some.cuda()], ref[some], norm_slack(X, ref)[some] + 3 * 2.0 ** -24 * ref[some], "scale")
    x = X.cuda()                      # in the input's place, and without the 8 bits
    b.rmsnorm_into(x, w.cuda(), Y=x, q=q, scale=scale, eps=0.0)
    assert torch.equal(x[some.cuda()], Y[some.cuda()])
    x = X.cuda()
    b.rmsnorm_into(x, w.cuda(), Y=x, eps=0.0)
    assert torch.equal(x[some.cuda()], Y[some.cuda()])


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("K", [40, 257, 1000, 2048, 5000, 16384, 16390, 40000])
def test_gradients_at_the_ends_of_the_range(K, dtype):
    """The same of the backward pass, dX in dY's or V's place too."""
    b = binding()
    V, w = rows_at_the_ends(K, dtype), (1.0 + 0.3 * normal(1, K, 6)[0]).to(dtype)
    V = V[(V != 0).any(1)]
    sizes = V.double().square().mean(1).sqrt()
    dY = (normal(len(V), K, 7).double() * sizes.clamp(1e-30, 1e30).unsqueeze(1)).to(dtype)   # (dX stays in range)
    ref, ref_w, mag, mag_w = norm_backward_reference(dY, V, w, None, 0.0)
    for into in ("other", "dY", "V"):
        given = dict(dY=dY.cuda(), V=V.cuda())
        dX, dw = given.get(into, torch.empty(len(V), K, dtype=dtype, device="cuda")), torch.empty(K, dtype=dtype, device="cuda")
        b.rmsnorm_backward_into(given["dY"], given["V"], w.cuda(), dX, dw=dw, eps=0.0)
        rounded(dX, ref, (2 * (K / 512 + 72) + 16) * 2.0 ** -24 * mag, "dX")
        rounded(dw, ref_w, (0.5 * (K / 512 + 72) + 20 + len(V)) * 2.0 ** -24 * mag_w, "dw")


@pytest.mark.parametrize("K", [40, 257, 1000, 5000, 20000])
def test_sums_of_the_gradient_past_float32(K):
    """Rows and gradients whose products, or their sum, leave fp32's range where the gradient itself does not."""
    b = binding()
    V, dY, w = normal(4, K, 8), normal(4, K, 9), 1.0 + 0.3 * normal(1, K, 10)[0]
    dY += 0.3 * V                      # (mean(g n) is of g's order)
    V[0] *= 1e14
    dY[0] *= 1e27
    V[1] *= 1e-5
    dY[1] *= 1e33
    V[2] *= 1e10
    dY[2] *= 1e36
    dX, dw = torch.empty(4, K, device="cuda"), torch.empty(K, device="cuda")
    b.rmsnorm_backward_into(dY.cuda(), V.cuda(), w.cuda(), dX, dw=dw)
    ref, ref_w, mag, mag_w = norm_backward_reference(dY, V, w, None, 1e-6)
    rounded(dX, ref, (2 * (K / 512 + 72) + 16) * 2.0 ** -24 * mag, "dX")
    rounded(dw, ref_w, (0.5 * (K / 512 + 72) + 24) * 2.0 ** -24 * mag_w, "dw")


# ------------------------------------------------------------------ no columns
@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_rows_of_no_columns_have_scales_of_zero(dtype):
    """A row of zeros has scale 0, one of no columns too; nothing beside the scales is written."""
    b = binding()
    X, w = torch.empty(5, 0, dtype=dtype, device="cuda"), torch.empty(0, dtype=dtype, device="cuda")
    scale = torch.full((7,), 55.0, device="cuda")
    b.rmsnorm_into(X, w, q=torch.empty(5, 0, dtype=torch.int8, device="cuda"), scale=scale[1:6])
    assert scale.tolist() == [55.0, 0.0, 0.0, 0.0, 0.0, 0.0, 55.0]
