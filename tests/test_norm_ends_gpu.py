"""The norm and its 8-bit rows where their arithmetic is at its limits: products a hair beside a tie."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu(cuda_device):
    yield


def binding():
    from dense_fp32_gemm_02_gb300 import binding
    return binding


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
