"""Activation checkpoints in 8 bits on the GPU, against their definition in 64 bits."""
import numpy as np
import pytest
import torch

from _layers import assert_close, device_matrix, quantise, values

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16]
# (rows, columns, padding of a row, offset of the first element)
SHAPES = [(1, 1, 0, 0), (1, 32, 0, 0), (3, 33, 0, 0), (5, 64, 0, 0), (7, 96, 8, 0), (2, 1000, 0, 0),
          (4, 1001, 3, 1), (33, 8, 0, 0), (65, 40, 8, 8), (9, 257, 0, 3), (2, 4104, 0, 0),
          (300, 31, 1, 0)]


@pytest.fixture(scope="module", autouse=True)
def _gpu(cuda_device):
    yield


def binding():
    from dense_fp32_gemm_02_gb300 import binding
    return binding


def inputs(M, K, dtype, seed=0):
    """Values over many magnitudes, zero blocks and exact powers of two among them."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g) * torch.exp2(torch.randint(-30, 30, (M, 1), generator=g).float())
    x[torch.rand(M, K, generator=g) < 0.05] = 0.0
    x[:, : min(K, 32)] *= (torch.rand(M, 1, generator=g) < 0.8).float()
    x[:, K // 2] = torch.exp2(torch.randint(-20, 20, (M,), generator=g).float())
    return x.to(dtype)


def int8_views(M, K, pad, offset):
    q = torch.full((M * (K + pad) + offset + 8,), 77, dtype=torch.int8, device="cuda")
    blocks = -(-K // 32)
    e = torch.full((M * (blocks + pad) + 8,), 77, dtype=torch.int8, device="cuda")
    return (q[offset:offset + M * (K + pad)].view(M, K + pad)[:, :K],
            e[:M * (blocks + pad)].view(M, blocks + pad)[:, :blocks], q, e)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_store_and_load_are_the_definition(shape, dtype):
    M, K, pad, offset = shape
    b = binding()
    x = inputs(M, K, dtype, seed=M * K)
    q, e, qflat, eflat = int8_views(M, K, pad, offset)
    b.act8_store_into(device_matrix(x, pad, offset), q, e)
    rq, re = quantise(x)
    assert torch.equal(q.cpu(), rq) and torch.equal(e.cpu(), re)
    # nothing around the two was written
    written = torch.zeros_like(qflat, dtype=torch.bool)
    written[offset:offset + M * (K + pad)].view(M, K + pad)[:, :K] = True
    assert bool((qflat[~written] == 77).all())
    assert int((eflat == 77).sum()) >= eflat.numel() - e.numel()
    back = device_matrix(torch.zeros(M, K, dtype=dtype), pad, offset)
    b.act8_load_into(q, e, back)
    assert torch.equal(back.cpu().double(), values(rq, re))      # exact in either type


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("K", [64, 67])
def test_special_values(K, dtype):
    b = binding()
    top = torch.finfo(dtype).max
    x = torch.zeros(9, K)
    x[0, 3] = float("nan")
    x[1, 5], x[1, 40] = float("inf"), 2.0
    x[2, 0] = -float("inf")
    x[3, :3] = torch.tensor([top, -top, 2.0 ** 120])
    x[4, 1], x[4, 2] = 127 * 2.0 ** 121, -(2.0 ** 121)
    x[5, 7] = 2.0 ** -126                 # the smallest normal number
    x[6, 7] = 2.0 ** -130                 # below: zero or one step of 2^-126
    x[7, :4] = torch.tensor([127.0, 0.5, 1.5, 2.5])      # ties go to the even neighbour
    x[8, :4] = torch.tensor([127.5, 64.0, -0.0, 1.0])    # just past 127 * 2^0
    x = x.to(dtype)
    q, e, _, _ = int8_views(9, K, 0, 0)
    b.act8_store_into(x.cuda(), q, e)
    rq, re = quantise(x)
    assert torch.equal(q.cpu(), rq) and torch.equal(e.cpu(), re)
    back = torch.empty(9, K, dtype=dtype, device="cuda")
    b.act8_load_into(q, e, back)
    back = back.cpu()
    assert torch.isnan(back[0, :32]).all() and torch.isnan(back[1, :32]).all()
    assert torch.isfinite(back[1, 32:]).all() and float(back[1, 40]) == 2.0
    assert torch.isfinite(back[3:]).all()
    dz = b.act8_grad_into(q, e, torch.ones(9, K, dtype=dtype, device="cuda"),
                          torch.empty(9, K, dtype=dtype, device="cuda"), act="relu").cpu()
    assert torch.isnan(dz[0, :32]).all() and torch.isfinite(dz[3:]).all()


def gelu(z):
    return z * 0.5 * torch.erfc(-z / 2 ** 0.5)


def gelu_slope(z):
    return 0.5 * torch.erfc(-z / 2 ** 0.5) + z * torch.exp(-z * z / 2) / (2 * np.pi) ** 0.5


ACTS = {"none": (lambda z: z, lambda z: torch.ones_like(z)),
        "relu": (torch.relu, lambda z: (z > 0).double()), "gelu": (gelu, gelu_slope)}


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", sorted(ACTS))
@pytest.mark.parametrize("shape", [(37, 256, 0, 0), (21, 203, 5, 1)])
def test_activation_and_its_gradient(shape, act, dtype):
    """The activation of the given values and the slope at the kept ones.  Phi is within
    1.5e-7 (the formula's error) plus a few fp32 roundings, 4e-7 in all, so z Phi(z) and
    the slope times dY are within that times |z| + 1 or |dY| (|z| + 1)."""
    M, K, pad, offset = shape
    b = binding()
    g = torch.Generator().manual_seed(5)
    z = (torch.randn(M, K, generator=g) * 3).to(dtype)
    dy = torch.randn(M, K, generator=g).to(dtype)
    q, e, _, _ = int8_views(M, K, pad, offset)
    y = device_matrix(torch.zeros(M, K, dtype=dtype), pad, offset)
    b.act8_store_into(device_matrix(z, pad, offset), q, e, act=act, Y=y)
    rq, re = quantise(z)
    assert torch.equal(q.cpu(), rq) and torch.equal(e.cpu(), re)
    f, slope = ACTS[act]
    kept = values(rq, re)
    dz = device_matrix(torch.zeros(M, K, dtype=dtype), pad, offset)
    b.act8_grad_into(q, e, device_matrix(dy, pad, offset), dz, act=act)
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24      # half a spacing
    for got, ref, size in ((y, f(z.double()), z.double().abs() + 1),
                           (dz, dy.double() * slope(kept), dy.double().abs() * (kept.abs() + 1))):
        err = (got.cpu().double() - ref).abs()
        assert bool((err <= 4e-7 * size + half * (ref.abs() + 4e-7 * size)).all()), float(err.max())


def test_gelu_gradient_against_differences():
    """(gelu(z + h) - gelu(z - h)) / 2h of the stored activation, h = 2^-6: off by h^2/6
    times the third derivative (under 1.6), 7e-5, and the rounding of two values of size
    under 4 over 2h, 4 * 2^-23 * 32 = 2e-5, to which the formula's 1.5e-7 * 4 * 64 adds 4e-5."""
    b = binding()
    z = (torch.randint(-127, 128, (64, 128)).float() / 32).cuda()     # kept exactly: |z| < 4
    z[:, ::32] = 127 / 32
    q, e = b.act8_empty(64, 128)
    y = torch.empty(2, 64, 128, device="cuda")
    h = 2.0 ** -6
    for i, s in enumerate((h, -h)):
        b.act8_store_into(z + s, q, e, act="gelu", Y=y[i])
    b.act8_store_into(z, q, e)
    back = b.act8_load_into(q, e, torch.empty_like(z))
    assert torch.equal(back, z)
    slope = b.act8_grad_into(q, e, torch.ones_like(z), torch.empty_like(z), act="gelu")
    assert float((slope - (y[0] - y[1]) / (2 * h)).abs().max()) <= 1.5e-4


def test_in_place_and_other_streams():
    b = binding()
    z = torch.randn(64, 128, device="cuda")
    q, e = b.act8_empty(64, 128)
    y = b.act8_empty(64, 128)
    want = torch.empty_like(z)
    b.act8_store_into(z, q, e, act="gelu", Y=want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    same = z.clone()
    torch.cuda.synchronize()
    b.act8_store_into(same, *y, act="gelu", Y=same, stream=side)
    b.act8_grad_into(*y, same, same, act="relu", stream=side)
    side.synchronize()
    assert torch.equal(y[0], q) and torch.equal(y[1], e)
    assert torch.equal(same, torch.where(b.act8_load_into(q, e, torch.empty_like(z)) > 0, want, 0.0))


WGRAD = [  # (M, K, N, padding, offset)
    (1, 1, 1, 0, 0), (1, 64, 64, 0, 0), (2, 33, 5, 3, 1), (63, 128, 96, 0, 0), (64, 256, 256, 8, 8),
    (65, 257, 127, 1, 0), (500, 96, 520, 0, 0), (513, 320, 8, 0, 3), (1025, 136, 264, 0, 0),
    (2300, 65, 300, 0, 0), (700, 1030, 700, 2, 2), (4111, 264, 40, 0, 0),
    # the float32 product's tiles of 160, 192 and 224 columns
    (72, 5000, 270, 1, 1), (72, 5000, 490, 0, 0), (72, 5000, 583, 1, 1)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("beta", [0.0, 0.5])
@pytest.mark.parametrize("shape", WGRAD)
def test_weight_gradient(shape, beta, dtype):
    M, K, N, pad, offset = shape
    b = binding()
    g = torch.Generator().manual_seed(M + K + N)
    x = torch.randn(M, K, generator=g) * torch.exp2(torch.randint(-3, 3, (M, 1), generator=g).float())
    dy = torch.randn(M, N, generator=g).to(dtype)
    start = torch.randn(K, N, generator=g).to(dtype)
    q, e, _, _ = int8_views(M, K, pad, offset)
    b.act8_store_into(x.cuda(), q, e)
    xv = values(q.cpu(), e.cpu())
    dw = device_matrix(start if beta else torch.full((K, N), float("nan"), dtype=dtype), pad, offset)
    b.act8_weight_grad_into(q, e, device_matrix(dy, pad, offset), dw, beta=beta)
    ref, mag = xv.t() @ dy.double(), xv.abs().t() @ dy.double().abs()
    if beta:
        ref, mag = ref + beta * start.double(), mag + beta * start.double().abs()
    assert_close(dw, ref, mag, M, f"dW {shape}")
    assert b.device_status() == b.SGEMM_OK


def test_weight_gradient_of_no_rows_and_of_a_nan_block():
    b = binding()
    dw = torch.ones(40, 24, device="cuda")
    q, e = b.act8_empty(0, 40)
    b.act8_weight_grad_into(q, e, torch.empty(0, 24, device="cuda"), dw, beta=2.0)
    assert bool((dw == 2).all())
    b.act8_weight_grad_into(q, e, torch.empty(0, 24, device="cuda"), dw)
    assert bool((dw == 0).all())
    x = torch.randn(100, 96, device="cuda")
    x[50, 40] = float("nan")
    q, e = b.act8_empty(100, 96)
    b.act8_store_into(x, q, e)
    dw = b.act8_weight_grad_into(q, e, torch.randn(100, 24, device="cuda"),
                                 torch.empty(96, 24, device="cuda"))
    assert torch.isnan(dw[32:64]).all()
    assert torch.isfinite(dw[:32]).all() and torch.isfinite(dw[64:]).all()


def test_weight_gradient_against_differences_and_repeats():
    """sum(dY * (x D)) is linear in D, so <dW, D> is its difference quotient; the loss is
    summed in 64 bits, so only dW's fp32 rounding (4e-6 of its norm) is between the two."""
    b = binding()
    x = torch.randn(900, 200, device="cuda")
    dy = torch.randn(900, 310, device="cuda")
    q, e = b.act8_empty(900, 200)
    b.act8_store_into(x, q, e)
    dw = b.act8_weight_grad_into(q, e, dy, torch.empty(200, 310, device="cuda"))
    again = b.act8_weight_grad_into(q, e, dy, torch.empty(200, 310, device="cuda"))
    assert torch.equal(dw, again)
    xv = values(q.cpu(), e.cpu())
    for seed in range(3):
        D = torch.randn(200, 310, generator=torch.Generator().manual_seed(seed)).double()
        loss = [(dy.cpu().double() * (xv @ (s * D))).sum() for s in (1.0, -1.0)]
        quotient = float(loss[0] - loss[1]) / 2
        have = float((dw.cpu().double() * D).sum())
        assert abs(have - quotient) <= 4e-6 * float(dw.double().norm() * D.norm())


def test_past_two_to_the_31_elements():
    """70000 x 32800 (2.3e9 elements, in both forms): the rows past the 2^31-th element are
    those of a call on them alone, bit for bit."""
    b = binding()
    for K, pad in ((32800, 0), (32801, 0)):
        M, tail = 70000, 300
        z = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
        g = torch.Generator(device="cuda")
        g.manual_seed(3)
        for r in range(0, M, 10000):
            z[r:r + 10000].normal_(generator=g)
        q, e = b.act8_empty(M, K)
        y = torch.empty_like(z)
        b.act8_store_into(z, q, e, act="gelu", Y=y)
        q2, e2 = b.act8_empty(tail, K)
        y2 = torch.empty(tail, K, dtype=torch.bfloat16, device="cuda")
        b.act8_store_into(z[-tail:], q2, e2, act="gelu", Y=y2)
        assert torch.equal(q[-tail:], q2) and torch.equal(e[-tail:], e2) and torch.equal(y[-tail:], y2)
        b.act8_grad_into(q, e, z, y, act="gelu")
        b.act8_grad_into(q2, e2, z[-tail:], y2, act="gelu")
        assert torch.equal(y[-tail:], y2)
        del z, q, e, y
    torch.cuda.empty_cache()


def test_weight_gradient_past_two_to_the_31_elements():
    """The columns of a 70000 x 32800 checkpoint one at a time would be the same sums: the
    last 64 against a call on a copy of them."""
    b = binding()
    M, K = 70000, 32800
    q = torch.randint(-127, 128, (M, K), dtype=torch.int8, device="cuda")
    e = torch.randint(-9, -5, (M, K // 32), dtype=torch.int8, device="cuda")
    dy = torch.randn(M, 40, device="cuda").to(torch.bfloat16)
    dw = b.act8_weight_grad_into(q, e, dy, torch.empty(K, 40, dtype=torch.bfloat16, device="cuda"))
    some = b.act8_weight_grad_into(q[:, -64:].contiguous(), e[:, -2:].contiguous(), dy,
                                   torch.empty(64, 40, dtype=torch.bfloat16, device="cuda"))
    # other splits of the contraction: equal up to fp32 sums, i.e. one rounding to bfloat16
    far = (dw[-64:].float() - some.float()).abs().max() / some.float().abs().max()
    assert float(far) <= 2.0 ** -7
    del q, e, dy
    torch.cuda.empty_cache()
