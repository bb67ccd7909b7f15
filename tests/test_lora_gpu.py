"""Low-rank adapters of many requests beside a shared projection, forward and backward,
on the GPU, against their formulas in 64 bits."""
import pytest
import torch

from _layers import (assert_close, device_matrix, device_stack, lora_backward_reference,
                     lora_reference, quantise, rank_of, row_ids, values)

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16]


@pytest.fixture(scope="module", autouse=True)
def _gpu(cuda_device):
    yield


def binding():
    from dense_fp32_gemm_02_gb300 import binding
    return binding


class Problem:
    """Inputs of one call on the CPU.  What no row may read is NaN: the stack past an
    adapter's rank, and adapters without rows."""

    def __init__(self, M, K, N, L, R, dtype, ids="runs", ranks=True, scale=True, bias=True, seed=0):
        g = torch.Generator().manual_seed(seed + M + K + N)
        r = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
        self.M, self.K, self.N, self.L, self.R, self.dtype = M, K, N, L, R, dtype
        self.X, self.W = r(M, K).to(dtype), (r(K, N) / max(K, 1) ** 0.5).to(dtype)
        self.A = (r(L, K, R) / max(K, 1) ** 0.5).to(dtype)
        self.B = (r(L, R, N) / max(R, 1) ** 0.5).to(dtype)
        self.dY = r(M, N).to(dtype)
        self.ids = row_ids(M, L, ids, seed)
        self.scale = torch.rand(L, generator=g) + 0.5 if scale else None
        self.ranks = torch.randint(0, R + 3, (L,), generator=g, dtype=torch.int32) if ranks else None
        self.bias = r(N).to(dtype) if bias else None
        for a in range(L):
            n = rank_of(self.ranks, a, R) if (self.ids == a).any() else 0
            self.A[a, :, n:], self.B[a, n:] = float("nan"), float("nan")

    def clean(self):
        """The stack with zeros in the place of what is not used."""
        return torch.nan_to_num(self.A), torch.nan_to_num(self.B)

    def on_gpu(self, pad, offset):
        d = {n: device_matrix(getattr(self, n), pad, offset) for n in ("X", "W", "dY")}
        d["A"], d["B"] = device_stack(self.A, pad, offset), device_stack(self.B, pad, offset)
        for n in ("ids", "scale", "ranks", "bias"):
            t = getattr(self, n)
            d[n] = None if t is None else t.cuda()
        return d

    def out(self, rows, cols, pad, offset, dtype=None):
        return device_matrix(torch.full((rows, cols), float("nan"), dtype=dtype or self.dtype), pad, offset)


def run_forward(p, pad=0, offset=0, H=True, stream=None):
    b, d = binding(), p.on_gpu(pad, offset)
    Y = p.out(p.M, p.N, pad, offset)
    h = p.out(p.M, p.R, pad, 0, torch.float32) if H else None
    b.lora_into(d["X"], d["W"], d["A"], d["B"], d["ids"], Y, scale=d["scale"], ranks=d["ranks"],
                bias=d["bias"], H=h, stream=stream)
    return Y, h


def check_forward(p, Y, h, what):
    A, B = p.clean()
    ref, href, mag, hmag = lora_reference(p.X, p.W, A, B, p.ids, p.scale, p.ranks, p.bias)
    assert_close(Y, ref, mag, p.K + p.R, f"Y {what}")
    if h is not None:
        assert_close(h, href, hmag, p.K, f"H {what}")
    b = binding()
    assert b.device_status() == b.SGEMM_OK


FORWARD = [  # (M, K, N, L, R, ids, padding, offset)
    (1, 1, 1, 1, 1, "single", 0, 0), (1, 64, 64, 2, 8, "single", 0, 0), (1, 1024, 1000, 3, 16, "none", 0, 0),
    (2, 100, 77, 4, 5, "mixed", 3, 1), (5, 256, 512, 1, 128, "single", 0, 0), (8, 1000, 1030, 8, 16, "mixed", 0, 0),
    (9, 513, 2049, 3, 20, "outside", 0, 0), (16, 2048, 256, 40, 8, "mixed", 8, 8),
    (17, 520, 264, 5, 33, "mixed", 0, 0), (32, 640, 328, 3, 64, "runs", 0, 0), (33, 300, 300, 2, 7, "runs", 1, 3),
    (64, 512, 1024, 32, 16, "mixed", 0, 0), (100, 65, 130, 3, 17, "outside", 0, 0),
    (128, 512, 256, 2, 16, "single", 0, 0), (129, 256, 384, 1, 100, "runs", 0, 0),
    (256, 200, 264, 3, 64, "runs", 8, 8), (300, 1000, 520, 4, 24, "runs", 0, 0),
    (400, 520, 264, 3, 16, "none", 0, 0), (513, 128, 513, 2, 128, "runs", 0, 1),
    (700, 264, 300, 6, 40, "mixed", 0, 0), (1100, 520, 776, 3, 16, "runs", 0, 0),
    (1025, 2056, 264, 2, 65, "runs", 0, 0), (64, 64, 4100, 4, 8, "mixed", 0, 0),
    (64, 4100, 520, 0, 1, "none", 0, 0), (40, 4100, 1032, 3, 8, "mixed", 4, 4), (200, 3000, 264, 2, 20, "runs", 0, 0),
    (16, 5000, 264, 5, 24, "mixed", 0, 0), (3, 9000, 72, 3, 128, "mixed", 0, 0), (300, 64, 64, 0, 1, "none", 0, 0), (7, 96, 40, 0, 1, "none", 0, 0), (600, 32, 8, 500, 4, "mixed", 0, 0),
    (8, 3000, 3016, 3, 8, "mixed", 0, 0), (5, 4100, 2300, 2, 16, "outside", 4, 4), (4, 4096, 7816, 2, 4, "runs", 0, 0),
    (3, 3000, 3017, 2, 8, "mixed", 1, 1)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("case", FORWARD)
def test_forward(case, dtype):
    M, K, N, L, R, ids, pad, offset = case
    p = Problem(M, K, N, L, R, dtype, ids, seed=3)
    check_forward(p, *run_forward(p, pad, offset, H=L > 0), case)


WIDTHS = [270, 390, 490, 583]   # of 5000 rows: the float32 products' tiles of 128, 160, 192 and 224 columns


@pytest.mark.parametrize("ids", ["mixed", "outside"])
@pytest.mark.parametrize("N", WIDTHS)
def test_forward_at_each_tile_width(N, ids):
    p = Problem(5000, 72, N, 3, 24, torch.float32, ids, ranks=False, seed=5)
    check_forward(p, *run_forward(p, 1, 1), N)
    p.A[1, 5, 3] = float("inf")     # the rank side of its rows' tiles in the epilogue
    ref, _, mag, _ = lora_reference(p.X, p.W, torch.where(p.A.isinf(), 0.0, p.A), p.B, p.ids, p.scale, p.ranks, p.bias)
    Y, _ = run_forward(p)
    clean = p.ids != 1
    assert_close(Y[clean.cuda()], ref[clean], mag[clean], p.K + p.R, f"Y {N}")


@pytest.mark.parametrize("M", [3, 40, 600, 1400])
@pytest.mark.parametrize("dtype", TYPES)
def test_forward_defaults(M, dtype):
    """No scale, no ranks, no bias, no H."""
    p = Problem(M, 136, 200, 3, 12, dtype, "runs", ranks=False, scale=False, bias=False)
    check_forward(p, *run_forward(p, H=False), "defaults")


@pytest.mark.parametrize("M", [6, 70, 900, 1700])
@pytest.mark.parametrize("ids", ["mixed", "runs"])
@pytest.mark.parametrize("dtype", TYPES)
def test_an_adapters_infinities_and_nans_stay_in_its_rows(M, ids, dtype):
    p = Problem(M, 128, 264, 3, 16, dtype, ids, ranks=False)
    p.A, p.B = torch.nan_to_num(p.A), torch.nan_to_num(p.B)
    p.A[1, 5, 3], p.B[1, 7] = float("nan"), float("inf")
    p.X[0, 9] = float("nan")             # a row's own NaN stays in that row
    Y, h = run_forward(p)
    A, B = p.A.clone(), p.B.clone()
    A[1], B[1] = 0, 0
    X = p.X.clone()
    X[0] = 0
    ref, _, mag, _ = lora_reference(X, p.W, A, B, p.ids, p.scale, None, p.bias)
    clean = p.ids != 1
    clean[0] = False
    assert_close(Y[clean.cuda()], ref[clean], mag[clean], 144, "rows of the other adapters")
    touched = (p.ids == 1)
    assert not torch.isfinite(Y.cpu()[touched].float()).any()
    assert torch.isnan(Y.cpu()[0].float()).all()


def test_empty_sizes():
    b = binding()
    e = lambda *s: torch.ones(*s, device="cuda")   # noqa: E731
    ids = torch.zeros(3, dtype=torch.int32, device="cuda")
    Y, H = e(3, 5), e(3, 2)
    bias = torch.randn(5, device="cuda")
    b.lora_into(e(3, 0), e(0, 5), e(1, 0, 2), e(1, 2, 5), ids, Y, bias=bias, H=H)     # K = 0
    assert torch.equal(Y, bias.expand(3, 5)) and bool((H == 0).all())
    b.lora_into(e(0, 4), e(4, 5), e(1, 4, 2), e(1, 2, 5), ids[:0], e(0, 5))           # M = 0
    x, a = torch.randn(3, 4, device="cuda"), torch.randn(1, 4, 2, device="cuda")
    b.lora_into(x, e(4, 0), a, e(1, 2, 0), ids, e(3, 0), H=H)                         # N = 0
    assert torch.allclose(H, x @ a[0], atol=1e-5)
    dA, dB = torch.full((1, 4, 2), 7.0, device="cuda"), torch.full((1, 2, 5), 7.0, device="cuda")
    b.lora_backward_into(e(0, 5), e(0, 4), e(4, 5), e(1, 4, 2), e(1, 2, 5), ids[:0], e(0, 2),
                         dX=e(0, 4), dA=dA, dB=dB)
    assert bool((dA == 0).all()) and bool((dB == 0).all())
    dX = torch.full((3, 4), 7.0, device="cuda")
    b.lora_backward_into(e(3, 0), x, e(4, 0), a, e(1, 2, 0), ids, H, dX=dX, dA=dA, dB=e(1, 2, 0))
    assert bool((dX == 0).all()) and bool((dA == 0).all())
    assert b.device_status() == b.SGEMM_OK


BACKWARD = [  # (M, K, N, L, R, ids, padding, offset, kept in 8 bits)
    (1, 1, 1, 1, 1, "single", 0, 0, False), (1, 64, 128, 2, 8, "single", 0, 0, True),
    (7, 100, 77, 4, 5, "mixed", 3, 1, False), (40, 264, 136, 3, 16, "none", 0, 0, False),
    (64, 256, 128, 1, 128, "single", 0, 0, False), (65, 130, 257, 3, 20, "outside", 0, 0, True),
    (130, 512, 264, 2, 33, "runs", 8, 8, False), (256, 128, 512, 3, 64, "runs", 0, 0, True),
    (300, 520, 1000, 4, 24, "runs", 0, 0, False), (515, 264, 300, 6, 40, "mixed", 1, 3, True),
    (1100, 136, 520, 3, 16, "runs", 0, 0, False), (2500, 72, 200, 2, 65, "runs", 0, 0, True),
    (600, 96, 64, 300, 4, "mixed", 0, 0, False), (1025, 2056, 264, 1, 100, "single", 0, 0, False)]


WIDE = [(5000, K, 72, 3, 24, "mixed", 1, 1, True) for K in WIDTHS]   # tile widths, as above


def run_backward(p, H, pad=0, offset=0, kept=None, stack=True, dx=True):
    b, d = binding(), p.on_gpu(pad, offset)
    dX = p.out(p.M, p.K, pad, offset) if dx else None
    dA = dB = None
    if stack:
        nan = lambda *s: torch.full(s, float("nan"), dtype=p.dtype)   # noqa: E731
        dA, dB = device_stack(nan(p.L, p.K, p.R), pad, offset), device_stack(nan(p.L, p.R, p.N), pad, offset)
    b.lora_backward_into(d["dY"], d["X"] if kept is None else kept, d["W"], d["A"], d["B"], d["ids"],
                         H, dX=dX, dA=dA, dB=dB, scale=d["scale"], ranks=d["ranks"])
    assert b.device_status() == b.SGEMM_OK
    return dX, dA, dB


@pytest.mark.parametrize("M", [5, 13, 30, 60, 200])
@pytest.mark.parametrize("dtype", TYPES)
def test_infinities_and_nans_of_x_and_w_stay_in_their_row_and_column(M, dtype):
    p = Problem(M, 200, 264, 2, 8, dtype, "mixed", ranks=False)
    p.X[1, 7], p.X[3, 150], p.W[100, 9], p.W[101, 70] = float("inf"), float("nan"), float("-inf"), float("nan")
    Y, _ = run_forward(p, H=False)
    rows, cols = torch.ones(M, dtype=torch.bool), torch.ones(264, dtype=torch.bool)
    rows[[1, 3]], cols[[9, 70]] = False, False
    X, W = p.X.nan_to_num(0, 0, 0), p.W.nan_to_num(0, 0, 0)
    A, B = p.clean()
    ref, _, mag, _ = lora_reference(X, W, A, B, p.ids, p.scale, p.ranks, p.bias)
    Y = Y.cpu()
    assert not torch.isfinite(Y[~rows]).any() and not torch.isfinite(Y[:, ~cols]).any()
    assert_close(Y[rows][:, cols], ref[rows][:, cols], mag[rows][:, cols], p.K + p.R, f"Y {M}")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("case", BACKWARD + WIDE)
def test_backward(case, dtype):
    M, K, N, L, R, ids, pad, offset, x8 = case
    p = Problem(M, K, N, L, R, dtype, ids, seed=8)
    X, kept = p.X, None
    if x8:
        q, e = quantise(p.X)
        X, kept = values(q, e), (q.cuda(), e.cuda())
    A, B = p.clean()
    H = lora_reference(X, p.W, A, B, p.ids, p.scale, p.ranks, None)[1].float()
    dX, dA, dB = run_backward(p, device_matrix(H, pad), pad, offset, kept)
    rX, rA, rB, mX, mA, mB = lora_backward_reference(p.dY, X, p.W, A, B, p.ids, H, p.scale, p.ranks)
    assert_close(dX, rX, mX, N + R, f"dX {case}")
    assert_close(dA, rA, mA, M + N, f"dA {case}")
    assert_close(dB, rB, mB, M + 1, f"dB {case}")


def test_backward_in_parts():
    """dX alone and the stack's gradients alone are those of the whole call, bit for bit."""
    p = Problem(333, 136, 200, 3, 24, torch.float32)
    A, B = p.clean()
    H = lora_reference(p.X, p.W, A, B, p.ids, p.scale, p.ranks, None)[1].float().cuda()
    dX, dA, dB = run_backward(p, H)
    assert torch.equal(run_backward(p, H, stack=False)[0], dX)
    _, a, b = run_backward(p, H, dx=False)
    assert torch.equal(a, dA) and torch.equal(b, dB)


def test_gradients_against_differences():
    """loss = sum(V * Y) is linear in X, in A and in B one at a time, so (loss(+D) -
    loss(-D)) / 2 along D is the gradient's inner product with D, up to the fp32 rounding
    of Y (4e-6 of its norm, times V's) and of the gradient (the same, times D's)."""
    p = Problem(1500, 136, 264, 3, 16, torch.float32, ranks=False, bias=False)
    p.A, p.B = torch.nan_to_num(p.A), torch.nan_to_num(p.B)
    _, h = run_forward(p)
    grads = dict(zip("XAB", run_backward(p, h)))
    V = p.dY.double()
    for name in "XAB":
        start = getattr(p, name)
        D = torch.randn(start.shape, generator=torch.Generator().manual_seed(1))
        loss, size = [], 0.0
        for s in (1.0, -1.0):
            setattr(p, name, s * D)
            Y = run_forward(p)[0].cpu().double()
            loss.append((V * Y).sum())
            size = max(size, float(V.norm() * Y.norm()))
        setattr(p, name, start)
        quotient = float(loss[0] - loss[1]) / 2
        if name in "AB":          # the plain projection does not depend on D
            assert size > 0
        have = float((grads[name].cpu().double() * D.double()).sum())
        assert abs(have - quotient) <= 4e-6 * (size + float(grads[name].double().norm() * D.norm())), name


@pytest.mark.parametrize("M", [4, 48, 700, 1500])
@pytest.mark.parametrize("dtype", TYPES)
def test_repeats_are_bitwise_equal_on_any_stream(M, dtype):
    p = Problem(M, 264, 520, 4, 24, dtype, "mixed")
    Y, h = run_forward(p)
    grads = run_backward(p, h)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        Y2, h2 = run_forward(p)
        grads2 = run_backward(p, h2)
    Y3, _ = run_forward(p, H=False, stream=side)
    side.synchronize()
    assert torch.equal(Y, Y2) and torch.equal(h, h2) and torch.equal(Y, Y3)
    assert all(torch.equal(a, b) for a, b in zip(grads, grads2))


@pytest.mark.parametrize("M", [4, 48, 700, 1500])
def test_capture_in_a_graph(M):
    """A forward call captured once and replayed on new inputs."""
    b = binding()
    p = Problem(M, 264, 520, 4, 24, torch.bfloat16, "mixed")
    d = p.on_gpu(0, 0)
    Y = p.out(M, p.N, 0, 0)
    call = lambda: b.lora_into(d["X"], d["W"], d["A"], d["B"], d["ids"], Y, scale=d["scale"],   # noqa: E731
                               ranks=d["ranks"], bias=d["bias"])
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    p.X = torch.randn(p.X.shape, generator=torch.Generator().manual_seed(9)).to(p.dtype)
    d["X"].copy_(p.X)
    Y.zero_()
    graph.replay()
    torch.cuda.synchronize()
    check_forward(p, Y, None, "replayed")


def test_host_threads_on_their_own_streams():
    """Calls of every path from four threads at once give what they give alone."""
    import threading
    problems = [Problem(M, 264, 520, 3, 16, dtype, "mixed", seed=M)
                for M, dtype in ((3, torch.float32), (40, torch.float32), (100, torch.bfloat16), (700, torch.bfloat16))]
    want = []
    for p in problems:
        Y, h = run_forward(p)
        want.append((Y, h, *run_backward(p, h)))
    torch.cuda.synchronize()
    errors = []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(10):
                    Y, h = run_forward(problems[i])
                    got = (Y, h, *run_backward(problems[i], h))
                    torch.cuda.current_stream().synchronize()
                    assert all(torch.equal(a, b) for a, b in zip(got, want[i]))
        except Exception as e:   # noqa: BLE001  (reported by the main thread)
            errors.append(f"problem {i}: {e!r}")

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(problems))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


def test_long_stacks_and_strides():
    """X, Y and the stack as slices of wider tensors whose strides pass 2^31 elements."""
    b = binding()
    K, N, R, M = 64, 72, 8, 300
    wide = torch.zeros(M * 8_000_000, dtype=torch.bfloat16, device="cuda")   # 4.8 GB
    X = torch.as_strided(wide, (M, K), (8_000_000, 1))
    X.copy_(torch.randn(M, K))
    stack = torch.zeros(3 * 1_500_000_000, dtype=torch.bfloat16, device="cuda")   # 9 GB
    A = torch.as_strided(stack, (3, K, R), (1_500_000_000, R, 1))
    B = torch.as_strided(stack, (3, R, N), (1_500_000_000, N, 1), storage_offset=4096)
    A.copy_(torch.randn(3, K, R))
    B.copy_(torch.randn(3, R, N))
    W = torch.randn(K, N).to(torch.bfloat16).cuda()
    ids = row_ids(M, 3, "mixed", 4).cuda()
    got = b.lora_into(X, W, A, B, ids, torch.empty(M, N, dtype=torch.bfloat16, device="cuda"))
    few = b.lora_into(X[-5:], W, A, B, ids[-5:], torch.empty(5, N, dtype=torch.bfloat16, device="cuda"))
    ref, _, mag, _ = lora_reference(X.cpu(), W.cpu(), A.cpu(), B.cpu(), ids.cpu(), None, None, None)
    assert_close(got, ref, mag, K + R, "wide strides")
    assert_close(few, ref[-5:], mag[-5:], K + R, "wide strides, few rows")
    del wide, stack
    torch.cuda.empty_cache()
