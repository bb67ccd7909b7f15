"""The norm, the 8-bit product and the gated block as a program uses them: one after the other, on streams, in graphs,
at once from several threads, on views; and what they refuse."""
import threading

import pytest
import torch

from _forward import (EPS, act_reference, gated_backward_reference, gated_reference, linear8_reference, norm_backward_reference,
                      norm_reference, norm_slack, rounded, rows8_reference, stream_of)
from test_layers_views_gpu import overlapping

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16]


@pytest.fixture(scope="module", autouse=True)
def _gpu(cuda_device):
    yield


def binding():
    from dense_fp32_gemm_02_gb300 import binding
    return binding


def rnd(*shape, dtype=torch.float32, seed=0, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def bytes_of(rows, cols, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randint(-127, 128, (rows, cols), generator=g, device="cuda", dtype=torch.int32).to(torch.int8)


def calls(M, K, N, dtype):
    """name -> (inputs that may change, outputs, call)."""
    b = binding()
    z = lambda *s, seed=1, scale=1.0: rnd(*s, dtype=dtype, seed=seed, scale=scale)   # noqa: E731
    X, R, w, S, Y = z(M, K), z(M, K, seed=2), z(K, seed=3), z(M, K), z(M, K)
    q, scale = torch.zeros(M, K, dtype=torch.int8, device="cuda"), torch.zeros(M, device="cuda")
    dY, dS, dX, dw = z(M, K, seed=4), z(M, K, seed=5), z(M, K), z(K)
    W8, ws, bias, Z = bytes_of(K, N, 6), torch.rand(N, device="cuda") + 0.1, z(N, seed=7), z(M, N)
    Wg, Wu, H, G, U, dH = z(K, N, seed=8, scale=0.05), z(K, N, seed=9, scale=0.05), z(M, N), z(M, N), z(M, N), z(M, N, seed=10)
    dWg, dWu = z(K, N), z(K, N)
    q0, s0 = bytes_of(M, K, 11), torch.rand(M, device="cuda") + 0.1
    return {
        "norm": ([X, R, w], [S, Y, q, scale], lambda **k: b.rmsnorm_into(X, w, Y=Y, q=q, scale=scale, R=R, S=S, **k)),
        "norm_backward": ([X, dY, w, dS], [dX, dw], lambda **k: b.rmsnorm_backward_into(dY, X, w, dX, dw=dw, dS=dS, **k)),
        "linear8": ([ws, bias], [Z], lambda **k: b.linear8_into((q0, s0), W8, ws, Z, bias=bias, **k)),
        "linear8_rows": ([X, ws], [Z], lambda **k: b.linear8_into(X, W8, ws, Z, **k)),
        "gated": ([X, Wg, Wu], [H, G, U], lambda **k: b.gated_into(X, Wg, Wu, H, G=G, U=U, **k)),
        "gated_backward": ([X, Wg, Wu, dH], [dX, dWg, dWu],
                           lambda **k: b.gated_backward_into(dH, X, Wg, Wu, G, U, dX=dX, dWg=dWg, dWu=dWu, **k)),
    }


NAMES = ["norm", "norm_backward", "linear8", "linear8_rows", "gated", "gated_backward"]
SHAPES = [(1, 264, 520), (8, 1024, 256), (20, 70, 130), (60, 264, 520), (300, 512, 264), (1100, 136, 200)]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("name", NAMES)
def test_captured_and_replayed(name, shape, dtype):
    """Two graphs of a call, replayed in turn with eager calls between, on new inputs: bit for bit what the call gives."""
    inputs, outputs, call = calls(*shape, dtype)[name]
    call()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
            call()
        graphs.append(g)
    for seed, g in enumerate((*graphs, *graphs)):
        for n, t in enumerate(inputs):
            t.copy_(rnd(*t.shape, seed=100 * seed + n))
        for t in outputs:
            t.fill_(55)
        call()
        torch.cuda.synchronize()
        want = [t.clone() for t in outputs]
        for t in outputs:
            t.fill_(77)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, t) for a, t in zip(want, outputs))
    assert binding().device_status() == 0


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("name", NAMES)
def test_on_a_stream_of_its_own(name, dtype):
    """Behind work of that stream that writes an input, without waiting for the host."""
    inputs, outputs, call = calls(300, 512, 264, dtype)[name]
    fresh = [rnd(*t.shape, seed=50 + n).to(t.dtype) for n, t in enumerate(inputs)]
    for t, x in zip(inputs, fresh):
        t.copy_(x)
    call()
    torch.cuda.synchronize()
    want = [t.clone() for t in outputs]
    stream = torch.cuda.Stream()
    for t in (*inputs, *outputs):
        t.fill_(3)
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        busy = torch.randn(4096, 4096, device="cuda")
        for _ in range(4):
            busy = busy @ busy * 1e-3
        for t, x in zip(inputs, fresh):
            t.copy_(x)
    call(stream=stream)
    with torch.cuda.stream(stream):
        got = [t.clone() for t in outputs]
        for t in inputs:      # the call's work is enqueued: what comes behind it may overwrite its inputs
            t.fill_(9)
    stream.synchronize()
    assert all(torch.equal(a, t) for a, t in zip(want, got))
    torch.cuda.synchronize()


def test_back_to_back_calls_that_depend_on_one_another():
    """A call's input is what the call before it wrote, with early launches on both sides, many times over."""
    b = binding()
    for M, K in ((1, 1024), (40, 512), (300, 512)):
        W8, ws = bytes_of(K, K, 1), torch.full((K,), 0.02 / K ** 0.5, device="cuda")
        w = torch.ones(K, device="cuda")
        Wg, Wu = rnd(K, K, seed=2, scale=K ** -0.5), rnd(K, K, seed=3, scale=K ** -0.5)

        def run():
            x = rnd(M, K, seed=4)
            y, q, s = torch.empty_like(x), torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
            for _ in range(20):
                b.rmsnorm_into(x, w, q=q, scale=s)
                b.linear8_into((q, s), W8, ws, y)
                b.linear8_into(y, W8, ws, x)
                b.gated_into(x, Wg, Wu, y)
                b.rmsnorm_into(y, w, Y=x)
            torch.cuda.synchronize()
            return x

        def slow():
            x = rnd(M, K, seed=4)
            y, q, s = torch.empty_like(x), torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
            for _ in range(20):
                for step in (lambda: b.rmsnorm_into(x, w, q=q, scale=s), lambda: b.linear8_into((q, s), W8, ws, y),
                             lambda: b.linear8_into(y, W8, ws, x), lambda: b.gated_into(x, Wg, Wu, y),
                             lambda: b.rmsnorm_into(y, w, Y=x)):
                    step()
                    torch.cuda.synchronize()
            return x
        assert torch.equal(run(), slow())


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_at_once_from_several_threads(dtype):
    sizes = [(1, 264, 520), (40, 512, 264), (300, 264, 520), (9, 70, 2000)]
    work = [calls(*s, dtype) for s in sizes]
    want = []
    for c in work:
        want.append({})
        for name in NAMES:
            c[name][2]()
            torch.cuda.synchronize()
            want[-1][name] = [t.clone() for t in c[name][1]]
    errors, start = [], threading.Barrier(len(sizes))

    def go(n):
        try:
            stream = torch.cuda.Stream()
            start.wait()
            for _ in range(20):
                for name in NAMES:
                    work[n][name][2](stream=stream)
                    stream.synchronize()
                    if not all(torch.equal(a, t) for a, t in zip(want[n][name], work[n][name][1])):
                        errors.append(f"{sizes[n]} {name}")
        except Exception as e:   # noqa: BLE001  (reported by the main thread)
            errors.append(repr(e))
    threads = [threading.Thread(target=go, args=(n,)) for n in range(len(sizes))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors[:5]
    assert binding().device_status() == 0


# ------------------------------------------------------------------ one after the other
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("M", [1, 7, 64, 700])
def test_a_served_block(M, dtype):
    """residual + norm -> rows in 8 bits -> gate and up projections in 8 bits -> activation -> down projection in 8
    bits, each step against its definition on what the step before gave."""
    b, K, N = binding(), 264, 520
    X, R, w = rnd(M, K, dtype=dtype, seed=1), rnd(M, K, dtype=dtype, seed=2), (1 + 0.2 * rnd(K, seed=3)).to(dtype)
    Wg, Wu, Wd = bytes_of(K, N, 4), bytes_of(K, N, 5), bytes_of(N, K, 6)
    sg, su, sd = (torch.rand(n, device="cuda") * 0.01 for n in (N, N, K))
    S, q, scale = torch.empty_like(X), torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    b.rmsnorm_into(X, w, q=q, scale=scale, R=R, S=S)
    V = stream_of(X.cpu(), R.cpu())
    assert torch.equal(S.cpu(), V)
    assert torch.equal(q.cpu(), rows8_reference(V.double() * w.cpu().double())[0])
    G, U = torch.empty(M, N, dtype=dtype, device="cuda"), torch.empty(M, N, dtype=dtype, device="cuda")
    b.linear8_into((q, scale), Wg, sg, G)
    b.linear8_into((q, scale), Wu, su, U)
    for got, W8, s in ((G, Wg, sg), (U, Wu, su)):
        ref, mag = linear8_reference(q, scale, W8, s, None)
        rounded(got, ref.cpu(), 4 * 2.0 ** -24 * mag.cpu(), "projection")
    H = (act_reference(G, "silu")[0] * U.double()).to(dtype)
    out = torch.empty(M, K, dtype=dtype, device="cuda")
    b.linear8_into(H, Wd, sd, out)
    ref, mag = linear8_reference(*rows8_reference(H.cpu()), Wd.cpu(), sd.cpu(), None)
    rounded(out, ref, 5 * 2.0 ** -24 * mag, "down")


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_a_trained_block(dtype):
    """residual + norm -> gated block -> down projection (the adapter layer without adapters), forward and backward,
    the gradients of the whole against differences of the whole in 64 bits (float32), and step by step."""
    b, M, K, N = binding(), 40, 24, 56
    X, R, w = rnd(M, K, dtype=dtype, seed=1), rnd(M, K, dtype=dtype, seed=2), (1 + 0.2 * rnd(K, seed=3)).to(dtype)
    Wg, Wu, Wd = (rnd(*s, dtype=dtype, seed=4 + n, scale=s[0] ** -0.5) for n, s in enumerate(((K, N), (K, N), (N, K))))
    e = lambda *s: torch.empty(*s, dtype=dtype, device="cuda")   # noqa: E731
    S, Y, H, G, U, O = e(M, K), e(M, K), e(M, N), e(M, N), e(M, N), e(M, K)
    none = X.new_empty(0, N, 1), X.new_empty(0, 1, K)
    b.rmsnorm_into(X, w, Y=Y, R=R, S=S)
    b.gated_into(Y, Wg, Wu, H, G=G, U=U)
    b.lora_into(H, Wd, *none, None, O)
    dO = rnd(M, K, dtype=dtype, seed=9)
    dH, dYn, dX, dw, dWg, dWu = e(M, N), e(M, K), e(M, K), e(K), e(K, N), e(K, N)
    b.lora_backward_into(dO, None, Wd, *none, None, None, dX=dH)
    b.gated_backward_into(dH, Y, Wg, Wu, G, U, dX=dYn, dWg=dWg, dWu=dWu)
    b.rmsnorm_backward_into(dYn, S, w, dX, dw=dw, dS=dO)      # the stream goes on past the block
    h, _, _, sh, _, _ = (t.cpu() for t in gated_reference(Y, Wg, Wu, "silu"))
    rounded(H, h, sh, "H")
    x, g, u, sx, sg, su = (t.cpu() for t in gated_backward_reference(dH, Y, Wg, Wu, G, U, "silu"))
    for got, ref, slack in ((dYn, x, sx), (dWg, g, sg), (dWu, u, su)):
        rounded(got, ref, slack, "gated gradient")
    ref, ref_w, mag, mag_w = norm_backward_reference(dYn.cpu(), S.cpu(), w.cpu(), dO.cpu(), EPS)
    rounded(dX, ref, 200 * 2.0 ** -24 * mag, "dX")
    rounded(dw, ref_w, 200 * 2.0 ** -24 * mag_w, "dw")
    if dtype != torch.float32:
        return
    at = [t.double().cpu() for t in (X, R, w, Wg, Wu, Wd)]

    def loss(X, R, w, Wg, Wu, Wd):
        V = X + R
        y = norm_reference(V, w, EPS)
        o = (act_reference(y @ Wg, "silu")[0] * (y @ Wu)) @ Wd
        return float(((o + V) * dO.double().cpu()).sum())
    for which, got in ((0, dX), (1, dX), (2, dw), (3, dWg), (4, dWu)):
        for n in range(0, got.numel(), 37):
            ends = []
            for step in (-1e-5, 1e-5):
                moved = [t.clone() for t in at]
                moved[which].view(-1)[n] += step
                ends.append(loss(*moved))
            # the difference's own error, and float32's through the block: sums of up to 56 terms of order 1
            assert abs((ends[1] - ends[0]) / 2e-5 - float(got.view(-1)[n])) < 2e-4


# ------------------------------------------------------------------ refusals
@pytest.mark.parametrize("name", NAMES)
def test_overlapping_rows_are_refused(name):
    b, M, K, N = binding(), 8, 64, 96
    z = lambda *s, **k: torch.zeros(*s, device="cuda", **k)   # noqa: E731
    i8 = lambda r, c: z(r, c, dtype=torch.int8)   # noqa: E731
    fn, given = {
        "norm": (b.rmsnorm_into, dict(X=z(M, K), w=z(K), Y=z(M, K), q=i8(M, K), scale=z(M), R=z(M, K), S=z(M, K))),
        "norm_backward": (b.rmsnorm_backward_into, dict(dY=z(M, K), V=z(M, K), w=z(K), dX=z(M, K), dw=z(K), dS=z(M, K))),
        "linear8": (lambda q, scale, **k: b.linear8_into((q, scale), **k),
                    dict(q=i8(M, K), scale=z(M), W=i8(K, N), wscale=z(N), Y=z(M, N))),
        "linear8_rows": (b.linear8_into, dict(X=z(M, K), W=i8(K, N), wscale=z(N), Y=z(M, N))),
        "gated": (b.gated_into, dict(X=z(M, K), Wg=z(K, N), Wu=z(K, N), H=z(M, N), G=z(M, N), U=z(M, N))),
        "gated_backward": (b.gated_backward_into, dict(dH=z(M, N), X=z(M, K), Wg=z(K, N), Wu=z(K, N), G=z(M, N), U=z(M, N),
                                                       dX=z(M, K), dWg=z(K, N), dWu=z(K, N))),
    }[name]
    fn(**given)
    launches = b.kernel_launch_count()
    for what, t in given.items():
        if t.dim() == 1:
            continue
        for view in overlapping(t.shape, t.dtype):
            with pytest.raises(ValueError, match=f"{what}: rows must not overlap"):
                fn(**{**given, what: view})
        with pytest.raises(ValueError, match=f"{what}: rows must be contiguous"):
            fn(**{**given, what: t.new_zeros(t.shape[1], t.shape[0]).t()})
        with pytest.raises(ValueError, match=f"{what} must be|must be"):
            fn(**{**given, what: t[:, :-1] if what not in ("X", "dY", "dH", "Y", "W", "Wg") else t[0]})
        if t.is_floating_point():
            if name != "linear8":      # (rows in 8 bits have no type that Y's could differ from)
                with pytest.raises(TypeError):
                    fn(**{**given, what: t.to(torch.bfloat16)})
            with pytest.raises((TypeError, ValueError)):
                fn(**{**given, what: t.cpu()})
    assert b.kernel_launch_count() == launches
    torch.cuda.synchronize()
    assert b.device_status() == b.SGEMM_OK


def test_what_must_be_given_together_and_at_least():
    b = binding()
    x, w = rnd(4, 64), rnd(64)
    q, s = torch.empty(4, 64, dtype=torch.int8, device="cuda"), torch.empty(4, device="cuda")
    with pytest.raises(ValueError, match="given together"):
        b.rmsnorm_into(x, w, q=q)
    with pytest.raises(ValueError, match="given together"):
        b.rmsnorm_into(x, w, Y=torch.empty_like(x), scale=s)
    with pytest.raises(ValueError, match="needs an output"):
        b.rmsnorm_into(x, w)
    with pytest.raises(ValueError, match="eps must be"):
        b.rmsnorm_into(x, w, Y=torch.empty_like(x), eps=-1.0)
    with pytest.raises(b.SgemmError):
        b.rmsnorm_into(x, w, Y=x, S=x)
    with pytest.raises(ValueError, match="given together"):
        b.gated_into(x, rnd(64, 8), rnd(64, 8), rnd(4, 8), G=rnd(4, 8))
    with pytest.raises(ValueError, match="act must be"):
        b.gated_into(x, rnd(64, 8), rnd(64, 8), rnd(4, 8), act="tanh")
    with pytest.raises(ValueError, match="pair"):
        b.linear8_into((q,), torch.empty(64, 8, dtype=torch.int8, device="cuda"), rnd(8), rnd(4, 8))
    with pytest.raises(b.SgemmError) as e:
        k = 131072
        b.linear8_into((torch.zeros(1, k, dtype=torch.int8, device="cuda"), rnd(1)), torch.zeros(k, 8, dtype=torch.int8, device="cuda"),
                       rnd(8), rnd(1, 8))
    assert e.value.status == b.SGEMM_ERR_TOO_LARGE
    assert b.device_status() == 0


def test_rows_past_2_31_elements():
    """Outputs whose last rows lie past 2^31 elements; the same last rows alone give the same."""
    b = binding()
    M, K, N = 530000, 64, 4104
    X, Wg, Wu = rnd(M, K, dtype=torch.bfloat16, seed=1), rnd(K, N, dtype=torch.bfloat16, seed=2), rnd(K, N, dtype=torch.bfloat16, seed=3)
    H = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    b.gated_into(X, Wg, Wu, H)
    few = b.gated_into(X[-300:], Wg, Wu, torch.empty(300, N, dtype=torch.bfloat16, device="cuda"))
    assert torch.equal(H[-300:], few)
    dX, dWg, dWu = torch.empty_like(X), torch.empty_like(Wg), torch.empty_like(Wu)
    b.gated_backward_into(H, X, Wg, Wu, H, H, dX=dX)
    few = b.gated_backward_into(H[-300:], X[-300:], Wg, Wu, H[-300:], H[-300:], dX=torch.empty(300, K, dtype=torch.bfloat16, device="cuda"))
    # (the ranges of the contraction may differ with the rows: one rounding of the output, and sums' order)
    ref, _, _, slack, _, _ = gated_backward_reference(H[-300:], X[-300:], Wg, Wu, H[-300:], H[-300:], "silu")
    rounded(dX[-300:], ref.cpu(), slack.cpu(), "dX")
    rounded(few[0], ref.cpu(), slack.cpu(), "dX of the last rows alone")
    W8, ws, q, s = bytes_of(K, N, 4), torch.rand(N, device="cuda"), bytes_of(M, K, 5), torch.rand(M, device="cuda")
    b.linear8_into((q, s), W8, ws, H)
    few = b.linear8_into((q[-300:], s[-300:]), W8, ws, torch.empty(300, N, dtype=torch.bfloat16, device="cuda"))
    assert torch.equal(H[-300:], few)
    assert b.device_status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("M", [1, 4, 33, 64, 65, 150, 300])
def test_calls_close_behind_one_another(M, dtype):
    """Each call reads what the one before it writes, and writes what an earlier one still reads: the same bits as with the
    device waited for after every call, in a stream and in a graph, where kernels start before the last one's end."""
    b, D, F = binding(), 520, 1000
    layers = [dict(w=(1 + 0.1 * rnd(D, seed=20 + i)).to(dtype), Wg=rnd(D, F, dtype=dtype, seed=30 + i) * 0.05,
                   Wu=rnd(D, F, dtype=dtype, seed=40 + i) * 0.05, Wd=bytes_of(F, D, 50 + i), Wq=bytes_of(D, D, 60 + i),
                   s=torch.rand(D, device="cuda") * 1e-3) for i in range(3)]
    X = rnd(M, D, dtype=dtype, seed=70)

    def e(*shape, t=dtype):
        return torch.empty(*shape, dtype=t, device="cuda")
    S, Y, A, O, dX, dV, H, G, U = (*(e(M, D) for _ in range(6)), *(e(M, F) for _ in range(3)))
    q, scale, dw, dWg, dWu = e(M, D, t=torch.int8), e(M, t=torch.float32), e(D), e(D, F), e(D, F)

    def chain(wait):
        S.copy_(X)
        O.zero_()
        for p in layers:
            for step in (lambda: b.rmsnorm_into(S, p["w"], q=q, scale=scale, R=O, S=S),
                         lambda: b.linear8_into((q, scale), p["Wq"], p["s"], A),
                         lambda: b.rmsnorm_into(A, p["w"], Y=Y, R=S, S=S),
                         lambda: b.gated_into(Y, p["Wg"], p["Wu"], H, G=G, U=U),
                         lambda: b.linear8_into(H, p["Wd"], p["s"], O),
                         lambda: b.gated_backward_into(H, Y, p["Wg"], p["Wu"], G, U, dX=dX, dWg=dWg, dWu=dWu),
                         lambda: b.rmsnorm_backward_into(dX, S, p["w"], dV, dw=dw, dS=O),
                         lambda: b.gated_into(dV, p["Wg"], p["Wu"], H)):
                step()
                if wait:
                    torch.cuda.synchronize()
        return [t.clone() for t in (S, O, H, dV, dw, dWg, dWu, A)]
    ref = chain(True)
    assert all(bool(torch.isfinite(t).all()) for t in ref)
    for _ in range(6):
        assert all(torch.equal(x, y) for x, y in zip(chain(False), ref))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = chain(False)
    for _ in range(4):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, ref))
    assert b.device_status() == 0
