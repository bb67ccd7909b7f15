"""Calls of the layers that meet: from threads at once, and one after another that CUDA refused."""
import ctypes
import subprocess

import pytest
import torch

from _forward import linear8_reference, rounded

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu(cuda_device):
    yield


def binding():
    from dense_fp32_gemm_02_gb300 import binding
    return binding


# ------------------------------------------------------------------ shared memory
# Calls from threads without the interpreter's lock between them: how many of each thread's were refused.
CALLER = """
#include <thread>
#include <vector>
struct Call { int M, N, K; const signed char *q, *W; const float *scale, *wscale; void *Y, *stream; int refused; };
using Entry = int (*)(int, int, int, int, const void *, int, const signed char *, int, const float *, const signed char *, int,
                      const float *, const void *, void *, int, void *);
extern "C" void call_at_once(Entry entry, Call *calls, int threads, int times) {
    std::vector<std::thread> all;
    for (int i = 0; i < threads; ++i)
        all.emplace_back([=] {
            Call &c = calls[i];
            for (int n = 0; n < times; ++n)
                c.refused += 0 != entry(0, c.M, c.N, c.K, nullptr, 0, c.q, c.K, c.scale, c.W, c.N, c.wscale, nullptr, c.Y, c.N, c.stream);
        });
    for (auto &t : all) t.join();
}
"""


class Call(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in "MNK"] + [(n, ctypes.c_void_p) for n in ("q", "W", "scale", "wscale", "Y", "stream")] + [
        ("refused", ctypes.c_int)]


def test_streamed_products_of_several_lengths_at_once(tmp_path):
    """Three and four rows by two lengths of the same kernel, that take 48 and 64 KB of shared memory, from threads at
    once: none lowers the limit under another's launch."""
    source, library = tmp_path / "caller.cpp", tmp_path / "libcaller.so"
    source.write_text(CALLER)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-pthread", "-o", str(library), str(source)], check=True)
    b, N = binding(), 32000
    shapes = ((4, 8192), (3, 4096), (4, 4096), (3, 8192))
    calls, work = (Call * len(shapes))(), []
    for n, (M, K) in enumerate(shapes):
        g = torch.Generator(device="cuda")
        g.manual_seed(n)
        q, W = (torch.randint(-127, 128, s, generator=g, device="cuda", dtype=torch.int32).to(torch.int8) for s in ((M, K), (K, N)))
        scale, ws = torch.rand(M, generator=g, device="cuda"), torch.rand(N, generator=g, device="cuda")
        Y = b.linear8_into((q, scale), W, ws, torch.empty(M, N, device="cuda"))
        ref, mag = linear8_reference(q, scale, W[:, :500], ws[:500], None)
        rounded(Y[:, :500], ref.cpu(), 4 * 2.0 ** -24 * mag.cpu(), "product")
        stream = torch.cuda.Stream()
        calls[n] = Call(M, N, K, q.data_ptr(), W.data_ptr(), scale.data_ptr(), ws.data_ptr(), Y.data_ptr(), stream.cuda_stream, 0)
        work.append((Y, Y.clone(), (q, W, scale, ws, stream)))
    torch.cuda.synchronize()
    ctypes.CDLL(str(library)).call_at_once(ctypes.cast(b.lib.sgemm_linear8, ctypes.c_void_p), calls, len(shapes), 3000)
    torch.cuda.synchronize()
    assert [c.refused for c in calls] == [0] * len(shapes)
    assert all(torch.equal(Y, want) for Y, want, _ in work)
    assert b.device_status() == 0


# ------------------------------------------------------------------ after a refused call
def refuse(call):
    """Makes `call(stream)` in a capture that has been invalidated, where CUDA refuses its launch."""
    driver = ctypes.CDLL("libcuda.so.1")
    stream = torch.cuda.Stream()
    handle, graph = ctypes.c_void_p(stream.cuda_stream), ctypes.c_void_p()
    assert driver.cuStreamBeginCapture_v2(handle, 1) == 0      # (thread-local mode)
    try:
        assert driver.cuStreamSynchronize(handle) != 0         # not permitted in a capture: invalidates it
        call(stream)
    finally:
        driver.cuStreamEndCapture(handle, ctypes.byref(graph))


def normal(rows, cols, seed, scale=1.0):
    g = torch.Generator()
    g.manual_seed(seed)
    return torch.randn(rows, cols, generator=g) * scale


def test_a_call_after_one_that_was_refused():
    """A launch that CUDA refuses fails its own call alone: the next one, of one kernel or of several, does its work."""
    b = binding()
    X, w = normal(40, 512, 1).cuda(), torch.ones(512, device="cuda")
    Wg, Wu = normal(512, 300, 2, 0.05).cuda(), normal(512, 300, 3, 0.05).cuda()
    e = torch.empty
    q8, e8 = e(40, 512, dtype=torch.int8, device="cuda"), e(40, 16, dtype=torch.int8, device="cuda")
    q, s, W8 = e(40, 512, dtype=torch.int8, device="cuda"), e(40, device="cuda"), torch.ones(512, 300, dtype=torch.int8, device="cuda")
    rows8, ones = b.rmsnorm_into(X, w, q=q, scale=s)[2:], torch.ones(300, device="cuda")
    calls = {
        "norm": ([e(40, 512, device="cuda")], lambda out, stream: b.rmsnorm_into(X, w, Y=out[0], stream=stream)),
        "gated": ([e(40, 300, device="cuda")], lambda out, stream: b.gated_into(X, Wg, Wu, out[0], stream=stream)),
        "linear8": ([e(40, 300, device="cuda")], lambda out, stream: b.linear8_into(rows8, W8, ones, out[0], stream=stream)),
        "sgemm": ([e(40, 300, device="cuda")], lambda out, stream: b.sgemm_into(X, Wg, out[0], stream=stream)),
        "act8": ([q8, e8], lambda out, stream: b.act8_store_into(X, out[0], out[1], stream=stream)),
    }
    for name, (out, call) in calls.items():
        call(out, None)
        want = [t.clone() for t in out]
        for refused in calls:
            with pytest.raises(b.SgemmError):
                refuse(lambda stream: calls[refused][1](calls[refused][0], stream))
            for t in out:
                t.fill_(55)
            call(out, None)               # raises nothing
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(out, want)), (name, refused)
    assert b.device_status() == 0
