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
