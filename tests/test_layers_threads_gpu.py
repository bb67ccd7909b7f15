"""Host threads whose layer calls need different amounts of shared memory of the same kernel."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_stacks_of_different_sizes_at_once(cuda_device):
    """Grouping the rows takes more shared memory the more adapters there are, past what a
    kernel has by default from 301 on: threads with 320, 700 and 1024 of them get what they get alone."""
    from dense_fp32_gemm_02_gb300 import binding as b
    M, K, N, R = 1500, 32, 40, 2
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")   # noqa: E731
    X, W = r(M, K), r(K, N)
    stacks = [(r(L, K, R), r(L, R, N), torch.randint(-1, L, (M,), generator=g, device="cuda", dtype=torch.int32))
              for L in (320, 1024, 700)]
    want = [b.lora_into(X, W, A, B, ids, torch.empty(M, N, device="cuda")) for A, B, ids in stacks]
    torch.cuda.synchronize()
    errors, start = [], threading.Barrier(len(stacks))

    def work(i):
        try:
            stream, Y = torch.cuda.Stream(), torch.empty(M, N, device="cuda")
            A, B, ids = stacks[i]
            start.wait()
            for _ in range(500):
                b.lora_into(X, W, A, B, ids, Y, stream=stream)
            stream.synchronize()
            assert torch.equal(Y, want[i])
        except Exception as e:   # noqa: BLE001  (reported by the main thread)
            errors.append(f"thread {i}: {e!r}")

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(stacks))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    assert b.device_status() == b.SGEMM_OK
