"""The range-checked build over the norm's, the 8-bit product's and the gated block's tests: their cases run again, in
a process of their own, on the library that checks every index; any found out of range makes device_status()
fail there."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


def test_every_index_stays_in_range(cuda_device):
    from dense_fp32_gemm_02_gb300 import build
    build.build(debug_bounds=True)
    env = dict(os.environ, SGEMM_LIBRARY="debug_bounds", PYTHONPATH=os.path.dirname(HERE))
    check = ("from dense_fp32_gemm_02_gb300 import binding; "
             "assert binding.lib.sgemm_debug_bounds_checks() == 1; import pytest, sys; "
             "sys.exit(pytest.main(['-q', '-m', 'gpu', '-p', 'no:cacheprovider', "
             "'test_norm_gpu.py', 'test_linear8_gpu.py', 'test_gated_gpu.py']))")
    r = subprocess.run([sys.executable, "-c", check], env=env, cwd=HERE, capture_output=True, text=True, timeout=1200)
    assert r.returncode == 0, r.stdout[-4000:] + "\n" + r.stderr[-4000:]
