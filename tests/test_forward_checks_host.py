"""The range-checked build checks the norm's, the 8-bit product's and the gated block's kernels, and their launches
keep the order of waits (on the CPU, from the sources; test_forward_bounds_gpu.py runs the checks)."""
import os
import re

import pytest

import test_layers_checks_host as layers

FILES = ["norm.cuh", "gated.cuh", "linear8.cuh", "byte_tiles.cuh", "byte_rows.cuh", "split_tiles.cuh", "gated_tiles.cuh", "pair_gemm.cuh"]


def functions():
    """name -> (is a kernel, body), of these files' functions and of the ones they call."""
    found = dict(layers.FUNCTIONS)
    for name in FILES:
        with open(os.path.join(layers.CSRC, name)) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for m in re.finditer(r"\n(?:template <[^\n]*>\n)?((?:static )?(?:__global__|__device__)[^;{}]*?)\b(\w+)\(([^;{}]*)\)\s*(?:-> [^{]*)?\{", text):
            depth, end = 1, m.end()
            while depth:
                depth += {"{": 1, "}": -1}.get(text[end], 0)
                end += 1
            head = re.sub(r"__(?:launch_bounds|cluster_dims)__\((?:[^()]|\((?:[^()]|\([^()]*\))*\))*\)", "", m.group(0))
            found[re.search(r"(\w+)\s*\(", head).group(1)] = ("__global__" in m.group(1), text[m.end():end])
    return found


FUNCTIONS = functions()
KERNELS = sorted(n for n, (kernel, _) in FUNCTIONS.items() if kernel and n not in layers.KERNELS)


def checks(name, seen=()):
    body = FUNCTIONS[name][1]
    return "SG_IN_RANGE" in body or any(
        checks(f, (*seen, name)) for f in FUNCTIONS if f != name and f not in seen and re.search(rf"\b{f}\b\s*[<(]", body))


def test_the_kernels_are_found():
    assert {"norm_kernel", "norm_backward_kernel", "norm_weight_kernel", "gated_stream_kernel", "gated_few_rows_kernel",
            "pair_finish_kernel", "gated_slopes_kernel", "byte_finish_kernel", "byte_expand_kernel", "byte_tiles_kernel", "byte_pitch_kernel",
            "pair_gemm_kernel", "byte_rows_kernel", "gated_parts_kernel", "split_tiles_kernel",
            "gated_tiles_kernel"} == set(KERNELS)


@pytest.mark.parametrize("kernel", KERNELS)
def test_every_kernel_checks_its_indices(kernel):
    assert checks(kernel), f"{kernel} asks SG_IN_RANGE about nothing"


def test_early_kernels_wait_before_they_let_the_next_one_start():
    """As for the layers' kernels; here a call's first kernel is launched early as well, and waits before it lets the
    second one start, so that all earlier work has ended by then."""
    never_first = {"byte_expand_kernel",      # X's form; W's, the call's first, waits
                   "split_tiles_kernel"}      # its parts of X are laid out first, by a kernel that waits
    for name in KERNELS:
        body = FUNCTIONS[name][1]
        wait, let = body.find("wait_prerequisites()"), body.find("launch_dependents()")
        if let >= 0 and name not in never_first:
            assert 0 <= wait < let, name
    for unit in ("norm.cu", "linear8.cu", "gated.cu", "pair_gemm.cu"):
        with open(os.path.join(layers.CSRC, unit)) as f:
            assert "<<<" not in f.read(), unit
