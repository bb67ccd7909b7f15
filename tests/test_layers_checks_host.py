"""The range-checked build checks the layer kernels too: every kernel of their sources, itself or
in the functions that it calls, asks SG_IN_RANGE about what it reads or writes (on the CPU, from
the sources; what the checks say at run time is test_layers_bounds_gpu.py's)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "dense_fp32_gemm_02_gb300", "csrc")
FILES = ["act8.cu", "lora.cuh", "rank_products.cuh", "rows.cuh", "parts_gemm.cuh"]


def functions():
    """name -> (is a kernel, body) of the functions of the layer sources."""
    found = {}
    for name in FILES:
        with open(os.path.join(CSRC, name)) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for m in re.finditer(r"\n(?:template <[^\n]*>\n)?((?:__global__|__device__)[^;{}]*?)\b(\w+)\(([^;{}]*)\)\s*\{", text):
            depth, end = 1, m.end()
            while depth:
                depth += {"{": 1, "}": -1}.get(text[end], 0)
                end += 1
            kernel = "__global__" in m.group(1)
            head = m.group(0)
            if kernel:   # the name is the word before the first parenthesis that no attribute owns
                head = re.sub(r"__(?:launch_bounds|cluster_dims)__\((?:[^()]|\([^()]*\))*\)", "", head)
            at = re.search(r"(\w+)\s*\(", head)
            found[at.group(1)] = (kernel, text[m.end():end])
    return found


FUNCTIONS = functions()


def checks(name, seen=()):
    body = FUNCTIONS[name][1]
    return "SG_IN_RANGE" in body or any(
        checks(f, (*seen, name)) for f in FUNCTIONS
        if f != name and f not in seen and re.search(rf"\b{f}\b\s*[<(]", body))


KERNELS = sorted(n for n, (kernel, _) in FUNCTIONS.items() if kernel)


def test_the_kernels_are_found():
    assert {"store_wide_kernel", "store_any_kernel", "read_wide_kernel", "read_any_kernel", "parts_kernel",
            "group_rows_kernel", "pack_stack_kernel", "rank_finish_kernel", "stack_tile_kernel",
            "stack_finish_kernel", "stream_rows_kernel", "few_rows_kernel", "few_rows_rank_kernel",
            "few_rows_finish_kernel", "parts_gemm_kernel", "finish_kernel"} == set(KERNELS)


@pytest.mark.parametrize("kernel", KERNELS)
def test_every_kernel_checks_its_indices(kernel):
    assert checks(kernel), f"{kernel} asks SG_IN_RANGE about nothing"


def test_local_arrays_read_as_vectors_are_aligned():
    """A local array that is read or written through a vector pointer has the vector's alignment
    (in registers it makes no difference, in local memory it would)."""
    size = {"uint2": 8, "uint4": 16, "float2": 8, "float4": 16}
    seen = 0
    for name in FILES:
        with open(os.path.join(CSRC, name)) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for m in re.finditer(r"reinterpret_cast<(?:const )?(\w+) \*>\((\w+)\)", text):
            vector, array = m.group(1), m.group(2)
            local = list(re.finditer(rf"(alignas\((\d+)\) )?\b(?:T|E|float|bf16|uint32_t|signed char) {array}\[", text[:m.start()]))
            if vector not in size or not local:
                continue
            seen += 1
            assert int(local[-1].group(2) or 0) >= size[vector], f"{name}: {array} as {vector}"
    assert seen >= 3


def test_early_kernels_wait_before_they_let_the_next_one_start():
    """A call's first kernel may let the second start only when all earlier work has ended, that
    is behind its own wait.  The others: launched plainly (so that wait is the launch's), or never
    first in a call."""
    plain, never_first = {"stream_rows_kernel", "few_rows_kernel"}, {"few_rows_rank_kernel"}
    for name in KERNELS:
        body = FUNCTIONS[name][1]
        wait, let = body.find("wait_prerequisites()"), body.find("launch_dependents()")
        if let >= 0 and name not in plain | never_first:
            assert 0 <= wait < let, name
    with open(os.path.join(CSRC, "lora.cu")) as f:
        text = f.read()
    for name in ("stream", "kernel"):     # what forward_few_rows calls those two
        assert re.search(rf"\b{name}<<<", text)
    assert "launch_early(stream" not in text and "launch_early(kernel" not in text.replace("launch_early(kernel, grid", "")
