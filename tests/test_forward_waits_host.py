"""The early launches of the norm's, the 8-bit product's and the gated block's calls, from the sources: what each kernel
that may start beside the one before it does ahead of its wait (host_state.h)."""
import os
import re

from test_forward_checks_host import FUNCTIONS, KERNELS
from test_layers_checks_host import CSRC


def body(name):
    return re.sub(r"\s+", " ", FUNCTIONS[name][1])


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"\s+", " ", re.sub(r"//[^\n]*", "", f.read()))


def test_the_form_for_weights_of_the_bytes_layout_waits_first():
    """byte_expand_kernel<false> is a call's first kernel where the rows come in 8 bits: its wait is its first statement,
    and it alone writes what X's form adds to; X's form waits before that one write, and its first block's wait is its end."""
    text = body("byte_expand_kernel")
    assert text.lstrip().startswith("if (!ROWS) sg::wait_prerequisites(); sg::launch_dependents();")
    assert text.index("*large = 0") < text.index("if (!ROWS) return;") < text.rindex("sg::wait_prerequisites();") < text.index("atomicExch(large, 1)")
    assert text.count("wait_prerequisites") == 2


def test_the_order_of_the_long_int8_product():
    """W's form is launched before X's, which relies on it, and after the rows' own kernel."""
    text = source("linear8.cu")
    rows, w, x, product = (text.index(s) for s in ("sgh::rows8(c.type", "expand(byte_expand_kernel<false>", "expand(byte_expand_kernel<true>",
                                                    "sgq::run<T, sgq::BYTES>"))
    assert rows < w < x < product


def test_kernels_that_start_beside_the_one_before_end_after_it():
    """gated_parts_kernel beside: its first block waits at the end.  split_tiles_kernel: the warp that reads what the
    kernel before it wrote waits, in every block, and it is launched behind a kernel that waits.  byte_finish_kernel reads
    inputs alone before its wait."""
    text = body("gated_parts_kernel")
    assert text.lstrip().startswith("constexpr int PARTS = sizeof(T) == 4 ? 3 : 1; if (!beside) sg::wait_prerequisites(); sg::launch_dependents();")
    assert text.rstrip(" }").endswith("if (beside && blockIdx.x == 0) sg::wait_prerequisites();")
    text = body("split_tiles_kernel")
    assert text.index("wait_prerequisites()") < text.index("&mX, bar") and text.count("&mX") == 1
    gated = source("gated.cu")
    split = gated[gated.index("int forward_split("):gated.index("int forward_tiles(")]
    assert split.index("pack(none, none, X, false") < split.index("sgh::launch(\"gated, W split")
    assert "pack(Wg, Wu, X, true" in gated and gated.index("gated_slopes_kernel<T>") < gated.index("pack(Wg, Wu, X, true")
    text = body("byte_finish_kernel")
    wait = text.index("} sg::wait_prerequisites();")
    assert "partial" not in text[:wait] and "Y[" not in text[:wait] and "if (ranges == 0) sg::wait_prerequisites();" in text[:wait]


def test_every_kernel_waits():
    for name in KERNELS:
        assert "wait_prerequisites()" in FUNCTIONS[name][1], name
