"""Properties of the kernels' sources that no run on one GPU can show (CPU)."""

import glob
import os
import re

from tensor_core_dense_fp16_gb300 import build as tcbuild

CSRC = os.path.join(os.path.dirname(tcbuild.__file__), "csrc")


def sources():
    files = sorted(glob.glob(os.path.join(CSRC, "*.cu*")) + glob.glob(os.path.join(CSRC, "*.h")))
    assert files
    return {os.path.basename(f): open(f, encoding="utf-8").read() for f in files}


def code(text):
    """The text without its comments."""
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def test_no_load_is_multicast():
    """An operand may be memory of another GPU, where a multicast load is not
    safe: every CTA loads for itself (commits may be multicast)."""
    for name, text in sources().items():
        for call in re.findall(r"asm volatile\((.*?)\);", code(text), flags=re.S):
            assert not ("cp.async.bulk" in call and "multicast" in call), name


def kernel(text, name):
    """A kernel's body."""
    start = text.index("{", text.index(name + "("))
    depth, i = 1, start + 1
    while depth:
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        i += 1
    return text[start:i]


def test_sums_beside_a_product_read_behind_a_fence_from_l2():
    """The column sums do not wait for the launches before them: what these
    wrote is read with loads that cannot meet an older line."""
    text = code(sources()["hgemm_linear.cu"])
    for name in ("column_sums_kernel", "column_sums_thin_kernel"):
        body = kernel(text, name)
        loop = body.index("for (")
        assert 0 <= body.find("fence_gpu()") < loop, name
        assert "__ldg" not in body and body.count("ld_gpu_16(") == 1, name
        # dy and the old sums, and nothing else in global memory
        assert not re.search(r"\bdy\s*\[|\*\s*\(?\s*dy\b|\bout\s*\[[^\]]*\]\s*\+|\*o\s*\+", body), name
        assert "ld_gpu_f32(" in body, name


BLOCK = ("hgemm_linear.cu", "hgemm_linear_any.cu", "hgemm_linear_small.cu", "hgemm_linear_wave.cu", "hgemm_norm.cu",
         "hgemm_ckpt8.cu", "linear_epilogue.cuh", "kernel_common.cuh")


def test_no_operand_is_read_through_the_non_coherent_path():
    """That path needs memory which nobody writes while the kernel lives, and
    these kernels start while the launch before them may still write."""
    for name in BLOCK:
        text = code(sources()[name])
        for what in (r"__ldg", r"ld\.global\.nc", r"const\s+\w+\s*\*\s*__restrict__"):
            assert not re.search(what, text), (name, what)


# what addresses global memory itself, by file
ADDRESSING = {
    "linear_epilogue.cuh": ("lin_fetch", "lin_row64"),
    "hgemm_linear.cu": ("linear_empty_kernel", "linear_rows_kernel", "column_sums_kernel", "column_sums_thin_kernel"),
    "hgemm_linear_small.cu": ("fetch_rows", "put_rows"),
    "hgemm_linear_any.cu": ("any_columns", "any_copy_edge", "linear_any_kernel"),
    "hgemm_linear_wave.cu": ("sum_rows",),
    "hgemm_norm.cu": ("layernorm_forward_kernel", "layernorm_backward_ring_kernel", "layernorm_partials_kernel"),
    "hgemm_ckpt8.cu": ("ckpt8_save_vec_kernel", "ckpt8_save_kernel", "ckpt8_load_vec_kernel", "ckpt8_load_kernel"),
}


def test_the_checking_build_checks_what_addresses_global_memory():
    """Without a check in it, a kernel passes the checking build whatever its
    indices are."""
    files = sources()
    for name, functions in ADDRESSING.items():
        for f in functions:
            body = kernel(code(files[name]), f)
            assert re.search(r"HG_DBG_(INDEX|ALIGN)\(|dbg_row\(|any_inside\(", body), (name, f)
