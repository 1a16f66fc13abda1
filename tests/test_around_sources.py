"""Properties of the sources of the operators around the feed-forward block
that no run on one GPU can show (CPU)."""

import re

from test_block_sources import code, kernel, sources

FILES = ("hgemm_residual_norm.cu", "hgemm_adamw.cu", "hgemm_experts.cu", "row_sums.cuh")

# what addresses global memory itself, by file
ADDRESSING = {
    "hgemm_residual_norm.cu": ("residual_norm_rows_kernel", "residual_norm_long_kernel", "residual_norm_ring_kernel",
                               "residual_norm_sums_kernel", "residual_norm_means_kernel",
                               "residual_norm_partials_kernel", "residual_norm_backward_kernel"),
    "hgemm_adamw.cu": ("adamw_eight", "adamw_bytes", "adamw_load_kernel"),
    "hgemm_experts.cu": ("experts_router_kernel", "put_unit", "experts_queue_kernel", "experts_sum_kernel"),
}


def test_no_operand_is_read_through_the_non_coherent_path():
    for name in FILES:
        text = code(sources()[name])
        for what in (r"__ldg", r"ld\.global\.nc", r"const\s+\w+\s*\*\s*__restrict__"):
            assert not re.search(what, text), (name, what)


def test_the_checking_build_checks_what_addresses_global_memory():
    files = sources()
    for name, functions in ADDRESSING.items():
        for f in functions:
            body = kernel(code(files[name]), f)
            assert re.search(r"HG_DBG_(INDEX|ALIGN)\(|dbg_row\(|piece\.(load|store)\(|put_unit", body), (name, f)


def test_every_kernel_waits_for_the_launch_before_it():
    """Programmatic launches overlap the one before: each kernel waits for it,
    and lets the next one start only after that."""
    for name in FILES[:3]:
        text = code(sources()[name])
        for k in re.findall(r"__global__[^{;]*?(\w+_kernel)\s*\(", text):
            body = kernel(text, k)
            waits = [m.start() for m in re.finditer(r"grid_dependency_wait\(\)", body)]
            starts = [m.start() for m in re.finditer(r"grid_launch_dependents\(\)", body)]
            assert waits and len(waits) == len(starts), k
            assert all(w < s for w, s in zip(waits, starts)), k


def test_what_is_read_before_the_wait_goes_past_l1():
    """The second product's routing and weights are read before its wait, behind
    a fence, with accesses that go to L2."""
    text = code(sources()["hgemm_experts.cu"])
    queue = kernel(text, "experts_queue_kernel")
    assert "fence_gpu()" in queue[:queue.index("find_entries<")]
    entries = kernel(text, "find_entries")
    assert "ld_gpu_s32(a.ws_chosen" in entries and "a.ws_chosen[" not in entries
    assert "copy(to, w0, true)" in queue and "copy(to + Cfg::ROWS, w1, true)" in queue
    assert re.search(r"if \(weights\)\s*cp_async_16\(to, p, bytes\);", queue)
    assert ".cg" in kernel(code(sources()["ptx.cuh"]), "cp_async_16")
