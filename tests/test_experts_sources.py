"""The experts' sources: the checking build's checks where the products address
global memory (CPU)."""

import re

from test_block_sources import code, kernel, sources


def test_the_products_copies_are_checked_on_both_paths():
    """Weights and tokens are copied by one function, for aligned rows and for
    any: each path checks the place in the row before it copies, by the end of
    the part that the block multiplies."""
    copy = kernel(kernel(code(sources()["hgemm_experts.cu"]), "experts_queue_kernel"), "auto copy = [&]")
    any_rows, aligned = copy.split("} else {")
    assert "if constexpr (ANY)" in any_rows
    for path, check in ((any_rows, r"HG_DBG_INDEX\(fk\b.*?fend \+ 7\)"), (aligned, r"dbg_row\(p\b.*?fend, 16\)")):
        found = re.search(check, path, flags=re.S)
        assert found and found.start() < path.index("copy_16("), check


def test_each_function_that_addresses_global_memory_checks_itself():
    """A call of another function that checks is no check."""
    text = code(sources()["hgemm_experts.cu"])
    for f in ("experts_router_kernel", "put_unit", "experts_queue_kernel", "experts_sum_kernel"):
        assert re.search(r"HG_DBG_(INDEX|ALIGN)\(|dbg_row\(", kernel(text, f)), f
