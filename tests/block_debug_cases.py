"""The feed-forward block's operators on every kernel, run by
tests/test_block_debug_gpu.py in a process that loads the -DHGEMM_DEBUG build
(HGEMM_LIBRARY_VARIANT=debug): no device-side check may fire, and the results
are the reference's."""

import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
sys.path.insert(0, os.path.join(ROOT, "tests"))


def main() -> int:
    assert os.environ.get("HGEMM_LIBRARY_VARIANT") == "debug"
    from tensor_core_dense_fp16_gb300 import build
    build.build(debug=True)
    import numpy as np
    import tensor_core_dense_fp16_gb300 as tc
    import test_block_gpu as cases

    tc.load()
    assert tc.hgemm_debug_build() == 1, "the debug variant was not loaded"

    def clean(what):
        st = tc.hgemm_device_status()
        assert st == tc.HGEMM_OK, f"{what}: status {st}, check code {tc.hgemm_debug_code()}"

    for name, path in cases.PATHS.items():
        tc.hgemm_force_path(path)
        try:
            for M, N, K in ((300, 264, 520), (129, 72, 200)):
                cases.run_linear(M, N, K, "gelu", keep=True)
                cases.run_dgrad(M, N, K, "silu")
                cases.run_wgrad(M, N, K, accumulate=True)
        finally:
            tc.hgemm_force_path(-1)
        clean(name)
    # one row, few rows, small weights of many rows, odd sizes and alignments
    for M, N, K in ((1, 264, 520), (7, 65, 77), (20, 2048, 1032), (100, 136, 4104)):
        cases.run_linear(M, N, K, "gelu")
        cases.run_dgrad(M, K, N, "gelu")
        clean(f"few rows {M}x{N}x{K}")
    cases.run_wgrad(2100, 200, 136)
    for pad, offset in ((3, 0), (1, 1), (8, 4)):
        cases.run_linear(150, 131, 77, "silu", keep=True, pad=pad, offset=offset)
        cases.run_dgrad(150, 131, 77, "silu", pad=pad, offset=offset)
        cases.run_wgrad(150, 131, 77, pad=pad, offset=offset)
    cases.run_linear(150, 131, 2049, "gelu", keep=True)
    cases.run_linear(150, 131, 1544, "gelu")
    clean("odd sizes")
    for M, D in ((1, 4096), (70, 264), (40, 1000), (30, 2048), (20, 4096), (9, 8192), (5, 16384), (7, 20001)):
        cases.run_layernorm(M, D)
        clean(f"layer norm {M}x{D}")
    rng = np.random.default_rng(3)
    for M, N in ((257, 1000), (33, 63), (5, 20001)):
        cases.run_ckpt8(cases.rng_half(rng, (M, N), 2), name="gelu")
        clean(f"8-bit form {M}x{N}")
    print("debug build: the block's operators clean")
    return 0


if __name__ == "__main__":
    sys.exit(main())
