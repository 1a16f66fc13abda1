"""The operators around the feed-forward block on every kernel, run by
tests/test_around_debug_gpu.py in a process that loads the -DHGEMM_DEBUG build
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
    import tensor_core_dense_fp16_gb300 as tc
    import test_adamw_gpu as adamw
    import test_experts_gpu as experts
    import test_residual_norm_gpu as norms

    tc.load()
    assert tc.hgemm_debug_build() == 1, "the debug variant was not loaded"

    def clean(what):
        st = tc.hgemm_device_status()
        assert st == tc.HGEMM_OK, f"{what}: status {st}, check code {tc.hgemm_debug_code()}"

    for m, d in ((1, 4096), (70, 264), (33, 1000), (9, 2048), (20, 4104), (3, 8192), (2, 16384), (2, 20001), (40, 77),
                 (700, 128), (650, 1024)):
        for post, pre in (("rms", "rms"), ("layer", "layer"), ("none", "layer"), ("rms", "none"), ("none", "none")):
            norms.run_forward(m, d, post, pre)
            norms.run_backward(m, d, post, pre)
        clean(f"norms {m}x{d}")
    for pad, offset in ((8, 0), (3, 0), (1, 1), (8, 4)):
        norms.run_forward(40, 264, "layer", "rms", pad=pad, offset=offset)
        norms.run_backward(40, 264, "rms", "layer", pad=pad, offset=offset)
    clean("norms' pitches")
    for n in (1, 63, 64, 2047, 2049, 10000, 300001):
        for bits in (8, 32):
            adamw.run([adamw.make(n, bits), adamw.make(n, bits, master=False, grad="float32", offset=1)])
        adamw.test_load(n, 0)
        clean(f"AdamW {n}")
    adamw.run([adamw.make(3 << 20, 8), adamw.make(8 << 20, 8, grad="float32")])
    clean("AdamW, several chunks a step")
    for m, d, f, e, k in experts.SHAPES:
        experts.run(m, d, f, e, k, gated=m % 2 == 0, bias=True)
        clean(f"experts {m} {d} {f} {e} {k}")
    for pad, offset in ((8, 0), (3, 0), (1, 1), (8, 4)):
        experts.run(12, 136, 72, 6, 2, bias=True, pad=pad, offset=offset)
    clean("experts' pitches")
    print("debug build: the operators around the block clean")
    return 0


if __name__ == "__main__":
    sys.exit(main())
