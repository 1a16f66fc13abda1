"""AdamW's 8-bit states rounded at random: the codes bit for bit, the random
numbers' evenness, and states that follow their gradients over thousands of
steps (GPU only)."""

import numpy as np
import pytest

import around_reference as ref
import rounding_reference as rounded
import tensor_core_dense_fp16_gb300 as tc
from gpu_helpers import torch_cuda
from test_adamw_gpu import HYPER, Array, make, same, table
from test_block_gpu import done

pytestmark = pytest.mark.gpu

RANDOM = tc.HGEMM_ROUND_RANDOM


def check_states(tensors, step, grad_scale=1.0, forms=rounded):
    for i, (t, _) in enumerate(tensors):
        h = {k: a.host for k, a in t.items()}
        what = f"tensor {i} of {h['grad'].size}: "
        if "m_scales" not in h:
            m, v = ref.adamw_states(h["grad"], h["m"], h["v"], HYPER["beta1"], HYPER["beta2"], grad_scale)
            same(t["m"].get(), m, what + "m")
            same(t["v"].get(), v, what + "v")
            continue
        m, v = ref.adamw_states(h["grad"], ref.kept_m(h["m"], h["m_scales"]), ref.kept_v(h["v"], h["v_scales"]),
                                HYPER["beta1"], HYPER["beta2"], grad_scale)
        for name, x in (("m", m), ("v", v)):
            codes, scales = getattr(forms, "keep_" + name)(x, step)
            same(t[name + "_scales"].get(), scales, what + name + " scales")
            same(t[name].get(), codes, what + name + " codes")


def run(tensors, step=3, grad_scale=1.0, stream=None):
    tc.hgemm_adamw_rounded(table(tensors), step=step, grad_scale=grad_scale, stream=stream, rounding=RANDOM, **HYPER)
    torch_cuda().cuda.synchronize()
    done()
    check_states(tensors, step, grad_scale)


@pytest.mark.parametrize("n", [1, 7, 8, 63, 64, 65, 200, 2047, 2048, 2049, 10000, 300001])
@pytest.mark.parametrize("master,grad", [(True, "float16"), (False, "float16"), (True, "float32"), (False, "float32")])
def test_codes(n, master, grad):
    run([make(n, 8, master=master, grad=grad)])


@pytest.mark.parametrize("n", [64, 1000, 5000])
@pytest.mark.parametrize("offset", [1, 4, 8])
def test_alignment_does_not_matter(n, offset):
    run([make(n, 8, offset=offset), make(n, 8, master=False, grad="float32", offset=offset)])


@pytest.mark.parametrize("step,grad_scale", [(1, 1.0), (2, 2.0 ** -10), ((1 << 31) + 5, 3.0), (1 << 40, 0.0)])
def test_step_numbers(step, grad_scale):
    run([make(1000, 32), make(1000, 8, master=False)], step, grad_scale)


@pytest.mark.parametrize("count", [17, 97, 400])
def test_many_tensors_of_both_kinds(count):
    rng = np.random.default_rng(count)
    run([make(int(rng.choice([0, 1, 64, 130, 2048, 3000])), int(rng.choice([8, 32])), seed=i,
              offset=int(rng.choice([0, 0, 1]))) for i in range(count)], stream=torch_cuda().cuda.Stream())


def test_several_chunks_a_step():
    run([make(4000000, 8), make(1, 8), make(1200007, 8, grad="float32"), make(5000, 8)])


def test_zero_infinite_and_nan_groups_and_values_at_the_ends():
    n = 64 * 6 + 5
    g = np.random.default_rng(1).standard_normal(n).astype(np.float32)
    g[:64] = 0
    g[64:128] *= 1e-18                        # v below 2^-100
    g[130], g[200] = np.inf, np.nan
    g[256:320] = 1                            # every value the group's largest
    g[320:384] = 1e-7                         # v below its least code next to one large value
    g[320] = 1
    t, d = make(n, 8)
    for name in ("m", "v"):
        t[name] = Array(np.zeros_like(t[name].host))
        t[name + "_scales"] = Array(np.zeros_like(t[name + "_scales"].host))
    t["grad"] = Array(g)
    for step in range(1, 40):
        tc.hgemm_adamw_rounded(table([(t, d)]), step=step, rounding=RANDOM, **HYPER)
        done()
        check_states([(t, d)], step)
        m, v = t["m"].get(), t["v"].get()
        assert (m[256:320] == 127).all() and (v[256:320] == 255).all()
        assert (v[321:384] == 1).all() and (v[:64] == 0).all() and (m[:64] == 0).all()
        for name in ("m", "v", "m_scales", "v_scales", "weight", "master"):
            t[name].host = t[name].get()


def test_a_graph_takes_the_devices_step_number():
    torch = torch_cuda()
    tensors = [make(1000 + 8 * i, 8 if i % 2 else 32, seed=i) for i in range(5)]
    plan = table(tensors)
    device = torch.zeros(16, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            tc.hgemm_adamw_rounded(plan, 123.0, 0.9, 0.999, 1e-8, dynamic=device, rounding=RANDOM)
    for step in (1, 2, 70000):
        device.copy_(tc.hgemm_adamw_dynamic(1e-2, 1.0, step))
        graph.replay()
        torch.cuda.synchronize()
        done()
        check_states(tensors, step)
        for t, _ in tensors:
            for a in t.values():
                a.host = a.get()


def test_to_nearest_where_nothing_is_said():
    class Nearest:
        keep_m = staticmethod(lambda m, step: ref.keep_m(m))
        keep_v = staticmethod(lambda v, step: ref.keep_v(v))

    tensors = [make(3000, 8), make(300, 8, offset=1)]
    tc.hgemm_adamw(table(tensors), step=3, **HYPER)
    done()
    check_states(tensors, 3, forms=Nearest)


@pytest.mark.parametrize("step", [1, 2, 1000])
def test_the_random_numbers_are_even(step):
    """2^16 equal values a part of the way p between two codes, next to their
    groups' largest: up with probability p, a value's neighbours independent of
    it. A fraction of n trials is within 6·√(p(1−p)/n) of its probability with
    all but 2e-9; p is known to within 2^-12 of a part (m's random numbers, FP32
    roundings)."""
    n = 1 << 16
    for name, code, part in (("m", 20, 0.3), ("m", -61, 0.9), ("v", 231, 0.02), ("v", 120, 0.5), ("v", 3, 0.8)):
        zeros = np.zeros(n, np.float16)
        t = {"grad": zeros, "weight": zeros, "m": np.zeros(n, np.int8), "v": np.zeros(n, np.uint8),
             "m_scales": np.zeros(n // 64, np.float32), "v_scales": np.zeros(n // 64, np.float32)}
        # a gradient g from states of zero: m = g/10 and v = g²/1000, up to FP32
        if name == "m":
            g = np.full(n, (code + part) / 127, np.float32)
        else:
            low, high = (2.0 ** ((c - 255) // 8) * (1 + ((c - 255) % 8) / 8) for c in (code, code + 1))
            g = np.full(n, np.sqrt(low + part * (high - low)), np.float32)
        g[::64] = 1
        t["grad"] = g
        t = {k: Array(a) for k, a in t.items()}
        tc.hgemm_adamw_rounded(table([(t, 0.0)]), step=step, rounding=RANDOM, **HYPER)
        done()
        codes = t[name].get().astype(np.int64).reshape(-1, 64)[:, 1:]
        assert ((codes == code) | (codes == code + 1)).all()
        up = codes == code + 1
        for got, p in ((up, part), (up[:, 1:] & up[:, :-1], part * part), (up[:, 3:] & up[:, :-3], part * part)):
            assert abs(got.mean() - p) < 6 * (p * (1 - p) / got.size) ** 0.5 + 2.0 ** -11, (name, code, got.mean(), p)


def test_states_follow_their_gradients_for_2000_steps():
    """A training run's recurrence, through the optimizer that training uses:
    after step 100 a quarter of the values' gradients stay as they are, a quarter
    fall by 10, a quarter grow by 3 and a quarter are 0, side by side in every
    group, next to states in 32 bits.

    v: a value's kept v is its formula's in the mean, since each rounding is. Its
    spread: a step moves v by (1 − β2)·(g² − v) and the group's scale likewise,
    c ≤ 3 times (1 − β2)·v together in the mean, of which a rounding to codes d ≤
    1/8 apart leaves a variance of at most d·c·(1 − β2)·v². While gradients stay
    the recurrence forgets them with β2²: d·c/2 = 0.19 of v². Where v falls they
    fall no faster than v, and 1900 steps add d·c·1.9 = 0.71 to that: a standard
    deviation of 0.95 at most, and of the mean of n = 1024 values 0.03. Six of
    those: 0.18.

    m of gradients that ended 1900 steps ago: a code of at most 127 falls to
    0.9^1900 of itself in the mean, 0 but for a probability below 1e-80.

    The update m/√v where gradients stay or grow: half of v's relative
    deviation, √0.19/2 = 0.22, and m's, whose roundings (variance at most 1/4 of
    a squared code, 5.3 of them by β1² = 0.81) are 1.15 codes of 1/127 of the
    group's largest, itself at most 4.5 deviations of the grown values': 0.04 of
    a deviation of theirs, 0.12 of the others'. Together below 0.26; a
    linearisation of 1/√v of that spread is short by no more than a quarter of
    it. Held to 0.33 of the update's norm."""
    from tensor_core_dense_fp16_gb300.feedforward import AdamW
    torch = torch_cuda()
    n, steps = 4096, 2000
    g = torch.Generator(device="cuda").manual_seed(11)
    p = torch.zeros(n, dtype=torch.float16, device="cuda")
    opt = AdamW({"p": p}, lr=1e-6, bits=8)
    m = torch.zeros(n, dtype=torch.float64, device="cuda")
    v = torch.zeros(n, dtype=torch.float64, device="cuda")
    scale = torch.ones(n, device="cuda")
    for step in range(1, steps + 1):
        if step == 101:
            scale = torch.tensor([1, 0.1, 3, 0], device="cuda").repeat(n // 4)
        grad = torch.randn(n, generator=g, device="cuda") * scale
        opt.step({"p": grad})
        m = 0.9 * m + 0.1 * grad.double()
        v = 0.999 * v + 0.001 * grad.double().square()
    done()
    t = {k: x.cpu().numpy() for k, x in opt.tensors[0].items() if hasattr(x, "cpu")}
    kept_m, kept_v = ref.kept_m(t["m"], t["m_scales"]), ref.kept_v(t["v"], t["v_scales"]).astype(np.float64)
    m, v = m.cpu().numpy(), v.cpu().numpy()
    for i, what in enumerate(("as they were", "a tenth", "three times", "none")):
        off = (kept_v / v)[i::4].mean() - 1
        assert abs(off) < 0.18, f"gradients {what}: kept v is {1 + off:.2f} times its formula's in the mean"
    assert (t["m"][3::4] == 0).all()
    update, want = kept_m / np.sqrt(kept_v), m / np.sqrt(v)
    for i in (0, 2):
        off = np.linalg.norm((update - want)[i::4]) / np.linalg.norm(want[i::4])
        assert off < 0.33, (i, off)


def test_equal_runs_are_equal():
    from tensor_core_dense_fp16_gb300.feedforward import AdamW
    torch = torch_cuda()

    def go():
        g = torch.Generator(device="cuda").manual_seed(2)
        ps = {n: torch.randn(s, generator=g, device="cuda").half() for n, s in (("a", (40, 65)), ("b", (3000,)))}
        opt = AdamW(ps, lr=1e-2, bits=8)
        for _ in range(5):
            opt.step({n: torch.randn(q.shape, generator=g, device="cuda") for n, q in ps.items()})
        return [t[k] for t in opt.tensors for k in ("weight", "master", "m", "v", "m_scales", "v_scales")]

    for a, b in zip(go(), go()):
        assert torch.equal(a, b)
    done()
