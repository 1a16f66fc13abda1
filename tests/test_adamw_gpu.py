"""AdamW over many tensors: the states bit for bit (their operations are
defined one by one), parameters within the bounds around_reference derives
(GPU only)."""

import numpy as np
import pytest

import around_reference as ref
import tensor_core_dense_fp16_gb300 as tc
from block_reference import half_rounding
from gpu_helpers import torch_cuda
from test_block_gpu import check, done

pytestmark = pytest.mark.gpu

HYPER = dict(lr=1e-2, beta1=0.9, beta2=0.999, eps=1e-8)
GUARD = 64  # bytes of 0x5A on either side of every array


class Array:
    """A device array `offset` elements off a 256-byte boundary, guarded on both sides."""

    def __init__(self, host, offset=0):
        torch = torch_cuda()
        self.host, self.at = host, GUARD * 4 + offset * host.itemsize
        raw = np.full(self.at + host.nbytes + GUARD, 0x5A, np.uint8)
        raw[self.at:self.at + host.nbytes] = np.frombuffer(host.tobytes(), np.uint8)
        self.raw = torch.from_numpy(raw).cuda()
        dtype = getattr(torch, str(host.dtype))
        self.tensor = torch.empty(0, dtype=dtype, device="cuda")
        if host.size:
            # (a view of another type needs an address that is a multiple of its size, which `at` is)
            self.tensor = self.raw[self.at:self.at + host.nbytes].view(dtype)

    def get(self):
        raw = self.raw.cpu().numpy()
        body = raw[self.at:self.at + self.host.nbytes].tobytes()
        raw[self.at:self.at + self.host.nbytes] = 0x5A
        assert (raw == 0x5A).all(), "written outside the array"
        return np.frombuffer(body, self.host.dtype)


def make(n, bits=32, weight=True, master=True, grad="float16", offset=0, decay=0.1, seed=0, scale=1.0):
    """One tensor: {name: Array}, its decay."""
    rng = np.random.default_rng(seed + n)
    spread = np.repeat(np.exp(1.5 * rng.standard_normal(-(-n // 64))), 64)[:n]

    def values(s):
        return (rng.standard_normal(n) * np.exp(rng.standard_normal(n)) * spread * s * scale).astype(np.float32)

    p = (0.5 * rng.standard_normal(n)).astype(np.float32)
    t = {"grad": values(0.02).astype(grad)}
    if weight:
        t["weight"] = p.astype(np.float16)
    if master:
        t["master"] = p
    m, v = values(0.01), np.square(values(0.02))
    if bits == 8:
        t["m"], t["m_scales"] = ref.keep_m(m)
        t["v"], t["v_scales"] = ref.keep_v(v)
    else:
        t["m"], t["v"] = m, v
    # (offsets in elements of each array, so that none but the element's own alignment is left)
    return {k: Array(a, offset) for k, a in t.items()}, decay


def table(tensors):
    return tc.hgemm_adamw_tensors([{**{k: a.tensor for k, a in t.items()}, "weight_decay": d} for t, d in tensors])


def same(got, want, what):
    got, want = np.asarray(got), np.asarray(want, got.dtype)
    bad = got.view(np.uint8 if got.itemsize == 1 else np.uint32) != want.view(
        np.uint8 if got.itemsize == 1 else np.uint32)
    if got.dtype.kind == "f":
        bad &= ~(np.isnan(got) & np.isnan(want)) & ~((got == 0) & (want == 0))
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} differ, first {np.argwhere(bad)[0]}: " \
                          f"{got[bad][0]} for {want[bad][0]}"


def check_step(tensors, step, grad_scale=1.0, hyper=HYPER):
    """The arrays against a step from their host values."""
    for i, (t, decay) in enumerate(tensors):
        h = {k: a.host for k, a in t.items()}
        n = h["grad"].size
        eight = "m_scales" in h
        m = ref.kept_m(h["m"], h["m_scales"]) if eight else h["m"]
        v = ref.kept_v(h["v"], h["v_scales"]) if eight else h["v"]
        m1, v1 = ref.adamw_states(h["grad"], m, v, hyper["beta1"], hyper["beta2"], grad_scale)
        what = f"tensor {i} of {n}: "
        if eight:
            for name, form, x in (("m", ref.keep_m, m1), ("v", ref.keep_v, v1)):
                codes, scales = form(x)
                same(t[name + "_scales"].get(), scales, what + name + " scales")
                same(t[name].get(), codes, what + name + " codes")
        else:
            same(t["m"].get(), m1, what + "m")
            same(t["v"].get(), v1, what + "v")
        p = h["master"] if "master" in h else h["weight"]
        want, bound = ref.adamw(p, h["grad"], m, v, decay=decay, step=step, grad_scale=grad_scale, **hyper)
        if "master" in t:
            got = t["master"].get()
            check(got, want, bound, what + "master")
            if "weight" in t:
                same(t["weight"].get().astype(np.float32), got.astype(np.float16).astype(np.float32), what + "weight")
        else:
            check(t["weight"].get(), want, bound + half_rounding(np.abs(want) + bound) * 1.001, what + "weight")
        assert (t["grad"].get() == h["grad"]).all()


def run(tensors, step=3, grad_scale=1.0, stream=None):
    tc.hgemm_adamw(table(tensors), step=step, grad_scale=grad_scale, stream=stream, **HYPER)
    done()
    check_step(tensors, step, grad_scale)


SIZES = [1, 7, 8, 63, 64, 65, 200, 2047, 2048, 2049, 4096, 10000, 300001]


@pytest.mark.parametrize("n", SIZES)
@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("weight,master", [(True, True), (True, False), (False, True)])
@pytest.mark.parametrize("grad", ["float16", "float32"])
def test_one_tensor(n, bits, weight, master, grad):
    run([make(n, bits, weight, master, grad)])


@pytest.mark.parametrize("n", [64, 1000, 5000])
@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("offset", [1, 4, 8])
def test_alignment(n, bits, offset):
    run([make(n, bits, offset=offset), make(n, bits, master=False, grad="float32", offset=offset)])


@pytest.mark.parametrize("count", [2, 15, 16, 17, 100, 383, 384, 385, 1000])
def test_many_tensors(count):
    rng = np.random.default_rng(count)
    run([make(int(rng.choice([0, 1, 64, 130, 2048, 3000])), int(rng.choice([8, 32])), master=bool(rng.random() < 0.5),
              grad=str(rng.choice(["float16", "float32"])), offset=int(rng.choice([0, 0, 1])), seed=i,
              decay=float(rng.choice([0, 0.1]))) for i in range(count)])


@pytest.mark.parametrize("step,grad_scale", [(1, 1.0), (2, 2.0 ** -10), (100000, 3.0), (1 << 40, 0.0)])
def test_step_and_scale(step, grad_scale):
    run([make(1000, 32), make(1000, 8, master=False)], step, grad_scale)


def test_the_forms_steps_and_ends():
    """Every code of v, both ends, and what lies between two codes."""
    n = 64 * 8
    v = np.zeros(n, np.float32)
    all_codes = ref.kept_v(np.arange(256).astype(np.uint8), np.ones(4, np.float32))
    v[:256] = all_codes
    v[0:256:64] = 1.0                                           # (a group's largest)
    v[256:512] = np.float32(1.0625) * all_codes                 # halfway between many of them
    v[256::64] = np.float32(3e-12)
    v[300:310] = np.float32(2.0 ** -34) * v[256]
    codes, scales = ref.keep_v(v)
    zeros = np.zeros(n, np.float16)
    t = {"grad": zeros, "weight": zeros, "m": np.zeros(n, np.int8), "m_scales": np.zeros(8, np.float32), "v": codes,
         "v_scales": scales}
    tensors = [({k: Array(a) for k, a in t.items()}, 0.0)]
    run(tensors)


def test_zero_tiny_infinite_and_nan_groups():
    n = 64 * 7 + 5
    g = np.random.default_rng(1).standard_normal(n).astype(np.float32)
    g[:64] = 0
    g[64:128] *= 1e-18      # v below 2^-100
    g[130], g[200], g[300] = np.inf, np.nan, -np.inf
    g[330] = 1e25           # v beyond FP32
    g[448:] = 0
    for bits in (8, 32):
        (t, d), = [make(n, bits)]
        for name in ("m", "v"):
            t[name] = Array(np.zeros_like(t[name].host))
            if bits == 8:
                t[name + "_scales"] = Array(np.zeros_like(t[name + "_scales"].host))
        t["grad"] = Array(g)
        tc.hgemm_adamw(table([(t, d)]), step=2, **HYPER)
        done()
        m, v = ref.adamw_states(g, np.zeros(n, np.float32), np.zeros(n, np.float32), 0.9, 0.999, 1.0)
        if bits == 8:
            for name, form, x in (("m", ref.keep_m, m), ("v", ref.keep_v, v)):
                codes, scales = form(x)
                same(t[name + "_scales"].get(), scales, name)
                same(t[name].get(), codes, name)
        else:
            same(t["m"].get(), m, "m")
            same(t["v"].get(), v, "v")
        p = t["master"].get()
        bad = ~np.isfinite(p)
        assert bad[[130, 200, 300]].all() and not bad[:128].any() and not bad[448:].any()
        # a value is its own: what spoils one leaves its neighbours' parameters alone
        spoilt = np.zeros(n, bool)
        spoilt[[130, 200, 300, 330]] = True
        assert not bad[~spoilt].any()


def test_steps_in_a_row():
    """What a step leaves is what the next one reads, for 20 steps, against the
    reference carried along in the same forms."""
    rng = np.random.default_rng(4)
    n = 3000
    for bits in (8, 32):
        (t, d), = [make(n, bits, seed=9)]
        plan = table([(t, d)])
        for step in range(1, 21):
            g = (rng.standard_normal(n) * 0.05).astype(np.float16)
            t["grad"].tensor.copy_(torch_cuda().from_numpy(g))
            t["grad"].host = g
            tc.hgemm_adamw(plan, step=step, **HYPER)
            done()
            check_step([(t, d)], step)
            for a in t.values():
                a.host = a.get()


@pytest.mark.parametrize("count", [3, 40])
def test_dynamic_values_in_a_graph(count):
    """A captured step follows the device's learning rate, gradient scale and
    step number, and its skip leaves everything as it was."""
    torch = torch_cuda()
    tensors = [make(1000 + 8 * i, 8 if i % 2 else 32, seed=i) for i in range(count)]
    plan = table(tensors)
    device = torch.zeros(16, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            tc.hgemm_adamw(plan, 123.0, 0.9, 0.999, 1e-8, dynamic=device)
    for step, lr, scale, skip in ((1, 1e-2, 0.5, False), (2, 1e-2, 1.0, True), (2, 3e-3, 2.0, False),
                                  (70000, 1e-2, 1.0, False)):
        device.copy_(tc.hgemm_adamw_dynamic(lr, scale, step, skip))
        graph.replay()
        torch.cuda.synchronize()
        done()
        if skip:
            for t, _ in tensors:
                for a in t.values():
                    assert a.get().tobytes() == a.host.tobytes()
        else:
            # lr and 1 − β^step in FP32 on the device are within 2^-21 of theirs in 64 bits, which the
            # update's bound has room for
            check_step(tensors, step, scale, {**HYPER, "lr": float(np.float32(lr))})
        for t, _ in tensors:
            for a in t.values():
                a.host = a.get()


def test_another_stream():
    run([make(100000, 8), make(5000, 32)], stream=torch_cuda().cuda.Stream())


@pytest.mark.parametrize("n", [1, 63, 64, 1000, 300001])
@pytest.mark.parametrize("offset", [0, 1])
def test_load(n, offset):
    rng = np.random.default_rng(n)
    m, ms = ref.keep_m(rng.standard_normal(n).astype(np.float32))
    v, vs = ref.keep_v(np.square(rng.standard_normal(n)).astype(np.float32))
    a = [Array(x, offset) for x in (m, ms, v, vs, np.zeros(n, np.float32), np.zeros(n, np.float32))]
    p = [x.tensor for x in a]
    tc.hgemm_adamw_load(*p, n)
    done()
    same(a[4].get(), ref.kept_m(m, ms), "m")
    same(a[5].get(), ref.kept_v(v, vs), "v")
    p[4].zero_(), p[5].zero_()
    tc.hgemm_adamw_load(None, None, p[2], p[3], None, p[5], n)
    tc.hgemm_adamw_load(p[0], p[1], None, None, p[4], None, n)
    done()
    same(a[4].get(), ref.kept_m(m, ms), "m")
    same(a[5].get(), ref.kept_v(v, vs), "v")


@pytest.mark.parametrize("bits,sizes", [(8, (1000003, 2048, 64 * 900 + 8, 5)), (8, (4000000, 1, 1200007, 5000, 65)),
                                        (8, (20000001, 777, 100000)), (32, (5000009, 3, 300000, 2049))])
def test_several_chunks_a_step(bits, sizes):
    """Tables large enough for steps of two, four and eight chunks, whose
    tensors end inside one."""
    tensors = [make(n, bits, master=i % 2 == 0, grad="float32" if i % 3 == 2 else "float16")
               for i, n in enumerate(sizes)]
    run(tensors)


def test_a_table_keeps_its_tensors():
    """The caller's dicts may be changed for the next table: a gradient that the
    first one points to stays alive with it."""
    import gc
    import weakref
    torch = torch_cuda()
    t = {"grad": torch.zeros(64, dtype=torch.float16, device="cuda"), "master": torch.zeros(64, device="cuda"),
         "m": torch.zeros(64, device="cuda"), "v": torch.zeros(64, device="cuda")}
    held = weakref.ref(t["grad"])
    first = tc.hgemm_adamw_tensors([t])
    t["grad"] = torch.zeros(64, dtype=torch.float16, device="cuda")
    gc.collect()
    assert held() is not None
    del first
    gc.collect()
    assert held() is None


def test_other_gradients_in_a_table():
    """set_gradients steps as a table of the new gradients does, of the other
    type too; what it refuses leaves the table as it was."""
    torch = torch_cuda()
    tensors = [make(1000, 8), make(5000, 32, grad="float32"), make(77, 32, master=False)]
    plan = table(tensors)
    run_with = [Array((a["grad"].host * 0.5).astype("float32" if i == 0 else "float16"))
                for i, (a, _) in enumerate(tensors)]
    good = [a.tensor for a in run_with]
    for bad, error in (([good[0], good[1]], ValueError), ([good[0], good[1], good[2][:70]], ValueError),
                       ([good[0], good[1], good[2].double()], TypeError), ([good[0], good[1], good[2].cpu()], ValueError),
                       ([good[0], good[1], tensors[2][0]["weight"].tensor], tc.HgemmError)):
        before, grads = bytes(plan.table), plan.grads
        with pytest.raises(error):
            plan.set_gradients(bad)
        assert bytes(plan.table) == before and plan.grads is grads
    plan.set_gradients(good)
    for (t, _), g in zip(tensors, run_with):
        t["grad"] = g
    tc.hgemm_adamw(plan, step=3, **HYPER)
    done()
    check_step(tensors, 3)
    empty = tc.hgemm_adamw_tensors([])
    empty.set_gradients([])
    tc.hgemm_adamw(empty, 1e-3)


def test_refusals():
    torch = torch_cuda()
    f, h = torch.zeros(128, device="cuda"), torch.zeros(128, dtype=torch.float16, device="cuda")
    with pytest.raises(tc.HgemmError) as err:  # m is v
        tc.hgemm_adamw_tensors([dict(weight=h, grad=h.clone(), m=f, v=f)])
    assert err.value.status == tc.HGEMM_ERR_ALIAS
    ok = dict(weight=h, grad=h.clone(), m=f, v=f.clone())
    with pytest.raises(tc.HgemmError):  # the same tensor twice
        tc.hgemm_adamw_tensors([ok, ok])
    with pytest.raises(ValueError):
        tc.hgemm_adamw_tensors([{**ok, "m": torch.zeros(128)}])
    with pytest.raises(ValueError):
        tc.hgemm_adamw_tensors([{**ok, "m": f[:64]}])
    plan = tc.hgemm_adamw_tensors([ok])
    for kw in (dict(lr=float("nan")), dict(beta1=1.0), dict(beta2=-0.1), dict(eps=-1.0), dict(step=0),
               dict(grad_scale=float("inf"))):
        with pytest.raises(tc.HgemmError):
            tc.hgemm_adamw(plan, **{**HYPER, **kw})
    with pytest.raises(ValueError):
        tc.hgemm_adamw(plan, **HYPER, dynamic=torch.zeros(16, dtype=torch.uint8))
