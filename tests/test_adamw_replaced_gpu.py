"""The optimizer's states, master copies and decays replaced between steps, as
restoring a checkpoint or a schedule does (GPU only)."""

import pytest

import tensor_core_dense_fp16_gb300 as tc
from gpu_helpers import torch_cuda
from test_block_gpu import done

pytestmark = pytest.mark.gpu

SHAPES = {"a": (40, 64), "b": (77,), "none": (0,)}


def optimizer(bits, master, seed=1):
    from tensor_core_dense_fp16_gb300.feedforward import AdamW
    torch = torch_cuda()
    g = torch.Generator(device="cuda").manual_seed(seed)
    ps = {n: torch.randn(*s, generator=g, device="cuda").half() for n, s in SHAPES.items()}
    return AdamW(ps, lr=0.1, bits=bits, master=master, weight_decay=0.1)


def gradients(step):
    torch = torch_cuda()
    g = torch.Generator(device="cuda").manual_seed(100 + step)
    return {n: torch.randn(*s, generator=g, device="cuda") * 0.01 for n, s in SHAPES.items()}


def states(opt):
    return [{n: x for n, x in t.items() if n != "weight_decay" and x is not None} for t in opt.tensors]


def equal(one, other):
    torch = torch_cuda()
    done()
    for a, b in zip(states(one), states(other)):
        for n in a:
            assert torch.equal(a[n], b[n]), n


# how a tensor of an entry comes to hold what `new` holds
def put(t, name, new):
    t[name] = new.clone()


def move(t, name, new):
    t[name].data = new.clone()


def write(t, name, new):
    t[name].copy_(new)


@pytest.mark.parametrize("how", [put, move, write])
@pytest.mark.parametrize("bits,master", [(8, True), (8, False), (32, True), (32, False)])
def test_a_checkpoint_put_back(bits, master, how):
    """Three steps, their start put back into the same optimizer, three others:
    what the others give from that start. The old tensors stay as they are."""
    torch = torch_cuda()
    one, other = optimizer(bits, master), optimizer(bits, master)
    one.step(gradients(0))
    other.step(gradients(0))
    start = [{n: x.clone() for n, x in s.items()} for s in states(one)]
    for i in (1, 2, 3):
        one.step(gradients(i))
    done()
    kept = [{n: x for n, x in s.items()} if how is put else {} for s in states(one)]
    after = [{n: x.clone() for n, x in s.items()} for s in kept]
    for t, s in zip(one.tensors, start):
        for n, x in s.items():
            how(t, n, x)
    one.steps = 1
    for i in (4, 5, 6):
        one.step(gradients(i))
        other.step(gradients(i))
    equal(one, other)
    for a, b in zip(kept, after):
        for n in a:
            assert torch.equal(a[n], b[n]), f"the replaced {n} was written"


@pytest.mark.parametrize("name", ["weight", "master", "m", "v", "m_scales", "v_scales"])
@pytest.mark.parametrize("how", [put, move])
def test_each_alone(name, how):
    one, other = optimizer(8, True), optimizer(8, True)
    for opt in (one, other):
        opt.step(gradients(0))
    done()
    old = one.tensors[0][name].data
    how(one.tensors[0], name, one.tensors[0][name])
    old.view(torch_cuda().uint8).fill_(7)
    for opt in (one, other):
        opt.step(gradients(1))
    equal(one, other)
    assert (old.view(torch_cuda().uint8) == 7).all()


def test_decays():
    one, other = optimizer(32, True), optimizer(32, True)
    one.step(gradients(0))
    one.tensors[0]["weight_decay"], one.tensors[1]["weight_decay"] = 0.3, 0.2
    one.step(gradients(1))
    other.step(gradients(0))
    other.plan = None
    other.tensors[0]["weight_decay"], other.tensors[1]["weight_decay"] = 0.3, 0.2
    other.step(gradients(1))
    equal(one, other)


def test_a_state_that_does_not_fit_is_refused():
    torch = torch_cuda()
    one, other = optimizer(32, True), optimizer(32, True)
    for opt in (one, other):
        opt.step(gradients(0))
    good = one.tensors[0]["m"]
    for bad, error in ((good[:64], ValueError), (good.half(), TypeError), (good.cpu(), ValueError), (None, ValueError),
                       (one.tensors[0]["v"], tc.HgemmError)):
        one.tensors[0]["m"] = bad
        for _ in range(2):
            with pytest.raises(error):
                one.step(gradients(1))
    one.tensors[0]["m"] = good
    assert one.steps == 1
    for opt in (one, other):
        opt.step(gradients(1))
    equal(one, other)
    assert torch.cuda.is_available()


def test_tensors_of_another_device_than_the_current_one():
    """The step runs on the current device: a table that says another is refused
    before anything is launched."""
    torch = torch_cuda()
    t = {"grad": torch.ones(64, device="cuda"), "master": torch.ones(64, device="cuda"),
         "m": torch.zeros(64, device="cuda"), "v": torch.zeros(64, device="cuda")}
    plan = tc.hgemm_adamw_tensors([t])
    assert plan.device == torch.cuda.current_device()
    plan.device += 1
    for stream in (None, torch.cuda.Stream(), 0):
        with pytest.raises(ValueError, match="current device"):
            tc.hgemm_adamw(plan, 0.1, stream=stream)
    done()
    assert (t["master"] == 1).all() and (t["m"] == 0).all()
    plan.device -= 1
    tc.hgemm_adamw(plan, 0.1)
    done()
    assert (t["master"] != 1).all()
