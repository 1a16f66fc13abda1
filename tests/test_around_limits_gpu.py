"""The operators around the feed-forward block where sizes and callers meet
their limits: offsets past 32 bits, calls at once on several streams, several
captured graphs, empty batches (GPU only)."""

import numpy as np
import pytest

import around_reference as ref
import tensor_core_dense_fp16_gb300 as tc
from gpu_helpers import torch_cuda
from test_block_gpu import check
from test_block_gpu import done as status_ok

pytestmark = pytest.mark.gpu


def done():
    """All streams have come to their end, without an error."""
    torch_cuda().cuda.synchronize()
    status_ok()


def normal(g, *shape, scale=1.0, shift=0.0):
    return (torch_cuda().randn(*shape, generator=g, device="cuda") * scale + shift).half()


def generator(seed):
    return torch_cuda().Generator(device="cuda").manual_seed(seed)


def bits(t):
    torch = torch_cuda()
    return t.contiguous().view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


class Norms:
    """A forward and a backward call on their own buffers."""

    def __init__(self, m, d, kind, seed, tile=None):
        torch = torch_cuda()
        g = generator(seed)
        rows = tile or m

        def matrix(scale=1.0):
            t = normal(g, rows, d, scale=scale)
            return t if rows == m else t.repeat(-(-m // rows), 1)[:m].contiguous()

        self.m, self.d, self.kind = m, d, kind
        self.x, self.y, self.dz, self.dh = matrix(), matrix(), matrix(0.1), matrix(0.1)
        self.gate, self.post, self.pre = (normal(g, d, scale=0.2, shift=1) for _ in range(3))
        self.z, self.h, self.dx, self.dy = (torch.empty_like(self.x) for _ in range(4))
        self.stats = torch.empty(4, m, device="cuda")
        self.sums = [torch.empty(d, device="cuda") for _ in range(5)]
        self.work = torch.empty(tc.hgemm_residual_norm_backward_workspace_size(m, d), dtype=torch.uint8, device="cuda")

    def __call__(self, stream=None):
        m, d, kind = self.m, self.d, self.kind
        tc.hgemm_residual_norm_forward(self.x, d, 0.5, self.y, d, self.gate, kind, self.post, None, kind, self.pre,
                                       None, 1e-5, self.z, d, self.h, d, self.stats, m, d, stream)
        tc.hgemm_residual_norm_backward(self.dz, d, self.dh, d, self.z, d, self.y, d, 0.5, self.gate, kind, self.post,
                                        None, kind, self.pre, self.stats, self.dx, d, self.dy, d, *self.sums,
                                        self.work, m, d, stream=stream)

    def results(self):
        return [self.z, self.h, self.stats, self.dx, self.dy, *self.sums]


class Steps:
    """AdamW on its own tensors, from the same state at every call."""

    def __init__(self, n, eight, seed, count=3):
        torch = torch_cuda()
        g = generator(seed)
        self.tensors, self.start = [], []
        for i in range(count):
            p = normal(g, n + 8 * i)
            t = {"grad": normal(g, n + 8 * i, scale=0.02), "weight": p}
            for name, dtype in (("m", torch.int8), ("v", torch.uint8)):
                t[name] = torch.zeros(n + 8 * i, dtype=dtype if eight else torch.float32, device="cuda")
                if eight:
                    t[name + "_scales"] = torch.zeros(-(-(n + 8 * i) // 64), device="cuda")
            self.tensors.append(t)
            self.start.append(p.clone())
        self.plan = tc.hgemm_adamw_tensors(self.tensors)

    def __call__(self, stream=None):
        torch = torch_cuda()
        with torch.cuda.stream(stream or torch.cuda.current_stream()):
            for t, p in zip(self.tensors, self.start):
                t["weight"].copy_(p)
                for name in ("m", "v", "m_scales", "v_scales"):
                    if name in t:
                        t[name].zero_()
        for step in (1, 2):
            tc.hgemm_adamw(self.plan, 1e-2, step=step, stream=stream)

    def results(self):
        return [t[n] for t in self.tensors for n in t if n != "grad"]


class Experts:
    def __init__(self, m, d, f, e, k, seed):
        torch = torch_cuda()
        g = generator(seed)
        self.sizes, self.k = (m, d, f, e), k
        self.x, self.r, self.wr = normal(g, m, d), normal(g, m, d), normal(g, e, d, scale=2 * d ** -0.5)
        self.w1, self.w2 = normal(g, e, 2 * f, d, scale=d ** -0.5), normal(g, e, d, f, scale=max(1, f) ** -0.5)
        self.y = torch.empty_like(self.x)
        self.chosen = torch.empty(m, k, dtype=torch.int32, device="cuda")
        self.share = torch.empty(m, k, device="cuda")
        self.work = torch.empty(tc.hgemm_experts_workspace_size(m, d, f, e, k), dtype=torch.uint8, device="cuda")

    def __call__(self, stream=None):
        m, d, f, e = self.sizes
        tc.hgemm_experts(self.x, d, self.wr, d, self.w1, d, None, self.w2, f, None, tc.HGEMM_ACT_SILU, True, self.k,
                         True, self.r, d, self.y, d, self.chosen, self.share, self.work, m, d, f, e, stream=stream)

    def results(self):
        return [self.y, self.chosen, self.share]


def several():
    return [Norms(900, 1024, tc.HGEMM_NORM_LAYER, 1), Experts(1, 1024, 1536, 8, 2, 2), Steps(300000, True, 3),
            Norms(700, 2048, tc.HGEMM_NORM_RMS, 4), Experts(24, 512, 520, 16, 4, 5), Steps(5000, False, 6),
            Norms(300, 77, tc.HGEMM_NORM_LAYER, 7), Experts(40, 264, 136, 4, 4, 8)]


def alone(work):
    """Each one's results by itself, copied."""
    want = []
    for w in work:
        w()
        done()
        want.append([t.clone() for t in w.results()])
    return want


def wipe(work):
    for w in work:
        for t in w.results():
            t.view(torch_cuda().uint8).fill_(0x5A)
    torch_cuda().cuda.synchronize()


def equal(work, want, what):
    for i, (w, results) in enumerate(zip(work, want)):
        for j, (a, b) in enumerate(zip(w.results(), results)):
            assert (bits(a) == bits(b)).all(), f"{what}: {type(w).__name__} {i}, result {j}"


def test_calls_at_once_on_their_own_streams():
    """Eight streams, each with an operator of its own, ten rounds without a
    wait: the bits of calls made one by one."""
    torch = torch_cuda()
    work = several()
    want = alone(work)
    wipe(work)
    streams = [torch.cuda.Stream() for _ in work]
    for _ in range(10):
        for w, s in zip(work, streams):
            w(s)
    done()
    equal(work, want, "streams")


def test_one_behind_the_other_without_a_wait():
    """All operators on one stream, each launched while the one before runs."""
    work = several()
    want = alone(work)
    wipe(work)
    for _ in range(5):
        for w in work:
            w()
    done()
    equal(work, want, "one stream")


def test_two_graphs_in_turn_and_at_once():
    """A graph of four operators each, replayed in turn on one stream, then on
    two at once."""
    torch = torch_cuda()
    work = several()
    want = alone(work)
    graphs = []
    for half in (work[:4], work[4:]):
        s = torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            for w in half:
                w(s)
        graphs.append((graph, s))
    wipe(work)
    for _ in range(3):
        for graph, _ in graphs:
            graph.replay()
    done()
    equal(work, want, "in turn")
    wipe(work)
    for _ in range(3):
        for graph, s in graphs:
            with torch.cuda.stream(s):
                graph.replay()
    done()
    equal(work, want, "at once")


def test_calls_from_two_threads():
    import threading
    torch = torch_cuda()
    work = several()
    want = alone(work)
    wipe(work)
    errors = []

    def go(half):
        try:
            s = torch.cuda.Stream()
            for _ in range(5):
                for w in half:
                    w(s)
            s.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=go, args=(half,)) for half in (work[:4], work[4:])]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    done()
    equal(work, want, "threads")


@pytest.mark.parametrize("kind", [tc.HGEMM_NORM_RMS, tc.HGEMM_NORM_LAYER])
@pytest.mark.parametrize("d", [8192, 4099])
def test_rows_past_32_bit_offsets(d, kind):
    """More than 2^31 values: a tile of rows over and over gives the tile's own
    results over and over, and a column's sum is the tiles' sums."""
    torch = torch_cuda()
    tile = 2000
    m = (2 ** 31 // d) // tile * tile + 2 * tile
    small, big = Norms(tile, d, kind, 11), Norms(m, d, kind, 11, tile=tile)
    small()
    big()
    done()
    for a, b in zip(small.results()[:5], big.results()[:5]):
        if a is small.stats:
            assert (bits(b).view(4, -1, tile) == bits(a).view(4, 1, tile)).all()
        else:
            for i in range(0, m, tile):  # (a tile at a time: comparisons take memory)
                assert torch.equal(bits(b[i:i + tile]), bits(a)), f"rows from {i}"
    # Σ dH: the terms are exact, so that a sum is off by at most the number of
    # additions a value passes through (m at most) times 2^-24 of Σ |terms|; in
    # any tree no deeper than 2·m/160 + 1000 rows a slice and the slices, which
    # is what the kernels have.
    tiles = m // tile
    terms = small.dh.double()
    deep = 2 * m / 160 + 1000
    off = (big.sums[4].double() - tiles * terms.sum(0)).abs()
    assert (off <= deep * 2.0 ** -24 * tiles * terms.abs().sum(0)).all()


def test_a_tensor_of_the_largest_size():
    """2^31 − 1 values with 8-bit states, and read back: a block of values over
    and over gives its own results over and over."""
    torch = torch_cuda()
    n, tile = 2 ** 31 - 1, 1 << 20
    g = generator(12)

    def make(size):
        def over(t):
            return t if size == tile else t.repeat(-(-size // tile))[:size].contiguous()
        groups = -(-size // 64)
        g.manual_seed(12)
        t = {"weight": over(normal(g, tile)), "grad": over(normal(g, tile, scale=0.02)),
             "m": torch.zeros(size, dtype=torch.int8, device="cuda"),
             "v": torch.zeros(size, dtype=torch.uint8, device="cuda"),
             "m_scales": torch.zeros(groups, device="cuda"), "v_scales": torch.zeros(groups, device="cuda")}
        out = [torch.empty(size, device="cuda") for _ in range(2)]
        plan = tc.hgemm_adamw_tensors([t])
        for step in (1, 2):
            tc.hgemm_adamw(plan, 1e-2, step=step)
        tc.hgemm_adamw_load(t["m"], t["m_scales"], t["v"], t["v_scales"], *out, size)
        done()
        return [t["weight"], t["m"], t["v"], *out], [t["m_scales"], t["v_scales"]]

    values, scales = make(tile)
    many, many_scales = make(n)
    last = n - n % tile
    for a, b in zip(values, many):
        for i in range(0, last, tile):
            assert torch.equal(bits(b[i:i + tile]), bits(a)), f"values from {i}"
        # (the last group has one value less, which may be its largest)
        whole = n // 64 * 64
        assert torch.equal(bits(b[last:whole]), bits(a[:whole - last]))
    for a, b in zip(scales, many_scales):
        assert torch.equal(bits(b[:last // 64]).view(-1, tile // 64), bits(a).view(1, -1).expand(last // tile, -1))


def test_experts_past_32_bit_offsets():
    """512 experts of 2·4096×1024: 2^32 values of W1, 2^31 of W2; the first and
    the last experts against the formulas in 64 bits."""
    torch = torch_cuda()
    m, d, f, e, k = 2, 1024, 4096, 512, 2
    w = Experts(m, d, f, e, k, 13)
    w.wr.zero_()
    # row i's largest logits are those of experts e−1−i and i
    for i in range(m):
        w.wr[e - 1 - i] = w.x[i] / 64
        w.wr[i] = w.x[i] / 128
    w()
    done()
    chosen = w.chosen.cpu().numpy()
    assert (chosen == [[e - 1 - i, i] for i in range(m)]).all()
    used = sorted(set(chosen.ravel().tolist()))
    host = {n: getattr(w, n)[used].cpu().numpy() for n in ("wr", "w1", "w2")}
    local = np.searchsorted(used, chosen)
    _, _, s, es, want, bound = ref.experts(w.x.cpu().numpy(), host["wr"], host["w1"], None, host["w2"], None, "silu",
                                           True, True, w.r.cpu().numpy(), local)
    check(w.share.cpu().numpy(), s, es, "share")
    check(w.y.cpu().numpy(), want, bound, "y")


def test_an_empty_batch_through_a_stack():
    from tensor_core_dense_fp16_gb300.feedforward import AdamW, ExpertFeedForward, FeedForward, FeedForwardStack
    torch = torch_cuda()
    g = generator(14)
    d, f = 64, 128
    blocks = [FeedForward(normal(g, d, shift=1), None, normal(g, f, d), normal(g, f), normal(g, d, f), normal(g, d),
                          norm="rms", post="layer", post_gamma=normal(g, d, shift=1), gate=normal(g, d))
              for _ in range(2)]
    stack = FeedForwardStack(blocks)
    x = torch.empty(0, d, dtype=torch.float16, device="cuda")
    y, saved = stack.forward(x)
    dx, grads = stack.backward(y, saved)
    assert y.shape == dx.shape == (0, d)
    for b, gr in zip(blocks, grads):
        assert set(gr.named()) == set(b.parameters())
        for n, t in gr.named().items():
            assert (t == 0).all(), n
        before = {n: p.clone() for n, p in b.parameters().items()}
        AdamW(b.parameters(), lr=1e-2, weight_decay=0.0).step(gr.named())
        done()
        for n, p in b.parameters().items():
            assert torch.equal(p, before[n]), n
    experts = ExpertFeedForward(normal(g, 4, d), normal(g, 4, 2 * f, d), normal(g, 4, d, f))
    y, chosen, share = experts(x, residual=x, choices=True)
    assert y.shape == (0, d) and chosen.shape == share.shape == (0, 2)
