"""The class AdamW: every parameter's own step number, in eager and captured steps and in checkpoints."""

import pytest
import torch

from tests import adamw_states as S
from tests.gpu_common import get_ss1

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
LR, BETAS, EPS, DECAY = 1e-2, (0.9, 0.999), 1e-8, 0.01


@pytest.fixture(scope="module")
def ops():
    get_ss1()
    from structured_compressed_linear_b200 import ops
    return ops


def _grad(n, t):
    return torch.randn(n, generator=torch.Generator().manual_seed(t)) * 1e-3


class Plain:
    """One parameter's steps on the CPU, with a step number of its own."""

    def __init__(self, p, bits):
        self.p, self.bits, self.t = p, bits, 0
        self.m = self.v = torch.zeros_like(p)

    def step(self, g):
        self.t += 1
        self.p, m, v, root = S.plain_step(self.p, g, self.m, self.v, self.t, LR, BETAS, EPS, DECAY)
        if self.bits == 8:
            m = S.decode(*S.encode(m, False, self.t))
            v = S.decode(*S.encode(root, True, self.t))
            v = v * v
        self.m, self.v = m, v


@pytest.mark.parametrize("bits", [32, 8])
def test_late_parameters_start_at_step_one(ops, bits):
    """Parameters that join at steps 1, 6 and 20, and one that pauses: each bit for bit as if it were alone."""
    sizes, T = [300, 513, 77, 1000], 26
    start = [torch.randn(n, generator=torch.Generator().manual_seed(n)) * 0.02 for n in sizes]
    ps = [p.cuda().requires_grad_() for p in start]
    opt = ops.AdamW(ps, lr=LR, betas=BETAS, eps=EPS, weight_decay=DECAY, state_bits=bits)
    plain = [Plain(p.clone(), bits) for p in start]
    assert opt.steps == 0
    opt.step()                                     # nobody has a gradient: nothing happens
    assert opt.steps == 0 and opt.counts() == [0] * 4
    for t in range(1, T + 1):
        there = [True, t >= 6, t >= 20, t % 3 != 0]
        for i, p in enumerate(ps):
            p.grad = _grad(sizes[i], 100 * t + i).cuda() if there[i] else None
            if there[i]:
                plain[i].step(_grad(sizes[i], 100 * t + i))
        opt.step()
        torch.cuda.synchronize()
        for i, p in enumerate(ps):
            assert torch.equal(p.detach().cpu(), plain[i].p), (t, i)
    assert opt.counts() == [x.t for x in plain] and opt.steps == T
    other = ops.AdamW([p.detach().clone() for p in ps], lr=LR, state_bits=bits)
    other.load_state_dict(opt.state_dict())
    assert other.counts() == opt.counts()


def test_first_step_of_a_late_parameter(ops):
    """The first update is lr * sign(gradient), whatever the others' step number (eps and rounding aside)."""
    a, b = (torch.zeros(64, device="cuda", requires_grad=True) for _ in range(2))
    opt = ops.AdamW([a, b], lr=LR, weight_decay=0.0)
    for t in range(100):
        a.grad = torch.ones(64, device="cuda")
        opt.step()
    b.grad = torch.full((64,), -0.5, device="cuda")
    opt.step()
    # three roundings of the quotient's terms and the float32 factors': 2^-21 in all, and eps / 0.5
    assert ((b.detach() - LR).abs() <= LR * (2.0 ** -20 + 2 * EPS)).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_replays_are_counted(ops, bits):
    """Eager steps, then replays of a captured one, then eager ones again: the same bits as eager steps throughout,
    the same step numbers, and a checkpoint that goes on from there."""
    n = 3000
    start = torch.randn(n, generator=torch.Generator().manual_seed(1)) * 0.02
    runs = []
    for captured in (False, True):
        p = start.cuda().to(BF16).requires_grad_()
        opt = ops.AdamW([p], lr=LR, betas=BETAS, eps=EPS, weight_decay=DECAY, state_bits=bits, master=True)
        p.grad = torch.zeros(n, dtype=BF16, device="cuda")
        grad = [_grad(n, t).to(BF16).cuda() for t in range(1, 31)]
        for t in range(1, 6):
            p.grad.copy_(grad[t - 1])
            opt.step()
        if captured:
            factors = torch.zeros(ops.ADAMW_FACTORS, device="cuda")
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                opt.step(factors=factors)
            assert opt.steps == 5                  # capturing runs nothing
        for t in range(6, 21):
            p.grad.copy_(grad[t - 1])
            if captured:
                factors.copy_(ops.adamw_factors(t, LR, BETAS, EPS, DECAY))
                graph.replay()
            else:
                opt.step()
        assert opt.steps == 20 and opt.state_dict()["steps"] == 20
        for t in range(21, 26):
            p.grad.copy_(grad[t - 1])
            opt.step()
        assert opt.counts() == [25]
        q = p.detach().clone().requires_grad_()
        second = ops.AdamW([q], lr=LR, betas=BETAS, eps=EPS, weight_decay=DECAY, state_bits=bits, master=True)
        second.load_state_dict(opt.state_dict())
        for t in range(26, 31):
            q.grad = grad[t - 1]
            second.step()
        torch.cuda.synchronize()
        assert second.counts() == [30]
        runs.append([x.detach().clone() for x in (p, q, *opt.master, *second.master, *second.exp_avg, *second.exp_avg_sq)])
    for a, b in zip(*runs):
        assert torch.equal(a, b)


def test_replays_on_another_stream_are_counted(ops):
    """A replay that waits behind other work on a stream of its own is part of the count."""
    p = torch.zeros(64, device="cuda", requires_grad=True)
    p.grad = torch.ones(64, device="cuda")
    opt = ops.AdamW([p], lr=LR)
    factors = ops.adamw_factors(1, LR).cuda()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        opt.step(factors=factors)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)              # about ten milliseconds
        graph.replay()
    assert opt.steps == 1
    torch.cuda.synchronize()


def test_eager_steps_with_factors(ops):
    """step(factors=...) without a graph, 8 bits: as without factors."""
    n = 700
    runs = []
    for given in (False, True):
        p = (torch.randn(n, generator=torch.Generator().manual_seed(2)) * 0.02).cuda().requires_grad_()
        opt = ops.AdamW([p], lr=LR, state_bits=8)
        for t in range(1, 16):
            p.grad = _grad(n, t).cuda()
            opt.step(factors=ops.adamw_factors(t, LR).cuda() if given else None)
        torch.cuda.synchronize()
        assert opt.steps == 15
        runs.append([p.detach().clone(), *opt.exp_avg, *opt.exp_avg_sq])
    assert all(torch.equal(a, b) for a, b in zip(*runs))


def test_refusals(ops):
    a, b = (torch.zeros(64, device="cuda", requires_grad=True) for _ in range(2))
    opt = ops.AdamW([a, b])
    a.grad = torch.ones(64, device="cuda")
    factors = ops.adamw_factors(1).cuda()
    with torch.cuda.graph(torch.cuda.CUDAGraph()):
        with pytest.raises(ValueError):
            opt.step()                             # captured without factors
        opt.step(factors=factors)
    with torch.cuda.graph(torch.cuda.CUDAGraph()):
        b.grad = a.grad
        a.grad.add_(0)                             # something to capture
        with pytest.raises(ValueError):
            opt.step(factors=factors)              # a second graph with other parameters
    b.grad = None
    opt.step()
    b.grad = a.grad
    with pytest.raises(ValueError):
        opt.step(factors=factors)                  # a is at step 1, b at 0
    with pytest.raises(ValueError):
        opt.load_state_dict(dict(opt.state_dict(), counts=[1]))
    before = a.detach().clone(), opt.counts()
    b.grad = torch.ones(128, device="cuda")[::2]
    with pytest.raises(ValueError):
        opt.step()                                 # b's gradient is not contiguous: a is not updated either
    torch.cuda.synchronize()
    assert torch.equal(a.detach(), before[0]) and opt.counts() == before[1]
    old = {k: v for k, v in opt.state_dict().items() if k != "counts"}
    opt.load_state_dict(dict(old, steps=7))
    assert opt.counts() == [7, 7] and opt.steps == 7


@pytest.mark.parametrize("bits", [32, 8])
def test_a_state_of_other_parameters_changes_nothing(ops, bits):
    """States whose tensors would only broadcast, or that are short of some, are refused before anything is copied."""
    def make(sizes, master=True):
        ps = [torch.ones(n, dtype=BF16, device="cuda", requires_grad=True) for n in sizes]
        opt = ops.AdamW(ps, state_bits=bits, master=master)
        for p in ps:
            p.grad = torch.ones_like(p)
        opt.step()
        return opt

    def tensors(opt):
        return [t.clone() for part in (opt.exp_avg, opt.exp_avg_sq, opt.master, *(opt.scales or ())) for t in part]
    mine, good = make((600, 300)), make((600, 300)).state_dict()
    before = tensors(mine)
    bad = [make((600, 1)).state_dict(), make((600, 300), master=False).state_dict(), dict(good, exp_avg_sq=good["exp_avg_sq"][:1]),
           dict(good, master=good["master"][:1]), dict(good, exp_avg_sq=[t.double() for t in good["exp_avg_sq"]]),
           dict(good, state_bits=40 - bits), dict(good, counts=[3])]
    if bits == 8:
        bad += [dict(good, scales=(good["scales"][0], good["scales"][1][:1])), dict(good, scales=None),
                dict(good, scales=(good["scales"][0], [t[:1] for t in good["scales"][1]]))]
    for i, state in enumerate(bad):
        for x in (state["exp_avg"][0], state["exp_avg_sq"][0]):
            x.add_(1)                              # what a partial load would bring in
        with pytest.raises(ValueError):
            mine.load_state_dict(state)
        assert all(torch.equal(a, b) for a, b in zip(before, tensors(mine))), i
        assert mine.counts() == [1, 1]
    mine.load_state_dict(good)


def test_a_tensor_given_twice_is_refused(ops):
    """Whatever is written may be given once only, whichever list it is in; gradients may be shared; empty tensors have no address."""
    def new(k, dt=F32):
        return [torch.zeros(300, dtype=dt, device="cuda") for _ in range(k)]
    P, (g,), M, V, W = new(2, BF16), new(1, BF16), new(2), new(2), new(2)
    eight, sc = new(4, torch.uint8), [torch.zeros(2, device="cuda") for _ in range(4)]
    G = [g, g]
    for bad in (lambda: ops.adamw_step(P, G, M, M), lambda: ops.adamw_step(P, G, [M[0], M[0]], V), lambda: ops.adamw_step(P, G, M, [V[0], M[0]]),
                lambda: ops.adamw_step(P, G, M, V, master=[W[0], W[0]]), lambda: ops.adamw_step(P, G, M, V, master=[None, M[1]]),
                lambda: ops.adamw_step(P[:1], G[:1], M[:1], V[:1], master=V[:1]),
                lambda: ops.adamw_step(P, G, eight[:2], eight[2:], scales=(sc[:2], sc[:2])),
                lambda: ops.adamw_step(P, G, eight[:2], eight[:2], scales=(sc[:2], sc[2:]))):
        with pytest.raises(ValueError, match="twice"):
            bad()
    torch.cuda.synchronize()
    assert not any(t.any() for t in (*P, *M, *V, *W, *eight, *sc))
    empty = [torch.zeros(0, device="cuda") for _ in range(3)]
    ops.adamw_step(empty, empty, empty, empty)
    ops.adamw_step([*P, empty[0]], [*G, empty[0]], [*M, empty[0]], [*V, empty[0]], master=[W[0], None, None])
    flat = torch.zeros(1000, device="cuda")        # neighbours touch, but do not overlap; a gradient that is its parameter
    ops.adamw_step([flat[:100]], [flat[:100]], [flat[100:200]], [flat[200:300]])
    ops.adamw_step([flat[:100], flat[300:400]], [flat[800:900], flat[850:950]], [flat[100:200], flat[400:500]], [flat[200:300], flat[500:600]])
    with pytest.raises(ValueError, match="overlaps"):
        ops.adamw_step([flat[:100]], [flat[300:400]], [flat[99:199]], [flat[200:300]])
    with pytest.raises(ValueError, match="overlaps"):
        ops.adamw_step([flat[:100]], [flat[50:150]], [flat[400:500]], [flat[200:300]])
