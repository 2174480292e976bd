"""8-bit AdamW states over many steps (ss1_adamw_step, ss1_adamw_step_ex): bit for bit the CPU form of their
definition, and 2000 steps beside float32 moments, within the bounds that test_adamw_states.py derives."""

import math

import pytest
import torch

from tests import adamw_states as S
from tests.gpu_common import get_ss1
from tests.test_adamw_states import bounds

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
LR, BETAS, EPS, DECAY = 1e-3, (0.9, 0.999), 1e-8, 0.01


@pytest.fixture(scope="module")
def ops():
    get_ss1()
    from structured_compressed_linear_b200 import ops
    return ops


def _start(sizes, seed, dtype=F32):
    """Parameters and 8-bit states of a run that is under way: (p, [m codes, root codes], [m scales, root scales])."""
    gen = torch.Generator().manual_seed(seed)
    p = [(torch.randn(n, generator=gen) * 0.02).to(dtype) for n in sizes]
    m = [S.encode(torch.randn(n, generator=gen) * 1e-3, False, 1) for n in sizes]
    r = [S.encode(torch.randn(n, generator=gen).abs() * 1e-3, True, 1) for n in sizes]
    return p, [[x[0] for x in m], [x[0] for x in r]], [[x[1] for x in m], [x[1] for x in r]]


SIZES = [1, 7, 8, 255, 256, 257, 8193, 20000]


@pytest.mark.parametrize("shift", [0, 3])
@pytest.mark.parametrize("t", [9, 10, 11, 12, 1000, (1 << 32) + 5])
def test_a_step_equals_the_definition(ops, t, shift):
    """One step of several tensors, on both sides of the change of rounding, aligned and not: codes, scales and
    parameters; and the same again from the same state."""
    p, codes, scales = _start(SIZES, 1)
    g = [torch.randn(n, generator=torch.Generator().manual_seed(n)) * 1e-3 for n in SIZES]

    def place(ts, dt):
        flat = torch.zeros(sum(SIZES) + 64 * len(SIZES), dtype=dt, device="cuda")
        out, at = [], shift
        for x in ts:
            out.append(flat[at:at + x.numel()])
            out[-1].copy_(x)
            at += x.numel() + (shift if shift else -x.numel() % 64)
        return out
    runs = []
    for _ in range(2):
        P, M, R = place(p, F32), place(codes[0], torch.uint8), place(codes[1], torch.uint8)
        sc = tuple([x.cuda() for x in s] for s in scales)
        ops.adamw_step(P, place(g, F32), M, R, step=t, lr=LR, betas=BETAS, eps=EPS, weight_decay=DECAY, scales=sc)
        torch.cuda.synchronize()
        runs.append([x.cpu() for x in (*P, *M, *R, *sc[0], *sc[1])])
    assert all(torch.equal(a, b) for a, b in zip(*runs))
    k = len(SIZES)
    for i in range(k):
        m, r = S.decode(codes[0][i], scales[0][i]), S.decode(codes[1][i], scales[1][i])
        new, m1, _, root = S.plain_step(p[i], g[i], m, r * r, t, LR, BETAS, EPS, DECAY)
        for at, want in ((0, new), (k, S.encode(m1, False, t)[0]), (2 * k, S.encode(root, True, t)[0]),
                         (3 * k, S.encode(m1, False, t)[1]), (4 * k, S.encode(root, True, t)[1])):
            assert torch.equal(runs[0][at + i], want), (SIZES[i], at)


def test_nan_infinity_and_zero(ops):
    """Past the nearest steps: a block of zeros stays zero, a NaN stays one, an infinity saturates; other blocks are as without."""
    n = 256 * 4
    p, codes, scales = _start([n], 2)
    codes[0][0][:256] = codes[1][0][:256] = 0
    g = torch.randn(n, generator=torch.Generator().manual_seed(3)) * 1e-3
    g[:256] = 0
    bad = g.clone()
    bad[300], bad[600] = float("nan"), float("inf")
    out = []
    for grad in (g, bad):
        P, M, R = p[0].cuda(), codes[0][0].cuda(), codes[1][0].cuda()
        sc = tuple([x[0].cuda()] for x in scales)
        ops.adamw_step([P], [grad.cuda()], [M], [R], step=500, scales=sc)
        torch.cuda.synchronize()
        out.append([x.cpu() for x in (P, M, R)])
    assert not out[0][1][:256].any() and not out[0][2][:256].any()
    for a, b in zip(*out):
        assert torch.equal(a[:256], b[:256]) and torch.equal(a[768:], b[768:])
    assert out[1][0].isnan().sum() == 2 and int(out[1][1][300]) & 0x7F == 0x7F and int(out[1][2][300]) == 0x7F
    assert int(out[1][1][600]) & 0x7F == 0x7E and int(out[1][2][600]) == 0x7E


def test_positive_roots_stay_positive(ops):
    """Zero gradients, 500 steps past the nearest ones: the moments shrink, and no positive root becomes 0."""
    p, codes, scales = _start([4096], 4)
    M, R = codes[0][0].cuda(), codes[1][0].cuda()
    sc = tuple([x[0].cuda()] for x in scales)
    P, G = torch.zeros(4096, device="cuda"), torch.zeros(4096, device="cuda")
    before = S.decode(codes[1][0], scales[1][0])
    for t in range(11, 511):
        ops.adamw_step([P], [G], [M], [R], step=t, betas=(0.9, 0.99), weight_decay=0.0, scales=sc)
    torch.cuda.synchronize()
    held = S.decode(R.cpu(), sc[1][0].cpu())
    assert (held[before > 0] > 0).all() and P.isfinite().all()
    # 0.99^250 = 0.081 of the roots on average; each deviates by a variance of at most 500 * 0.005 / 8, 4096 of them together
    # by 5 * sqrt(0.32 / 4096) = 4.4 % of their sum's largest terms; the smallest code's floor is 2^-9 of a block's largest
    ratio = float(held.double().sum() / before.double().sum()) / 0.99 ** 250
    assert 0.85 <= ratio <= 1.15, ratio


def test_captured_steps_count_on(ops):
    """A captured step with the number on the device, replayed, equals eager steps; and what has no number is refused."""
    n = 5000
    runs = []
    p, codes, scales = _start([n], 5, BF16)
    g = [(torch.randn(n, generator=torch.Generator().manual_seed(6)) * 1e-3).to(BF16).cuda()]

    def make():
        return ([x.cuda() for x in p], [codes[0][0].cuda()], [codes[1][0].cuda()], tuple([s[0].cuda()] for s in scales),
                [p[0].float().cuda()])
    A, B = make(), make()
    factors, number = ops.adamw_factors(1).cuda(), torch.full((1,), 8, dtype=torch.int64, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        number.add_(1)
        ops.adamw_step(B[0], g, B[1], B[2], master=B[4], scales=B[3], factors=factors, device_step=number)
    for t in range(9, 15):
        ops.adamw_step(A[0], g, A[1], A[2], step=t, master=A[4], scales=A[3])
        factors.copy_(ops.adamw_factors(t))
        graph.replay()
        torch.cuda.synchronize()
        assert int(number) == t
        for a, b in zip((*A[0], *A[1], *A[2], *A[3][0], *A[3][1], *A[4]), (*B[0], *B[1], *B[2], *B[3][0], *B[3][1], *B[4])):
            assert torch.equal(a, b), t
        runs.append(A[2][0].clone())
    assert any(not torch.equal(a, b) for a, b in zip(runs, runs[1:]))
    for bad in (dict(factors=factors), dict(device_step=number), dict(factors=factors, device_step=number.int()),
                dict(factors=factors, device_step=number.cpu())):
        with pytest.raises(ValueError):
            ops.adamw_step(A[0], g, A[1], A[2], scales=A[3], **bad)


@pytest.mark.parametrize("beta2", [0.95, 0.99, 0.999])
@pytest.mark.parametrize("kind", S.KINDS)
def test_many_steps_follow_float32_moments(ops, kind, beta2):
    n, steps, betas = 16384, 2000, (0.9, beta2)
    zeros = torch.zeros(n, device="cuda")
    P = [torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")]
    m32, v32 = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    m8, r8 = torch.zeros(n, dtype=torch.uint8, device="cuda"), torch.zeros(n, dtype=torch.uint8, device="cuda")
    sc = ([torch.zeros(n // 256, device="cuda")], [torch.zeros(n // 256, device="cuda")])
    sums = torch.zeros(2, 2, dtype=torch.float64, device="cuda")
    for t, g in enumerate(S.gradients(kind, n, steps), 1):
        G = [g.cuda()]
        for x in P:
            x.copy_(zeros)
        ops.adamw_step(P[:1], G, [m8], [r8], step=t, lr=1.0, betas=betas, eps=1e-12, weight_decay=0.0, scales=sc)
        ops.adamw_step(P[1:], G, [m32], [v32], step=t, lr=1.0, betas=betas, eps=1e-12, weight_decay=0.0)
        both = torch.stack([x.double().square().mean() for x in P])
        sums[0] += both
        if t > steps - steps // 10:
            sums[1] += both
    sums = sums.cpu()
    root = S.decode(r8.cpu(), sc[1][0].cpu()) / v32.cpu().sqrt()
    got = (math.sqrt(sums[0, 0] / sums[0, 1]), math.sqrt(sums[1, 0] / sums[1, 1]), float(root.median()))
    for ratio, bound in zip(got, bounds(kind, beta2)):
        assert abs(ratio - 1) <= bound, got
