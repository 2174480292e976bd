"""One AdamW step over many tensors (ss1_adamw_step).

Every float32 operation of the step is rounded on its own, so a step equals the same formula written
with elementwise torch operations on the CPU bit for bit, codes and scales of the 8-bit states among
them. Against float64 (float32 states) the new moments are off by at most 3 roundings of their terms
(4 u (|b1 m| + |(1 - b1) g|)), and the parameter by u per operation: 2 u |p| + 12 u |update|, with
the update's own terms, plus half a step of the parameter's type.
"""

import math

import pytest
import torch

from tests.gpu_common import get_ss1

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
LR, BETAS, EPS, DECAY = 1e-3, (0.9, 0.999), 1e-8, 0.01


@pytest.fixture(scope="module")
def ops():
    get_ss1()
    from structured_compressed_linear_b200 import ops
    return ops


# ---- the formula with elementwise operations, on the CPU ------------------------------------------

def encode(values, positive):
    n = values.numel()
    v = torch.nn.functional.pad(values.reshape(-1), (0, -n % 256)).reshape(-1, 256)
    mantissa, exponent = torch.frexp(v.abs().amax(1))
    exponent = torch.where(mantissa == 0, -999, exponent)   # nothing but zeros: the smallest scale
    scale = torch.ldexp(torch.ones_like(mantissa), (exponent - torch.where(mantissa <= 0.875, 9, 8)).clamp(min=-126))
    codes = (v / scale[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    if positive:
        codes = torch.where(v > 0, codes.clamp(min=1), codes)
    return codes.reshape(-1)[:n], scale


def decode(codes, scale):
    return codes.reshape(-1).view(torch.float8_e4m3fn).float() * scale.repeat_interleave(256)[:codes.numel()]


def plain_step(p, g, m, v, t, lr=LR, betas=BETAS, eps=EPS, decay=DECAY, grad_scale=1.0):
    """New (p, m, v, sqrt v) in float32."""
    def f(x):
        return torch.tensor(x, dtype=F32)
    b1, b2 = betas
    g = g.float() * f(grad_scale)
    m = m * f(b1) + g * f(1 - b1)
    v = v * f(b2) + (g * g) * f(1 - b2)
    root = torch.sqrt(v.double()).float()   # correctly rounded (the CPU's float32 sqrt is not in every lane)
    den = root * f(1 / math.sqrt(1 - b2 ** t)) + f(eps)
    return p.float() * f(1 - lr * decay) - (m / den) * f(lr / (1 - b1 ** t)), m, v, root


def _tensors(sizes, pt, gt, seed, gscale=1e-3):
    gen = torch.Generator().manual_seed(seed)
    return ([(torch.randn(n, generator=gen) * 0.02).to(pt) for n in sizes],
            [(torch.randn(n, generator=gen) * gscale).to(gt) for n in sizes])


def _cuda(ts):
    return [t.cuda() for t in ts]


SIZES = [1, 7, 8, 255, 256, 257, 8191, 8192, 8193, 20000]
TYPES = [(BF16, BF16, True), (BF16, BF16, False), (BF16, F32, True), (F32, F32, False), (F32, BF16, False)]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("pt,gt,with_master", TYPES)
def test_steps_match_the_formula(ops, bits, pt, gt, with_master):
    """Three steps from zero states, bit for bit; the first two also against float64."""
    p, _ = _tensors(SIZES, pt, gt, 1)
    master = [t.float() + 1e-5 for t in p] if with_master else None
    state = F32 if bits == 32 else torch.uint8
    zeros = [[torch.zeros(n, dtype=state) for n in SIZES] for _ in range(2)]
    scales = None if bits == 32 else tuple([torch.zeros(-(-n // 256)) for n in SIZES] for _ in range(2))
    P, M, Z = _cuda(p), _cuda(master) if master else None, [_cuda(z) for z in zeros]
    S = None if scales is None else tuple(_cuda(s) for s in scales)
    for t in (1, 2, 3):
        _, g = _tensors(SIZES, pt, gt, 10 + t)
        ops.adamw_step(P, _cuda(g), Z[0], Z[1], step=t, lr=LR, betas=BETAS, eps=EPS, weight_decay=DECAY, grad_scale=0.5, master=M,
                       scales=S)
        torch.cuda.synchronize()
        for i in range(len(SIZES)):
            if bits == 32:
                m, v = zeros[0][i], zeros[1][i]
            else:
                m = decode(zeros[0][i], scales[0][i])
                r = decode(zeros[1][i], scales[1][i])
                v = r * r
            old = master[i] if master else p[i]
            new, m1, v1, root = plain_step(old, g[i], m, v, t, grad_scale=0.5)
            g64 = g[i].double() * 0.5
            tol_m = 4 * U * (0.9 * m.double().abs() + 0.1 * g64.abs())
            assert ((m1.double() - (0.9 * m.double() + 0.1 * g64)).abs() <= tol_m).all()
            if master:
                master[i] = new
                assert torch.equal(M[i].cpu(), new)
            p[i] = new.to(pt)
            assert torch.equal(P[i].cpu(), p[i]), (t, SIZES[i])
            if bits == 32:
                zeros[0][i], zeros[1][i] = m1, v1
            else:
                zeros[0][i], scales[0][i] = encode(m1, False)
                zeros[1][i], scales[1][i] = encode(root, True)
                assert torch.equal(S[0][i].cpu(), scales[0][i]) and torch.equal(S[1][i].cpu(), scales[1][i])
            assert torch.equal(Z[0][i].cpu(), zeros[0][i]) and torch.equal(Z[1][i].cpu(), zeros[1][i]), (t, SIZES[i])


def test_against_float64(ops):
    n, t = 50000, 7
    (p,), (g,) = _tensors([n], F32, F32, 3)
    gen = torch.Generator().manual_seed(4)
    m, v = torch.randn(n, generator=gen) * 1e-3, (torch.randn(n, generator=gen) * 1e-3).square()
    P, Mo, V = p.cuda(), m.cuda(), v.cuda()
    ops.adamw_step([P], [g.cuda()], [Mo], [V], step=t, lr=LR, betas=BETAS, eps=EPS, weight_decay=DECAY)
    p, g, m, v = (x.double() for x in (p, g, m, v))
    m1, v1 = 0.9 * m + 0.1 * g, 0.999 * v + 0.001 * g * g
    size = (0.9 * m.abs() + 0.1 * g.abs()) / (1 - 0.9 ** t) / ((v1 / (1 - 0.999 ** t)).sqrt() + EPS) * LR
    p1 = p * (1 - LR * DECAY) - LR * m1 / (1 - 0.9 ** t) / ((v1 / (1 - 0.999 ** t)).sqrt() + EPS)
    assert ((Mo.cpu().double() - m1).abs() <= 4 * U * (0.9 * m.abs() + 0.1 * g.abs())).all()
    assert ((V.cpu().double() - v1).abs() <= 5 * U * v1).all()
    assert ((P.cpu().double() - p1).abs() <= 3 * U * p.abs() + 14 * U * size).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_unaligned_tensors_and_guards(ops, bits):
    """Tensors at odd offsets of one buffer (the scalar loads): the same bits, and nothing between them is touched."""
    sizes, pad = [300, 513, 1], 3
    (p, g) = _tensors(sizes, BF16, BF16, 5)
    state = F32 if bits == 32 else torch.uint8

    def run(shift):
        def place(ts, dt):
            flat = torch.full((sum(sizes) + (len(sizes) + 1) * 64,), 9, dtype=dt, device="cuda")
            out, at = [], 64 if not shift else 64 + pad
            for t in ts:
                out.append(flat[at:at + t.numel()])
                out[-1].copy_(t)
                at += t.numel() + (-t.numel() % 64 if not shift else pad)
            return out, flat
        P, pf = place(p, BF16)
        G, gf = place(g, BF16)
        Ms, mf = place([torch.zeros(n) for n in sizes], state)
        Vs, vf = place([torch.zeros(n) for n in sizes], state)
        sc = None if bits == 32 else tuple([torch.zeros(-(-n // 256), device="cuda") for n in sizes] for _ in range(2))
        for t in (1, 2):
            ops.adamw_step(P, G, Ms, Vs, step=t, scales=sc)
        torch.cuda.synchronize()
        inside = sum(t.numel() for t in P)
        for flat, views in ((pf, P), (mf, Ms), (vf, Vs)):
            kept = (flat == 9).sum().item() - sum((v == 9).sum().item() for v in views)
            assert kept == flat.numel() - inside
        return [x.clone() for x in (*P, *Ms, *Vs)] + ([] if sc is None else [s.clone() for part in sc for s in part])
    for a, b in zip(run(False), run(True)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("count", [32, 33, 440, 441, 900])
def test_many_tensors(ops, count):
    """Table sizes on both sides of a launch's limits, empty tensors among them."""
    sizes = [(37 * i) % 700 for i in range(count)]
    p, g = _tensors(sizes, F32, F32, 6)
    P, Z = _cuda(p), [[torch.zeros(n, device="cuda") for n in sizes] for _ in range(2)]
    ops.adamw_step(P, _cuda(g), Z[0], Z[1], step=1)
    torch.cuda.synchronize()
    for i, n in enumerate(sizes):
        assert torch.equal(P[i].cpu(), plain_step(p[i], g[i], torch.zeros(n), torch.zeros(n), 1)[0]), i


def test_zero_tiny_and_nonfinite_gradients(ops):
    """8-bit states: an all-zero block, subnormal moments, one block's NaN and infinity leave the others alone."""
    n = 256 * 6
    p = torch.randn(n, generator=torch.Generator().manual_seed(8)) * 0.02
    g = torch.randn(n, generator=torch.Generator().manual_seed(9)) * 1e-3
    g[256:512] = 0.0
    g[512:768] *= 1e-36
    clean = g.clone()
    g[800], g[1100] = float("nan"), float("inf")
    out = []
    for grad in (clean, g):
        P, Mc, Vc = p.cuda(), torch.zeros(n, dtype=torch.uint8, device="cuda"), torch.zeros(n, dtype=torch.uint8, device="cuda")
        S = ([torch.zeros(6, device="cuda")], [torch.zeros(6, device="cuda")])
        ops.adamw_step([P], [grad.cuda()], [Mc], [Vc], step=1, scales=S)
        torch.cuda.synchronize()
        out.append([t.cpu() for t in (P, Mc, Vc, S[0][0], S[1][0])])
        z = torch.zeros(n)
        new, m, v, root = plain_step(p, grad, z, z, 1)
        assert torch.equal(out[-1][0].nan_to_num(7.0), new.nan_to_num(7.0))
        for want, codes, sc in ((encode(m, False), out[-1][1], out[-1][3]), (encode(root, True), out[-1][2], out[-1][4])):
            keep = torch.ones(6, dtype=torch.bool)
            if grad is g:
                keep[3] = keep[4] = False    # a block with a NaN or an infinity has no scale to agree on
            assert torch.equal(codes.reshape(6, 256)[keep], want[0].reshape(6, 256)[keep]) and torch.equal(sc[keep], want[1][keep])
    assert not out[0][1][256:512].any() and not out[0][2][256:512].any()
    a, b = (o[0].reshape(6, 256) for o in out)
    assert torch.equal(a[[0, 1, 2, 5]], b[[0, 1, 2, 5]]) and b[3].isnan().sum() == 1 and b[4].isnan().sum() == 1
    tiny = out[0][2][512:768]
    assert (tiny[clean[512:768].float().square() * 1e-3 > 0] >= 1).all()


def test_positive_roots_stay_positive(ops):
    """With zero gradients a moment only shrinks by beta: a positive root never becomes 0 by rounding to its code."""
    n = 2048
    gen = torch.Generator().manual_seed(10)
    codes, scale = encode(torch.randn(n, generator=gen) * 1e-3, False)
    rcodes, rscale = encode(torch.rand(n, generator=gen) * 1e-3, True)
    M, V, S = codes.cuda(), rcodes.cuda(), ([scale.cuda()], [rscale.cuda()])
    P, G = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    for t in range(1, 200):
        ops.adamw_step([P], [G], [M], [V], step=t, betas=(0.5, 0.5), scales=S)
        if t <= 60:   # roots of 2^-28 and more have v >= 2^-(56 + 60) there; past 2^-149 v itself is 0 in float32
            assert (V[rcodes.cuda() > 0] > 0).all()
    torch.cuda.synchronize()
    assert P.isfinite().all()


def test_device_factors_and_graph(ops):
    """A captured step replayed with new factors equals the eager steps."""
    n = 5000
    (p,), (g,) = _tensors([n], BF16, BF16, 12)
    mk = lambda: ([p.clone().cuda()], [p.float().cuda()], [torch.zeros(n, device="cuda")], [torch.zeros(n, device="cuda")])  # noqa: E731
    A, B = mk(), mk()
    G = [g.cuda()]
    factors = ops.adamw_factors(1, lr=1e-2).cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.adamw_step(B[0], G, B[2], B[3], master=B[1], factors=factors)
    for t in (1, 2, 3):
        lr = 1e-2 / t
        ops.adamw_step(A[0], G, A[2], A[3], step=t, lr=lr, master=A[1])
        factors.copy_(ops.adamw_factors(t, lr=lr))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(A, B):
            assert torch.equal(a[0], b[0])


def test_optimizer_class(ops):
    """AdamW over mixed parameters: skips those without a gradient, resumes from a state_dict."""
    gen = torch.Generator().manual_seed(13)

    def make():
        gen.manual_seed(13)
        return [(torch.randn(*s, generator=gen) * 0.02).to(t).cuda().requires_grad_()
                for s, t in (((64, 48), BF16), ((77,), F32), ((8, 300), BF16), ((5,), F32))]
    for bits in (32, 8):
        runs = []
        for resume in (False, True):
            ps = make()
            opt = ops.AdamW(ps, lr=1e-2, state_bits=bits, master=True)
            for t in range(4):
                if resume and t == 2:
                    old, opt = opt, ops.AdamW(ps, lr=1e-2, state_bits=bits, master=True)
                    opt.load_state_dict(old.state_dict())
                for i, p in enumerate(ps):
                    p.grad = None if i == 3 and t < 2 else torch.randn(p.shape, generator=torch.Generator().manual_seed(t)).to(p.dtype).cuda()
                opt.step()
            assert opt.steps == 4
            runs.append([p.detach().clone() for p in ps] + opt.exp_avg)
        for a, b in zip(*runs):
            assert torch.equal(a, b)
        fresh = make()
        assert all(not torch.equal(a, b) for a, b in zip(runs[0], fresh))
    with pytest.raises(ValueError):
        ops.AdamW([fresh[0], fresh[0]])
    with pytest.raises(ValueError):
        ops.AdamW(fresh, state_bits=16)


def test_refusals_change_nothing(ops):
    (p,), (g,) = _tensors([300], BF16, BF16, 14)
    P, G, M, V = p.cuda(), g.cuda(), torch.zeros(300, device="cuda"), torch.zeros(300, device="cuda")
    eight = torch.zeros(300, dtype=torch.uint8, device="cuda")
    sc = [torch.zeros(2, device="cuda")]
    for bad in (lambda: ops.adamw_step([P], [G], [M[:-1]], [V]), lambda: ops.adamw_step([P], [G, G], [M], [V]),
                lambda: ops.adamw_step([P], [G], [eight], [eight]), lambda: ops.adamw_step([P], [G], [M], [V], scales=(sc, sc)),
                lambda: ops.adamw_step([P], [G], [eight], [eight], scales=([sc[0][:1]], sc)),
                lambda: ops.adamw_step([P], [G.half()], [M], [V]), lambda: ops.adamw_step([P], [G.cpu()], [M], [V]),
                lambda: ops.adamw_step([P], [G], [M], [V], master=[M[::2]]), lambda: ops.adamw_step([P], [G], [M], [V], betas=(1.0, 0.9)),
                lambda: ops.adamw_step([P], [G], [M], [V], step=0), lambda: ops.adamw_step([P.float()], [G], [M], [V], master=[V]),
                lambda: ops.adamw_step([P], [G], [M], [V], factors=M[:3]), lambda: ops.adamw_step([P, P], [G, G], [M, V], [V, M])):
        with pytest.raises((ValueError, TypeError, RuntimeError)):
            bad()
    torch.cuda.synchronize()
    assert torch.equal(P.cpu(), p) and not M.any() and not V.any()


def test_offsets_past_32_bits(ops):
    """One tensor of more than 2^31 elements, 8-bit states: its end steps like a small tensor."""
    n, last = 2 ** 31 + 256 * 40 + 77, 256 * 20 + 77
    P = torch.full((n,), 0.5, dtype=BF16, device="cuda")
    G = torch.full((n,), 1e-3, dtype=BF16, device="cuda")
    (g,) = _tensors([last], BF16, BF16, 15)[1]
    G[-last:] = g.cuda()
    S = [torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2)]
    sc = tuple([torch.zeros(-(-n // 256), device="cuda")] for _ in range(2))
    ops.adamw_step([P], [G], [S[0]], [S[1]], step=1, scales=sc)
    torch.cuda.synchronize()
    p = torch.full((last,), 0.5, dtype=BF16)
    new, m, v, root = plain_step(p, g, torch.zeros(last), torch.zeros(last), 1)
    assert torch.equal(P[-last:].cpu(), new.to(BF16))
    for codes, scales, (wc, ws) in ((S[0], sc[0][0], encode(m, False)), (S[1], sc[1][0], encode(root, True))):
        assert torch.equal(codes[-last:].cpu(), wc) and torch.equal(scales[-(-(-last // 256)):].cpu(), ws)
