"""Low-rank adapters of many requests (ss1_adapter_*) against the formulas in float64.

Tolerances, with u = 2^-24 and h = finfo(type).eps / 2 of the output's type. A product of C terms
adds at most 16 terms at a time into a float32 sum, by additions that are off by at most 2 u of what
they give, so it is off by at most p(C) = 2 u (C / 16 + 32) times the sum of the magnitudes |terms|
(the 32 covers the partial sums of threads, CTAs and shares). The second product of each chain
takes H or G as two bf16 parts, which leaves out at most 2^-17 of each. So
  H   : p(K) sum|x a|                                                       =: eH
  out : h |out| + s (sum_r eH |b| + (p(R) + 2^-17) sum_r |H b|) + 2 u (|Y| + |out|)
  G   : s p(N) sum|dy b|                                                    =: eG
  dX  : h |dX| + sum_r eG |a| + (p(R) + 2^-17) sum_r |G a| + 2 u (|dX_in| + |dX|)
  dA  : h |dA| + sum_m eG |x| + (p(rows) + 2^-17) sum_m |G x|
  dB  : h |dB| + s (p(rows) + 2^-17 + 2 u) sum_m |dy H|
"""

import pytest
import torch

from tests.gpu_common import get_ss1

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


@pytest.fixture(scope="module")
def ops():
    get_ss1()
    from structured_compressed_linear_b200 import ops
    return ops


def p(C):
    return 2 * U * (C / 16 + 32)


def _half(t):
    return torch.finfo(t).eps / 2


def _inputs(M, K, N, R, n, t, seed):
    g = torch.Generator().manual_seed(seed)
    d = {"X": torch.randn(M, K, generator=g).to(t), "A": (torch.randn(n, R, K, generator=g) * K ** -0.5).to(t),
         "B": (torch.randn(n, N, R, generator=g) * 0.05).to(t), "Y": torch.randn(M, N, generator=g).to(t),
         "dY": torch.randn(M, N, generator=g).to(t), "dX": torch.randn(M, K, generator=g).to(t),
         "scale": 0.5 + torch.rand(n, generator=g), "H": torch.randn(M, R, generator=g)}
    return {k: v.cuda() for k, v in d.items()}


def _index(kind, M, n, seed):
    if kind == "one":
        return None
    g = torch.Generator().manual_seed(seed)
    if kind == "random":
        idx = torch.randint(-1, n, (M,), generator=g)
    elif kind == "sorted":
        idx = torch.sort(torch.randint(-1, n, (M,), generator=g))[0]
    elif kind == "none":
        idx = torch.full((M,), -1)
    elif kind == "last":
        idx = torch.full((M,), n - 1)
    elif kind == "outside":
        idx = torch.randint(-1, n, (M,), generator=g)
        idx[::3] = n
        idx[1::7] = 2 ** 31 - 1
        idx[2::11] = -2 ** 31
    return idx.to(torch.int32).cuda()


def _groups(index, M, n):
    index = torch.zeros(M, dtype=torch.int32, device="cuda") if index is None else index
    return [(a, torch.nonzero(index == a)[:, 0]) for a in range(n)]


def _close(got, want, tol, what):
    off = (got.double() - want).abs()
    bad = ~(off <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((off / tol.clamp(min=1e-300)).max()):.3g} x tolerance"


def check_forward(ops, d, index, use_scale=True, plan=None, out=None):
    t, (M, K), (n, N, R) = d["X"].dtype, d["X"].shape, d["B"].shape
    got, H = ops.adapter_forward(d["X"], d["A"], d["B"], d["Y"], index, d["scale"] if use_scale else None, keep=True, plan=plan, out=out)
    torch.cuda.synchronize()
    x, A, B = d["X"].double(), d["A"].double(), d["B"].double()
    want, wantH = d["Y"].double().clone(), torch.zeros(M, R, dtype=torch.float64, device="cuda")
    eH, tol = torch.zeros_like(wantH), torch.zeros_like(want)
    for a, rows in _groups(index, M, n):
        s = d["scale"][a].double() if use_scale else 1.0
        wantH[rows] = x[rows] @ A[a].T
        eH[rows] = p(K) * (x[rows].abs() @ A[a].abs().T)
        want[rows] += s * (wantH[rows] @ B[a].T)
        tol[rows] = s * (eH[rows] @ B[a].abs().T + (p(R) + 2.0 ** -17) * (wantH[rows].abs() @ B[a].abs().T))
    tol += _half(t) * want.abs() + 2 * U * (d["Y"].double().abs() + want.abs())
    some = torch.zeros(M, dtype=torch.bool, device="cuda")
    for _, rows in _groups(index, M, n):
        some[rows] = True
    _close(H, wantH, eH, "H")
    _close(got[some], want[some], tol[some], "out")
    assert torch.equal(got[~some], d["Y"][~some]) and not H[~some].any()
    return got, H


def check_backward(ops, d, index, use_scale=True, use_dx=True, plan=None):
    t, (M, K), (n, N, R) = d["X"].dtype, d["X"].shape, d["B"].shape
    args = (d["dY"], d["X"], d["A"], d["B"], d["H"], d["dX"] if use_dx else None, index, d["scale"] if use_scale else None, plan)
    dX, dA, dB = ops.adapter_backward(*args)
    again = ops.adapter_backward(*args)
    torch.cuda.synchronize()
    for a, b in zip((dX, dA, dB), again):
        assert torch.equal(a, b)
    x, A, B, dy, H = (d[k].double() for k in ("X", "A", "B", "dY", "H"))
    base = d["dX"].double() if use_dx else torch.zeros_like(x)
    want, tol = base.clone(), torch.zeros_like(x)
    some = torch.zeros(M, dtype=torch.bool, device="cuda")
    for a, rows in _groups(index, M, n):
        some[rows] = True
        s = d["scale"][a].double() if use_scale else torch.ones((), dtype=torch.float64, device="cuda")
        G = s * (dy[rows] @ B[a])
        eG = s * p(N) * (dy[rows].abs() @ B[a].abs())
        want[rows] += G @ A[a]
        tol[rows] = eG @ A[a].abs() + (p(R) + 2.0 ** -17) * (G.abs() @ A[a].abs())
        wa, q = G.T @ x[rows], p(rows.numel()) + 2.0 ** -17
        _close(dA[a], wa, _half(t) * wa.abs() + eG.T @ x[rows].abs() + q * (G.abs().T @ x[rows].abs()), f"dA[{a}]")
        wb = s * (dy[rows].T @ H[rows])
        _close(dB[a], wb, _half(t) * wb.abs() + s * (q + 2 * U) * (dy[rows].abs().T @ H[rows].abs()), f"dB[{a}]")
        if rows.numel() == 0:
            assert not dA[a].any() and not dB[a].any()
    tol += _half(t) * want.abs() + 2 * U * (base.abs() + want.abs())
    _close(dX[some], want[some], tol[some], "dX")
    assert torch.equal(dX[~some], d["dX"][~some] if use_dx else torch.zeros_like(dX[~some]))
    return dX, dA, dB


# (M, K, N, R, count, index): one row and few rows, tiles that end inside, every rank's padding, odd sizes, adapters
# without rows, more adapters than rows
CASES = [
    (1, 256, 512, 16, 1, "one"), (1, 4096, 4096, 16, 3, "random"), (3, 64, 8, 1, 2, "random"), (48, 1024, 768, 16, 24, "random"),
    (64, 512, 256, 8, 5, "sorted"), (65, 512, 256, 8, 5, "random"), (127, 256, 384, 4, 1, "one"), (128, 256, 384, 32, 1, "one"),
    (129, 256, 384, 16, 2, "sorted"), (300, 768, 2304, 32, 4, "random"), (333, 1000, 776, 12, 7, "sorted"),
    (500, 640, 1288, 64, 3, "random"), (400, 512, 1024, 128, 2, "sorted"), (260, 520, 264, 100, 2, "random"),
    (333, 1001, 770, 6, 5, "sorted"), (70, 77, 91, 5, 3, "random"), (200, 8, 8, 2, 40, "random"), (150, 256, 256, 16, 6, "none"),
    (150, 256, 256, 16, 6, "last"), (140, 256, 264, 16, 6, "outside"), (1024, 1024, 1024, 16, 200, "random"),
    (2000, 512, 512, 8, 1, "one"), (130, 256, 256, 16, 1024, "random"),
]


@pytest.mark.parametrize("t", [BF16, F32])
@pytest.mark.parametrize("M,K,N,R,n,kind", CASES)
def test_forward(ops, M, K, N, R, n, kind, t):
    check_forward(ops, _inputs(M, K, N, R, n, t, M + K + R), _index(kind, M, n, M))


@pytest.mark.parametrize("t", [BF16, F32])
@pytest.mark.parametrize("M,K,N,R,n,kind", CASES)
def test_backward(ops, M, K, N, R, n, kind, t):
    check_backward(ops, _inputs(M, K, N, R, n, t, M + 2 * K + R), _index(kind, M, n, M))


@pytest.mark.parametrize("t", [BF16, F32])
@pytest.mark.parametrize("M", [40, 300])
def test_optional_arguments(ops, M, t):
    """No scale, no incoming dX, a plan made beforehand, out = Y, and each gradient alone."""
    d, index = _inputs(M, 384, 512, 16, 4, t, 3), _index("random", M, 4, 5)
    plan = ops.adapter_plan(index, 4)
    out, H = check_forward(ops, d, index, use_scale=False, plan=plan)
    want, _ = check_forward(ops, d, index)
    Y = d["Y"].clone()
    assert ops.adapter_forward(d["X"], d["A"], d["B"], Y, index, d["scale"], out=Y) is Y
    assert torch.equal(Y, want)
    check_backward(ops, d, index, use_scale=False, use_dx=False)
    full = check_backward(ops, d, index)
    with_plan = check_backward(ops, d, index, plan=plan)
    for a, b in zip(full, with_plan):
        assert torch.equal(a, b)
    for need in ((True, False, False), (False, True, False), (False, False, True), (False, True, True), (True, False, True)):
        got = ops.adapter_backward(d["dY"], d["X"], d["A"], d["B"], d["H"], d["dX"], index, d["scale"], need=need)
        for g, w, n in zip(got, full, need):
            assert torch.equal(g, w) if n else g is None


@pytest.mark.parametrize("M,n", [(1, 1), (31, 4), (1000, 3), (5000, 1024), (40000, 17)])
def test_plan_lists_the_rows(ops, M, n):
    index = _index("outside", M, n, M)
    plan = ops.adapter_plan(index, n)
    torch.cuda.synchronize()
    data = plan.data.cpu().view(torch.int32)
    head, tiles = 2 * ((n + 2 + 3) // 4 * 4), M // 128 + n + 1
    first, rows = data[:n + 2], data[head + 4 * tiles:head + 4 * tiles + M]
    idx = index.cpu()
    group = torch.where((idx >= 0) & (idx < n), idx, n)
    order = torch.argsort(group.long(), stable=True)
    assert torch.equal(rows.long(), order)
    counts = torch.bincount(group.long(), minlength=n + 1)
    assert torch.equal(first[1:].long(), counts.cumsum(0)) and first[0] == 0
    per = [0] + [-(-int(c) // 128) for c in counts]
    assert torch.equal(data[head // 2:head // 2 + n + 2].long(), torch.tensor(per).cumsum(0))
    got = data[head:head + 4 * tiles].reshape(-1, 4)
    want = [(a if a < n else -1, int(first[a]) + i, min(128, int(counts[a]) - i)) for a in range(n + 1) for i in range(0, int(counts[a]), 128)]
    assert [tuple(r[:3].tolist()) for r in got[:len(want)]] == want and not got[len(want):, 2].any()


def test_nothing_crosses_rows(ops):
    """A NaN row and an infinite adapter reach only what their formulas reach."""
    for M, t in ((20, BF16), (300, BF16), (20, F32)):
        d, index = _inputs(M, 256, 384, 16, 4, t, 7), _index("random", M, 4, 9)
        index[3] = 0
        clean, cleanH = ops.adapter_forward(d["X"], d["A"], d["B"], d["Y"], index, d["scale"], keep=True)
        d["X"][3, 17] = float("nan")
        d["A"][2, 1, 5] = float("inf")
        out, H = ops.adapter_forward(d["X"], d["A"], d["B"], d["Y"], index, d["scale"], keep=True)
        keep = (index != 2)
        keep[3] = False
        assert torch.equal(out[keep], clean[keep]) and torch.equal(H[keep], cleanH[keep]) and out[3].isnan().all()
        d["dY"][5, 2] = float("nan")
        index[5] = 1
        dX, dA, dB = ops.adapter_backward(d["dY"], d["X"], d["A"], d["B"], d["H"], d["dX"], index, d["scale"])
        rows = (index != 2)
        rows[5] = False
        assert dX[rows].isfinite().all() and dX[5].isnan().all()
        assert dA[3].isfinite().all() and dB[3].isfinite().all() and dB[2].isfinite().all()


def test_unaligned_bases_and_guards(ops):
    """bf16 tensors that start off a 16-byte boundary, and what lies around the outputs."""
    M, K, N, R, n = 140, 256, 264, 16, 3
    d, index = _inputs(M, K, N, R, n, BF16, 13), _index("random", M, n, 14)

    def shifted(t, by=1):
        flat = torch.full((t.numel() + 2 * by + 6,), 5.0, dtype=t.dtype, device="cuda")
        flat[by:by + t.numel()] = t.reshape(-1)
        return flat[by:by + t.numel()].view(t.shape), flat
    s = {k: shifted(v)[0] for k, v in d.items() if k not in ("scale", "H")}
    s.update(scale=d["scale"], H=d["H"])
    y, flat = shifted(d["Y"], 3)
    check_forward(ops, s, index)
    check_backward(ops, s, index)
    ops.adapter_forward(s["X"], s["A"], s["B"], y, index, d["scale"], out=y)
    torch.cuda.synchronize()
    assert (flat[:3] == 5).all() and (flat[3 + y.numel():] == 5).all()


def test_no_rows(ops):
    d = _inputs(0, 64, 32, 8, 2, BF16, 1)
    index = torch.zeros(0, dtype=torch.int32, device="cuda")
    out, H = ops.adapter_forward(d["X"], d["A"], d["B"], d["Y"], index, d["scale"], keep=True)
    assert out.shape == (0, 32) and H.shape == (0, 8)
    dX, dA, dB = ops.adapter_backward(d["dY"], d["X"], d["A"], d["B"], d["H"], None, index, d["scale"])
    torch.cuda.synchronize()
    assert dX.shape == (0, 64) and not dA.any() and not dB.any()
    ops.adapter_plan(index, 2)
    torch.cuda.synchronize()


def test_streams_and_graph(ops):
    """Two calls at once on two streams, and a captured one replayed with other inputs."""
    cases = [(_inputs(M, 512, 768, 16, 3, BF16, M), _index("random", M, 3, M)) for M in (24, 400)]
    want = [(ops.adapter_forward(d["X"], d["A"], d["B"], d["Y"], i, d["scale"]),
             *ops.adapter_backward(d["dY"], d["X"], d["A"], d["B"], d["H"], d["dX"], i, d["scale"])) for d, i in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(5):
        for k, ((d, i), s) in enumerate(zip(cases, streams)):
            got[k] = (ops.adapter_forward(d["X"], d["A"], d["B"], d["Y"], i, d["scale"], stream=s),
                      *ops.adapter_backward(d["dY"], d["X"], d["A"], d["B"], d["H"], d["dX"], i, d["scale"], stream=s))
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    for d, i in cases:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = ops.adapter_forward(d["X"], d["A"], d["B"], d["Y"], i, d["scale"])
            grads = ops.adapter_backward(d["dY"], d["X"], d["A"], d["B"], d["H"], d["dX"], i, d["scale"])
        i.copy_(i.flip(0))
        d["X"].mul_(0.5)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ops.adapter_forward(d["X"], d["A"], d["B"], d["Y"], i, d["scale"]))
        for a, b in zip(grads, ops.adapter_backward(d["dY"], d["X"], d["A"], d["B"], d["H"], d["dX"], i, d["scale"])):
            assert torch.equal(a, b)


def test_gradients_against_differences(ops):
    """Through the forward's own formula in float64, each entry moved by h."""
    M, K, N, R, n, h = 5, 6, 7, 2, 2, 1e-6
    d, index = _inputs(M, K, N, R, n, F32, 21), _index("random", M, n, 3)
    _, H = ops.adapter_forward(d["X"], d["A"], d["B"], d["Y"], index, d["scale"], keep=True)
    got = ops.adapter_backward(d["dY"], d["X"], d["A"], d["B"], H, None, index, d["scale"])

    def loss(x, A, B):
        total = 0.0
        for a, rows in _groups(index, M, n):
            total = total + ((x[rows] @ A[a].T @ B[a].T) * d["dY"][rows].double()).sum() * d["scale"][a].double()
        return total
    at = [d[k].double() for k in ("X", "A", "B")]
    for i, g in enumerate(got):
        want = torch.empty(at[i].numel(), dtype=torch.float64, device="cuda")
        for j in range(want.numel()):
            ends = []
            for s in (h, -h):
                moved = [v.clone() for v in at]
                moved[i].reshape(-1)[j] += s
                ends.append(loss(*moved))
            want[j] = (ends[0] - ends[1]) / (2 * h)
        # the loss is bilinear at most in each: no error of the method; float32 products of terms below 10
        _close(g.reshape(-1), want, torch.full_like(want, 10 * p(16) + 1e-8), f"gradient {i}")


def test_refusals(ops):
    d, index = _inputs(6, 64, 32, 8, 2, BF16, 1), _index("random", 6, 2, 1)
    X, A, B, Y, s = d["X"], d["A"], d["B"], d["Y"], d["scale"]
    other = ops.adapter_plan(_index("random", 7, 2, 1), 2)
    for bad in (lambda: ops.adapter_forward(X, A, B, Y), lambda: ops.adapter_forward(X, A[:, :, :-1], B, Y, index),
                lambda: ops.adapter_forward(X, A, B[:, :, :-1], Y, index), lambda: ops.adapter_forward(X, A, B, Y[:-1], index),
                lambda: ops.adapter_forward(X, A, B, Y, index.long()), lambda: ops.adapter_forward(X, A, B, Y, index[:-1]),
                lambda: ops.adapter_forward(X, A, B, Y, index, s.double()), lambda: ops.adapter_forward(X, A, B, Y, index, s[:1]),
                lambda: ops.adapter_forward(X.float(), A, B, Y, index), lambda: ops.adapter_forward(X, A, B, Y, index, plan=other),
                lambda: ops.adapter_forward(X, A, B, Y, index, out=X[:, :32]), lambda: ops.adapter_forward(X, A, B, Y.t(), index),
                lambda: ops.adapter_forward(X, A.repeat(1, 17, 1), B.repeat(1, 1, 17), Y, index),
                lambda: ops.adapter_backward(d["dY"], X, A, B, None, None, index), lambda: ops.adapter_plan(index.float(), 2),
                lambda: ops.adapter_backward(d["dY"], X, A, B, d["H"].to(BF16), None, index),
                lambda: ops.adapter_backward(d["dY"], X, A, B, d["H"], d["dX"].float(), index), lambda: ops.adapter_plan(index, 0)):
        with pytest.raises((ValueError, TypeError, RuntimeError)):
            bad()


@pytest.mark.parametrize("M,K,N,R,n", [(300, 256, 264, 12, 3), (140, 264, 256, 64, 2), (300, 77, 91, 5, 3)])
def test_each_gradient_alone(ops, M, K, N, R, n):
    """Ranks that are padded, widened or neither, on both paths: a gradient does not depend on which others are asked for."""
    d, index = _inputs(M, K, N, R, n, BF16, 31), _index("random", M, n, 32)
    full = check_backward(ops, d, index)
    for need in ((True, False, False), (False, True, False), (False, False, True), (True, True, False), (False, True, True)):
        got = ops.adapter_backward(d["dY"], d["X"], d["A"], d["B"], d["H"], d["dX"], index, d["scale"], need=need)
        for g, w, asked in zip(got, full, need):
            assert torch.equal(g, w) if asked else g is None


@pytest.mark.parametrize("t", [BF16, F32])
def test_many_rows(ops, t):
    """More rows than the plan keeps in registers, adapters that share runs of tiles and one that has many runs."""
    M, n = 40000, 6
    d = _inputs(M, 64, 72, 8, n, t, 41)
    index = _index("random", M, n, 42)
    index[:30000] = 4
    check_forward(ops, d, index)
    check_backward(ops, d, index)


def test_offsets_past_32_bits(ops):
    """Y of more than 2^31 elements: the last rows, in the forward and the backward pass."""
    M, K, N, R, n = 263000, 256, 8192, 8, 2
    assert M * N > 2 ** 31
    X = torch.randn(M, K, dtype=BF16, device="cuda")
    Y = torch.randn(M, N, dtype=BF16, device="cuda")
    g = torch.Generator().manual_seed(1)
    A = (torch.randn(n, R, K, generator=g) * K ** -0.5).to(BF16).cuda()
    B = (torch.randn(n, N, R, generator=g) * 0.05).to(BF16).cuda()
    index = (torch.arange(M, device="cuda") % 3 - 1).to(torch.int32)
    rows = torch.tensor([0, 1, 2, M // 2, M - 3, M - 2, M - 1], device="cuda")
    out, H = ops.adapter_forward(X, A, B, Y, index, keep=True)
    dX, dA, dB = ops.adapter_backward(Y, X, A, B, H, None, index, need=(True, False, False))
    torch.cuda.synchronize()
    for m in rows.tolist():
        a = int(index[m])
        if a < 0:
            assert torch.equal(out[m], Y[m]) and not dX[m].any()
            continue
        G = Y[m].double() @ B[a].double()
        wantx = G @ A[a].double()
        eG = p(N) * (Y[m].double().abs() @ B[a].double().abs())
        tol = _half(BF16) * wantx.abs() + eG @ A[a].double().abs() + (p(R) + 2.0 ** -17) * (G.abs() @ A[a].double().abs())
        _close(dX[m], wantx, tol, f"dX[{m}]")
        h = X[m].double() @ A[a].T.double()
        wanto = Y[m].double() + B[a].double() @ h
        eH = p(K) * (X[m].double().abs() @ A[a].T.double().abs())
        tolo = _half(BF16) * wanto.abs() + B[a].double().abs() @ eH + (p(R) + 2.0 ** -17) * (B[a].double().abs() @ h.abs()) + 2 * U * wanto.abs()
        _close(out[m], wanto, tolo, f"out[{m}]")
