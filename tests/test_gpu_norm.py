"""Layer norm's forward and backward pass (ss1_layernorm_*) against the formulas in float64.

Tolerances, with u = 2^-24 and h = finfo(type).eps / 2 of the output's type. A sum over a row adds at
most 40 terms in a thread (K / 1024 for rows past the register kernels) and up to 11 partial sums
in trees: n <= 64 roundings for every K here, so a sum is off by at most n u times the sum of the
magnitudes. That makes
  mean : n u mean|x|;  xhat: n u (mean|x| rstd + |xhat|) (the deviations' sum of squares has
         relative error (n + 3) u, its root half of that);
  Y    : h |y| + n u (|w| (|xhat| + mean|x| rstd) + |y|);
  dX   : h |dx| + n u rstd (|g| + mean|g| + |xhat| mean|g xhat|);
  dw,db: h |dw| + n u sum|dy xhat|, since a column adds M / (CTAs x groups) rows in a thread, then up to
         8 groups and parts / 32 + 5 partial sums: also <= 64 here.
"""

import pytest
import torch

from tests.gpu_common import get_ss1

pytestmark = pytest.mark.gpu

U, N = 2.0 ** -24, 64
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ops():
    get_ss1()
    from structured_compressed_linear_b200 import ops
    return ops


def _half(t):
    return torch.finfo(t).eps / 2


def _inputs(M, K, xt, wt, seed, offset=0.5):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g) + offset * torch.randn(M, 1, generator=g)
    if M > 4:
        x[3] *= 20.0
    w, b = 1 + 0.1 * torch.randn(K, generator=g), 0.1 * torch.randn(K, generator=g)
    dy = torch.randn(M, K, generator=g)
    return x.to(xt).cuda(), w.to(wt).cuda(), b.to(wt).cuda(), dy.to(xt).cuda()


def _reference(x, eps):
    x = x.double()
    mean = x.mean(1)
    rstd = 1 / torch.sqrt((x - mean[:, None]).square().mean(1) + eps)
    return mean, rstd


def _close(got, want, tol, what):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float(((got.double() - want).abs() / tol).max()):.3g} x tolerance"


# every kernel: a warp a row with 1 .. 5 units, a CTA a row with 1, 2, 4 units, past the registers; vector and
# scalar rows; one row, several CTAs of rows, a ragged last CTA
SHAPES = [(1, 1), (3, 7), (9, 256), (17, 257), (8, 512), (5, 768), (33, 1021), (130, 1024), (40, 1280), (7, 1288), (16, 4096),
          (3, 5000), (2, 8192), (3, 8200), (2, 16384), (2, 20003), (2, 32768), (3, 32776), (1, 33001)]


@pytest.mark.parametrize("M,K", SHAPES)
@pytest.mark.parametrize("xt,wt", [(BF16, BF16), (BF16, F32), (F32, F32)])
def test_forward(ops, M, K, xt, wt):
    x, w, b, _ = _inputs(M, K, xt, wt, M + K)
    Y, mean, rstd = ops.layernorm_forward(x, w, b, eps=1e-5)
    torch.cuda.synchronize()
    m, r = _reference(x, 1e-5)
    size = x.double().abs().mean(1)
    _close(mean, m, N * U * size, "mean")
    _close(rstd, r, N * U * r * (1 + size * r), "rstd")
    xhat = (x.double() - m[:, None]) * r[:, None]
    want = xhat * w.double() + b.double()
    tol = _half(xt) * want.abs() + N * U * (w.double().abs() * (xhat.abs() + (size * r)[:, None]) + want.abs() + b.double().abs())
    _close(Y, want, tol, "Y")


@pytest.mark.parametrize("M,K", SHAPES + [(2051, 1021), (3000, 1280), (5000, 64)])
@pytest.mark.parametrize("xt,wt", [(BF16, BF16), (BF16, F32), (F32, F32)])
def test_backward(ops, M, K, xt, wt):
    x, w, _, dy = _inputs(M, K, xt, wt, M + 2 * K)
    m, r = _reference(x, 1e-5)
    m, r = m.float(), r.float()
    dX, dw, db = ops.layernorm_backward(dy, x, m, r, w)
    again = ops.layernorm_backward(dy, x, m, r, w)
    torch.cuda.synchronize()
    xh = (x.double() - m.double()[:, None]) * r.double()[:, None]
    d = dy.double()
    g = d * w.double()
    want = r.double()[:, None] * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    mags = g.abs() + g.abs().mean(1, keepdim=True) + xh.abs() * (g * xh).abs().mean(1, keepdim=True)
    _close(dX, want, _half(xt) * want.abs() + N * U * r.double()[:, None] * mags, "dX")
    for got, terms, name in ((dw, d * xh, "dweight"), (db, d, "dbias")):
        _close(got, terms.sum(0), _half(wt) * terms.sum(0).abs() + N * U * terms.abs().sum(0), name)
    for a, b in zip((dX, dw, db), again):
        assert torch.equal(a, b)          # the column sums have one order


def test_large_mean_keeps_its_digits(ops):
    """Rows far from zero: the variance comes from the deviations."""
    x = (torch.randn(8, 1024, generator=torch.Generator().manual_seed(1)) * 1e-2 + 100.0).cuda()
    Y, mean, rstd = ops.layernorm_forward(x)
    m, r = _reference(x, 1e-5)
    xhat = (x.double() - m[:, None]) * r[:, None]
    _close(Y, xhat, N * U * (xhat.abs() + 100.0 * r[:, None]), "Y")


def test_without_weights_and_constant_rows(ops):
    x = torch.full((4, 96), 3.0, dtype=BF16, device="cuda")
    Y, mean, rstd = ops.layernorm_forward(x, eps=1e-5)
    assert torch.equal(Y, torch.zeros_like(Y)) and torch.equal(mean, torch.full_like(mean, 3.0))
    b = torch.arange(96, device="cuda").to(BF16)
    assert torch.equal(ops.layernorm_forward(x, None, b)[0], b.expand(4, 96))
    dX, dw, db = ops.layernorm_backward(torch.ones_like(x), x, mean, rstd)
    assert torch.equal(dw, torch.zeros_like(dw)) and torch.equal(db, torch.full_like(db, 4.0))
    assert dX.abs().max() <= 2 ** -20 / 1e-5 ** 0.5
    one = torch.tensor([[5.0]], device="cuda")            # K = 1: the deviation is 0
    assert ops.layernorm_forward(one)[0].item() == 0.0


def test_no_rows_and_parts(ops):
    x = torch.zeros(0, 64, dtype=BF16, device="cuda")
    Y, mean, rstd = ops.layernorm_forward(x)
    assert Y.shape == (0, 64) and mean.numel() == 0
    dX, dw, db = ops.layernorm_backward(x, x, mean, rstd)
    torch.cuda.synchronize()
    assert dX.shape == (0, 64) and not dw.any() and not db.any()
    x, w, _, dy = _inputs(50, 320, BF16, BF16, 3)
    m, r = (t.float() for t in _reference(x, 1e-5))
    full = ops.layernorm_backward(dy, x, m, r, w)
    for need in ((True, False, False), (False, True, False), (False, False, True), (False, True, True)):
        for got, want, n in zip(ops.layernorm_backward(dy, x, m, r, w, need), full, need):
            assert torch.equal(got, want) if n else got is None


def test_nan_and_infinity_stay_in_their_row(ops):
    x, w, b, dy = _inputs(40, 1280, BF16, BF16, 5)
    clean = ops.layernorm_forward(x, w, b)[0]
    x[7, 100], x[21, 3] = float("nan"), float("inf")
    Y = ops.layernorm_forward(x, w, b)[0]
    rows = torch.ones(40, dtype=torch.bool, device="cuda")
    rows[7] = rows[21] = False
    assert torch.equal(Y[rows], clean[rows]) and Y[7].isnan().all() and Y[21].isnan().any()


@pytest.mark.parametrize("K", [1, 4, 8, 512])
def test_mean_that_overflows_behind_the_rows_end(ops, K):
    """(0 - mean) rstd is past float32 here, and nothing behind the row's end may come of it. K is a power of two, so
    that mean is x, xhat 0 and dX = rstd (dy - mean(dy)): the sum over K is the one rounding that counts."""
    x = torch.full((3, K), 2.0 ** 66, device="cuda")
    dy = torch.randn(3, K, generator=torch.Generator().manual_seed(K)).cuda()
    Y, mean, rstd = ops.layernorm_forward(x, eps=2.0 ** -124)
    assert bool((Y == 0).all()) and bool((mean == 2.0 ** 66).all()) and bool(((rstd / 2.0 ** 62 - 1).abs() <= 4 * U).all())
    dX, dw, db = ops.layernorm_backward(dy, x, mean, rstd)
    d = dy.double()
    scale = rstd.double()[:, None]
    _close(dX, scale * (d - d.mean(1, keepdim=True)), N * U * scale * (d.abs() + d.abs().mean(1, keepdim=True)), "dX")
    assert bool((dw == 0).all())
    _close(db, d.sum(0), N * U * d.abs().sum(0), "db")


@pytest.mark.parametrize("K", [1280, 1021])
def test_outputs_end_where_they_end(ops, K):
    """Unaligned bases (the scalar kernels) and guard elements around the outputs, through the C entry points."""
    from structured_compressed_linear_b200 import ss1
    M, lib = 37, ss1.lib()
    x, w, b, dy = _inputs(M, K, F32, F32, 9)
    want = ops.layernorm_forward(x, w, b)
    flat = torch.full((M * K + 6,), 7.0, device="cuda")
    shifted = torch.empty(M * K + 1, device="cuda")
    shifted[1:] = x.reshape(-1)
    st = torch.cuda.current_stream().cuda_stream
    assert lib.ss1_layernorm_forward(shifted.data_ptr() + 4, w.data_ptr(), b.data_ptr(), flat.data_ptr() + 12, None, None, M, K,
                                     1e-5, 1, 1, st) == 0
    torch.cuda.synchronize()
    assert (flat[:3] == 7).all() and (flat[-3:] == 7).all()
    _close(flat[3:-3].reshape(M, K), want[0].double(), 2 * N * U * (want[0].double().abs() + 2), "shifted Y")


def test_other_stream_and_graph(ops):
    x, w, b, dy = _inputs(300, 768, BF16, BF16, 11)
    want = ops.layernorm_forward(x, w, b)
    back = ops.layernorm_backward(dy, x, want[1], want[2], w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ops.layernorm_forward(x, w, b, stream=side)
    gback = ops.layernorm_backward(dy, x, got[1], got[2], w, stream=side)
    side.synchronize()
    for a, c in zip((*want, *back), (*got, *gback)):
        assert torch.equal(a, c)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = ops.layernorm_forward(x, w, b)
        z = ops.layernorm_backward(dy, x, y[1], y[2], w)
    x.copy_(x.flip(0))
    dy.copy_(dy.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    want = ops.layernorm_forward(x, w, b)
    for a, c in zip((*want, *ops.layernorm_backward(dy, x, want[1], want[2], w)), (*y, *z)):
        assert torch.equal(a, c)


def test_autograd_and_differences(ops):
    """LayerNormFunction's gradients against central differences of a float64 loss."""
    M, K, h = 3, 40, 1e-6
    g = torch.Generator().manual_seed(2)
    x, w, b, t = (torch.randn(*s, generator=g).cuda() for s in ((M, K), (K,), (K,), (M, K)))
    leaves = [v.clone().requires_grad_() for v in (x, w, b)]
    (ops.LayerNormFunction.apply(*leaves, 1e-5) * t).sum().backward()

    def loss(x, w, b):
        m, r = _reference(x, 1e-5)
        return (((x - m[:, None]) * r[:, None] * w + b) * t.double()).sum()
    at = [v.double() for v in (x, w, b)]
    for i, leaf in enumerate(leaves):
        want = torch.empty_like(at[i]).reshape(-1)
        for j in range(want.numel()):
            ends = []
            for s in (h, -h):
                moved = [v.clone() for v in at]
                moved[i].reshape(-1)[j] += s
                ends.append(loss(*moved))
            want[j] = (ends[0] - ends[1]) / (2 * h)
        # float32 arithmetic (N u per unit of the terms, which are below 100 here) beside the differences' 1e-8
        _close(leaf.grad.reshape(-1), want, 100 * N * U + 1e-7, f"leaf {i}")


def test_refusals(ops):
    x, w, b, dy = _inputs(4, 64, BF16, BF16, 1)
    m, r = (t.float() for t in _reference(x, 1e-5))
    for bad in (lambda: ops.layernorm_forward(x.t()), lambda: ops.layernorm_forward(x[0]), lambda: ops.layernorm_forward(x.half()),
                lambda: ops.layernorm_forward(x, w[:-1]), lambda: ops.layernorm_forward(x, w, b.float()),
                lambda: ops.layernorm_forward(x.float(), w), lambda: ops.layernorm_forward(x, out=x),
                lambda: ops.layernorm_forward(x, w.cpu()), lambda: ops.layernorm_backward(dy[:3], x, m, r, w),
                lambda: ops.layernorm_backward(dy.float(), x, m, r, w), lambda: ops.layernorm_backward(dy, x, m.double(), r, w)):
        with pytest.raises((ValueError, TypeError)):
            bad()
    with pytest.raises(RuntimeError):
        ops.layernorm_forward(x, eps=-1.0)


def test_offsets_past_32_bits(ops):
    """More than 2^31 elements: the last rows of both passes."""
    M, K = 1_680_000, 1288
    assert M * K > 2 ** 31
    x = torch.randn(M, K, dtype=BF16, device="cuda")
    rows = torch.tensor([0, M // 2, M - 2, M - 1], device="cuda")
    Y, mean, rstd = ops.layernorm_forward(x)
    dX, _, db = ops.layernorm_backward(x, x, mean, rstd)
    few = x[rows]
    fewY, m, r = ops.layernorm_forward(few)
    assert torch.equal(Y[rows], fewY) and torch.equal(mean[rows], m) and torch.equal(rstd[rows], r)
    assert torch.equal(dX[rows], ops.layernorm_backward(few, few, m, r)[0])
    # column sums over 1.68 M rows: a thread adds M / (148 * 3) of them, ten times the rows of the bound above
    want, size = x.sum(0, dtype=torch.float64), x.abs().sum(0, dtype=torch.float64)
    _close(db, want, _half(BF16) * want.abs() + (M / 444 + 32) * U * size, "dbias")
