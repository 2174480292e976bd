"""Layer norm with a float32 bias and no weight beside bf16 rows: the bias's gradient keeps float32's digits."""

import pytest
import torch

from tests.gpu_common import get_ss1

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ops():
    get_ss1()
    from structured_compressed_linear_b200 import ops
    return ops


@pytest.mark.parametrize("M,K", [(1, 8), (7, 33), (300, 768), (5, 8200), (400, 1280)])
def test_gradient_of_a_float32_bias(ops, M, K):
    """Against float64. A sum of M terms in float32 is off by at most M u sum |dy|, u = 2^-24; one rounded to bf16 on the way
    would be off by up to 2^-9 of itself."""
    gen = torch.Generator().manual_seed(M + K)
    x = torch.randn(M, K, generator=gen).to(BF16).cuda()
    b = torch.randn(K, generator=gen).cuda().requires_grad_()
    dy = torch.randn(M, K, generator=gen).to(BF16).cuda()
    y = ops.LayerNormFunction.apply(x, None, b, 1e-5)
    y.backward(dy)
    want, size = dy.double().sum(0), dy.double().abs().sum(0)
    assert b.grad.dtype == F32
    assert ((b.grad.double() - want).abs() <= M * 2.0 ** -24 * size).all()
    _, mean, rstd = ops.layernorm_forward(x, None, b)
    dX, dw, db = ops.layernorm_backward(dy, x, mean, rstd, weight_dtype=F32)
    assert dX.dtype == BF16 and dw.dtype == F32 and torch.equal(db, b.grad)
    assert torch.equal(db.to(BF16), ops.layernorm_backward(dy, x, mean, rstd)[2])
    xhat = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    # xhat itself is off by 3 u of its terms' size
    assert ((dw.double() - (dy.double() * xhat).sum(0)).abs() <= (M + 3) * 2.0 ** -24 * (dy.double() * xhat).abs().sum(0)
            + 2.0 ** -23 * (dy.double() * mean.double()[:, None] * rstd.double()[:, None]).abs().sum(0)).all()


def test_refusals(ops):
    x = torch.randn(4, 16, device="cuda")
    w = torch.ones(16, device="cuda")
    _, mean, rstd = ops.layernorm_forward(x, w)
    for bad in (dict(weight_dtype=BF16), dict(weight=w, weight_dtype=BF16), dict(weight_dtype=torch.float16)):
        with pytest.raises(ValueError):
            ops.layernorm_backward(x, x, mean, rstd, **bad)
    xb = x.to(BF16)
    wb = w.to(BF16)
    with pytest.raises(ValueError):
        ops.layernorm_backward(xb, xb, mean, rstd, wb, weight_dtype=F32)
    ops.layernorm_backward(xb, xb, mean, rstd, wb, weight_dtype=BF16)
