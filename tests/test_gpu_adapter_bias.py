"""Adapters' gradients over very many rows and very many columns: terms of one sign, whose sums a tensor core's truncating
additions would leave too small by more the more of them there are.

What is looked at is the mean of (result - the rounded float64 value) / value over all elements: rounding to bf16 falls out of
it, a sum that is too small by a share e shows up as -e. At most 64 tiles of 128 rows go into one sum in
tensor memory, 512 additions (16 rows each), and 4096 columns, 256 additions. Each is truncated by less than 2^-23 of a sum
that grows evenly, so e <= 512 / 2 * 2^-23 = 2^-15; float32 sums of the parts that were taken out add 2^-20 at
most (16 of them, rounded). G, H: their second bf16 parts are rounded, not truncated."""

import pytest
import torch

from tests.gpu_common import get_ss1

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
BOUND = 2.0 ** -15 + 2.0 ** -20


@pytest.fixture(scope="module")
def ops():
    get_ss1()
    from structured_compressed_linear_b200 import ops
    return ops


def _positive(gen, M, C):
    """Values of one sign, sizes that differ by row and column."""
    out = torch.empty(M, C, dtype=BF16, device="cuda")
    col = 1 + torch.rand(C, generator=gen, device="cuda")
    for a in range(0, M, 4096):
        b = min(M, a + 4096)
        out[a:b] = (torch.rand(b - a, C, generator=gen, device="cuda") * (1 + torch.rand(b - a, 1, generator=gen, device="cuda")) * col).to(BF16)
    return out


def _products(U, P):
    """U^T P in float64, rows in pieces."""
    return sum(U[a:a + 4096].double().T @ P[a:a + 4096].double() for a in range(0, U.shape[0], 4096))


def _bias(got, want):
    return float(((got.double() - want.to(BF16).double()) / want).mean())


@pytest.mark.parametrize("M,C,R", [(65536, 8192, 16), (33000, 14336, 32), (262144, 1024, 16)])
def test_many_rows_of_one_adapter(ops, M, C, R):
    gen = torch.Generator(device="cuda").manual_seed(1)
    U = _positive(gen, M, C)
    H = torch.rand(M, R, generator=gen, device="cuda")
    small = torch.zeros(M, 64, dtype=BF16, device="cuda")
    A, B = torch.zeros(1, R, 64, dtype=BF16, device="cuda"), torch.zeros(1, C, R, dtype=BF16, device="cuda")
    _, _, dB = ops.adapter_backward(U, small, A, B, H, need=(False, False, True))
    assert abs(_bias(dB[0], _products(U, H))) <= BOUND
    # dA of the same matrix as X: G = dY B with one column for each rank, so G is dY's first columns
    dY = _positive(gen, M, 64)
    A, B = torch.zeros(1, R, C, dtype=BF16, device="cuda"), torch.zeros(1, 64, R, dtype=BF16, device="cuda")
    B[0, :R] = torch.eye(R)
    _, dA, _ = ops.adapter_backward(dY, U, A, B, None, need=(False, True, False))
    assert abs(_bias(dA[0].T, _products(U, dY[:, :R]))) <= BOUND


@pytest.mark.parametrize("M,N,R", [(20000, 32768, 16), (300, 131072, 64), (20000, 14336, 32), (19000, 8256, 128)])
def test_many_columns(ops, M, N, R):
    """G alone: dX = G A with one column for each rank."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    dY = _positive(gen, M, N)
    B = torch.rand(1, N, R, generator=gen, device="cuda").to(BF16)
    K = max(64, R)
    A, X = torch.zeros(1, R, K, dtype=BF16, device="cuda"), torch.zeros(M, K, dtype=BF16, device="cuda")
    A[0, :, :R] = torch.eye(R)
    dX, _, _ = ops.adapter_backward(dY, X, A, B, None, need=(True, False, False))
    want = torch.cat([dY[a:a + 4096].double() @ B[0].double() for a in range(0, M, 4096)])
    assert abs(_bias(dX[:, :R], want)) <= BOUND


def test_sums_that_are_taken_out_more_than_once(ops):
    """A CTA's columns span several pieces, the last one short: values, against the float64 product, row by row."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    M, N, R, K = 19000, 3 * 4096 + 72, 40, 64
    dY = torch.randn(M, N, generator=gen, device="cuda").to(BF16)
    B = torch.randn(1, N, R, generator=gen, device="cuda").to(BF16)
    A, X = torch.zeros(1, R, K, dtype=BF16, device="cuda"), torch.zeros(M, K, dtype=BF16, device="cuda")
    A[0, :, :R] = torch.eye(R)
    dX, _, _ = ops.adapter_backward(dY, X, A, B, None, need=(True, False, False))
    for a in range(0, M, 4096):
        want = dY[a:a + 4096].double() @ B[0].double()
        size = dY[a:a + 4096].double().abs() @ B[0].double().abs()
        # half a step of bf16, the second parts' 2^-17, and 2^-23 a addition of a sum no larger than `size`
        assert ((dX[a:a + 4096, :R].double() - want).abs() <= (2.0 ** -8 + 2.0 ** -17) * want.abs() + 260 * 2.0 ** -23 * size).all()
    assert not dX[:, R:].any()
