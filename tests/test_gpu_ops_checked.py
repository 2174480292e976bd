"""The operators around a projection through the bounds-checked debug build (libss1_checked.so): on each kernel
path the results must be those of the normal build, bit for bit, and no index test may fail."""

import pytest
import torch

from tests.gpu_common import get_ss1

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def both():
    ss1 = get_ss1()
    from structured_compressed_linear_b200 import build, ops
    build.build(checked=True)
    ss1.load_library(ss1.CHECKED_LIB_PATH)

    def run(fn):
        ss1.use_library(ss1.LIB_PATH)
        try:
            want = fn(ops)
            torch.cuda.synchronize()
            ss1.use_library(ss1.CHECKED_LIB_PATH)
            assert ss1.bounds_check() == (True, 0)
            got = fn(ops)
            torch.cuda.synchronize()
            checked, record = ss1.bounds_check()
        finally:
            ss1.use_library(ss1.LIB_PATH)
        assert checked and record == 0, f"out-of-range access: site {record >> 48}, index {record & ((1 << 48) - 1)}"
        for a, b in zip(want, got):
            assert torch.equal(a, b)
    yield run
    ss1.use_library(ss1.LIB_PATH)


@pytest.mark.parametrize("t", [BF16, F32])
@pytest.mark.parametrize("M,K", [(1, 1), (9, 257), (130, 1280), (700, 1021), (300, 4096), (5, 8200), (3, 33001)])
def test_layernorm(both, M, K, t):
    g = torch.Generator().manual_seed(M + K)
    x, dy = (torch.randn(M, K, generator=g).to(t).cuda() for _ in range(2))
    w, b = (torch.randn(K, generator=g).to(t).cuda() for _ in range(2))

    def run(ops):
        Y, m, r = ops.layernorm_forward(x, w, b)
        return Y, m, r, *ops.layernorm_backward(dy, x, m, r, w)
    both(run)


@pytest.mark.parametrize("t", [BF16, F32])
@pytest.mark.parametrize("M,K,N,R,n", [(1, 256, 512, 16, 1), (40, 512, 256, 16, 9), (300, 768, 1288, 32, 4), (333, 1001, 770, 6, 5),
                                       (200, 264, 520, 100, 3), (2000, 256, 256, 8, 2)])
def test_adapters(both, M, K, N, R, n, t):
    g = torch.Generator().manual_seed(M + K)

    def make(*shape):
        return torch.randn(*shape, generator=g).to(t).cuda()
    X, A, B, Y, dY, dX = make(M, K), make(n, R, K), make(n, N, R), make(M, N), make(M, N), make(M, K)
    index = None if n == 1 else torch.randint(-1, n + 1, (M,), generator=g).to(torch.int32).cuda()
    scale = torch.rand(n, generator=g).cuda()

    def run(ops):
        out, H = ops.adapter_forward(X, A, B, Y, index, scale, keep=True)
        return out, H, *ops.adapter_backward(dY, X, A, B, H, dX, index, scale)
    both(run)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("t", [BF16, F32])
def test_adamw(both, bits, t):
    sizes = [1, 255, 257, 8193, 30000] + [13] * 50
    gen = torch.Generator().manual_seed(3)
    p, g = ([torch.randn(n, generator=gen).to(t).cuda() for n in sizes] for _ in range(2))

    def run(ops):
        P = [x.clone() for x in p]
        state = F32 if bits == 32 else torch.uint8
        S = [[torch.zeros(n, dtype=state, device="cuda") for n in sizes] for _ in range(2)]
        sc = None if bits == 32 else tuple([torch.zeros(-(-n // 256), device="cuda") for n in sizes] for _ in range(2))
        ops.adamw_step(P, g, *S, scales=sc)
        return (*P, *S[0], *S[1], *(() if sc is None else (*sc[0], *sc[1])))
    both(run)
