"""Adapters of prompt-sized batches in a captured graph, replayed while the rows' adapters, the tables and the inputs change
in place: what kernels read before they wait for the one in front of them has to be this replay's, not the last one's."""

import pytest
import torch

from tests.gpu_common import get_ss1

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def ops():
    get_ss1()
    from structured_compressed_linear_b200 import ops
    return ops


@pytest.mark.parametrize("M,K,N,R,n", [(300, 256, 384, 16, 4), (1000, 512, 768, 12, 5), (2000, 256, 512, 64, 3), (600, 264, 256, 128, 2)])
@pytest.mark.parametrize("own_plan", [False, True])
def test_replays_follow_their_inputs(ops, M, K, N, R, n, own_plan):
    gen = torch.Generator(device="cuda").manual_seed(M + R)

    def new(*shape, dtype=BF16):
        return torch.randn(*shape, generator=gen, device="cuda").to(dtype)
    X, A, B, Y, dY, dX = new(M, K), new(n, R, K), new(n, N, R), new(M, N), new(M, N), new(M, K)
    scale = torch.rand(n, generator=gen, device="cuda")
    index = torch.zeros(M, dtype=torch.int32, device="cuda")

    def run():
        plan = ops.adapter_plan(index, n) if own_plan else None
        out, H = ops.adapter_forward(X, A, B, Y, index, scale, keep=True, plan=plan)
        return (out, H, *ops.adapter_backward(dY, X, A, B, H, dX, index, scale, plan))
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for turn in range(12):
        kind = turn % 4
        if kind == 0:       # every row another adapter, some none
            index.copy_(torch.randint(-1, n + 1, (M,), generator=gen, device="cuda").int())
        elif kind == 1:     # all rows one adapter
            index.fill_(turn % n)
        elif kind == 2:     # the same rows in another order, and other tables
            index.copy_(index.flip(0))
            A.copy_(new(n, R, K))
            B.copy_(new(n, N, R))
        else:               # nobody has one
            index.fill_(-1)
        for t in (X, Y, dY, dX):
            t.copy_(new(*t.shape))
        graph.replay()
        mine = [t.clone() for t in got]
        graph.replay()      # at once again: the same bits
        torch.cuda.synchronize()
        want = run()
        torch.cuda.synchronize()
        for a, b, c in zip(mine, got, want):
            assert torch.equal(a, c) and torch.equal(b, c), turn
    # and the last eager result against float64, loosely: the bounds proper are test_gpu_adapter.py's
    index.copy_(torch.arange(M, device="cuda").int() % n)
    out, H = run()[:2]
    a = index.long()
    wantH = torch.einsum("mk,mrk->mr", X.double(), A.double()[a])
    assert ((H.double() - wantH).abs().amax(1) <= 1e-4 * wantH.abs().amax(1)).all()
    want = Y.double() + scale.double()[a][:, None] * torch.einsum("mr,mnr->mn", wantH, B.double()[a])
    assert ((out.double() - want).abs().amax(1) <= 2 ** -8 * want.abs().amax(1)).all()
