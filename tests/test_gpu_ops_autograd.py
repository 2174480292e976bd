"""The operators beside autograd: what is written in place is known to it, and what has no derivative is refused."""

import pytest
import torch

from tests.gpu_common import get_ss1

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def libs():
    ss1 = get_ss1()
    from structured_compressed_linear_b200 import ops
    return ss1, ops


def _leaves(*shapes, t=F32):
    gen = torch.Generator().manual_seed(1)
    return [torch.randn(*s, generator=gen).to(t).cuda().requires_grad_() for s in shapes]


@pytest.mark.parametrize("bits", [32, 8])
def test_backward_after_a_step_is_refused(libs, bits):
    """The graph saved weights that the step has changed since: torch's own in-place check has to see it."""
    ss1, ops = libs
    M, K, N, R = 40, 256, 128, 8
    x, w, b, Wc, A, B = _leaves((M, K), (K,), (K,), (N, K // 2), (1, R, K), (1, N, R))
    layer = ss1.SS1Layer(K, N, 2, 128, 128, 3)
    for chosen in ([w], [Wc], [A], [B]):
        h = ops.LayerNormFunction.apply(x, w, b, 1e-5)
        y = ops.AdaptedSS1Function.apply(h, Wc, layer, A, B)
        opt = ops.AdamW(chosen, state_bits=bits)
        chosen[0].grad = torch.ones_like(chosen[0])
        opt.step()
        with pytest.raises(RuntimeError, match="inplace|in-place|modified"):
            y.sum().backward()
    for leaf in (x, w, b, Wc, A, B):
        leaf.grad = None
    ops.AdaptedSS1Function.apply(ops.LayerNormFunction.apply(x, w, b, 1e-5), Wc, layer, A, B).sum().backward()
    assert all(leaf.grad is not None for leaf in (x, w, b, Wc, A, B))
    layer.close()


def test_versions_of_what_is_written(libs):
    """adamw_step: parameters, masters, moments and scales, not gradients; `out` of the forward passes, not their inputs."""
    _, ops = libs
    n = 300
    P, G = torch.zeros(n, dtype=BF16, device="cuda"), torch.ones(n, dtype=BF16, device="cuda")
    W = torch.zeros(n, device="cuda")
    M, V = (torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2))
    sc = tuple([torch.zeros(2, device="cuda")] for _ in range(2))
    all_of = [P, W, M, V, sc[0][0], sc[1][0]]
    before = [t._version for t in all_of]
    ops.adamw_step([P], [G], [M], [V], master=[W], scales=sc)
    assert all(t._version > v for t, v in zip(all_of, before)) and G._version == 0
    x, a, b, y = (t.detach() for t in _leaves((5, 64), (1, 8, 64), (1, 32, 8), (5, 32)))
    out = torch.empty_like(x)
    ops.layernorm_forward(x, out=out)
    assert out._version == 1
    assert ops.adapter_forward(x, a, b, y)._version == 0 and y._version == 0
    ops.adapter_forward(x, a, b, y, out=y)
    assert y._version == 1 and x._version == a._version == b._version == 0


def test_a_backward_pass_that_saved_out_is_refused(libs):
    _, ops = libs
    x, a, b, y = _leaves((5, 64), (1, 8, 64), (1, 32, 8), (5, 32))
    z = y * 2.0
    loss = z.square().sum()                       # saves z
    with torch.no_grad():
        ops.adapter_forward(x, a, b, z, out=z)
    with pytest.raises(RuntimeError, match="inplace|in-place|modified"):
        loss.backward()


def test_second_derivatives_are_refused(libs):
    """create_graph=True is fine for a first derivative; a second one through the operators is an error, not a missing term."""
    ss1, ops = libs
    M, K, N, R = 40, 256, 128, 8
    x, w, b, Wc, A, B = _leaves((M, K), (K,), (K,), (N, K // 2), (1, R, K), (1, N, R))
    layer = ss1.SS1Layer(K, N, 2, 128, 128, 3)
    for make, leaf in ((lambda: ops.LayerNormFunction.apply(x, w, b, 1e-5), w),
                       (lambda: ops.AdaptedSS1Function.apply(x, Wc, layer, A, B), A),
                       (lambda: ss1.SS1Function.apply(x, Wc, layer), Wc)):
        y = make()
        plain, = torch.autograd.grad(y.square().sum(), leaf)
        first, = torch.autograd.grad(make().square().sum(), leaf, create_graph=True)
        assert torch.equal(plain, first.detach())
        with pytest.raises(RuntimeError, match="once_differentiable|differentiat"):
            first.square().sum().backward()
    layer.close()


def test_scale_has_no_gradient(libs):
    ss1, ops = libs
    x, Wc, A, B, scale = _leaves((8, 256), (128, 128), (1, 8, 256), (1, 128, 8), (1,))
    layer = ss1.SS1Layer(256, 128, 2, 128, 128, 3)
    with torch.no_grad():
        y = ops.AdaptedSS1Function.apply(x, Wc, layer, A, B, None, scale)
    z = ops.AdaptedSS1Function.apply(x, Wc, layer, A, B, None, scale)
    assert torch.equal(y, z)
    with pytest.raises(ValueError, match="scale"):
        z.sum().backward()
    ops.AdaptedSS1Function.apply(x, Wc, layer, A, B, None, scale.detach()).sum().backward()
    assert A.grad is not None and scale.grad is None
    layer.close()
