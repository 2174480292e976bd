"""The operators' binding on CPU: calls that reach its checks and no device."""

import pytest
import torch


@pytest.fixture(scope="module")
def ops():
    from structured_compressed_linear_b200 import build
    build.build()
    from structured_compressed_linear_b200 import ops
    return ops


class Stream:
    """What the binding reads of a torch.cuda.Stream of another device."""
    device = torch.device("cuda", 1)


def _calls(ops):
    x, i = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int32)
    A, B, Y = torch.zeros(1, 2, 8), torch.zeros(1, 6, 2), torch.zeros(4, 6)
    return [(ops.layernorm_forward, dict(X=x)), (ops.layernorm_backward, dict(dY=x, X=x, mean=x[:, 0], rstd=x[:, 0])),
            (ops.adapter_plan, dict(index=i, count=2)), (ops.adapter_forward, dict(X=x, A=A, B=B, Y=Y)),
            (ops.adapter_backward, dict(dY=Y, X=x, A=A, B=B, H=None)),
            (ops.adamw_step, dict(params=[x], grads=[x], exp_avg=[x], exp_avg_sq=[x]))]


def test_every_argument_by_name(ops):
    """Named arguments, the first among them, reach the same check as positional ones: CPU tensors are refused."""
    for fn, kw in _calls(ops):
        for call in (lambda: fn(**kw), lambda: fn(*kw.values())):
            with pytest.raises(ValueError, match="CUDA"):
                call()
        for call in (lambda: fn(**kw, stream=Stream()), lambda: fn(*kw.values(), stream=Stream())):
            with pytest.raises(ValueError, match="the stream is on cuda:1"):
                call()
        with pytest.raises(TypeError):
            fn(**dict(list(kw.items())[1:]))     # the first one is missing
    ops.adamw_step(params=[], grads=[], exp_avg=[], exp_avg_sq=[])


def test_size_caches_are_bounded(ops):
    """Ragged batches have ever new sizes; what is remembered of them stays bounded."""
    from structured_compressed_linear_b200 import ss1
    L = ss1.load_library()
    for cached, args in ((ops._norm_workspace, (64,)), (ops._plan_bytes, (3,))):
        for M in range(1, 5000):
            cached(L, M, *args)
        assert cached.cache_info().currsize <= 4096
    assert ops._adapter_workspace.cache_parameters()["maxsize"] == 4096


def test_an_optimizer_of_nothing(ops):
    opt = ops.AdamW([])
    opt.step()
    opt.zero_grad()
    assert opt.counts() == [] and opt.steps == 0
    opt.load_state_dict(opt.state_dict())
