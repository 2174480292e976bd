"""A bounded wait of the adapters' tensor-core kernels that runs out: the kernel returns, says so, and leaves NaN in what it
was computing and nowhere else. No GPU fault is involved: one CTA does not announce finished products, and waits end after 5 ms."""

import pytest
import torch

from tests.gpu_common import get_ss1

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
TIMEOUT = -6


@pytest.fixture(scope="module")
def libs():
    ss1 = get_ss1()
    from structured_compressed_linear_b200 import ops
    return ss1, ops


def _call(ss1, ops, d, index, out, **change):
    """ss1_test_adapter_timeout's status."""
    M, K = d["X"].shape
    n, N, R = d["B"].shape
    code = int(ss1._dtype_code(d["X"].dtype))
    ad = ops._ADAPTERS.pack(d["A"].data_ptr(), d["B"].data_ptr(), 0, index.data_ptr() if index is not None else 0, 0, K, N, R, n, code)
    size = ops._adapter_workspace(ss1.lib(), M, K, N, R, n, code, True)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    args = dict(ad=ad, dY=d["dY"].data_ptr(), X=d["X"].data_ptr(), H=d["H"].data_ptr(), dX_in=d["dX"].data_ptr(), dX=out[0].data_ptr(),
                dA=out[1].data_ptr(), dB=out[2].data_ptr(), M=M, ws=ws.data_ptr(), size=size, site=1, limit=1000,
                st=torch.cuda.current_stream().cuda_stream)
    status = ss1.lib().ss1_test_adapter_timeout(*dict(args, **change).values())
    torch.cuda.synchronize()            # the kernels returned
    return status


def _inputs(M, K, N, R, n, dtype=BF16):
    g = torch.Generator().manual_seed(M + R)
    d = {"X": torch.randn(M, K, generator=g), "A": torch.randn(n, R, K, generator=g) * K ** -0.5, "B": torch.randn(n, N, R, generator=g),
         "dY": torch.randn(M, N, generator=g), "dX": torch.randn(M, K, generator=g)}
    d = {k: v.to(dtype).cuda() for k, v in d.items()}
    d["H"] = torch.randn(M, R, generator=g).cuda()
    return d


@pytest.mark.parametrize("M,K,N,R,n", [(700, 512, 768, 16, 3), (300, 264, 4352, 64, 1), (260, 256, 512, 128, 2), (140, 64, 64, 12, 1)])
@pytest.mark.parametrize("site", [1, 2, 3])
def test_a_wait_that_runs_out(libs, site, M, K, N, R, n):
    ss1, ops = libs
    d = _inputs(M, K, N, R, n)
    index = None if n == 1 else (torch.arange(M) * n // M).int().cuda()       # adapter 0's rows first
    good = ops.adapter_backward(d["dY"], d["X"], d["A"], d["B"], d["H"], d["dX"], index)
    torch.cuda.synchronize()
    assert ops.adapter_status() == (0, 0)
    got = tuple(torch.zeros_like(t) for t in good)
    assert _call(ss1, ops, d, index, got, site=site, limit=5_000_000) == 0
    assert ops.adapter_status() == (TIMEOUT, (4 << 8) | 0x80 | site)
    assert ops.adapter_status() == (0, 0)
    first = min(M, 128)                        # the first tile, all of adapter 0
    dX, dA, dB = got
    if site == 1:
        assert dX[:first].isnan().all() and torch.equal(dX[first:], good[0][first:])
        assert dA[0].isnan().all() and torch.equal(dA[1:], good[1][1:]) and torch.equal(dB, good[2])
    elif site == 2:
        some = dB[0, :min(N, 256)]
        assert some.isnan().all() and not dB[:, 256:].isnan().any()
        assert torch.equal(dX, good[0]) and torch.equal(dA, good[1]) and torch.equal(dB[:, 256:], good[2][:, 256:])
    else:
        some = dA[0, :, :min(K, 256)]
        assert some.isnan().all() and not dA[:, :, 256:].isnan().any()
        assert torch.equal(dX, good[0]) and torch.equal(dB, good[2]) and torch.equal(dA[:, :, 256:], good[1][:, :, 256:])
    again = ops.adapter_backward(d["dY"], d["X"], d["A"], d["B"], d["H"], d["dX"], index)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(again, good)) and ops.adapter_status(0) == (0, 0)


def test_refusals(libs):
    ss1, ops = libs
    d = _inputs(140, 64, 64, 12, 1)
    out = tuple(torch.zeros_like(d[k]) for k in ("dX", "A", "B"))
    for bad in (dict(site=0), dict(site=4), dict(limit=0), dict(limit=2_000_000_001), dict(dX=None), dict(dA=None), dict(dB=None), dict(M=0)):
        assert _call(ss1, ops, d, None, out, **bad) == -1, bad
    assert _call(ss1, ops, d, None, out, dY=d["dY"].data_ptr() + 2) == -8      # not the tensor-core kernels' alignment
    odd = _inputs(140, 64, 64, 12, 1, torch.float32)
    assert _call(ss1, ops, odd, None, tuple(torch.zeros_like(odd[k]) for k in ("dX", "A", "B"))) == -8
    assert not any(t.any() for t in out) and ops.adapter_status() == (0, 0)
