"""The operators together, as a model uses them: layer norm, an SS1 projection with adapters beside it,
the gradients of all of them, and AdamW; and a decode step captured into one graph."""

import numpy as np
import pytest
import torch

import oracle as O
from tests.gpu_common import get_ss1, to_np64

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def libs():
    ss1 = get_ss1()
    from structured_compressed_linear_b200 import ops
    return ss1, ops


def _block(seed, M, K, N, R, n, c, t):
    g = torch.Generator().manual_seed(seed)
    return {"x": torch.randn(M, K, generator=g).to(t), "w": (1 + 0.1 * torch.randn(K, generator=g)).to(t),
            "b": (0.1 * torch.randn(K, generator=g)).to(t), "Wc": (torch.randn(N, K // c, generator=g) * K ** -0.5).to(t),
            "A": (torch.randn(n, R, K, generator=g) * K ** -0.5).to(t), "B": (torch.randn(n, N, R, generator=g) * 0.2).to(t),
            "dY": torch.randn(M, N, generator=g).to(t)}


@pytest.mark.parametrize("M,K,N,c,BK,BN,t", [(200, 256, 384, 2, 128, 128, F32), (300, 1024, 384, 2, 128, 128, BF16)])
def test_block_gradients(libs, M, K, N, c, BK, BN, t):
    """Gradients of norm -> SS1 + adapters against float64 autograd of the definition. float32: 1e-4 of each
    row's largest value, the layer's own bound; bf16: its 2e-2 (the norm's output and the layer's are
    rounded to bf16 in between)."""
    ss1, ops = libs
    R, n, seed = 16, 3, 5
    d = _block(1, M, K, N, R, n, c, t)
    index = torch.randint(-1, n, (M,), generator=torch.Generator().manual_seed(2)).to(torch.int32)
    scale = torch.tensor([0.5, 1.0, 2.0])
    layer = ss1.SS1Layer(K, N, c, BK, BN, seed)
    leaf = {k: d[k].cuda().requires_grad_() for k in ("x", "w", "b", "Wc", "A", "B")}
    h = ops.LayerNormFunction.apply(leaf["x"], leaf["w"], leaf["b"], 1e-5)
    y = ops.AdaptedSS1Function.apply(h, leaf["Wc"], layer, leaf["A"], leaf["B"], index.cuda(), scale.cuda())
    y.backward(d["dY"].cuda())
    torch.cuda.synchronize()

    H, g = O.ss1_tables(K, N, c, BK, BN, seed)
    ref = {k: d[k].double().requires_grad_() for k in leaf}
    x = ref["x"]
    mean = x.mean(1, keepdim=True)
    rstd = 1 / torch.sqrt((x - mean).square().mean(1, keepdim=True) + 1e-5)
    hn = (x - mean) * rstd * ref["w"] + ref["b"]
    cols = torch.from_numpy(H.astype(np.int64))                              # [N / BN, K]
    signs = torch.from_numpy(g.astype(np.float64))
    full = torch.cat([ref["Wc"][i * BN:(i + 1) * BN][:, cols[i]] * signs[i] for i in range(N // BN)])
    out = hn @ full.T
    for a in range(n):
        rows = torch.nonzero(index == a)[:, 0]
        out = out.index_add(0, rows, scale[a].double() * (hn[rows] @ ref["A"][a].T) @ ref["B"][a].T)
    out.backward(d["dY"].double())
    tol = 1e-4 if t == F32 else 2e-2

    def close(got, want, what):
        got, want = got.detach().double().cpu(), want.detach()
        got, want = got.reshape(-1, got.shape[-1]), want.reshape(-1, want.shape[-1])
        off = ((got - want).abs().amax(1) / want.abs().amax(1).clamp(min=1e-30)).max()
        assert off <= tol, f"{what}: {off:.3g}"
    close(y, out, "Y")
    for k in leaf:
        close(leaf[k].grad, ref[k].grad, k)
    layer.close()


def test_training_step_updates_every_parameter(libs):
    """One step of AdamW (8-bit states, float32 master copies) on the block's gradients."""
    ss1, ops = libs
    M, K, N = 96, 512, 256
    d = _block(3, M, K, N, 8, 2, 2, BF16)
    layer = ss1.SS1Layer(K, N, 2, 128, 128, 9)
    leaf = {k: d[k].cuda().requires_grad_() for k in ("w", "b", "Wc", "A", "B")}
    before = {k: v.detach().clone() for k, v in leaf.items()}
    opt = ops.AdamW(leaf.values(), lr=1e-2, weight_decay=0.0, state_bits=8, master=True)
    index = (torch.arange(M) % 2).to(torch.int32).cuda()
    h = ops.LayerNormFunction.apply(d["x"].cuda(), leaf["w"], leaf["b"], 1e-5)
    ops.AdaptedSS1Function.apply(h, leaf["Wc"], layer, leaf["A"], leaf["B"], index).backward(d["dY"].cuda())
    grads = {k: v.grad.clone() for k, v in leaf.items()}
    opt.step()
    torch.cuda.synchronize()
    for i, (k, v) in enumerate(leaf.items()):
        # the first step is lr * sign(gradient), up to eps and rounding
        g = grads[k].double()
        moved = opt.master[i].double() - before[k].double()
        big = g.abs() > 1e-4
        assert big.any() and ((moved[big] + 1e-2 * g[big].sign()).abs() <= 1e-2 * (1e-4 + 1e-3)).all(), k
        assert torch.equal(v.detach(), opt.master[i].to(BF16))
    layer.close()


def test_decode_step_in_one_graph(libs):
    """norm -> projection -> adapters for a batch of single tokens, captured once and replayed on new tokens."""
    ss1, ops = libs
    M, K, N, n = 16, 1024, 512, 4
    d = _block(7, M, K, N, 16, n, 2, BF16)
    layer = ss1.SS1Layer(K, N, 2, 128, 128, 11)
    x, w, b, Wc, A, B = (d[k].cuda() for k in ("x", "w", "b", "Wc", "A", "B"))
    index = (torch.arange(M) % (n + 1) - 1).to(torch.int32).cuda()

    def step():
        h = ops.layernorm_forward(x, w, b)[0]
        y = layer.forward(h, Wc)
        return ops.adapter_forward(h, A, B, y, index, out=y)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step()
    for seed in (1, 2):
        x.copy_(torch.randn(M, K, generator=torch.Generator().manual_seed(seed)).to(BF16))
        index.copy_(index.roll(seed))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, step())
    Hh, g = O.ss1_tables(K, N, 2, 128, 128, 11)
    hn = ops.layernorm_forward(x, w, b)[0]
    want = O.ss1_forward(to_np64(hn), to_np64(Wc), Hh, g, 128)
    idx = index.cpu().numpy()
    for m in range(M):
        if idx[m] >= 0:
            want[m] += to_np64(B[idx[m]]) @ (to_np64(A[idx[m]]) @ to_np64(hn[m]))
    off = np.abs(to_np64(y) - want).max(1) / np.abs(want).max(1)
    assert off.max() <= 2e-2
    layer.close()
