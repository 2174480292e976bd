"""Refusals of the operators around a projection, on CPU: every call here returns before it touches a
device (the addresses are made up and never read)."""

import ctypes
import re

import pytest
import torch

from tests.conftest import ROOT


@pytest.fixture(scope="module")
def lib():
    from structured_compressed_linear_b200 import build
    build.build()
    from structured_compressed_linear_b200 import ss1
    return ss1.load_library()


P = 0x10000   # a made-up, 256-byte aligned address


def test_layernorm_forward(lib):
    f = lib.ss1_layernorm_forward
    ok = dict(X=P, w=P, b=P, Y=P, mean=P, rstd=P, M=4, K=8, eps=1e-5, dtype=0, wt=1, st=None)

    def call(**change):
        return f(*dict(ok, **change).values())
    assert call(M=0) == 0                     # no rows: nothing to do
    assert call(M=0, X=None, Y=None) == 0
    for bad in (dict(M=-1), dict(K=0), dict(K=(1 << 30) + 1), dict(M=1 << 31), dict(dtype=2), dict(wt=7), dict(eps=-1e-5),
                dict(eps=float("nan")), dict(X=None), dict(Y=None), dict(dtype=1, wt=0)):
        assert call(**bad) == -1, bad
    for bad in (dict(X=P + 1), dict(Y=P + 1), dict(w=P + 2), dict(b=P + 2), dict(mean=P + 2), dict(rstd=P + 1)):
        assert call(**bad) == -5, bad


def test_layernorm_backward(lib):
    n = ctypes.c_size_t()
    assert lib.ss1_layernorm_backward_workspace(4000, 64, ctypes.byref(n)) == 0 and n.value > 0
    assert lib.ss1_layernorm_backward_workspace(-1, 64, ctypes.byref(n)) == -1
    assert lib.ss1_layernorm_backward_workspace(1, 0, ctypes.byref(n)) == -1
    assert lib.ss1_layernorm_backward_workspace(1, 1, None) == -1
    lib.ss1_layernorm_backward_workspace(4000, 64, ctypes.byref(n))
    ok = dict(dY=P, X=P, mean=P, rstd=P, w=P, dX=P, dw=P, db=P, M=4000, K=64, dtype=0, wt=0, ws=P, size=n.value, st=None)

    def call(**change):
        return lib.ss1_layernorm_backward(*dict(ok, **change).values())
    assert call(dX=None, dw=None, db=None) == 0
    assert call(M=0, dw=None, db=None) == 0
    for bad in (dict(dY=None), dict(X=None), dict(mean=None), dict(rstd=None), dict(ws=None), dict(size=n.value - 1), dict(M=-1),
                dict(K=0), dict(dtype=3), dict(wt=-1)):
        assert call(**bad) == -1, bad
    for bad in (dict(dY=P + 1), dict(X=P + 1), dict(dX=P + 1), dict(w=P + 1), dict(dw=P + 1), dict(db=P + 1), dict(mean=P + 2),
                dict(ws=P + 8)):
        assert call(**bad) == -5, bad


def _adapters(**change):
    from structured_compressed_linear_b200 import ops
    fields = dict(A=P, B=P, scale=P, index=P, plan=None, K=64, N=32, R=8, count=3, dtype=0)
    return ops._ADAPTERS.pack(*(v or 0 for v in dict(fields, **change).values()))


BAD_ADAPTERS = [dict(R=0), dict(R=129), dict(count=0), dict(count=1025), dict(K=0), dict(N=0), dict(K=(1 << 24) + 1), dict(dtype=2),
                dict(index=None), dict(A=None), dict(B=None), dict(count=1024, R=128, K=1 << 24)]


def test_adapter_plan(lib):
    n = ctypes.c_size_t()
    assert lib.ss1_adapter_plan_bytes(1000, 7, ctypes.byref(n)) == 0 and n.value >= 4000
    for M, count in ((-1, 1), (1, 0), (1, 1025), ((1 << 30) + 1, 1)):
        assert lib.ss1_adapter_plan_bytes(M, count, ctypes.byref(n)) == -1
    assert lib.ss1_adapter_plan_bytes(1, 1, None) == -1
    lib.ss1_adapter_plan_bytes(10, 2, ctypes.byref(n))
    assert lib.ss1_adapter_plan(None, 10, 2, P, n.value, None) == -1
    assert lib.ss1_adapter_plan(P, 10, 2, None, n.value, None) == -1
    assert lib.ss1_adapter_plan(P, 10, 2, P, n.value - 1, None) == -1
    assert lib.ss1_adapter_plan(P, 10, 0, P, n.value, None) == -1
    assert lib.ss1_adapter_plan(P, 10, 2, P + 16, n.value, None) == -5
    assert lib.ss1_adapter_plan(P + 2, 10, 2, P, n.value, None) == -5


def test_adapter_forward(lib):
    f = ctypes.c_size_t()
    assert lib.ss1_adapter_workspace(4, 64, 32, 8, 3, 0, ctypes.byref(f), None) == 0
    assert lib.ss1_adapter_workspace(4, 64, 32, 129, 3, 0, ctypes.byref(f), None) == -1
    ok = dict(X=P, Y=P, out=P, H=P, M=4, ws=P, size=f.value, st=None)

    def call(ad=None, **change):
        ad = _adapters(**(ad or {}))
        return lib.ss1_adapter_forward(ad, *dict(ok, **change).values())
    assert call(M=0) == 0
    assert lib.ss1_adapter_forward(None, *ok.values()) == -1
    for bad in BAD_ADAPTERS:
        assert call(ad=bad) == -1, bad
    for bad in (dict(X=None), dict(Y=None), dict(out=None), dict(ws=None), dict(size=f.value - 1), dict(M=-1)):
        assert call(**bad) == -1, bad
    for bad in (dict(X=P + 1), dict(Y=P + 1), dict(out=P + 1), dict(H=P + 2), dict(ws=P + 16)):
        assert call(**bad) == -5, bad
    for bad in (dict(A=P + 1), dict(B=P + 1), dict(scale=P + 2), dict(index=P + 1), dict(plan=P + 16)):
        assert call(ad=bad) == -5, bad


def test_adapter_backward(lib):
    b = ctypes.c_size_t()
    assert lib.ss1_adapter_workspace(4, 64, 32, 8, 3, 0, None, ctypes.byref(b)) == 0
    ok = dict(dY=P, X=P, H=P, dX_in=P, dX=P, dA=P, dB=P, M=4, ws=P, size=b.value, st=None)

    def call(ad=None, **change):
        ad = _adapters(**(ad or {}))
        return lib.ss1_adapter_backward(ad, *dict(ok, **change).values())
    assert call(dX_in=None, dX=None, dA=None, dB=None) == 0
    for bad in BAD_ADAPTERS:
        assert call(ad=bad) == -1, bad
    for bad in (dict(dY=None), dict(X=None), dict(H=None), dict(dX=None), dict(ws=None), dict(size=b.value - 1), dict(M=-1)):
        assert call(**bad) == -1, bad
    for bad in (dict(dY=P + 1), dict(X=P + 1), dict(H=P + 2), dict(dX_in=P + 1), dict(dX=P + 1), dict(dA=P + 1), dict(dB=P + 1),
                dict(ws=P + 128)):
        assert call(**bad) == -5, bad


def test_adamw(lib):
    import numpy as np

    from structured_compressed_linear_b200 import ops
    hyper = ops._AdamWHyper(1e-3, 0.9, 0.999, 1e-8, 0.01, 1.0, 1)

    def call(bits=32, count=1, h=hyper, factors=None, **change):
        t = np.zeros(1, ops._ADAMW_TENSOR)
        t[0] = (P, P, 0, P, P, P, P, 10, 0, 0)
        for k, v in change.items():
            t[k] = v
        return lib.ss1_adamw_step(t.ctypes.data, count, bits, ctypes.byref(h) if h is not None else None, factors, None)
    assert call(count=0) == 0
    assert call(numel=0, param=0, grad=0, exp_avg=0, exp_avg_sq=0) == 0
    assert call(count=-1) == -1 and call(bits=16) == -1 and call(h=None) == -1
    assert lib.ss1_adamw_step(None, 1, 32, ctypes.byref(hyper), None, None) == -1
    for bad in (dict(numel=-1), dict(numel=(1 << 40) + 1), dict(param_dtype=2), dict(grad_dtype=-1), dict(param=0), dict(grad=0),
                dict(exp_avg=0), dict(exp_avg_sq=0), dict(master=P, param_dtype=1), dict(bits=8, avg_scale=0),
                dict(bits=8, sq_scale=0)):
        assert call(**bad) == -1, bad
    for bad in (dict(param=P + 1), dict(grad=P + 1), dict(master=P + 2), dict(exp_avg=P + 2), dict(exp_avg_sq=P + 1),
                dict(bits=8, avg_scale=P + 2), dict(bits=8, sq_scale=P + 1), dict(factors=P + 2)):
        assert call(**bad) == -5, bad
    inf, nan = float("inf"), float("nan")
    for k, v in (("lr", nan), ("lr", inf), ("beta1", 1.0), ("beta1", -0.1), ("beta2", 1.0), ("beta2", nan), ("eps", -1e-9),
                 ("eps", inf), ("weight_decay", nan), ("grad_scale", inf), ("step", 0)):
        h = ops._AdamWHyper(1e-3, 0.9, 0.999, 1e-8, 0.01, 1.0, 1)
        setattr(h, k, v)
        assert call(h=h) == -1, (k, v)
        assert lib.ss1_adamw_factors(ctypes.byref(h), P) == -1
    assert lib.ss1_adamw_factors(ctypes.byref(hyper), None) == -1


def test_adamw_factors(lib):
    from structured_compressed_linear_b200 import ops
    got = ops.adamw_factors(3, 2e-3, (0.8, 0.95), 1e-7, 0.1, 0.5).tolist()
    want = [0.8, 0.2, 0.95, 0.05, 1 - 2e-4, 2e-3 / (1 - 0.8 ** 3), 1 / (1 - 0.95 ** 3) ** 0.5, 1e-7, 0.5]
    assert torch.tensor(got).allclose(torch.tensor(want), rtol=2 ** -22, atol=0)


def test_constants_match_header():
    import os

    from structured_compressed_linear_b200 import ops
    text = open(os.path.join(ROOT, "include", "ss1.h")).read()

    def const(name):
        return int(re.search(rf"#define\s+{name}\s+(\d+)", text).group(1))
    assert const("SS1_ADAPTER_MAX_RANK") == ops.ADAPTER_MAX_RANK
    assert const("SS1_ADAPTER_MAX_COUNT") == ops.ADAPTER_MAX_COUNT
    assert const("SS1_ADAMW_BLOCK") == ops.ADAMW_BLOCK
    assert const("SS1_ADAMW_FACTORS") == ops.ADAMW_FACTORS


def test_structs_match_header(tmp_path):
    """The binding's structures have the C compiler's layout."""
    import os
    import shutil
    import subprocess

    from structured_compressed_linear_b200 import ops
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc not available")
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include "ss1.h"\n#define AT(t, f) (int)offsetof(t, f)\nint main(void) {\n'
                   '  printf("%d %d %d %d %d %d %d\\n", (int)sizeof(ss1_adapters), AT(ss1_adapters, K), AT(ss1_adapters, dtype),\n'
                   '         (int)sizeof(ss1_adamw_tensor), AT(ss1_adamw_tensor, numel), AT(ss1_adamw_tensor, grad_dtype),\n'
                   '         (int)sizeof(ss1_adamw_hyper));\n  return 0;\n}\n')
    exe = tmp_path / "layout"
    subprocess.run([gcc, "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True).stdout.split()]
    f = ops._ADAMW_TENSOR.fields
    assert got == [ops._ADAPTERS.size, 40, 64, ops._ADAMW_TENSOR.itemsize,
                   f["numel"][1], f["grad_dtype"][1], ctypes.sizeof(ops._AdamWHyper)]


def test_binding_refuses_cpu_tensors():
    from structured_compressed_linear_b200 import ops
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        ops.layernorm_forward(x)
    with pytest.raises(ValueError):
        ops.layernorm_backward(x, x, x[:, 0], x[:, 0])
    with pytest.raises(ValueError):
        ops.adapter_plan(torch.zeros(4, dtype=torch.int32), 2)
    with pytest.raises(ValueError):
        ops.adapter_forward(x, torch.zeros(1, 2, 8), torch.zeros(1, 6, 2), torch.zeros(4, 6))
    with pytest.raises(ValueError):
        ops.adamw_step([x], [x], [x], [x])
    ops.adamw_step([], [], [], [])     # no tensors: nothing to do
