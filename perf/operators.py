"""Workloads of the operators around a projection: layer norm, low-rank adapters, AdamW.

Each case is one pass through one operator. `run` computes it in a plain form (elementary torch
operations in float32, rounded once at the end) where `own` is false, and through the package's
entry points where it is true. `exact` gives the same outputs in float64.

Operators and their definitions:
  ln_fwd       Y = (X - mean) * rstd * weight + bias over the rows of X [M, K]; also mean, rstd
  ln_bwd       dX, dweight, dbias from dY, X, mean, rstd, weight
  adapter_fwd  out[m] = Y[m] + scale[a] * (X[m] A[a]^T) B[a]^T with a = index[m]; index -1: out[m] = Y[m]
  adapter_bwd  dX[m] + G[m] A[a], dA[a] = sum G[m]^T X[m], dB[a] = scale[a] sum dY[m]^T H[m], with
               G[m] = scale[a] dY[m] B[a] and H = X A^T kept by the forward pass
  adamw        one AdamW step over many tensors, in place; the moments in float32 or, in blocks of
               256, as E4M3 codes of the first moment and of the root of the second one, with one
               power-of-two scale a block
"""

import math

import numpy as np
import torch

own = False

BLOCK = 256          # elements that share one scale of an 8-bit state
LR, BETA1, BETA2, EPS, DECAY, STEP = 1e-3, 0.9, 0.999, 1e-8, 0.01, 10
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # a decode batch of 16 rows of a 4096-wide model in front of its projections: latency
        {"name": "ln fwd decode", "op": "ln_fwd", "M": 16, "K": 4096, "x": "bf16", "w": "bf16"},
        # GPT-2-Large rows (16 sequences of 1024), a training batch with outlier rows
        {"name": "ln fwd large", "op": "ln_fwd", "M": 16384, "K": 1280, "x": "bf16", "w": "bf16"},
        # its backward pass, with the column sums over all rows; float32 weights beside bf16 rows
        {"name": "ln bwd large", "op": "ln_bwd", "M": 16384, "K": 1280, "x": "bf16", "w": "fp32"},
        # odd row count and width in float32: no row after the first starts on a vector boundary
        {"name": "ln bwd odd", "op": "ln_bwd", "M": 2051, "K": 1021, "x": "fp32", "w": "fp32"},
        # decode: 48 requests of one token each, 24 adapters, on a 4096 x 4096 projection
        {"name": "adapter fwd decode", "op": "adapter_fwd", "M": 48, "K": 4096, "N": 4096, "R": 16, "adapters": 24,
         "rows": "single", "dtype": "bf16", "keep": False},
        # prefill of ragged requests, some without an adapter, on the widest projection
        {"name": "adapter fwd prefill", "op": "adapter_fwd", "M": 4096, "K": 4096, "N": 14336, "R": 16, "adapters": 8,
         "rows": "ragged", "dtype": "bf16", "keep": False},
        # float32, odd everywhere: the general path
        {"name": "adapter fwd odd", "op": "adapter_fwd", "M": 333, "K": 1001, "N": 770, "R": 6, "adapters": 5,
         "rows": "ragged", "dtype": "fp32", "keep": True},
        # fine-tuning one adapter on a 4096 x 4096 projection, 4096 tokens
        {"name": "adapter bwd one", "op": "adapter_bwd", "M": 4096, "K": 4096, "N": 4096, "R": 16, "adapters": 1,
         "rows": "one", "dtype": "bf16"},
        # fine-tuning four adapters at once on GPT-2-Small's widest attention projection, 8192 tokens
        {"name": "adapter bwd many", "op": "adapter_bwd", "M": 8192, "K": 768, "N": 2304, "R": 32, "adapters": 4,
         "rows": "ragged", "dtype": "bf16"},
        # the adapter pairs of a small model's 12 blocks and their norms: many small tensors, latency
        {"name": "adamw adapters", "op": "adamw", "sizes": "6144*24 18432*12 24576*12 768*24 1021*8", "p": "bf16",
         "g": "bf16", "master": True, "bits": 32},
        # GPT-2-Small's compressed projections (c = 2), float32 throughout
        {"name": "adamw small model", "op": "adamw", "sizes": "884736*12 294912*12 1179648*24 768*25", "p": "fp32",
         "g": "fp32", "master": False, "bits": 32},
        # one Llama-3-8B block's seven compressed projections (c = 2), bf16 weights, 8-bit states
        {"name": "adamw 8-bit block", "op": "adamw", "sizes": "8388608*2 2097152*2 29360128*3 4096*2", "p": "bf16",
         "g": "bf16", "master": True, "bits": 8},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_bwd", "adapter_fwd", "adapter_bwd", "adamw"])
    if op in ("ln_fwd", "ln_bwd"):
        K = _log(rng, 64, 8192)
        K = K if rng.random() < 0.4 else (K + 63) // 64 * 64
        M = _log(rng, 1, max(2, min(32768, 20_000_000 // K)))
        x, w = rng.choice([("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32")])
        return {"op": op, "M": M, "K": K, "x": x, "w": w}
    if op in ("adapter_fwd", "adapter_bwd"):
        dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
        top = 8192 if dtype == "bf16" else 1024
        K, N = _log(rng, 256, top), _log(rng, 256, top)
        if rng.random() < 0.75:
            K, N = (K + 63) // 64 * 64, (N + 63) // 64 * 64
        M = _log(rng, 1, max(2, min(8192 if dtype == "bf16" else 1024, 50_000_000 // (K + N))))
        R = rng.choice([4, 8, 8, 16, 16, 16, 32, 5, 12, 64])
        adapters = min(M, rng.choice([1, 2, 3, 8, 16, 32]))
        rows = "one" if adapters == 1 else rng.choice(["ragged", "single"])
        case = {"op": op, "M": M, "K": K, "N": N, "R": R, "adapters": adapters, "rows": rows, "dtype": dtype}
        return dict(case, keep=rng.random() < 0.5) if op == "adapter_fwd" else case
    kinds = [(_log(rng, 64, 4_000_000), rng.randint(1, 12)) for _ in range(rng.randint(1, 6))]
    p, g, master = rng.choice([("bf16", "bf16", True), ("bf16", "bf16", False), ("bf16", "fp32", True),
                               ("fp32", "fp32", False)])
    return {"op": "adamw", "sizes": " ".join("%d*%d" % k for k in kinds), "p": p, "g": g, "master": master,
            "bits": rng.choice([32, 8])}


def _sizes(case):
    return [int(n) for part in case["sizes"].split() for n in [part.split("*")[0]] * int(part.split("*")[1])]


def _index(case, seed):
    """One adapter a row: requests of ragged lengths in order, or every row a request of its own."""
    M, n = case["M"], case["adapters"]
    if case["rows"] == "one":
        return None
    rng = np.random.RandomState(seed % (1 << 31))
    if case["rows"] == "single":
        return rng.randint(0, n, M).astype(np.int32)
    cuts = np.sort(rng.randint(0, M + 1, 2 * n - 1))
    lengths = np.diff(np.concatenate([[0], cuts, [M]]))
    who = rng.randint(-1, n, 2 * n)                      # -1: a request without an adapter
    return np.repeat(who, lengths).astype(np.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)

    op = case["op"]
    if op in ("ln_fwd", "ln_bwd"):
        M, K, xt, wt = case["M"], case["K"], DTYPES[case["x"]], DTYPES[case["w"]]
        X = normal(M, K) + normal(M, 1, std=0.5)
        X[torch.rand(M, generator=gen, device="cuda") < 0.01] *= 20.0
        s = {"case": case, "X": X.to(xt), "weight": (1.0 + normal(K, std=0.1)).to(wt), "bias": normal(K, std=0.1, dtype=wt)}
        if op == "ln_bwd":
            x = s["X"].double()
            mean = x.mean(1)
            s["mean"] = mean.float()
            s["rstd"] = (1.0 / torch.sqrt((x - mean[:, None]).square().mean(1) + 1e-5)).float()
            s["dY"] = normal(M, K, dtype=xt)
        return s
    if op in ("adapter_fwd", "adapter_bwd"):
        M, K, N, R, n, t = case["M"], case["K"], case["N"], case["R"], case["adapters"], DTYPES[case["dtype"]]
        index = _index(case, seed)
        s = {"case": case, "X": normal(M, K, dtype=t), "A": normal(n, R, K, std=K ** -0.5, dtype=t),
             "B": normal(n, N, R, std=0.05, dtype=t),
             "index": None if index is None else torch.from_numpy(index).cuda(),
             "scale": 0.5 + torch.rand(n, generator=gen, device="cuda") * 1.5}
        if op == "adapter_fwd":
            s["Y"] = normal(M, N, dtype=t)
        else:
            s["dY"], s["dX"] = normal(M, N, dtype=t), normal(M, K, dtype=t)
            s["H"] = _products(s["X"].double(), s["A"].double(), s["index"]).float()
        return s
    pt, gt, sizes = DTYPES[case["p"]], DTYPES[case["g"]], _sizes(case)
    starts = np.concatenate([[0], np.cumsum([(n + 63) // 64 * 64 for n in sizes])]).tolist()   # aligned views of one buffer
    total = starts[-1]

    def views(flat):
        return [flat[a:a + n] for a, n in zip(starts, sizes)]

    w = normal(total, std=0.02)
    s = {"case": case, "p_flat": w.to(pt), "g": views(normal(total, std=1e-3, dtype=gt))}
    s["p"] = views(s["p_flat"])
    if case["master"]:
        s["master_flat"] = w
        s["master"] = views(w)
    first, second = normal(total, std=3e-4), normal(total, std=1e-3).square()
    if case["bits"] == 32:
        s["m_flat"], s["v_flat"] = first, second
        s["m"], s["v"] = views(first), views(second)
        return s
    blocks = [-(-n // BLOCK) for n in sizes]
    bstart = np.concatenate([[0], np.cumsum(blocks)]).tolist()
    for name, values in (("m", first), ("r", second.sqrt())):
        codes, scales = _encode(_blocked(views(values)), name == "r")
        s[name + "_scale_flat"] = scales
        s[name + "_scale"] = [scales[a:a + b] for a, b in zip(bstart, blocks)]
        s[name + "_flat"] = torch.zeros(total, dtype=torch.uint8, device="cuda")
        s[name] = views(s[name + "_flat"])
        _unblock(codes, s[name])
    return s


# ---- plain forms ---------------------------------------------------------------------------

def _pick(table, index, M):
    """What each row's adapter has in `table` [n, ...]; 0 where it has none."""
    if index is None:
        return table[0].expand(M, *table.shape[1:])
    some = (index >= 0).reshape(-1, *[1] * (table.dim() - 1))
    return torch.where(some, table[index.clamp(min=0).long()], 0)


def _mask(index, n, like):
    """[M, n, 1]: whether row m goes to adapter a."""
    if index is None:
        return torch.ones(like.shape[0], 1, 1, dtype=torch.bool, device=like.device)
    return (index[:, None] == torch.arange(n, device=like.device)[None, :])[:, :, None]


def _products(x, table, index):
    """[M, R] = x[m] table[a]^T with a = index[m], from one product with every adapter's rows."""
    n, R, K = table.shape
    every = (x @ table.reshape(n * R, K).T).reshape(-1, n, R)
    return torch.where(_mask(index, n, x), every, 0).sum(1)


def _spread(h, index, n):
    """[M, n * R]: h[m] in the columns of row m's adapter, 0 in the others'."""
    return torch.where(_mask(index, n, h), h[:, None, :], 0).reshape(h.shape[0], -1)


def _blocked(tensors):
    """[blocks, BLOCK] float32: every tensor, the last block of each filled up with zeros."""
    return torch.cat([torch.nn.functional.pad(t.float(), (0, -t.numel() % BLOCK)) for t in tensors]).reshape(-1, BLOCK)


def _unblock(blocks, tensors):
    flat = blocks.reshape(-1)
    starts = np.concatenate([[0], np.cumsum([-(-t.numel() // BLOCK) * BLOCK for t in tensors])]).tolist()
    [t.copy_(flat[a:a + t.numel()]) for a, t in zip(starts, tensors)]


def _encode(values, positive):
    """(E4M3 codes as uint8, scales) of [blocks, BLOCK]: the scale is the smallest power of two (from
    2^-126 on) that brings the block's largest magnitude to 448 or below. A positive value never
    becomes 0 where `positive` is asked for: it takes at least the smallest code."""
    mantissa, exponent = torch.frexp(values.abs().amax(1))
    e = (exponent - torch.where(mantissa <= 0.875, 9, 8)).clamp(min=-126)
    scales = torch.ldexp(torch.ones_like(mantissa), e)
    codes = (values / scales[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    if positive:
        codes = torch.where(values > 0, codes.clamp(min=1), codes)
    return codes, scales


def _decode(codes, scales):
    return codes.view(torch.float8_e4m3fn).float() * scales[:, None]


def _blocked_codes(tensors):
    return torch.cat([torch.nn.functional.pad(t, (0, -t.numel() % BLOCK)) for t in tensors]).reshape(-1, BLOCK)


def _adamw(s):
    case = s["case"]
    g = _blocked(s["g"])
    p = _blocked(s["master"] if case["master"] else s["p"])
    if case["bits"] == 32:
        m, v = _blocked(s["m"]), _blocked(s["v"])
    else:
        m = _decode(_blocked_codes(s["m"]), torch.cat(s["m_scale"]))
        r = _decode(_blocked_codes(s["r"]), torch.cat(s["r_scale"]))
        v = r * r
    m = m * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + (g * g) * (1 - BETA2)
    root = torch.sqrt(v)
    denominator = root * (1 / math.sqrt(1 - BETA2 ** STEP)) + EPS
    p = p * (1 - LR * DECAY) - (m / denominator) * (LR / (1 - BETA1 ** STEP))
    if case["master"]:
        _unblock(p, s["master"])
    _unblock(p, s["p"])
    if case["bits"] == 32:
        _unblock(m, s["m"])
        _unblock(v, s["v"])
        return
    for name, values in (("m", m), ("r", root)):
        codes, scales = _encode(values, name == "r")
        s[name + "_scale_flat"].copy_(scales)
        _unblock(codes, s[name])


def _adamw_out(s):
    """The updated parameters and moments; 8-bit moments as the values that they stand for."""
    out = {"p": s["p_flat"]}
    if s["case"]["master"]:
        out["master"] = s["master_flat"]
    if s["case"]["bits"] == 32:
        return dict(out, m=s["m_flat"], v=s["v_flat"])
    return dict(out, m=_decode(_blocked_codes(s["m"]), s["m_scale_flat"]),
                root=_decode(_blocked_codes(s["r"]), s["r_scale_flat"]))


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "ln_fwd":
        x = s["X"].float()
        mean = x.mean(1, keepdim=True)
        rstd = 1.0 / torch.sqrt((x - mean).square().mean(1, keepdim=True) + 1e-5)
        y = (x - mean) * rstd * s["weight"].float() + s["bias"].float()
        return {"Y": y.to(s["X"].dtype), "mean": mean[:, 0], "rstd": rstd[:, 0]}
    if op == "ln_bwd":
        xhat = (s["X"].float() - s["mean"][:, None]) * s["rstd"][:, None]
        dy = s["dY"].float()
        g = dy * s["weight"].float()
        dx = (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True)) * s["rstd"][:, None]
        wt = s["weight"].dtype
        return {"dX": dx.to(s["X"].dtype), "dweight": (dy * xhat).sum(0).to(wt), "dbias": dy.sum(0).to(wt)}
    if op in ("adapter_fwd", "adapter_bwd"):
        t, n, index, M = s["X"].dtype, case["adapters"], s["index"], case["M"]
        x, A, B = s["X"].float(), s["A"].float(), s["B"].float()
        wide_b = B.transpose(1, 2).reshape(-1, B.shape[1])           # [n * R, N]
        scale = _pick(s["scale"], index, M)[:, None]
    if op == "adapter_fwd":
        h = _products(x, A, index)
        out = (s["Y"].float() + _spread(h * scale, index, n) @ wide_b).to(t)
        return {"out": out, "H": h} if case["keep"] else {"out": out}
    if op == "adapter_bwd":
        dy = s["dY"].float() * scale
        g = _spread(_products(dy, B.transpose(1, 2), index), index, n)
        dx = s["dX"].float() + g @ A.reshape(-1, A.shape[2])
        da = (g.T @ x).reshape(A.shape)
        db = (_spread(s["H"], index, n).T @ dy).reshape(n, case["R"], -1).transpose(1, 2)
        return {"dX": dx.to(t), "dA": da.to(t), "dB": db.to(t)}
    _adamw(s)
    return _adamw_out(s)


# ---- the package's entry points --------------------------------------------------------------

def _own(s):
    from structured_compressed_linear_b200 import ops
    case, op = s["case"], s["case"]["op"]
    if op == "ln_fwd":
        Y, mean, rstd = ops.layernorm_forward(s["X"], s["weight"], s["bias"], eps=1e-5)
        return {"Y": Y, "mean": mean, "rstd": rstd}
    if op == "ln_bwd":
        dX, dw, db = ops.layernorm_backward(s["dY"], s["X"], s["mean"], s["rstd"], s["weight"])
        return {"dX": dX, "dweight": dw, "dbias": db}
    if op == "adapter_fwd":
        if case["keep"]:
            out, H = ops.adapter_forward(s["X"], s["A"], s["B"], s["Y"], index=s["index"], scale=s["scale"], keep=True)
            return {"out": out, "H": H}
        return {"out": ops.adapter_forward(s["X"], s["A"], s["B"], s["Y"], index=s["index"], scale=s["scale"])}
    if op == "adapter_bwd":
        dX, dA, dB = ops.adapter_backward(s["dY"], s["X"], s["A"], s["B"], s["H"], s["dX"], index=s["index"],
                                          scale=s["scale"])
        return {"dX": dX, "dA": dA, "dB": dB}
    states = (s["m"], s["v"]) if case["bits"] == 32 else (s["m"], s["r"])
    scales = None if case["bits"] == 32 else (s["m_scale"], s["r_scale"])
    ops.adamw_step(s["p"], s["g"], states[0], states[1], step=STEP, lr=LR, betas=(BETA1, BETA2), eps=EPS,
                   weight_decay=DECAY, master=s["master"] if case["master"] else None, scales=scales)
    return _adamw_out(s)


def run(state):
    return _own(state) if own else _plain(state)


# ---- what a pass cannot do without -----------------------------------------------------------

def work(case):
    op, size = case["op"], {"bf16": 2, "fp32": 4}
    if op == "ln_fwd":
        M, K = case["M"], case["K"]
        return {"bytes": 2 * M * K * size[case["x"]] + 2 * K * size[case["w"]] + 8 * M, "flops": 8 * M * K}
    if op == "ln_bwd":
        M, K = case["M"], case["K"]
        return {"bytes": 3 * M * K * size[case["x"]] + 3 * K * size[case["w"]] + 8 * M, "flops": 14 * M * K}
    if op in ("adapter_fwd", "adapter_bwd"):
        M, K, N, R, n, e = case["M"], case["K"], case["N"], case["R"], case["adapters"], size[case["dtype"]]
        few = 0 if case["rows"] == "one" else 4 * M                  # the index
        # the adapters that rows name: all of them once there are many rows a piece
        n = n if case["rows"] != "single" else n * (1 - (1 - 1 / n) ** M)
        pair = n * R * (K + N) * e
        if op == "adapter_fwd":
            kept = 4 * M * R if case["keep"] else 0
            return {"bytes": M * K * e + pair + 2 * M * N * e + kept + few, "flops": 2 * M * R * (K + N)}
        return {"bytes": M * N * e + 3 * M * K * e + 2 * pair + 4 * M * R + few, "flops": 4 * M * R * (K + N)}
    n = sum(_sizes(case))
    state = 16 if case["bits"] == 32 else 4 + 16 / BLOCK
    each = 2 * size[case["p"]] + size[case["g"]] + (8 if case["master"] else 0) + state
    if case["master"]:
        each -= size[case["p"]]                                      # a parameter with a master copy is only written
    return {"bytes": n * each, "flops": 16 * n}


# ---- the definition in 64 bits -----------------------------------------------------------------

def _e4m3_64(values):
    """[blocks, BLOCK] float64 rounded to E4M3 multiples of each block's power-of-two scale; a positive
    value takes at least the smallest code."""
    top = values.abs().amax(1, keepdim=True)
    exponent = torch.ceil(torch.log2(top / 448.0).clamp(min=-126))
    exponent = torch.where(top > 448.0 * torch.exp2(exponent), exponent + 1, exponent)
    exponent = torch.where((top <= 448.0 * torch.exp2(exponent - 1)) & (exponent > -126), exponent - 1, exponent)
    unit = torch.exp2(exponent)
    q = values / unit
    place = torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(place - 3)
    q = torch.round(q / step) * step                                  # ties to even
    return torch.where(values > 0, q.clamp(min=2.0 ** -9), q) * unit


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "ln_fwd":
        x = s["X"].double()
        var, mean = torch.var_mean(x, 1, correction=0)
        rstd = torch.rsqrt(var + 1e-5)
        y = torch.addcmul(s["bias"].double(), (x - mean[:, None]) * rstd[:, None], s["weight"].double())
        return {"Y": y, "mean": mean, "rstd": rstd}
    if op == "ln_bwd":
        # d/dx of the row's normalisation as the projection off the vectors (1) and (xhat)
        x, dy, w = s["X"].double(), s["dY"].double(), s["weight"].double()
        xhat = (x - s["mean"].double()[:, None]) * s["rstd"].double()[:, None]
        u = torch.stack([torch.ones_like(xhat), xhat], 2)             # [M, K, 2]
        along = torch.einsum("mk,mkj->mj", dy * w, u) / case["K"]
        dx = (dy * w - torch.einsum("mkj,mj->mk", u, along)) * s["rstd"].double()[:, None]
        return {"dX": dx, "dweight": torch.einsum("mk,mk->k", dy, xhat), "dbias": dy.sum(0)}
    if op in ("adapter_fwd", "adapter_bwd"):
        x, A, B, n = s["X"].double(), s["A"].double(), s["B"].double(), case["adapters"]
        index = torch.zeros(case["M"], dtype=torch.int32, device="cuda") if s["index"] is None else s["index"]
        H = torch.zeros(case["M"], case["R"], dtype=torch.float64, device="cuda")
        if op == "adapter_fwd":
            out = s["Y"].double()
            for a in range(n):
                rows = torch.nonzero(index == a)[:, 0]
                H[rows] = x[rows] @ A[a].T
                out[rows] += H[rows] @ (B[a].T * s["scale"][a].double())
            return {"out": out, "H": H} if case["keep"] else {"out": out}
        dx, dA, dB = s["dX"].double(), torch.zeros_like(A), torch.zeros_like(B)
        for a in range(n):
            rows = torch.nonzero(index == a)[:, 0]
            dy = s["dY"][rows].double()
            G = (dy @ B[a]) * s["scale"][a].double()
            dx[rows] += G @ A[a]
            dA[a] = G.T @ x[rows]
            dB[a] = (dy.T @ s["H"][rows].double()) * s["scale"][a].double()
        return {"dX": dx, "dA": dA, "dB": dB}
    # AdamW, tensor by tensor, into buffers laid out like the state's
    gap = {k: torch.zeros_like(s[k + "_flat"], dtype=torch.float64) for k in ("p", "master", "m", "v") if k + "_flat" in s}
    out, kept, at = {}, {"root": []}, 0
    for i, n in enumerate(_sizes(case)):
        g, p = s["g"][i].double(), s["master" if case["master"] else "p"][i].double()
        if case["bits"] == 32:
            m, v = s["m"][i].double(), s["v"][i].double()
        else:
            spread = [s[k][i].view(torch.float8_e4m3fn).double() * s[k + "_scale"][i].double().repeat_interleave(BLOCK)[:n]
                      for k in ("m", "r")]
            m, v = spread[0], spread[1].square()
        m, v = m + (g - m) * (1 - BETA1), v + (g.square() - v) * (1 - BETA2)
        mhat, vhat = m / (1 - BETA1 ** STEP), v / (1 - BETA2 ** STEP)
        p = p - LR * DECAY * p - LR * mhat / (vhat.sqrt() + EPS)
        for k, value in (("p", p), ("master", p), ("m", m), ("v", v)):
            if k in gap and (case["bits"] == 32 or k in ("p", "master")):
                gap[k][at:at + n] = value
        if case["bits"] == 8:
            kept["root"].append(_e4m3_64(torch.nn.functional.pad(v.sqrt(), (0, -n % BLOCK)).reshape(-1, BLOCK)))
        at += (n + 63) // 64 * 64
    # the gaps between the tensors stay as they were
    inside = torch.zeros(at, dtype=torch.bool, device="cuda")
    at = 0
    for n in _sizes(case):
        inside[at:at + n] = True
        at += (n + 63) // 64 * 64
    for k in ("p", "master") + (("m", "v") if case["bits"] == 32 else ()):
        if k in gap:
            out[k] = torch.where(inside, gap[k], s[k + "_flat"].double())
    if case["bits"] == 32:
        return out
    # A first moment is a 4-bit fraction times 0.9 plus an 8-bit fraction (bf16) times 0.1: about one in a
    # hundred lies exactly half way between two codes, and the rounding of 0.9 decides. So its codes
    # have no value apart from float32's arithmetic.
    return dict(out, m=None, root=torch.cat(kept["root"]))
