"""The 8-bit AdamW states on the CPU, bit for bit as include/ss1.h defines them: codes, scales, and how a step rounds."""

import math

import numpy as np
import torch

BLOCK, NEAREST = 256, 10


def _mix(x):
    x = (x ^ x >> np.uint32(16)) * np.uint32(0x9E3779B9)
    x = (x ^ x >> np.uint32(15)) * np.uint32(0xBB67AE85)
    return x ^ x >> np.uint32(16)


def random_words(t, n):
    """uint32 [n]: step t's random word of each element."""
    with np.errstate(over="ignore"):
        key = _mix(np.array([(t & 0xFFFFFFFF)], np.uint32) * np.uint32(0x9E3779B9) + np.uint32((t >> 32) & 0xFFFFFFFF) * np.uint32(0xBB67AE85)
                   + np.uint32(0x3C6EF373))
        lane = np.arange(-(-n // 8), dtype=np.uint64)
        bits = _mix(lane.astype(np.uint32) ^ (key + (lane >> np.uint64(32)).astype(np.uint32) * np.uint32(0x9E3779B9)))
        out = np.empty((bits.size, 8), np.uint32)
        for i in range(8):
            out[:, i] = bits
            bits = bits * np.uint32(0xB7E15165) + np.uint32(0x243F6A89)
    return out.reshape(-1)[:n]


def neighbours(x, words):
    """One of the two E4M3 values around each x (float32, |x| <= 448), by the words' upper 20 bits."""
    shift = torch.where(x.abs() < 2.0 ** -6, torch.copysign(torch.full_like(x, 2.0 ** -6), x), torch.zeros_like(x))
    bits = (x + shift).numpy().view(np.uint32)
    with np.errstate(over="ignore"):
        y = torch.from_numpy(((bits + (words >> np.uint32(12))) & np.uint32(0xFFF00000)).view(np.float32)) - shift
    return torch.where(x == x, y, x)


def encode(values, positive, t):
    """(codes, scales) of float32 values as step t holds them; `positive`: roots."""
    n = values.numel()
    v = torch.nn.functional.pad(values.reshape(-1), (0, -n % BLOCK)).reshape(-1, BLOCK)
    mantissa, exponent = torch.frexp(v.abs().amax(1))
    exponent = torch.where(mantissa == 0, -999, exponent)
    scale = torch.ldexp(torch.ones_like(mantissa), (exponent - torch.where(mantissa <= 0.875, 9, 8)).clamp(min=-126))
    x = (v / scale[:, None]).reshape(-1)[:n]
    if t > NEAREST:
        words = random_words(t, n)
        with np.errstate(over="ignore"):
            x = neighbours(x.contiguous(), words if positive else words * np.uint32(0xBB67AE85))
    codes = x.to(torch.float8_e4m3fn).view(torch.uint8)
    if positive:
        codes = torch.where(values.reshape(-1) > 0, codes.clamp(min=1), codes)
    return codes, scale


def decode(codes, scale):
    return codes.reshape(-1).view(torch.float8_e4m3fn).float() * scale.repeat_interleave(BLOCK)[:codes.numel()]


def plain_step(p, g, m, v, t, lr, betas, eps, decay):
    """New (p, m, v, sqrt v), every float32 operation rounded on its own."""
    def f(x):
        return torch.tensor(x, dtype=torch.float32)
    b1, b2 = betas
    m = m * f(b1) + g * f(1 - b1)
    v = v * f(b2) + (g * g) * f(1 - b2)
    root = torch.sqrt(v.double()).float()
    den = root * f(1 / math.sqrt(1 - b2 ** t)) + f(eps)
    return p * f(1 - lr * decay) - (m / den) * f(lr / (1 - b1 ** t)), m, v, root


#: Gradients of a long run, by step: each element has a size of its own.
KINDS = ("constant", "normal", "shrinking")


def gradients(kind, n, steps, seed=0):
    """Yields float32 gradients [n]: one value for ever, normal ones, or normal ones that shrink tenfold over the run."""
    gen = torch.Generator().manual_seed(seed)
    size = torch.randn(n, generator=gen).exp() * 1e-3
    sign = torch.randn(n, generator=gen).sign()
    for t in range(steps):
        if kind == "constant":
            yield size * sign
        else:
            yield size * torch.randn(n, generator=gen) * (0.1 ** (t / steps) if kind == "shrinking" else 1.0)
