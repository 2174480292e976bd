"""How the 8-bit AdamW states round, on the CPU form of their definition: that their random words are even, that a value is
held as it is on average, and that 2000 steps follow AdamW with float32 moments.

Bounds. Codes lie s <= 1/8 of the value apart. A step moves a root by a share d of itself, E|d| <= (1 - beta2) / 2
(E|g^2 / v - 1| <= 1 for a normal gradient), and rounding a move of d to codes s apart adds a variance of at most d s. A
deviation decays by 1 - beta2 a step, so its variance settles at or below (1 - beta2) / 2 / 8 / (2 (1 - beta2)) = 1/32, and the
mean square of 1 / root lies at most 3/32 above the undisturbed one, its root 4.7 %. The first moment's rounding, s^2 / 6 at
most a step, settles at 1/384 / (1 - beta1^2) = 1.4 % of the square, 0.7 % of the root; it is largest where g^2 is
beside v, so the two do not add up in full: 5 % over a run. A root that only shrinks (gradients that fall faster than
beta2 can follow: tenfold in 2000 steps at 0.999) has nothing that pulls it back: variance t (1 - beta2) / 2 / 8,
1/8 at the end, 3/16 of the square, 9 %, and where v is far below its largest the codes are coarser: 15 % there."""

import math

import numpy as np
import pytest
import torch

from tests import adamw_states as S


def test_words_are_even():
    """4096 steps of 16,384 elements: means within 5 standard errors, no correlation with the next step or the next element."""
    n, first, steps = 16384, 11, 1024
    u = np.stack([S.random_words(t, n) for t in range(first, first + steps)])
    with np.errstate(over="ignore"):
        for w in (u, u * np.uint32(0xBB67AE85)):
            x = (w >> np.uint32(12)) / 2.0 ** 20 - 0.5
            sd = math.sqrt(1 / 12)
            assert abs(x.mean()) <= 5 * sd / math.sqrt(x.size)
            assert np.abs(x.mean(0)).max() <= 5.5 * sd / math.sqrt(steps)      # 16,384 elements' own means
            for a, b in ((x[1:], x[:-1]), (x[:, 1:], x[:, :-1])):
                assert abs((a * b).mean()) * 12 <= 5 / math.sqrt(a.size)
            few = (x > 0.495).mean(0) * steps                                  # rare events: Poisson counts
            assert abs(few.mean() - 0.005 * steps) <= 0.05 and 0.9 <= few.var() / few.mean() <= 1.1


def test_words_of_far_places():
    """Steps past 2^32 and the words' independence of the length asked for."""
    assert np.array_equal(S.random_words(17, 100), S.random_words(17, 10000)[:100])
    assert not np.array_equal(S.random_words(17, 64), S.random_words(17 + (1 << 32), 64))


@pytest.mark.parametrize("x", [0.0, 1.0, 1.03, 300.0, 447.9, 448.0, 0.0156, 0.0157, 0.003, 0.0001, -1.03, -0.003, -447.9])
def test_a_value_is_held_as_it_is_on_average(x):
    n = 1 << 18
    y = S.neighbours(torch.full((n,), x), S.random_words(11, n))
    v = float(torch.tensor(x))
    kinds = y.unique()
    assert len(kinds) <= 2 and torch.equal(kinds.to(torch.float8_e4m3fn).float(), kinds)
    gap = float(kinds.max() - kinds.min())
    assert gap <= max(abs(v) / 8, 2.0 ** -9)
    if v in kinds.tolist():
        assert len(kinds) == 1
    # a share p of n draws: within 5 standard errors, and the 20 bits' step
    assert abs(float(y.double().mean()) - v) <= gap * (5 * 0.5 / math.sqrt(n) + 2.0 ** -20) + 2.0 ** -30


def test_not_finite_values_stay_so():
    x = torch.tensor([float("nan"), float("inf"), -float("inf")] * 8)
    y = S.neighbours(x, S.random_words(99, 24))
    assert torch.equal(y.nan_to_num(7.0), x.nan_to_num(7.0))


def run(kind, beta2, steps=2000, n=8192):
    """r.m.s. updates of 8-bit over float32 moments: of the run, and of its last tenth; the held roots' median ratio."""
    betas, eps = (0.9, beta2), 1e-12
    zero = torch.zeros(n)
    m32, v32 = zero, zero
    m8, r8 = zero, zero
    sums = np.zeros((2, 2))
    for t, g in enumerate(S.gradients(kind, n, steps), 1):
        p32, m32, v32, root = S.plain_step(zero, g, m32, v32, t, 1.0, betas, eps, 0.0)
        p8, m, v, r = S.plain_step(zero, g, m8, r8 * r8, t, 1.0, betas, eps, 0.0)
        m8, r8 = S.decode(*S.encode(m, False, t)), S.decode(*S.encode(r, True, t))
        both = np.array([float(p8.double().square().mean()), float(p32.double().square().mean())])
        sums[0] += both
        if t > steps - steps // 10:
            sums[1] += both
    return math.sqrt(sums[0, 0] / sums[0, 1]), math.sqrt(sums[1, 0] / sums[1, 1]), float((r8 / root).median())


def bounds(kind, beta2):
    """Of a run's r.m.s. ratio, of its last tenth's, and of the median root, each around 1."""
    falls = kind == "shrinking" and beta2 == 0.999
    return 0.05, 0.15 if falls else 0.05, 0.05


@pytest.mark.parametrize("beta2", [0.95, 0.99, 0.999])
@pytest.mark.parametrize("kind", S.KINDS)
def test_many_steps_follow_float32_moments(kind, beta2):
    got = run(kind, beta2)
    for ratio, bound in zip(got, bounds(kind, beta2)):
        assert abs(ratio - 1) <= bound, got


def test_refusals():
    """ss1_adamw_step_ex's own refusals (before it touches a device; the addresses are made up), and the constant's copies."""
    import ctypes
    import os
    import re

    from structured_compressed_linear_b200 import build, ops, ss1
    from tests.conftest import ROOT
    build.build()
    lib, P = ss1.load_library(), 0x10000
    hyper = ops._AdamWHyper(1e-3, 0.9, 0.999, 1e-8, 0.01, 1.0, 1)
    t = np.zeros(1, ops._ADAMW_TENSOR)
    t[0] = (P, P, 0, P, P, P, P, 10, 0, 0)

    def call(bits, factors, number, count=1, h=hyper):
        return lib.ss1_adamw_step_ex(t.ctypes.data, count, bits, ctypes.byref(h) if h else None, factors, number, None)
    assert call(8, P, P, count=0) == 0 and call(8, P, P, count=0, h=None) == 0
    assert call(32, None, P) == -1 and call(8, None, P) == -1          # a number without factors
    assert call(8, P, None) == -1                                      # factors without a number
    assert lib.ss1_adamw_step(t.ctypes.data, 1, 8, ctypes.byref(hyper), P, None) == -1
    assert call(8, P, P + 4) == -5 and call(8, P + 2, P) == -5
    assert call(8, None, None, h=None) == -1
    text = open(os.path.join(ROOT, "include", "ss1.h")).read()
    assert int(re.search(r"#define\s+SS1_ADAMW_NEAREST\s+(\d+)", text).group(1)) == ops.ADAMW_NEAREST == S.NEAREST


def test_overlaps():
    """Memory that a step writes may not overlap anything else of it (made-up addresses; refused before a device is touched)."""
    from structured_compressed_linear_b200 import build, ops, ss1
    import ctypes
    build.build()
    lib = ss1.load_library()
    hyper = ops._AdamWHyper(1e-3, 0.9, 0.999, 1e-8, 0.01, 1.0, 1)
    OVERLAP, K = -9, 1 << 20
    assert lib.ss1_strerror(OVERLAP) != lib.ss1_strerror(12345)

    def call(bits, *rows, factors=None):
        t = np.zeros(len(rows), ops._ADAMW_TENSOR)
        for i, row in enumerate(rows):
            t[i] = (*(K * a + b for a, b in row[:7]), 1000, *row[7:])
        return lib.ss1_adamw_step_ex(t.ctypes.data, len(rows), bits, ctypes.byref(hyper), factors, None, None)

    def entry(first, **change):
        """Param, grad, master, moments and scales at megabytes first, first + 1, ..., bf16."""
        names = ("param", "grad", "master", "exp_avg", "exp_avg_sq", "avg_scale", "sq_scale")
        at = {k: (first + i, 0) for i, k in enumerate(names)}
        at.update(change)
        return (*(at[k] for k in names), 0, 0)
    a, none = entry(1), (0, 0)
    for bits, size in ((32, 4), (8, 1)):
        for k, n in (("param", 2000), ("grad", 2000), ("master", 4000), ("exp_avg", 1000 * size), ("exp_avg_sq", 1000 * size)):
            for other, m in (("param", 2000), ("exp_avg", 1000 * size), ("exp_avg_sq", 1000 * size)):
                if other == k:
                    continue
                at = dict(zip(("param", "grad", "master", "exp_avg", "exp_avg_sq"), a))[other]
                # on it, its last bytes, and from below into its first ones (a gradient on its parameter is allowed)
                shifts = [4 * ((m - 1) // 4), -4 * ((n - 1) // 4)] + ([0] if (k, other) != ("grad", "param") else [])
                for shift in shifts:
                    assert call(bits, entry(1, **{k: (at[0], shift)})) == OVERLAP, (bits, k, other, shift)
        assert call(bits, a, entry(20, param=(1, 0))) == OVERLAP and call(bits, a, entry(20, grad=(1, 0))) == OVERLAP
        assert call(bits, entry(20, param=(2, 0)), a) == OVERLAP          # another entry's gradient
        assert call(bits, a, entry(20, exp_avg=(4, 4 * ((1000 * size - 1) // 4)))) == OVERLAP
        assert call(bits, entry(20), a, entry(40, master=(23, 0))) == OVERLAP
    assert call(8, entry(1, sq_scale=(6, 0))) == OVERLAP and call(8, a, entry(20, avg_scale=(6, 12))) == OVERLAP
    assert call(8, entry(1, master=none, avg_scale=(4, 996))) == OVERLAP
