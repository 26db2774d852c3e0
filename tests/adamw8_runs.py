"""Long runs of the AdamW step with 8-bit moments, against the fp64 step: the
gradients and what has to hold, for the oracle's codes (CPU) and the kernels'.

`step(G, t)` advances the run by one step; `read()` gives its weights and held
moments (W, M, V) in fp64.  Weights start at 0, without decay, so that they are
the sum of all updates.  Gradients are of order 1 and eps (1e-8) is nothing
beside them.  What each bound rests on:

steady gradient    Rounding to a code is unbiased (to 2^-17 of a step of 1/8, a
    bias below 1e-3 with b1 <= 0.95), and the recurrence of M is linear: its mean is the
    exact M.  A rounding's variance is at most a quarter of a squared step of
    m'/8, so the relative variance s of M satisfies
    s (1 - b1^2 257/256) <= 1/256; the mean of n elements is within 5 standard errors.
    Of V: a rounding's variance is at most the distance moved times a step.  While
    it builds up it moves by 1/t of itself and gains at most 1/(8 t) of relative
    variance a step, which the 2/t that it forgets holds below 1/16, and less
    later.  An update goes with V^-1/2, whose mean is 1 + 3/8 of that variance: 2.5 %
    too much at most, 5 % allowed.  One element: a quarter's standard deviation
    of V (an eighth of the update) over a third of the run, 6 of them and M's
    own (0.2, but independent every 20 steps): 30 %.
no more gradient   The rest of the way is a sum of b1^k m0 V_k^-1/2.  M stays
    unbiased and never grows.  V gains (1 - b2)/8 of relative variance a step: with
    b2 = 0.999 nothing before M is gone, with b1 = b2 = 0.95 the sum grows from
    1/(1 - 0.9747) to at most 1/(1 - 0.9747 (1 + 3/8 0.05/8)) = 1.10 of itself, plus
    the sums' own scatter (0.4 of one element over the square root of 512 at least: 9 % for 5 of
    them): 0.8 to 1.3.  One element goes 5 times its way only where M goes down
    fewer than 8 of its codes in 100 steps, each with a probability of 0.4 or more:
    1e-13.
"""
import math

import numpy as np

from oracle import adamw as oa

LR, EPS = 1e-3, 1e-8
BUILD_UP = 50                      # steps with random gradients before they end
BETAS = [(0.9, 0.999), (0.95, 0.999), (0.95, 0.95), (0.9, 0.95)]


def exact(W, M, V, first, steps, b1, b2, G=None):
    """fp64 AdamW over steps first + 1 .. first + steps with a constant gradient (none: 0)."""
    G = 0 * W if G is None else G
    for t in range(first + 1, first + steps + 1):
        W, M, V = oa.adamw_step(W, G, M, V, t=t, lr=LR, beta1=b1, beta2=b2, eps=EPS)
    return W


def steady(step, read, n, steps, b1, b2):
    rng = np.random.default_rng(41)
    g = np.float64(np.float32(rng.uniform(0.5, 2, n) * rng.choice([-1, 1], n)))
    for t in range(1, steps + 1):
        step(g, t)
    W, M, _ = read()
    var = (1 / 256) / (1 - b1 * b1 * 257 / 256)
    mean = float(np.mean(M / g))
    assert abs(mean - 1) <= 5 * math.sqrt(var / n) + 1e-3, mean
    way = W / exact(0 * g, 0 * g, 0 * g, 0, steps, b1, b2, g)
    assert abs(float(np.mean(way)) - 1) <= 0.05, np.mean(way)
    assert np.all(np.abs(way - 1) <= 0.3), (way.min(), way.max())


def gradient_ends(step, read, n, steps, b1, b2, live):
    """live: share of each block's elements that go on (at its start)."""
    rng = np.random.default_rng(43)
    dead = np.arange(n) % 256 >= live * 256
    for t in range(1, BUILD_UP + 1):
        step(np.float64(np.float32(rng.standard_normal(n))), t)
    W0, M0, V0 = read()
    for t in range(BUILD_UP + 1, BUILD_UP + steps + 1):
        step(np.where(dead, 0.0, np.float64(np.float32(rng.standard_normal(n)))) if live else np.zeros(n), t)
    W, M, _ = read()
    left = exact(W0, M0, V0, BUILD_UP, steps, b1, b2) - W0
    way = (W - W0)[dead]
    left = left[dead]
    assert np.all(np.isfinite(W))
    ratio = float(np.sum(way * np.sign(left)) / np.sum(np.abs(left)))
    assert 0.8 <= ratio <= 1.3, ratio
    assert np.abs(way).max() <= 5 * np.abs(left).max(), (np.abs(way).max(), np.abs(left).max())
    if live:
        assert np.all(M[dead] == 0)
