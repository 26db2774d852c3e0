"""Some thousand steps of the oracle's 8-bit moments with noise against fp64
AdamW, and the noise bits and codes of the first moment."""
import adamw8_runs as runs
import numpy as np
import pytest

from oracle import adamw as oa

N, STEPS = 1024, 2000


def _run(b1, b2, seed=3):
    s = dict(W=np.zeros(N), st=(*oa.first_codes(np.zeros(N)), *oa.second_codes(np.zeros(N))))

    def step(G, t):
        s["W"], s["st"] = oa.adamw8_step(s["W"], G, s["st"], t=t, noise_seed=seed, lr=runs.LR, beta1=b1, beta2=b2, eps=runs.EPS)

    def read():
        m8, ms, v8, vs = s["st"]
        return s["W"], oa.first_moment(m8, ms), oa.second_moment(v8, vs)
    return step, read


@pytest.mark.parametrize("b1,b2", runs.BETAS)
def test_steady_gradient(b1, b2):
    runs.steady(*_run(b1, b2), N, STEPS, b1, b2)


@pytest.mark.parametrize("live", [0, 0.5])
@pytest.mark.parametrize("b1,b2", runs.BETAS)
def test_gradient_ends(b1, b2, live):
    runs.gradient_ends(*_run(b1, b2), N, STEPS, b1, b2, live)


def test_nearest_first_codes_stick():
    # why the first moment needs noise: without gradient 0.95 x 9 and 0.95 x 10 go back to where they were
    m = np.full(256, 9.0)
    m[1:] = 10.0
    c, s = oa.first_codes(m)
    again, s2 = oa.first_codes(np.float32(0.95) * np.float32(oa.first_moment(c, s)))
    np.testing.assert_array_equal(again, c)
    assert s[0] == s2[0]


def test_first_noise_bits():
    n = 1 << 18
    m = oa.first_noise(np.arange(n), seed=7, step=3, index=2)
    v, w = oa.noise(np.arange(n), seed=7, step=3, index=2)
    others = [v, w, oa.first_noise(np.arange(n), seed=7, step=4, index=2), oa.first_noise(np.arange(n), seed=7, step=3, index=3)]
    # as for the other words: mean, variance and correlations within 5 standard errors
    for x in (m, m[::2], m[1::2]):
        assert abs(x.mean() - 32767.5) < 5 * 65536 / np.sqrt(12 * x.size)
        assert abs(x.var() / (65536 ** 2 / 12) - 1) < 5 * np.sqrt(0.8 / x.size)
    for x, y in [(m, o) for o in others] + [(m[:-1], m[1:]), (m[:-2], m[2:]), (m[::2], m[1::2]), (m[:-256], m[256:])]:
        assert abs(np.corrcoef(x, y)[0, 1]) < 5 / np.sqrt(min(x.size, y.size))


@pytest.mark.parametrize("base", [2.0, 2.0 ** -9])
def test_stochastic_first_codes_are_unbiased(base):
    # m stands at a share p above a code (a normal one, or 5 of the steps below the normal ones)
    n = 1 << 16
    bits = oa.first_noise(np.arange(n), seed=1, step=1, index=0)
    for p in (0.01, 0.3, 0.75):
        for sign in (1, -1):
            m = np.full(n, sign * ((8 if base > 1 else 5) + p) * base)
            m[::256] = 2.0 ** 7                           # fixes the scale at 1
            c, s = oa.first_codes(m, bits)
            keep = np.arange(n) % 256 != 0
            assert np.all(s == 127)
            up = np.mean(np.abs(oa.first_moment(c, s)[keep]) / base - (8 if base > 1 else 5))
            assert abs(up - p) < 5 * np.sqrt(p * (1 - p) / keep.sum())
            assert np.all(np.signbit(oa.first_moment(c, s)[keep]) == (sign < 0))


def test_stochastic_first_codes_of_special_values():
    x = np.zeros(300, dtype=np.float32)
    x[:5] = [np.nan, np.inf, -np.inf, 3.0, -0.0]
    bits = np.full(300, 65535)
    codes, s = oa.first_codes(x, bits)
    assert list(codes[:3]) == [127] * 3 and codes[4] == 128 and codes[5] == 0 and s[0] == 128 - 7 and s[1] == 1
    # a value whose code the noise carries over the top of its binade
    x[:] = 0
    x[0] = np.float32(255.9)
    codes, s = oa.first_codes(x, bits)
    assert oa.first_moment(codes, s)[0] == 256.0
