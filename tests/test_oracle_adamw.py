"""Pins of the AdamW oracle: hand-worked steps, the identity-basis SOAP step,
the 8-bit formats against torch's types and a search over all codes, and the
quality of the noise bits."""
import numpy as np
import torch

from oracle import adamw as oa
from oracle import soap as osoap


def test_first_step_by_hand():
    # t = 1: the corrected moments are g and g^2, so each weight moves by lr against the gradient's sign
    W, G = np.array([1.0, -2.0, 0.5]), np.array([0.3, -4.0, 0.0])
    w, m, v = oa.adamw_step(W, G, 0 * W, 0 * W, t=1, lr=0.1, eps=0.0 + 1e-30, weight_decay=0.5)
    np.testing.assert_allclose(w, [0.95 * 1 - 0.1, 0.95 * -2 + 0.1, 0.95 * 0.5], rtol=1e-12)
    np.testing.assert_allclose(m, 0.1 * G, rtol=1e-12)
    np.testing.assert_allclose(v, 0.001 * G * G, rtol=1e-12)


def test_second_step_by_hand():
    # b1 = b2 = 1/2, gradients 2 then 0: m = 1/2, v = 1, corrections 3/4; step = lr (2/3) / sqrt(4/3)
    w, m, v = oa.adamw_step([0.0], [2.0], [0.0], [0.0], t=1, lr=1.0, beta1=0.5, beta2=0.5, eps=0.0)
    w, m, v = oa.adamw_step(w, [0.0], m, v, t=2, lr=1.0, beta1=0.5, beta2=0.5, eps=0.0)
    np.testing.assert_allclose((m[0], v[0]), (0.5, 1.0), rtol=1e-15)
    np.testing.assert_allclose(w[0], -1.0 - (2 / 3) / np.sqrt(4 / 3), rtol=1e-14)


def test_is_soap_with_identity_bases():
    rng = np.random.default_rng(3)
    W, G, M = (rng.standard_normal((6, 5)) for _ in range(3))
    V = rng.random((6, 5))
    ref = osoap.soap_step(W, G, M, V, t=4, lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
    w, m, v = oa.adamw_step(W, G, M, V, t=4, lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
    for a, b in ((w, ref["W"]), (m, ref["M"]), (v, ref["V"])):
        np.testing.assert_allclose(a, b, rtol=1e-12)


def test_first_values_are_e4m3():
    ref = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(oa.first_values(), ref)


def test_second_values_are_the_top_of_fp16():
    # 5 exponent and 3 mantissa bits are an fp16's upper bits without its sign; its exponent 31 goes on here
    bits = (np.arange(248) << 7).astype(np.uint16).view(np.float16).astype(np.float64)
    np.testing.assert_array_equal(oa.second_values()[:248], bits)
    assert oa.second_values()[248] == 2.0 ** 16


def _nearest(x, values):
    """Code of the nearest value by search, ties to the even code."""
    out = []
    for a in x:
        d = np.abs(values - a)
        best = np.flatnonzero(d == np.nanmin(d))
        out.append(int(best[best % 2 == 0][0] if best.size > 1 else best[0]))
    return np.array(out)


def test_codes_by_search():
    rng = np.random.default_rng(5)
    x = np.float32(np.exp(rng.uniform(-20, 0, 256)) * rng.choice([-1, 1], 256))
    x[:4] = [1.0, 0.28125, -0.265625, 2.0 ** -18]        # the largest, two ties, the last step above zero
    codes, s = oa.first_codes(x)
    assert s[0] == 127 - 7
    pos = oa.first_values()[:127]
    want = _nearest(np.abs(np.float64(x)) * 2.0 ** 7, pos) + 128 * (x < 0)
    np.testing.assert_array_equal(codes, want)
    v = np.abs(x) ** 2
    codes, s = oa.second_codes(v)
    assert s[0] == 127 - 15
    want = np.maximum(1, _nearest(np.float64(v) * 2.0 ** 15, oa.second_values()[:249]))
    np.testing.assert_array_equal(codes, want)


def test_codes_of_special_values():
    x = np.zeros(300, dtype=np.float32)
    x[:5] = [np.nan, np.inf, -np.inf, 3.0, -0.0]
    codes, s = oa.first_codes(x)
    assert list(codes[:3]) == [127] * 3 and codes[4] == 128 and s[0] == 128 - 7 and s[1] == 1
    codes, s = oa.second_codes(x)
    assert list(codes[:3]) == [255] * 3 and codes[4] == 0 and s[0] == 128 - 15 and s[1] == 1
    x = np.float32([2.0 ** 100, 1e-45])                   # a value far below the range keeps a code above zero
    assert oa.second_codes(x)[0][1] == 1


def test_codes_of_held_values_do_not_change():
    for values, codes in ((oa.first_values(), oa.first_codes), (oa.second_values(), oa.second_codes)):
        # a block whose largest value is that of the scale's top binade holds its own values exactly
        top = 128.0 if np.nanmin(values) < 0 else 2.0 ** 15
        x = np.where(np.abs(values) < 2 * top, values, 0.0)
        x = np.where(np.isnan(x), 0.0, x)
        x[0] = top
        c, s = codes(x)
        back = values[c] * np.ldexp(1.0, int(s[0]) - 127)
        np.testing.assert_array_equal(back, x)


def test_noise_bits():
    n = 1 << 18
    a, b = oa.noise(np.arange(n), seed=7, step=3, index=2)
    c, _ = oa.noise(np.arange(n), seed=7, step=4, index=2)
    d, _ = oa.noise(np.arange(n), seed=7, step=3, index=3)
    # mean and variance of a uniform 16-bit number: 5 standard errors (sigma / sqrt(n), sigma = 2^16 / sqrt(12))
    for x in (a, b, c, d, a[::2], a[1::2]):
        assert abs(x.mean() - 32767.5) < 5 * 65536 / np.sqrt(12 * x.size)
        assert abs(x.var() / (65536 ** 2 / 12) - 1) < 5 * np.sqrt(0.8 / x.size)
    # independent streams correlate by 1 / sqrt(n) at most (5 standard errors)
    for x, y in ((a, b), (a, c), (a, d), (a[:-1], a[1:]), (a[:-2], a[2:]), (a[::2], a[1::2]), (a[:-256], a[256:])):
        assert abs(np.corrcoef(x, y)[0, 1]) < 5 / np.sqrt(min(x.size, y.size))


def test_stochastic_codes_are_unbiased():
    # v stands at a share p above a code: it goes up in a share p of many draws (5 standard errors)
    n = 1 << 16
    bits, _ = oa.noise(np.arange(n), seed=1, step=1, index=0)
    for p in (0.01, 0.3, 0.75):
        v = np.full(n, (8 + p) * 2.0 ** 12)
        v[::256] = 2.0 ** 15                              # fixes the scale
        c, _ = oa.second_codes(v, bits)
        keep = np.arange(n) % 256 != 0
        base = c[keep].min()
        up = np.mean(c[keep] - base)
        assert abs(up - p) < 5 * np.sqrt(p * (1 - p) / keep.sum())


def test_clip_by_hand():
    norm, f = oa.clip([np.array([3.0]), np.array([[4.0]])], 1.0)
    assert norm == 5.0 and abs(f - 1 / 5.000001) < 1e-15
    assert oa.clip([np.array([3.0, 4.0])], 10.0) == (5.0, 1.0)
    norm, f = oa.clip([np.array([3.0, 4.0])], 1.0, scale=0.5)
    assert norm == 2.5 and abs(f - 0.5 / 2.500001) < 1e-15
