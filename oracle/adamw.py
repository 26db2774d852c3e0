"""AdamW for one tensor, its moments held in 8 bits, and clipping by the global
norm, in float64.

The step ("LLM Optimizers: From SGD and AdamW to SOAP, Muon, and Scalable
Training", sections 5 and 6), at step t >= 1:

    M = b1 M + (1 - b1) G ;  V = b2 V + (1 - b2) G * G
    W = (1 - lr wd) W - lr (M / (1 - b1^t)) / (sqrt(V / (1 - b2^t)) + eps)

The moments in 8 bits share one power-of-two scale in each block of 256
elements, taken from the exponent E of the block's largest finite magnitude
(biased, as an fp32 value has it):

    m: 4 exponent bits (bias 7), 3 mantissa bits and a sign, scale 2^(s - 127)
       with s = max(1, E - 7); the pattern 127 (or 255) is a NaN
    v: 5 exponent bits (bias 15), 3 mantissa bits, no sign, s = max(1, E - 15);
       255 stands for a value that is not finite; v > 0 has a code of at least 1

m and v go to the nearest code (ties to even) or, with noise bits u in 0..65535,
to the code above (in magnitude) where the distance from the code below, in
steps, plus (16 u + 8) / 2^20 reaches one.  The moments that a step rounds are
fp32 values, each product and sum of the recurrence rounded once
(``fp32_moments``): with few-bit codes and 16-bit gradients the exact sum is
often a tie of two codes, which only a stated order of roundings decides.

Clipping ("LLM Optimizers", section 7.4): factor = s min(1, c / (s ||G|| + 1e-6))
over all tensors of the list.
"""

import numpy as np

BLOCK = 256
M32, M64 = (1 << 32) - 1, (1 << 64) - 1


def adamw_step(W, G, M, V, *, t, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0,
               bias_correction=True):
    """(W, M, V) after one step; inputs are not modified."""
    W, G, M, V = (np.asarray(x, dtype=np.float64) for x in (W, G, M, V))
    M = beta1 * M + (1 - beta1) * G
    V = beta2 * V + (1 - beta2) * G * G
    c1, c2 = (1 - beta1 ** t, 1 - beta2 ** t) if bias_correction else (1.0, 1.0)
    D = (M / c1) / (np.sqrt(V / c2) + eps)
    return (1 - lr * weight_decay) * W - lr * D, M, V


def fp32_moments(G, M, V, beta1=0.9, beta2=0.999):
    """The new moments in the fixed order of fp32 roundings (float32 arrays)."""
    f = np.float32
    G, M, V = (np.asarray(x, dtype=f) for x in (G, M, V))
    with np.errstate(all="ignore"):
        m = f(beta1) * M + f(1 - beta1) * G
        v = f(beta2) * V + f(1 - beta2) * (G * G)
    return m, v


# ---------------------------------------------------------------- noise bits


def _words(elements, seed, step, index):
    z = (seed + step * 0x9E3779B97F4A7C15 + index * 0xBB67AE8584CAA73B) & M64
    for _ in range(2):
        z = ((z ^ (z >> 32)) * 0x6A09E667F3BCC909) & M64
    z ^= z >> 32
    k1, k2 = np.uint64(z & M32), np.uint64(z >> 32)
    low, a, b = np.uint64(M32), np.uint64(0x9E3779B9), np.uint64(0x6A09E667)
    pair = np.asarray(elements, dtype=np.uint64) >> np.uint64(1)
    x = ((pair & low) ^ k1) * a & low
    x ^= x >> np.uint64(16)
    x = (x * b + k2 + (pair >> np.uint64(32))) & low
    x ^= x >> np.uint64(15)
    x = x * a & low
    x ^= x >> np.uint64(16)
    y = ((x ^ k1) * b + k2) & low
    y ^= y >> np.uint64(16)
    z = ((x ^ k2) * a + k1) & low
    z ^= z >> np.uint64(16)
    return x, y, z


def _halves(words, elements):
    half = (np.asarray(elements, dtype=np.uint64) & np.uint64(1)) * np.uint64(16)
    return tuple(((w >> half) & np.uint64(0xFFFF)).astype(np.int64) for w in words)


def noise(elements, *, seed, step, index):
    """16 bits for each element's second moment and 16 for its bf16 weight."""
    return _halves(_words(elements, seed, step, index)[:2], elements)


def first_noise(elements, *, seed, step, index):
    """16 bits for each element's first moment."""
    return _halves(_words(elements, seed, step, index)[2:], elements)[0]


# ---------------------------------------------------------------- 8-bit codes


def first_values():
    """The value of each of the 256 codes of m, before the scale."""
    c = np.arange(256)
    e, f = (c >> 3) & 15, c & 7
    v = np.where(e > 0, (8 + f) * 2.0 ** (e - 10.0), f * 2.0 ** -9)
    v = np.where(c & 128, -v, v)
    v[[127, 255]] = np.nan
    return v


def second_values():
    """The value of each of the 256 codes of v, before the scale."""
    c = np.arange(256)
    e, f = c >> 3, c & 7
    v = np.where(e > 0, (8 + f) * 2.0 ** (e - 18.0), f * 2.0 ** -17)
    v[255] = np.nan
    return v


def scale_bytes(x, drop):
    """The scale byte of each block of 256 elements of the flat array x."""
    x = np.abs(np.asarray(x, dtype=np.float64).reshape(-1))
    x = np.where(np.isfinite(x), x, 0.0)
    full = np.zeros(-(-x.size // BLOCK) * BLOCK)
    full[:x.size] = x
    big = full.reshape(-1, BLOCK).max(1)
    E = np.where(big >= 2.0 ** -126, np.frexp(big)[1] - 1 + 127, 0)
    return np.maximum(1, E - drop).astype(np.uint8)


def per_element(scales, n):
    return np.ldexp(1.0, np.repeat(scales.astype(np.int64), BLOCK)[:n] - 127)


def _steps(x, bias):
    """|x| in units of its own code step, and the codes at whole numbers of steps."""
    e = np.where(x > 0, np.maximum(np.frexp(x)[1] - 1, 1 - bias), 1 - bias)
    return x / np.ldexp(1.0, e - 3), (e + bias - 1) * 8


def first_codes(m, bits=None):
    """(codes, scales) of the first moment; bits: noise for stochastic rounding."""
    m = np.asarray(m, dtype=np.float64).reshape(-1)
    s = scale_bytes(m, 7)
    y = m / per_element(s, m.size)
    ok = np.isfinite(y)
    n, base = _steps(np.abs(np.where(ok, y, 0.0)), 7)
    n = np.rint(n) if bits is None else np.floor(n + (16 * bits + 8) / 2.0 ** 20)
    c = n.astype(np.int64) + base + 128 * np.signbit(y)
    return np.where(ok, c, 127).astype(np.uint8), s


def second_codes(v, bits=None):
    """(codes, scales) of the second moment; bits: noise for stochastic rounding."""
    v = np.asarray(v, dtype=np.float64).reshape(-1)
    s = scale_bytes(v, 15)
    ok = np.isfinite(v)
    n, base = _steps(np.where(ok, np.maximum(v, 0.0), 0.0) / per_element(s, v.size), 15)
    n = np.rint(n) if bits is None else np.floor(n + (16 * bits + 8) / 2.0 ** 20)
    c = np.where(v > 0, np.maximum(1, n.astype(np.int64) + base), 0)
    return np.where(ok, c, 255).astype(np.uint8), s


def first_moment(codes, scales):
    return first_values()[codes] * per_element(scales, codes.size)


def second_moment(codes, scales):
    return second_values()[codes] * per_element(scales, codes.size)


def adamw8_step(W, G, state, *, t, noise_seed=None, index=0, beta1=0.9, beta2=0.999, **hyper):
    """(W, state) after one step with the moments held as codes, state = (M8, MS, V8, VS); with a noise_seed both are
    rounded stochastically.  W is formed from the new moments before they are rounded to codes."""
    m8, ms, v8, vs = state
    M, V = first_moment(m8, ms), second_moment(v8, vs)
    W = adamw_step(W, G, M, V, t=t, beta1=beta1, beta2=beta2, **hyper)[0]
    m, v = fp32_moments(G, M, V, beta1, beta2)
    mbits = vbits = None
    if noise_seed is not None:
        at = np.arange(m8.size)
        mbits = first_noise(at, seed=noise_seed, step=t, index=index)
        vbits = noise(at, seed=noise_seed, step=t, index=index)[0]
    return W, (*first_codes(m, mbits), *second_codes(v, vbits))


# ---------------------------------------------------------------- clipping


def clip(grads, max_norm, scale=1.0):
    """(norm, factor) of a list of gradients."""
    norm = abs(scale) * np.sqrt(sum(float(np.sum(np.asarray(g, dtype=np.float64) ** 2)) for g in grads))
    f = max_norm / (norm + 1e-6)
    return norm, scale * (1.0 if f >= 1 else f)
