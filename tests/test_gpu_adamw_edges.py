"""AdamW, 8-bit moments and clipping at the ends of what the formats and the
calls hold, against the fp64 oracle."""
import numpy as np
import pytest
from test_gpu_adamw import U, Flat, _dt, _np

from gpu_env import context
from oracle import adamw as oa

pytestmark = pytest.mark.gpu


def test_factor_is_rounded_once():
    """Norms that are whole numbers of 5 are exact; the factor is the fp32 value nearest to 1 / (norm + 1e-6)."""
    import torch
    ctx = context()
    got = []
    for c in range(1, 101):
        norm, factor = ctx.clip_grads([torch.tensor([3.0 * c, 4.0 * c], device="cuda")], 1.0, apply=False)
        assert float(norm) == 5.0 * c
        got.append(float(factor))
    want = np.float32(1.0 / (5.0 * np.arange(1, 101) + 1e-6))
    np.testing.assert_array_equal(np.float32(got), want)
# ---------------------------------------------------------------- the norm over fp32's range


def _norm_case(arrays, dtype, shift, scale=None):
    """Squares are taken in fp32 and eight of them added (8 u of the sum: 4 u of the norm), or in fp64 where they would
    leave fp32's range; the norm is rounded once more.  The factor is formed in fp64 and rounded once."""
    import torch
    ctx = context()
    G = Flat(arrays, _dt(dtype), shift)
    g0 = [_np(v) for v in G.views]
    s = None if scale is None else torch.tensor(scale, device="cuda")
    flag = torch.full((1,), 5, dtype=torch.int32, device="cuda")
    norm, factor = ctx.clip_grads(list(G.views), 1.0, apply=False, scale=s, nonfinite=flag)
    want, f = oa.clip(g0, 1.0, 1.0 if scale is None else float(np.float32(scale)))
    if want > np.finfo(np.float32).max:               # of 1e37: finite gradients whose norm fp32 does not hold
        assert int(flag) == 1 and np.isposinf(float(norm)) and float(factor) == 0
        return
    assert int(flag) == 0
    assert abs(float(norm) - want) <= 6 * U * want + 2.0 ** -150, (float(norm), want)
    assert abs(float(factor) - f) <= 6 * U * f, (float(factor), f)


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", [8e18, 1e19, 1e30, 1e37, 1e-19, 1e-22, 1e-30, 1e-38])
def test_norm_of_large_and_small_gradients(dtype, shift, size):
    rng = np.random.default_rng(1)
    _norm_case([size * rng.uniform(0.5, 1, n) for n in (8, 5000, 256, 3)], dtype, shift)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_norm_of_blocks_of_every_size(dtype):
    rng = np.random.default_rng(2)
    x = rng.standard_normal(256 * 40) * np.repeat(10.0 ** rng.uniform(-44, 19, 256 * 5), 8)
    _norm_case([x, x[:700] * 1e17], dtype, 0)
    _norm_case([x[:3001] * 1e-18, np.full(9, 1e-42), np.zeros(300)], dtype, 1)


def test_norm_with_a_scale_that_brings_it_back():
    """The scale is applied to the norm in fp64: gradients that were scaled up for fp16 may be large."""
    rng = np.random.default_rng(3)
    _norm_case([1e25 * rng.standard_normal(4000)], "f32", 0, 2.0 ** -80)
    _norm_case([1e-30 * rng.standard_normal(4000)], "f32", 0, 2.0 ** 90)


# ---------------------------------------------------------------- denominators at the ends of fp32


@pytest.mark.parametrize("device", [False, True])
@pytest.mark.parametrize("b2,eps,size", [(1 - 1e-7, 1e-10, 2e-16), (1 - 1e-10, 1e-9, 6e-15), (0.999, 1e-10, 2e-18), (0.999, 1.5e38, 1e18),
                                         (0.999, 2.0 ** 101, 1e18)])
def test_small_second_moments_and_large_eps(b2, eps, size, device):
    """The first step from zero moments: V = (1 - b2) g^2 around fp32's smallest normal number, divided by 1 - b2 again, beside
    eps; and a denominator whose reciprocal is below it.  The bounds of the steps of test_gpu_adamw.py."""
    import torch
    ctx = context()
    n = 2000
    rng = np.random.default_rng(4)
    g = np.float64(np.float32(size * np.exp(rng.uniform(-1, 1, n)) * rng.choice([-1, 1], n)))
    W, M, V = (torch.zeros(n, device="cuda") for _ in range(3))
    step, lr = 1, 1.0
    if device:
        step, lr = torch.tensor([1], device="cuda"), torch.tensor(1.0, device="cuda")
    ctx.adamw_step([dict(W=W, G=torch.from_numpy(g).float().cuda(), M=M, V=V)], step, lr=lr, beta2=b2, eps=eps)
    # V as fp32 holds it: below 2^-126 its own rounding is larger than u
    v = np.float64(np.float32(1 - b2) * np.float32(np.float32(g) * np.float32(g)))
    m = np.float64(np.float32(0.1) * np.float32(g))
    D = (m / 0.1) / (np.sqrt(v / (1 - b2)) + eps)
    got = _np(W)
    assert np.all(np.abs(got + D) <= U * 24 * np.abs(D) + 1e-45), np.max(np.abs(got + D) / np.abs(D)) / U


# ---------------------------------------------------------------- codes below the normal ones


def _low_codes(values, top):
    """A block whose scale is 1 (its largest value is `top`) and which holds `values`."""
    x = np.zeros(256, dtype=np.float32)
    x[0] = top
    x[1:1 + len(values)] = values
    assert np.all(np.float64(x[1:1 + len(values)]) == values)
    return x


def test_second_codes_next_to_ties():
    """V at one fp32 step from the middle between two codes: the nearest code is that of the value, not of the value
    rounded to the bits that an fp32 number of its size would have below 2^-126."""
    import torch
    ctx = context()
    near = [(c + 0.5) * (1 + s * 2.0 ** -23) * 2.0 ** -17 for c in range(1, 8) for s in (-1, 0, 1)]
    near = [float(np.float32(x)) for x in near] + [float(np.nextafter(np.float32((c + 0.5) * 2.0 ** -17), np.float32(s)))
                                                   for c in range(1, 8) for s in (0, 1)]
    for top in (2.0 ** 15, 2.0 ** 15 * 2.0 ** 100, 2.0 ** 15 * 2.0 ** -60):
        x = _low_codes(np.array(near) * (top / 2.0 ** 15), top)
        M, V = torch.zeros(256, device="cuda"), torch.from_numpy(x).cuda()
        d = ctx.adamw8_state(M)
        ctx.adamw8_pack([dict(M=M, V=V, **d)])
        np.testing.assert_array_equal(d["V8"].cpu().numpy(), oa.second_codes(x)[0])


def test_noise_next_to_a_code():
    """Values that the noise brings to less than one fp32 step below a code, and just to it."""
    import torch
    ctx = context()
    for kw, kind in ((dict(seed=3), "second"), (dict(noise=3), "second"), (dict(noise=3), "first")):
        at = np.arange(256)
        first = kind == "first"
        bits = oa.first_noise(at, seed=3, step=5, index=0) if first else oa.noise(at, seed=3, step=5, index=0)[0]
        # c + 1 - (16 bits + 8) / 2^20 is a code's border; a quarter of 2^-20 below it, at it, and above it
        border = (at % 6 + 2) - (16.0 * bits + 8) / 2 ** 20
        y = border + np.array([-0.5, 0.0, 0.5])[at % 3] / 2 ** 20
        unit, top = (2.0 ** -9, 2.0 ** 7) if first else (2.0 ** -17, 2.0 ** 15)
        x = np.float32(y * unit)
        x[0] = top
        X, Z = torch.from_numpy(x).cuda(), torch.zeros(256, device="cuda")
        d = ctx.adamw8_state(Z)
        ctx.adamw8_pack([dict(M=X if first else Z, V=Z if first else X, **d)], step=5, **kw)
        want = oa.first_codes(x, bits)[0] if first else oa.second_codes(x, bits)[0]
        np.testing.assert_array_equal(d["M8" if first else "V8"].cpu().numpy(), want)


def test_small_betas_keep_the_order_of_roundings():
    """rn(b M) with a beta that times the scale of M is below fp32's normal numbers: 8 eighths times b stand 2^-20 above the
    middle between two codes."""
    import torch
    ctx = context()
    b = 2.0 ** -41 * (17 / 16 + 2.0 ** -23)
    n = 512
    W, G = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    st = ctx.adamw8_state(W)
    st["M8"].copy_(torch.arange(n) % 8 + 8 * (torch.arange(n) // 8 % 15))
    st["V8"].copy_(torch.arange(n) % 248)
    st["MS"].fill_(40)
    st["VS"].fill_(41)
    c = {k: v.cpu().numpy() for k, v in st.items()}
    m0, v0 = oa.first_moment(c["M8"], c["MS"]), oa.second_moment(c["V8"], c["VS"])
    ctx.adamw8_step([dict(W=W, G=G, **st)], 1, beta1=b, beta2=b, noise=None)
    m, v = oa.fp32_moments(0 * m0, m0, v0, b, b)
    for key, (codes, scales) in (("M", oa.first_codes(m)), ("V", oa.second_codes(v))):
        np.testing.assert_array_equal(st[key + "S"].cpu().numpy(), scales)
        np.testing.assert_array_equal(st[key + "8"].cpu().numpy(), codes)


# ---------------------------------------------------------------- streams


def test_workspace_of_a_first_call_on_another_stream():
    """The workspace that a call on a given stream attaches is not memory that the current stream still writes."""
    import torch
    n = 1 << 20
    want = float(np.sqrt(n))
    G = torch.ones(n, device="cuda")
    s = torch.cuda.Stream()
    for _ in range(3):
        ctx = context()
        torch.cuda.synchronize()
        old = [torch.empty(k, dtype=torch.uint8, device="cuda") for k in (4096, 65536, 256 + 65536, 1 << 20)]
        torch.cuda._sleep(100_000_000)                 # some 50 ms
        for x in old:
            x.fill_(255)
        del old, x
        norm, _ = ctx.clip_grads([G], 1.0, apply=False, stream=s)
        torch.cuda.synchronize()
        assert float(norm) == want and ctx.device_status() == 0
