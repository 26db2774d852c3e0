"""AdamW over many tensors, 8-bit moments and gradient clipping on the GPU
against the fp64 oracle.

Tolerances count roundings (u = 2^-24, half a step of fp32 relative to the value):
  M'  the constant, the product and the sum round each term: 4 u (|b1 M| + |c1 g|)
  V'  the constant, g g, its product and the sum: 5 u V'
  W'  with D = rate (|b1 M| + |c1 g|) / den: rate (2: lr / correction, lr_scale),
      M' (4), rate M' (1), the square root of V' (2.5 + 2), root (1), den (1),
      the division (2), and the same for the decay (3 u |W|) and the sum:
      u (4 |W| + 16 D); bias corrections formed on the device from t log b in
      fp32 add 3 u for rate and 2 u for root: 24 D in all tests
  16-bit outputs: half a step more, 2^-8 (bf16) or 2^-11 (fp16) of the value, and
      fp16's subnormal half step 2^-25; stochastic bf16: the neighbour that the
      oracle's noise chooses, the other one only where the choice is within the
      fp32 tolerance of its border.
8-bit codes are taken of fp32 values with a fixed order of roundings and are equal."""
import math

import numpy as np
import pytest

from gpu_env import context
from oracle import adamw as oa
from oracle import muon as omuon

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
B1, B2, EPS = 0.9, 0.999, 1e-8


def _dt(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


def _np(t):
    return t.detach().double().cpu().numpy().reshape(-1)


class Flat:
    """Tensors as views of one buffer with untouched elements around each."""

    def __init__(self, arrays, dtype, shift):
        import torch
        self.lo, at = [], 0
        for a in arrays:
            at = -(-at // 64) * 64 + 64 + shift
            self.lo.append(at)
            at += a.size
        self.n = at + 64
        host = torch.full((self.n,), 7.0, dtype=torch.float64)
        for lo, a in zip(self.lo, arrays):
            host[lo:lo + a.size] = torch.from_numpy(np.asarray(a, dtype=np.float64).reshape(-1))
        self.buf = host.to(dtype).cuda()
        self.before = self.buf.clone()
        self.views = [self.buf[lo:lo + a.size] for lo, a in zip(self.lo, arrays)]

    def others_untouched(self):
        import torch
        inside = torch.zeros(self.n, dtype=torch.bool, device="cuda")
        for lo, v in zip(self.lo, self.views):
            inside[lo:lo + v.numel()] = True
        a, b = self.buf[~inside], self.before[~inside]
        return bool((a == b).all())


def _inputs(sizes, seed, zero=False):
    rng = np.random.default_rng(seed)
    out = []
    for n in sizes:
        s = 1e-3 * math.exp(rng.standard_normal())
        G = s * rng.standard_normal(n)
        M = 0.23 * s * rng.standard_normal(n)
        V = s * s * (0.25 + rng.random(n))
        if zero:
            M, V = 0 * M, 0 * V
        G[rng.random(n) < 0.05] = 0
        out.append([(0.02 * rng.standard_normal(n)), G, M, V])
    return out


def _check_w(got, w64, W, D, dtype, bits=None):
    """The new weights (as stored) against the fp64 step's."""
    tol = U * (4 * np.abs(W) + 24 * D) + 1e-45
    if dtype == "f32":
        assert np.all(np.abs(got - w64) <= tol), np.max(np.abs(got - w64) / tol)
    elif bits is None:
        half = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}[dtype]
        sub = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25}[dtype]
        assert np.all(np.abs(got - w64) <= tol * 1.01 + np.maximum(half * np.abs(w64), sub))
    else:
        step = np.ldexp(1.0, np.frexp(np.abs(w64))[1] - 8)
        n = np.abs(w64) / step
        up = np.floor(n + bits / 65536) * step * np.sign(w64)
        border = np.abs((n + bits / 65536) - np.rint(n + bits / 65536)) * step
        # the fp32 value's own rounding may cross the border: at most one step off, and only there
        off = np.abs(got - up)
        assert np.all(off[border > 2 * tol] == 0)
        assert np.all(off <= 1.01 * step)


def _adamw_case(sizes, *, w="f32", g="f32", copy=None, shift=0, device=False, seed=None, t=3, lr=1e-2, eps=EPS, bias=True,
                gscale=None, zero=False, ctx=None):
    import torch
    ctx = ctx or context()
    arrays = _inputs(sizes, 100 + len(sizes) + sizes[0], zero)
    W = Flat([a[0] for a in arrays], _dt(w), shift)
    G = Flat([a[1] for a in arrays], _dt(g), shift)
    M = Flat([a[2] for a in arrays], torch.float32, shift)
    V = Flat([a[3] for a in arrays], torch.float32, shift)
    C = Flat([a[0] for a in arrays], _dt(copy), shift) if copy else None
    wds = [0.1 * (i % 3) for i in range(len(sizes))]
    lrs = [1.0 - 0.25 * (i % 2) for i in range(len(sizes))]
    mats = [dict(W=W.views[i], G=G.views[i], M=M.views[i], V=V.views[i], copy=C.views[i] if C else None, lr_scale=lrs[i],
                 weight_decay=wds[i]) for i in range(len(sizes))]
    old = [[_np(x.views[i]) for x in (W, G, M, V)] for i in range(len(sizes))]
    kw = dict(lr=lr, beta1=B1, beta2=B2, eps=eps, bias_correction=bias, seed=seed)
    step = t
    if device:
        step = torch.tensor([t], device="cuda")
        kw["lr"] = torch.tensor(lr, device="cuda", dtype=torch.float32)
    if gscale is not None:
        kw["grad_scale"] = torch.tensor([gscale], device="cuda")
    ctx.adamw_step(mats, step, **kw)
    torch.cuda.synchronize()
    for x in (W, G, M, V, C):
        assert x is None or x.others_untouched()
    for i in range(len(sizes)):
        w0, g0, m0, v0 = old[i]
        g0 = np.float64(np.float32(g0) * np.float32(gscale)) if gscale is not None else g0
        w1, m1, v1 = oa.adamw_step(w0, g0, m0, v0, t=t, lr=lr * lrs[i], beta1=B1, beta2=B2, eps=eps, weight_decay=wds[i],
                                   bias_correction=bias)
        m32, v32 = oa.fp32_moments(g0, m0, v0, B1, B2)
        np.testing.assert_array_equal(_np(M.views[i]), m32)
        np.testing.assert_array_equal(_np(V.views[i]), v32)
        mag = B1 * np.abs(m0) + (1 - B1) * np.abs(g0)
        assert np.all(np.abs(_np(M.views[i]) - m1) <= 4 * U * mag)
        assert np.all(np.abs(_np(V.views[i]) - v1) <= 5 * U * v1)
        c1, c2 = (1 - B1 ** t, 1 - B2 ** t) if bias else (1, 1)
        D = lr * lrs[i] * mag / c1 / (np.sqrt(v1 / c2) + eps)
        bits = None
        if seed is not None and w == "bf16":
            bits = oa.noise(np.arange(sizes[i]), seed=seed, step=t, index=i)[1]
        _check_w(_np(W.views[i]), w1, w0, D, w, bits)
        if C:
            _check_w(_np(C.views[i]), w1, w0, D, copy)


SIZES = [1, 7, 255, 256, 257, 2048, 2049, 30011]


@pytest.mark.parametrize("shift", [0, 1, 4, 8])
@pytest.mark.parametrize("w,g,copy", [("f32", "f32", None), ("f32", "bf16", "bf16"), ("f32", "f16", "f16"), ("bf16", "bf16", None),
                                      ("bf16", "f32", None), ("f32", "bf16", None), ("bf16", "f16", None)])
def test_adamw_types_sizes_alignment(w, g, copy, shift):
    _adamw_case(SIZES, w=w, g=g, copy=copy, shift=shift)


@pytest.mark.parametrize("kw", [dict(device=True), dict(device=True, t=100000), dict(bias=False), dict(bias=False, device=True),
                                dict(t=1, zero=True), dict(t=1, zero=True, device=True), dict(gscale=0.37),
                                dict(w="bf16", seed=5), dict(w="bf16", seed=2 ** 63 + 11, t=70000, shift=1),
                                dict(w="bf16", seed=0, device=True, g="bf16"), dict(t=1 << 40), dict(eps=1e-3), dict(lr=0.0),
                                dict(eps=1e-12), dict(w="bf16", eps=1e-11, seed=3, shift=1), dict(gscale=0.37, shift=3, g="f16")])
def test_adamw_options(kw):
    _adamw_case([5000, 256, 3, 2048], **kw)


def test_adamw_many_tensors():
    """More tensors than one launch holds, most of them tiny."""
    rng = np.random.default_rng(0)
    _adamw_case([int(n) for n in rng.integers(1, 600, 700)], w="bf16", g="bf16", seed=9)


def test_adamw_skipped_tensors_keep_their_noise_place():
    """A tensor without gradient, or without elements, is left alone and takes no other's place in the noise."""
    import torch
    ctx = context()
    rng = np.random.default_rng(1)
    W = [torch.from_numpy(0.02 * rng.standard_normal(n)).cuda().to(torch.bfloat16) for n in (300, 0, 500)]
    G = [torch.from_numpy(rng.standard_normal(n)).cuda().float() for n in (300, 0, 500)]
    M, V = ([torch.zeros(n, device="cuda") for n in (300, 0, 500)] for _ in range(2))
    w0, w2 = _np(W[0]), _np(W[2])
    before = [x.clone() for x in (W[0], M[0], V[0])]
    ctx.adamw_step([dict(W=a, G=g, M=m, V=v) for a, g, m, v in zip(W, [None, G[1], G[2]], M, V)], 1, lr=1e-3, seed=3)
    for a, b in zip(before, (W[0], M[0], V[0])):
        assert torch.equal(a, b)
    w1, m1, v1 = oa.adamw_step(w2, _np(G[2]), 0 * w2, 0 * w2, t=1, lr=1e-3)
    D = 1e-3 * np.ones_like(w2)
    _check_w(_np(W[2]), w1, w2, D, "bf16", oa.noise(np.arange(500), seed=3, step=1, index=2)[1])
    assert w0.size == 300


def test_adamw_nonfinite_gradients_stay_where_they_are():
    import torch
    ctx = context()
    for n, shift in ((600, 0), (601, 1)):
        base = torch.zeros(n + 8, device="cuda")
        W, M, V = (base.clone()[shift:n + shift] for _ in range(3))
        G = torch.ones(n + 8, device="cuda")[shift:n + shift]
        G[5], G[300], G[301] = float("nan"), float("inf"), -float("inf")
        st = ctx.adamw8_state(W)
        W8 = W.clone() if shift == 0 else base.clone()[shift:n + shift]
        ctx.adamw_step([dict(W=W, G=G, M=M, V=V)], 1)
        ctx.adamw8_step([dict(W=W8, G=G, **st)], 1, seed=None)
        bad = torch.zeros(n, dtype=torch.bool, device="cuda")
        bad[[5, 300, 301]] = True
        for x in (W, W8):
            assert bool(torch.isnan(x[bad]).all()) and bool(torch.isfinite(x[~bad]).all())
        assert bool((torch.isnan(M) | torch.isinf(M))[bad].all()) and bool(torch.isfinite(M[~bad]).all())
        m, v = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
        ctx.adamw8_unpack([dict(M=m, V=v, **st)])
        for x in (m, v):
            assert bool(torch.isnan(x[bad]).all()) and bool(torch.isfinite(x[~bad]).all())


# ---------------------------------------------------------------- 8-bit moments


def _state(arrays, shift, seed=None):
    """Codes and scales by the oracle, as tensors `shift` bytes off their alignment."""
    import torch
    out = []
    for i, (_, _, m, v) in enumerate(arrays):
        (m8, ms), (v8, vs) = oa.first_codes(np.float32(m)), oa.second_codes(np.float32(v))
        d = {}
        for k, a in (("M8", m8), ("V8", v8), ("MS", ms), ("VS", vs)):
            full = torch.full((a.size + 64,), 99, dtype=torch.uint8, device="cuda")
            full[shift:shift + a.size] = torch.from_numpy(a).cuda()
            d[k], d["_" + k] = full[shift:shift + a.size], full
        out.append(d)
    return out


def _held(d):
    m8, v8, ms, vs = (d[k].cpu().numpy() for k in ("M8", "V8", "MS", "VS"))
    return oa.first_moment(m8, ms), oa.second_moment(v8, vs)


@pytest.mark.parametrize("shift", [0, 1, 8])
@pytest.mark.parametrize("w,g,copy,seed", [("f32", "f32", None, None), ("f32", "bf16", None, None), ("bf16", "bf16", None, 4),
                                           ("f32", "f16", "f16", 4), ("f32", "bf16", "bf16", 4), ("bf16", "f32", None, None)])
def test_adamw8_steps(w, g, copy, seed, shift):
    """Three steps; every step starts from the state that the one before left."""
    import torch
    ctx = context()
    arrays = _inputs(SIZES, 77)
    rng = np.random.default_rng(8)
    W = Flat([a[0] for a in arrays], _dt(w), shift)
    C = Flat([a[0] for a in arrays], _dt(copy), shift) if copy else None
    st = _state(arrays, shift)
    wds = [0.1 * (i % 2) for i in range(len(SIZES))]
    for t in (5, 6, 7):
        G = Flat([a[1] * rng.uniform(0.2, 3) * rng.choice([-1, 1], a[1].size) for a in arrays], _dt(g), shift)
        old = [(_np(W.views[i]), _np(G.views[i]), *_held(st[i])) for i in range(len(SIZES))]
        step = t if t != 6 else torch.tensor(t, device="cuda")
        ctx.adamw8_step([dict(W=W.views[i], G=G.views[i], copy=C.views[i] if C else None, weight_decay=wds[i],
                              **{k: st[i][k] for k in ("M8", "V8", "MS", "VS")}) for i in range(len(SIZES))],
                        step, lr=1e-2, beta1=B1, beta2=B2, eps=EPS, seed=seed)
        torch.cuda.synchronize()
        for i, n in enumerate(SIZES):
            w0, g0, m0, v0 = old[i]
            m32, v32 = oa.fp32_moments(g0, m0, v0, B1, B2)
            bits = (None, None) if seed is None else oa.noise(np.arange(n), seed=seed, step=t, index=i)
            (m8, ms), (v8, vs) = oa.first_codes(m32), oa.second_codes(v32, bits[0])
            for k, a in (("MS", ms), ("VS", vs), ("M8", m8), ("V8", v8)):
                np.testing.assert_array_equal(st[i][k].cpu().numpy(), a, err_msg=f"{k} of {n} at step {t}")
                full, s = st[i]["_" + k].cpu().numpy(), shift
                assert np.all(full[:s] == 99) and np.all(full[s + a.size:] == 99)
            w1, m1, v1 = oa.adamw_step(w0, g0, m0, v0, t=t, lr=1e-2, beta1=B1, beta2=B2, eps=EPS, weight_decay=wds[i])
            # the held moments are within half a code step of the exact ones (a step for the second with noise), the
            # step being 2^-3 of the binade and its floor 2^-9 or 2^-17 of the scale; 1.001 covers the fp32 values
            hm, hv = _held(st[i])
            sm, sv = oa.per_element(ms, n), oa.per_element(vs, n)
            stepm = np.maximum(np.ldexp(1.0, np.frexp(np.abs(m1) / sm)[1] - 4), 2.0 ** -9) * sm
            stepv = np.maximum(np.ldexp(1.0, np.frexp(v1 / sv)[1] - 4), 2.0 ** -17) * sv
            assert np.all(np.abs(hm - m1) <= 0.5 * 1.001 * stepm)
            assert np.all(np.abs(hv - v1) <= (1.0 if seed is not None else 0.5) * 1.001 * stepv + (v1 < sv * 2.0 ** -17) * stepv)
            mag = B1 * np.abs(m0) + (1 - B1) * np.abs(g0)
            D = 1e-2 * mag / (1 - B1 ** t) / (np.sqrt(v1 / (1 - B2 ** t)) + EPS)
            _check_w(_np(W.views[i]), w1, w0, D, w, bits[1] if w == "bf16" else None)
            if C:
                _check_w(_np(C.views[i]), w1, w0, D, copy)
        assert W.others_untouched() and (C is None or C.others_untouched())


def _extreme_blocks():
    rng = np.random.default_rng(2)
    x = rng.standard_normal(256 * 8).astype(np.float32)
    x[:256] *= 1e-38                                  # around the smallest normal number
    x[256:512] = 0
    x[512:768] *= np.float32(2.0) ** 120
    x[768:1024] *= np.exp(rng.uniform(-40, 0, 256)).astype(np.float32)   # a range that the formats do not hold
    x[1024:1028] = [np.nan, np.inf, -np.inf, 3e38]
    x[1280:1536] = np.float32(1e-45)                  # subnormal
    x[1536] = np.float32(3.4028235e38)
    x[1792:] = np.ldexp(1.0, rng.integers(-9, 8, 256)) * 1.0625  # halfway between two first-moment codes
    return x


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,shift", [(2048, 0), (2047, 0), (2045, 1), (1, 0), (257, 3)])
@pytest.mark.parametrize("seed", [None, 21])
def test_pack_and_unpack(dtype, n, shift, seed):
    import torch
    ctx = context()
    x = torch.from_numpy(_extreme_blocks()[:n]).to(_dt(dtype))
    M = torch.zeros(n + 64, dtype=_dt(dtype), device="cuda")[shift:shift + n]
    V = torch.zeros(n + 64, dtype=_dt(dtype), device="cuda")[shift:shift + n]
    M.copy_(x)
    V.copy_(x.abs() if n != 2045 else x)              # a negative second moment takes code 0
    d = {k: torch.full((s + 32,), 9, dtype=torch.uint8, device="cuda")[shift:shift + s]
         for k, s in (("M8", n), ("V8", n), ("MS", -(-n // 256)), ("VS", -(-n // 256)))}
    ctx.adamw8_pack([dict(M=M, V=V, **d)], seed=seed, step=12)
    bits = None if seed is None else oa.noise(np.arange(n), seed=seed, step=12, index=0)[0]
    (m8, ms), (v8, vs) = oa.first_codes(_np(M)), oa.second_codes(_np(V), bits)
    got = d["M8"].cpu().numpy()
    nan = np.isin(m8, (127, 255))
    assert np.all(np.isin(got[nan], (127, 255)))      # a NaN's sign says nothing
    np.testing.assert_array_equal(got[~nan], m8[~nan])
    for k, a in (("V8", v8), ("MS", ms), ("VS", vs)):
        np.testing.assert_array_equal(d[k].cpu().numpy(), a)
    for out in ("f32", "bf16"):
        a, b = (torch.full((n + 64,), 5.0, dtype=_dt(out), device="cuda")[shift:shift + n] for _ in range(2))
        ctx.adamw8_unpack([dict(M=a, V=b, **d)])
        for y, want in ((a, oa.first_moment(m8, ms)), (b, oa.second_moment(v8, vs))):
            want = torch.from_numpy(want).float().to(_dt(out)).double().numpy().reshape(-1)
            np.testing.assert_array_equal(_np(y), want)


def test_unpack_every_code_and_scale():
    import torch
    ctx = context()
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").repeat(255)
    scales = torch.arange(255, dtype=torch.uint8, device="cuda")        # 255 stands for no number
    m, v = (torch.empty(codes.numel(), device="cuda") for _ in range(2))
    ctx.adamw8_unpack([dict(M=m, V=v, M8=codes, V8=codes.clone(), MS=scales, VS=scales.clone())])
    c, s = codes.cpu().numpy(), scales.cpu().numpy()
    with np.errstate(over="ignore"):
        np.testing.assert_array_equal(m.cpu().numpy(), oa.first_moment(c, s).astype(np.float32))
        np.testing.assert_array_equal(v.cpu().numpy(), oa.second_moment(c, s).astype(np.float32))


def test_adamw8_second_moment_follows_a_small_gradient():
    """V decays by 0.1 % a step: with noise its mean over many elements follows, to the nearest it stays.  Each of
    n = 2^16 elements makes T = 200 independent choices; the mean's standard error stays below the largest code step
    (2^-3 of the value) times sqrt(T / (4 n)) = 0.0035; 5 of these."""
    import torch
    ctx = context()
    n, T = 1 << 16, 200
    v0 = 1.3e-6
    out = {}
    for seed in (None, 3):
        W, G, M = (torch.zeros(n, device="cuda") for _ in range(3))
        V = torch.full((n,), v0, device="cuda")
        st = ctx.adamw8_state(W)
        ctx.adamw8_pack([dict(M=M, V=V, **st)])
        ctx.adamw8_unpack([dict(M=M, V=V, **st)])
        held = float(V[0])
        lst = ctx.adamw8_tensors([dict(W=W, G=G, **st)])
        for t in range(1, T + 1):
            ctx.adamw8_step(lst, t, seed=seed)
        ctx.adamw8_unpack([dict(M=M, V=V, **st)])
        out[seed] = float(V.double().mean()) / held
    assert out[None] == 1.0
    assert abs(out[3] - 0.999 ** T) < 5 * 0.0035


# ---------------------------------------------------------------- clipping


@pytest.mark.parametrize("g,out", [("f32", "f32"), ("bf16", "f32"), ("f16", "f32"), ("bf16", None), ("f32", None), ("f16", "bf16"),
                                   ("f32", "f16")])
@pytest.mark.parametrize("shift,max_norm,scale", [(0, 0.5, None), (1, 0.5, 0.25), (3, 1e9, None), (0, math.inf, 2.0), (8, 0.0, None)])
def test_clip(g, out, shift, max_norm, scale):
    """norm: 8 squares added in fp32 (9 u), the rest in fp64, one rounding: 6 u; factor: two more roundings and the
    sum's, 10 u; out: that and one product, then the type's half step."""
    import torch
    ctx = context()
    arrays = [a[1] for a in _inputs(SIZES, 5)]
    G = Flat(arrays, _dt(g), shift)
    O = Flat([0 * a for a in arrays], _dt(out), shift) if out else None
    g0 = [_np(v) for v in G.views]
    s = None if scale is None else torch.tensor(scale, device="cuda")
    flag = torch.full((1,), 5, dtype=torch.int32, device="cuda")
    lst = ctx.clip_tensors([dict(G=G.views[i], out=O.views[i] if O else None) for i in range(len(SIZES))])
    norm, factor = ctx.clip_grads(lst, max_norm, scale=s, nonfinite=flag)
    want, f = oa.clip(g0, max_norm, 1.0 if scale is None else scale)
    assert abs(float(norm) - want) <= 6 * U * want and int(flag) == 0
    assert abs(float(factor) - f) <= 10 * U * abs(f)
    half, sub = {"f32": (U, 2.0 ** -150), "bf16": (2.0 ** -8, 2.0 ** -134), "f16": (2.0 ** -11, 2.0 ** -25)}[out or g]
    dst = O or G
    for a, v in zip(g0, dst.views):
        assert np.all(np.abs(_np(v) - f * a) <= (12 * U + half * (1 + 1e-6)) * np.abs(f * a) + sub * (1 + 1e-6))
    assert dst.others_untouched()
    if O:
        assert torch.equal(G.buf, G.before)
    again, _ = ctx.clip_grads(lst, max_norm, apply=False, scale=s)
    if O:
        assert float(again) == float(norm)            # the same order of sums, the same bits


def test_clip_factor_one_keeps_the_bits():
    import torch
    ctx = context()
    G = torch.randn(5000, device="cuda").to(torch.bfloat16)
    G[7] = -0.0
    before = G.clone()
    norm, factor = ctx.clip_grads([G], 1e6)
    assert float(factor) == 1.0 and torch.equal(G.view(torch.int16), before.view(torch.int16))


def test_clip_empty_and_nonfinite():
    import torch
    ctx = context()
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    for grads in ([], [None], [torch.zeros(0, device="cuda")], [torch.zeros(9, device="cuda")]):
        norm, factor = ctx.clip_grads(grads, 1.0, nonfinite=flag)
        assert float(norm) == 0.0 and float(factor) == 1.0 and int(flag) == 0
    for bad, f in ((float("nan"), None), (float("inf"), 0.0)):
        G = torch.ones(3000, device="cuda")
        G[2999] = bad
        norm, factor = ctx.clip_grads([G], 1.0, nonfinite=flag, apply=False)
        assert int(flag) == 1 and not math.isfinite(float(norm))
        assert math.isnan(float(factor)) if f is None else float(factor) == f


def test_clip_many_tensors():
    import torch
    ctx = context()
    rng = np.random.default_rng(4)
    sizes = [int(n) for n in rng.integers(1, 5000, 5000)]
    flat = torch.randn(sum(sizes), device="cuda")
    out = torch.zeros_like(flat)
    views = lambda t: list(torch.split(t, sizes))     # noqa: E731
    norm, factor = ctx.clip_grads([dict(G=a, out=b) for a, b in zip(views(flat), views(out))], 3.0)
    want = float(flat.double().norm())
    assert abs(float(norm) - want) <= 6 * U * want
    assert torch.equal(out, flat * factor)


# ---------------------------------------------------------------- as a program uses them


def test_graph_replay_with_new_scalars():
    """Clipping and both steps captured once; step, rate, skip and gradients change between replays."""
    import torch
    ctx = context()
    rng = np.random.default_rng(6)
    sizes = [5000, 257, 40000]

    def make():
        r = np.random.default_rng(6)
        W = [torch.from_numpy(0.02 * r.standard_normal(n)).float().cuda() for n in sizes]
        G = [torch.zeros(n, device="cuda", dtype=torch.bfloat16) for n in sizes]
        M, V = ([torch.zeros(n, device="cuda") for n in sizes] for _ in range(2))
        W8 = [w.to(torch.bfloat16) for w in W]
        st = [ctx.adamw8_state(w) for w in W8]
        return dict(W=W, G=G, M=M, V=V, W8=W8, st=st, step=torch.zeros(1, dtype=torch.int64, device="cuda"),
                    lr=torch.zeros(1, device="cuda"), skip=torch.zeros(1, dtype=torch.int32, device="cuda"))

    def call(s, stream=None):
        norm, factor = ctx.clip_grads(s["G"], 1.0, apply=False, nonfinite=s["skip"], stream=stream)
        ctx.adamw_step([dict(W=w, G=g, M=m, V=v) for w, g, m, v in zip(s["W"], s["G"], s["M"], s["V"])], s["step"], lr=s["lr"],
                       grad_scale=factor, skip=s["skip"], stream=stream)
        ctx.adamw8_step([dict(W=w, G=g, **c) for w, g, c in zip(s["W8"], s["G"], s["st"])], s["step"], lr=s["lr"],
                        grad_scale=factor, skip=s["skip"], seed=2, stream=stream)

    grads = [[torch.from_numpy(rng.standard_normal(n)).cuda().to(torch.bfloat16) for n in sizes] for _ in range(4)]
    grads[2][1][3] = float("inf")                     # this step is skipped
    a, b = make(), make()
    call(a)                                           # sets up the workspace; the step 0 inputs are rewritten
    a = make()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(a)
    for t in range(4):
        for s in (a, b):
            s["step"].fill_(t + 1)
            s["lr"].fill_(1e-2 / (t + 1))
            for x, y in zip(s["G"], grads[t]):
                x.copy_(y)
        before = [x.clone() for x in b["W"] + b["W8"]]
        graph.replay()
        call(b)
        torch.cuda.synchronize()
        for k in ("W", "M", "V", "W8"):
            for x, y in zip(a[k], b[k]):
                assert torch.equal(x, y), (k, t)
        for c, d in zip(a["st"], b["st"]):
            assert all(torch.equal(c[k], d[k]) for k in c)
        same = [torch.equal(x, y) for x, y in zip(before, b["W"] + b["W8"])]
        assert all(same) if t == 2 else not any(same)


def test_another_stream_and_a_list_kept():
    import torch
    ctx = context()
    n = 100000
    W = torch.randn(n, device="cuda")
    M, V = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    G = torch.randn(n, device="cuda")
    lst = ctx.adamw_tensors([dict(W=W, G=G, M=M, V=V)])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    W2, M2, V2 = W.clone(), M.clone(), V.clone()
    torch.cuda.synchronize()
    for t in (1, 2, 3):
        ctx.adamw_step(lst, t, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    for t in (1, 2, 3):
        ctx.adamw_step([dict(W=W2, G=G, M=M2, V=V2)], t)
    for a, b in ((W, W2), (M, M2), (V, V2)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("n", [70001, 256 * 9, 256 * 9 + 7, 256 * 9 + 8, 519, 264])
def test_every_alignment_gives_the_same_bits(n):
    """The same numbers at every offset from an aligned address, and with codes at an odd one, weights included."""
    import torch
    ctx = context()
    x = _inputs([n], 31)[0]
    res = []
    for shift in (*range(10), 100):
        def at(a, dtype, off=shift):
            full = torch.full((n + 64,), 3.0, device="cuda").to(dtype)
            t = full[off % 64:off % 64 + n]
            t.copy_(torch.from_numpy(np.asarray(a)))
            kept.append((full, off % 64))
            return t
        kept = []
        W, G, C = at(x[0], torch.bfloat16), at(x[1], torch.float16, shift + 3 if shift else 0), at(x[0], torch.float16)
        d = _state([x], 1 if shift == 100 else 0)[0]
        d = {k: d[k] for k in ("M8", "V8", "MS", "VS")}
        ctx.adamw8_step([dict(W=W, G=G, **d)], 4, seed=8)
        W32, M, V = at(x[0], torch.float32, 2 * shift), at(x[2], torch.float32), at(x[3], torch.float32)
        ctx.adamw_step([dict(W=W32, G=G, M=M, V=V, copy=C)], 4)
        e = {k: torch.zeros_like(v) for k, v in d.items()}
        if shift == 100:
            e = {k: torch.zeros(v.numel() + 1, dtype=torch.uint8, device="cuda")[1:] for k, v in d.items()}
        ctx.adamw8_pack([dict(M=M, V=V, **e)], seed=3, step=2)
        m, v, o = at(0 * x[0], torch.bfloat16), at(0 * x[0], torch.bfloat16), at(0 * x[0], torch.float32)
        ctx.adamw8_unpack([dict(M=m, V=v, **e)])
        _, factor = ctx.clip_grads([dict(G=G, out=o)], 1e-3)
        assert torch.equal(o, G.float() * factor)
        for full, off in kept:
            rest = torch.cat([full[:off], full[off + n:]])
            assert bool((rest == torch.full_like(rest, 3.0)).all())
        res.append([W, *d.values(), W32, M, V, C, *e.values(), m, v, G])
    for r in res[1:]:
        for a, b in zip(res[0], r):
            assert torch.equal(a, b)


def test_prepared_lists_are_the_calls_with_lists():
    """A list kept over steps gives the bits of a list made for each call, with other rates, steps and gradients."""
    import torch
    ctx = context()
    rng = np.random.default_rng(9)
    sizes = [int(n) for n in rng.integers(1, 3000, 120)]             # more than a launch with few parameters takes
    made = []
    for _ in range(2):
        r = np.random.default_rng(2)
        made.append([dict(W=torch.from_numpy(r.standard_normal(n)).cuda().to(torch.bfloat16), G=torch.zeros(n, device="cuda"),
                          weight_decay=0.1 * (i % 2)) for i, n in enumerate(sizes)])
    for m in made:
        for d in m:
            d.update(ctx.adamw8_state(d["W"]))
    kept = ctx.adamw8_tensors(made[0])
    for t in (1, 2, 3):
        for i, n in enumerate(sizes):
            g = torch.from_numpy(rng.standard_normal(n)).cuda().float()
            made[0][i]["G"].copy_(g)
            made[1][i]["G"].copy_(g)
        ctx.adamw8_step(kept, t, lr=1e-2 / t, seed=t)
        ctx.adamw8_step(made[1], t, lr=1e-2 / t, seed=t)
    for a, b in zip(*made):
        for k in ("W", "M8", "V8", "MS", "VS"):
            assert torch.equal(a[k], b[k])


def test_profile_counts_the_launches():
    import torch
    ctx = context()
    W = [torch.zeros(3000, device="cuda"), torch.zeros(5000, device="cuda", dtype=torch.bfloat16)]
    mats = [dict(W=w, G=torch.ones_like(w), M=torch.zeros(w.numel(), device="cuda"), V=torch.zeros(w.numel(), device="cuda"))
            for w in W]
    full = [dict(M=d["M"], V=d["V"], **ctx.adamw8_state(d["M"])) for d in mats]
    ctx.clip_grads([W[0]], 1.0)
    ctx.profile()
    ctx.adamw_step(mats, 1)                            # two pairs of types: two launches
    ctx.adamw8_pack(full)
    ctx.adamw8_unpack(full)
    ctx.clip_grads([d["G"] for d in mats], 1.0)        # the same: norm, norm, factor, scaling, scaling
    ctx.clip_grads([mats[0]["G"]], 1.0)                # few sums: norm, scaling
    got = ctx.profile_read()
    ctx.profile(False)
    assert got["adamw"][2] == 2 and got["moments"][2] == 2 and got["clip"][2] == 7
    assert all(got[k][0] > 0 for k in ("adamw", "moments", "clip"))


@pytest.mark.parametrize("shift", [0, 1, 5])
def test_steps_in_a_row(shift):
    """Twenty steps that nothing waits between give the bits of twenty with a wait after each: a step's words around a
    block are not seen again by the next step."""
    import torch
    ctx = context()
    sizes = [300007, 1000, 70001]
    res = []
    for wait in (True, False):
        arrays = _inputs(sizes, 13)
        W, G = Flat([a[0] for a in arrays], torch.bfloat16, shift), Flat([a[1] for a in arrays], torch.bfloat16, shift)
        W32, M, V = (Flat([a[k] for a in arrays], torch.float32, shift) for k in (0, 2, 3))
        st = _state(arrays, 0)
        l8 = ctx.adamw8_tensors([dict(W=w, G=g, **{k: d[k] for k in ("M8", "V8", "MS", "VS")})
                                 for w, g, d in zip(W.views, G.views, st)])
        l32 = ctx.adamw_tensors([dict(W=w, G=g, M=m, V=v) for w, g, m, v in zip(W32.views, G.views, M.views, V.views)])
        torch.cuda.synchronize()
        for t in range(1, 21):
            ctx.adamw8_step(l8, t, lr=1e-2, seed=1)
            ctx.adamw_step(l32, t, lr=1e-2)
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        res.append([W.buf, W32.buf, M.buf, V.buf, *(d[k] for d in st for k in ("M8", "V8", "MS", "VS"))])
    for a, b in zip(*res):
        assert torch.equal(a, b)


def test_two_streams_at_once():
    """Steps on different tensors run on two streams and need no workspace."""
    import torch
    ctx = context()
    n = 1 << 20
    x = torch.randn(n, device="cuda")
    res = []
    for both in (False, True):
        sets = [[dict(W=x.clone(), G=x.clone(), M=torch.zeros(n, device="cuda"), V=torch.zeros(n, device="cuda"))] for _ in range(2)]
        streams = [torch.cuda.Stream() for _ in range(2)] if both else [torch.cuda.current_stream()] * 2
        torch.cuda.synchronize()
        for t in range(1, 6):
            for m, s in zip(sets, streams):
                ctx.adamw_step(m, t, stream=s)
        torch.cuda.synchronize()
        res.append([m[0]["W"] for m in sets])
    for w in res[1]:
        assert torch.equal(w, res[0][0])


def test_a_training_step_of_a_whole_model():
    """bf16 gradients are clipped together into fp32; Muon takes the matrices, AdamW the rest."""
    import torch
    ctx = context()
    rng = np.random.default_rng(12)
    mats = [(256, 128), (128, 384)]
    rest = [1000, 128, 64 * 128]
    Wm = [torch.from_numpy(0.02 * rng.standard_normal(s)).float().cuda() for s in mats]
    Gm = [torch.from_numpy(rng.standard_normal(s)).cuda().to(torch.bfloat16) for s in mats]
    Om = [torch.zeros(s, device="cuda") for s in mats]
    Bm = [torch.zeros(s, device="cuda") for s in mats]
    W = [torch.from_numpy(0.02 * rng.standard_normal(n)).float().cuda() for n in rest]
    G = [torch.from_numpy(rng.standard_normal(n)).cuda().to(torch.bfloat16) for n in rest]
    M, V = ([torch.zeros(n, device="cuda") for n in rest] for _ in range(2))
    w0, wm0 = [_np(w) for w in W], [w.double().cpu().numpy() for w in Wm]
    norm, factor = ctx.clip_grads([dict(G=g, out=o) for g, o in zip(Gm, Om)] + [dict(G=g, out=None) for g in G], 1.0)
    ctx.muon_step(Wm, Om, Bm, lr=0.02, weight_decay=0.01)
    ctx.adamw_step([dict(W=w, G=g, M=m, V=v, weight_decay=0.1) for w, g, m, v in zip(W, G, M, V)], 1, lr=1e-3)
    assert ctx.device_status() == 0
    # the fp32 gradients are the bf16 ones times the factor, and Muon's momentum is made of them
    for g, o, b in zip(Gm, Om, Bm):
        assert torch.equal(o, g.float() * factor) and torch.equal(b, o)
    total = math.sqrt(sum(float((o.double() ** 2).sum()) for o in Om) + sum(float((g.double() ** 2).sum()) for g in G))
    assert abs(total - 1) < 2.0 ** -8                  # in place in bf16: half a step of each
    for w, wold, g in zip(W, w0, G):
        ref, _, _ = oa.adamw_step(wold, _np(g), 0 * wold, 0 * wold, t=1, lr=1e-3, weight_decay=0.1)
        assert np.all(np.abs(_np(w) - ref) <= U * (4 * np.abs(wold) + 24e-3))
    for w, wold, o in zip(Wm, wm0, Om):
        ref = omuon.muon_step(wold, o.double().cpu().numpy(), 0 * wold, lr=0.02, weight_decay=0.01, momentum=0.95)
        dw, dr = w.double().cpu().numpy() - wold, ref["W"] - wold
        assert np.linalg.norm(dw - dr) < 0.1 * np.linalg.norm(dr)    # bf16 Newton-Schulz; its own tests are tighter


def test_offsets_beyond_32_bits():
    """A tensor of 2^32 + 1000 elements: its last blocks are those of their own offsets."""
    import torch
    ctx = context()
    n, k = (1 << 32) + 1000, 3000
    W = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    G = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    st = ctx.adamw8_state(W)
    rng = np.random.default_rng(5)
    lo = (n - k) // 256 * 256
    W[lo:] = torch.from_numpy(0.02 * rng.standard_normal(n - lo)).cuda().to(torch.bfloat16)
    G[lo:] = torch.from_numpy(rng.standard_normal(n - lo)).cuda().to(torch.bfloat16)
    w0, g0 = _np(W[lo:]), _np(G[lo:])
    ctx.adamw8_step([dict(W=W, G=G, **st)], 2, lr=1e-2, seed=6)
    z = 0 * w0
    m32, v32 = oa.fp32_moments(g0, z, z, 0.9, 0.999)
    bits = oa.noise(np.arange(lo, n), seed=6, step=2, index=0)
    np.testing.assert_array_equal(st["M8"][lo:].cpu().numpy(), oa.first_codes(m32)[0])
    np.testing.assert_array_equal(st["V8"][lo:].cpu().numpy(), oa.second_codes(v32, bits[0])[0])
    w1, m1, v1 = oa.adamw_step(w0, g0, z, z, t=2, lr=1e-2)
    D = 1e-2 * np.abs(m1) / (1 - 0.9 ** 2) / (np.sqrt(v1 / (1 - 0.999 ** 2)) + 1e-8)
    _check_w(_np(W[lo:]), w1, w0, D, "bf16", bits[1])
    assert int(st["M8"][:1 << 20].max()) == 0
    norm, _ = ctx.clip_grads([G], 1.0, apply=False)
    want = math.sqrt(float((g0 ** 2).sum()))
    assert abs(float(norm) - want) <= 6 * U * want
