"""Both 8-bit moments rounded with noise: codes equal to the oracle's, long runs
against fp64 AdamW, and the ways to ask for it."""
import warnings

import adamw8_runs as runs
import numpy as np
import pytest
from test_gpu_adamw import B1, B2, EPS, SIZES, Flat, _check_w, _dt, _extreme_blocks, _held, _inputs, _np, _state

from gpu_env import context
from oracle import adamw as oa

pytestmark = pytest.mark.gpu

KEYS = ("M8", "V8", "MS", "VS")
N, STEPS = 64 * 256, 3000


def _run(b1, b2, seed=3):
    import torch
    ctx = context()
    W, G = torch.zeros(N, device="cuda"), torch.zeros(N, device="cuda")
    st = ctx.adamw8_state(W)
    lst = ctx.adamw8_tensors([dict(W=W, G=G, **st)])

    def step(g, t):
        G.copy_(torch.from_numpy(g))
        ctx.adamw8_step(lst, t, lr=runs.LR, beta1=b1, beta2=b2, eps=runs.EPS, noise=seed)

    def read():
        return (_np(W), *_held(st))
    return step, read


@pytest.mark.parametrize("b1,b2", runs.BETAS)
def test_steady_gradient(b1, b2):
    runs.steady(*_run(b1, b2), N, STEPS, b1, b2)


@pytest.mark.parametrize("live", [0, 0.5])
@pytest.mark.parametrize("b1,b2", runs.BETAS)
def test_gradient_ends(b1, b2, live):
    runs.gradient_ends(*_run(b1, b2), N, STEPS, b1, b2, live)


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("w,g,copy", [("f32", "f32", None), ("f32", "bf16", "bf16"), ("f32", "f16", "f16"), ("bf16", "bf16", None),
                                      ("bf16", "f16", None), ("bf16", "f32", None)])
def test_codes_and_weights(w, g, copy, shift):
    """Three steps; every step starts from the state that the one before left.  Codes and scales are equal to the oracle's;
    weights as in the steps with other roundings."""
    import torch
    ctx = context()
    seed = 11
    arrays = _inputs(SIZES, 77)
    rng = np.random.default_rng(8)
    W = Flat([a[0] for a in arrays], _dt(w), shift)
    C = Flat([a[0] for a in arrays], _dt(copy), shift) if copy else None
    st = _state(arrays, shift)
    for t in (5, 6, 7):
        G = Flat([a[1] * rng.uniform(0.2, 3) * rng.choice([-1, 1], a[1].size) for a in arrays], _dt(g), shift)
        old = [(_np(W.views[i]), _np(G.views[i]), *_held(st[i])) for i in range(len(SIZES))]
        step = t if t != 6 else torch.tensor(t, device="cuda")
        ctx.adamw8_step([dict(W=W.views[i], G=G.views[i], copy=C.views[i] if C else None, weight_decay=0.1,
                              **{k: st[i][k] for k in KEYS}) for i in range(len(SIZES))],
                        step, lr=1e-2, beta1=B1, beta2=B2, eps=EPS, noise=seed)
        for i, n in enumerate(SIZES):
            w0, g0, m0, v0 = old[i]
            m32, v32 = oa.fp32_moments(g0, m0, v0, B1, B2)
            at = np.arange(n)
            vbits, wbits = oa.noise(at, seed=seed, step=t, index=i)
            (m8, ms), (v8, vs) = oa.first_codes(m32, oa.first_noise(at, seed=seed, step=t, index=i)), oa.second_codes(v32, vbits)
            for k, a in (("MS", ms), ("VS", vs), ("M8", m8), ("V8", v8)):
                np.testing.assert_array_equal(st[i][k].cpu().numpy(), a, err_msg=f"{k} of {n} at step {t}")
                full = st[i]["_" + k].cpu().numpy()
                assert np.all(full[:shift] == 99) and np.all(full[shift + a.size:] == 99)
            w1, _, v1 = oa.adamw_step(w0, g0, m0, v0, t=t, lr=1e-2, beta1=B1, beta2=B2, eps=EPS, weight_decay=0.1)
            mag = B1 * np.abs(m0) + (1 - B1) * np.abs(g0)
            D = 1e-2 * mag / (1 - B1 ** t) / (np.sqrt(v1 / (1 - B2 ** t)) + EPS)
            _check_w(_np(W.views[i]), w1, w0, D, w, wbits if w == "bf16" else None)
            if C:
                _check_w(_np(C.views[i]), w1, w0, D, copy)
        assert W.others_untouched() and (C is None or C.others_untouched())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,shift", [(2048, 0), (2047, 1), (1, 0), (257, 3)])
def test_pack(dtype, n, shift):
    """Blocks at the ends of fp32's range, with NaN and infinities."""
    import torch
    ctx = context()
    x = torch.from_numpy(_extreme_blocks()[:n]).to(_dt(dtype))
    M, V = (torch.zeros(n + 64, dtype=_dt(dtype), device="cuda")[shift:shift + n] for _ in range(2))
    M.copy_(x)
    V.copy_(x.abs())
    if n > 300:
        V[1024:1027] = 1.0                                # a first moment that is not finite beside a second that is
    d = {k: torch.full((s + 32,), 9, dtype=torch.uint8, device="cuda")[shift:shift + s]
         for k, s in (("M8", n), ("V8", n), ("MS", -(-n // 256)), ("VS", -(-n // 256)))}
    ctx.adamw8_pack([dict(M=M, V=V, **d)], noise=21, step=12)
    at = np.arange(n)
    (m8, ms) = oa.first_codes(_np(M), oa.first_noise(at, seed=21, step=12, index=0))
    (v8, vs) = oa.second_codes(_np(V), oa.noise(at, seed=21, step=12, index=0)[0])
    for k, a in (("MS", ms), ("VS", vs), ("M8", m8), ("V8", v8)):
        np.testing.assert_array_equal(d[k].cpu().numpy(), a, err_msg=k)


def test_the_default_is_noise_of_seed_0_and_seed_is_the_earlier_form():
    import torch
    ctx = context()
    n = 5000
    g = torch.randn(n, device="cuda", generator=torch.Generator("cuda").manual_seed(1))

    def after(pack=False, **kw):
        W = torch.zeros(n, device="cuda", dtype=torch.bfloat16)
        st = ctx.adamw8_state(W)
        if pack:
            ctx.adamw8_pack([dict(M=g, V=g * g, **st)], step=3, **kw)
        else:
            for t in (1, 2, 3):
                ctx.adamw8_step([dict(W=W, G=g, **st)], t, **kw)
        return [W, *(st[k] for k in KEYS)]

    def same(a, b):
        return [torch.equal(x, y) for x, y in zip(a, b)]
    assert all(same(after(), after(noise=0)))
    assert not any(same(after(noise=5), after(noise=0))[:3])
    assert all(same(after(noise=None), after(seed=None)))
    with warnings.catch_warnings():
        warnings.simplefilter("ignore")
        assert not same(after(seed=5), after(noise=5))[1]  # the first moment goes to the nearest code
    # packing: nearest unless asked; V's codes are those of the same seed either way, M's differ
    assert all(same(after(True), after(True, noise=None)))
    w, m8, v8, ms, vs = same(after(True, noise=4), after(True, seed=4))
    assert v8 and ms and vs and not m8
    w, m8, v8, ms, vs = same(after(True), after(True, seed=4))
    assert m8 and not v8


def test_replayed_and_eager_steps_agree():
    """A captured step draws the noise of the step that it reads on the device."""
    import torch
    ctx = context()
    n = 70001
    gen = torch.Generator("cuda").manual_seed(4)
    gs = [torch.randn(n, device="cuda", generator=gen) for _ in range(4)]
    sets = []
    for _ in range(2):
        W, G = torch.zeros(n, device="cuda", dtype=torch.bfloat16), torch.zeros(n, device="cuda")
        st = ctx.adamw8_state(W)
        sets.append(dict(W=W, G=G, st=st, list=ctx.adamw8_tensors([dict(W=W, G=G, **st)]),
                         t=torch.zeros(1, dtype=torch.int64, device="cuda")))
    a, b = sets
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        ctx.adamw8_step(a["list"], a["t"], noise=9)
    for t, g in enumerate(gs, 1):
        for s in sets:
            s["G"].copy_(g)
            s["t"].fill_(t)
        graph.replay()
        ctx.adamw8_step(b["list"], b["t"], noise=9)
        assert torch.equal(a["W"], b["W"]) and all(torch.equal(a["st"][k], b["st"][k]) for k in KEYS)
