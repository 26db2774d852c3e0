"""Lists whose tensors differ in types and offsets, longer than one launch
holds: every tensor gets its own rates, noise and copy."""
import numpy as np
import pytest
from test_gpu_adamw import B1, B2, EPS, _check_w, _dt, _inputs, _np

from gpu_env import context
from oracle import adamw as oa

pytestmark = pytest.mark.gpu

TENSORS = 900
KEYS = ("M8", "V8", "MS", "VS")


def _drawn(seed):
    """Sizes, types and offsets of the list's tensors, and their arrays."""
    rng = np.random.default_rng(seed)
    sizes = [int(2 ** rng.uniform(0, 11.5)) for _ in range(TENSORS)]
    sizes[::97] = [0] * len(sizes[::97])
    kinds = [dict(w=rng.choice(["f32", "bf16"]), g=rng.choice(["f32", "bf16", "f16"]), copy=rng.choice(["", "bf16", "f16"]),
                  shift=[int(s) for s in rng.choice([0, 0, 0, 1, 3, 8], 7)], wd=0.1 * int(rng.integers(3)),
                  lr=float(rng.choice([1.0, 0.5])), none=rng.random() < 0.1) for _ in range(TENSORS)]
    return sizes, kinds, _inputs(sizes, seed)


class Place:
    """Tensors of one type in one buffer of elements that stay as they are."""

    def __init__(self, dtype):
        self.dtype, self.at, self.items = dtype, 64, []

    def take(self, array, shift):
        lo = -(-self.at // 64) * 64 + 64 + shift
        self.items.append((lo, array))
        self.at = lo + array.size
        return len(self.items) - 1

    def make(self):
        import torch
        fill = 99 if self.dtype == torch.uint8 else 7.0
        host = torch.full((self.at + 64,), fill, dtype=torch.float64)
        inside = torch.zeros(self.at + 64, dtype=torch.bool)
        for lo, a in self.items:
            host[lo:lo + a.size] = torch.from_numpy(np.asarray(a, dtype=np.float64))
            inside[lo:lo + a.size] = True
        self.buf, self.inside, self.fill = host.to(self.dtype).cuda(), inside.cuda(), fill

    def view(self, i):
        lo, a = self.items[i]
        return self.buf[lo:lo + a.size]

    def others_untouched(self):
        return bool((self.buf[~self.inside] == self.fill).all())


class Places:
    def __init__(self):
        import torch
        self.by = {k: Place(_dt(k)) for k in ("f32", "bf16", "f16")}
        self.by["u8"] = Place(torch.uint8)

    def take(self, kind, array, shift):
        p = self.by[kind]
        i = p.take(array, shift)
        return lambda: p.view(i)

    def make(self):
        for p in self.by.values():
            p.make()

    def others_untouched(self):
        return all(p.others_untouched() for p in self.by.values())


@pytest.mark.parametrize("seed", [None, 5])
def test_adamw(seed):
    ctx = context()
    sizes, kinds, arrays = _drawn(21)
    P, get = Places(), []
    for k, (w, g, m, v) in zip(kinds, arrays):
        s = k["shift"]
        c = P.take(k["copy"], w, s[4]) if k["w"] == "f32" and k["copy"] else None
        get.append((P.take(k["w"], w, s[0]), P.take(k["g"], g, s[1]), P.take("f32", m, s[2]), P.take("f32", v, s[3]), c))
    P.make()
    old = [[_np(f()) for f in x[:4]] for x in get]
    ctx.adamw_step([dict(W=x[0](), G=None if k["none"] else x[1](), M=x[2](), V=x[3](), copy=x[4] and x[4](),
                         lr_scale=k["lr"], weight_decay=k["wd"]) for x, k in zip(get, kinds)],
                   7, lr=1e-2, beta1=B1, beta2=B2, eps=EPS, seed=seed)
    assert P.others_untouched()
    for i, (x, k, (w0, g0, m0, v0)) in enumerate(zip(get, kinds, old)):
        if k["none"] or not w0.size:
            for f, a in zip((x[0], x[2], x[3]), (w0, m0, v0)):
                np.testing.assert_array_equal(_np(f()), a)
            continue
        m32, v32 = oa.fp32_moments(g0, m0, v0, B1, B2)
        np.testing.assert_array_equal(_np(x[2]()), m32)
        np.testing.assert_array_equal(_np(x[3]()), v32)
        bits = oa.noise(np.arange(w0.size), seed=seed, step=7, index=i)[1] if seed is not None and k["w"] == "bf16" else None
        _weights(k, x, 4, w0, g0, m0, v0, 7, bits)


def _weights(k, x, copy, w0, g0, m0, v0, t, bits):
    lr = 1e-2 * k["lr"]
    w1, _, v1 = oa.adamw_step(w0, g0, m0, v0, t=t, lr=lr, beta1=B1, beta2=B2, eps=EPS, weight_decay=k["wd"])
    D = lr * (B1 * np.abs(m0) + (1 - B1) * np.abs(g0)) / (1 - B1 ** t) / (np.sqrt(v1 / (1 - B2 ** t)) + EPS)
    _check_w(_np(x[0]()), w1, w0, D, k["w"], bits)
    if x[copy]:
        _check_w(_np(x[copy]()), w1, w0, D, k["copy"])


@pytest.mark.parametrize("noise", [None, 5])
def test_adamw8(noise):
    ctx = context()
    sizes, kinds, arrays = _drawn(22)
    P, get = Places(), []
    for k, (w, g, m, v) in zip(kinds, arrays):
        s = k["shift"]
        (m8, ms), (v8, vs) = oa.first_codes(np.float32(m)), oa.second_codes(np.float32(v))
        c = P.take(k["copy"], w, s[4]) if k["w"] == "f32" and k["copy"] else None
        get.append((P.take(k["w"], w, s[0]), P.take(k["g"], g, s[1]),
                    {n: P.take("u8", a, o) for n, a, o in zip(KEYS, (m8, v8, ms, vs), (s[2], s[3], s[5], s[6]))}, c))
    P.make()
    old = [[_np(x[0]()), _np(x[1]()), *(x[2][n]().cpu().numpy() for n in KEYS)] for x in get]
    ctx.adamw8_step([dict(W=x[0](), G=None if k["none"] else x[1](), copy=x[3] and x[3](), lr_scale=k["lr"], weight_decay=k["wd"],
                          **{n: f() for n, f in x[2].items()}) for x, k in zip(get, kinds)],
                    7, lr=1e-2, beta1=B1, beta2=B2, eps=EPS, noise=noise)
    assert P.others_untouched()
    for i, (x, k, (w0, g0, *codes)) in enumerate(zip(get, kinds, old)):
        if k["none"] or not w0.size:
            for f, a in zip((x[0], *x[2].values()), (w0, *codes)):
                np.testing.assert_array_equal(_np(f()), a)
            continue
        m8, v8, ms, vs = codes
        m0, v0 = oa.first_moment(m8, ms), oa.second_moment(v8, vs)
        m32, v32 = oa.fp32_moments(g0, m0, v0, B1, B2)
        at, mbits, vbits, wbits = np.arange(w0.size), None, None, None
        if noise is not None:
            mbits, (vbits, wbits) = oa.first_noise(at, seed=noise, step=7, index=i), oa.noise(at, seed=noise, step=7, index=i)
        (m8, ms), (v8, vs) = oa.first_codes(m32, mbits), oa.second_codes(v32, vbits)
        for n, a in zip(KEYS, (m8, v8, ms, vs)):
            np.testing.assert_array_equal(x[2][n]().cpu().numpy(), a, err_msg=f"{n} of tensor {i}")
        _weights(k, x, 3, w0, g0, m0, v0, 7, wbits if k["w"] == "bf16" else None)


@pytest.mark.parametrize("noise", [None, 5])
def test_pack_and_unpack(noise):
    ctx = context()
    sizes, kinds, arrays = _drawn(23)
    P, get = Places(), []
    for k, (_, _, m, v) in zip(kinds, arrays):
        s = k["shift"]
        nb = -(-m.size // 256)
        z = np.zeros(m.size)
        get.append((P.take(k["w"], m, s[0]), P.take(k["w"], v, s[1]),
                    {n: P.take("u8", a, o) for n, a, o in zip(KEYS, (z, z, np.zeros(nb), np.zeros(nb)), (s[2], s[3], s[5], s[6]))},
                    P.take(k["copy"] if k["copy"] == "bf16" else "f32", z, s[4]),
                    P.take(k["copy"] if k["copy"] == "bf16" else "f32", z, s[1])))
    P.make()
    codes = [{n: f() for n, f in x[2].items()} for x in get]
    ctx.adamw8_pack([dict(M=x[0](), V=x[1](), **c) for x, c in zip(get, codes)], noise=noise, step=7)
    ctx.adamw8_unpack([dict(M=x[3](), V=x[4](), **c) for x, c in zip(get, codes)])
    assert P.others_untouched()
    for i, (x, c) in enumerate(zip(get, codes)):
        m, v = _np(x[0]()), _np(x[1]())
        at, mbits, vbits = np.arange(m.size), None, None
        if noise is not None:
            mbits, vbits = oa.first_noise(at, seed=noise, step=7, index=i), oa.noise(at, seed=noise, step=7, index=i)[0]
        (m8, ms), (v8, vs) = oa.first_codes(m, mbits), oa.second_codes(v, vbits)
        for n, a in zip(KEYS, (m8, v8, ms, vs)):
            np.testing.assert_array_equal(c[n].cpu().numpy(), a, err_msg=f"{n} of tensor {i}")
        # a code has so few bits that bf16 holds its value, whose scale is far from the ends here
        np.testing.assert_array_equal(_np(x[3]()), oa.first_moment(m8, ms))
        np.testing.assert_array_equal(_np(x[4]()), oa.second_moment(v8, vs))


def test_clip():
    import torch
    ctx = context()
    sizes, kinds, arrays = _drawn(24)
    P, get = Places(), []
    for k, (_, g, _, _) in zip(kinds, arrays):
        s = k["shift"]
        get.append((P.take(k["g"], g, s[0]), P.take(k["copy"] or "f32", 0 * g, s[1]) if k["w"] == "f32" else None))
    P.make()
    old = [x[0]().clone() for x in get]
    norm, factor = ctx.clip_grads([None if k["none"] else dict(G=x[0](), out=x[1] and x[1]()) for x, k in zip(get, kinds)], 0.1)
    want, f = oa.clip([_np(g) for g, k in zip(old, kinds) if not k["none"]], 0.1)
    u = 2.0 ** -24
    assert abs(float(norm) - want) <= 6 * u * want and abs(float(factor) - f) <= 10 * u * f
    assert P.others_untouched()
    for x, g, k in zip(get, old, kinds):
        if k["none"]:
            assert torch.equal(x[0](), g) and (x[1] is None or not x[1]().any())
            continue
        out = x[1]() if x[1] else x[0]()
        assert torch.equal(out, (g.float() * factor).to(out.dtype))
        assert x[1] is None or torch.equal(x[0](), g)
