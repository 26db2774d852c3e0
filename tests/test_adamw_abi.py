"""Refusals of the AdamW, 8-bit-moment and clipping entry points, on the host:
every one comes before a launch, so none needs a GPU."""
import ctypes

import pytest
import torch

import matrix_aware_optimizers_muon_b200 as mo
from matrix_aware_optimizers_muon_b200 import _lib
from matrix_aware_optimizers_muon_b200 import build as mo_build

BAD = _lib.MO_ERR_INVALID_ARG


@pytest.fixture(scope="module")
def lib():
    mo_build.build()
    return _lib.load()


@pytest.fixture
def ctx(lib):
    h = ctypes.c_void_p()
    assert lib.mo_ctx_create(ctypes.byref(h), 0) == 0
    yield h
    lib.mo_ctx_destroy(h)


def _cfg(**kw):
    d = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, bias_correction=1, stochastic=0, seed=0)
    d.update(kw)
    return _lib.AdamWCfg(**d)


def _tensor(**kw):
    d = dict(numel=1000, W=1 << 20, G=2 << 20, M=3 << 20, V=4 << 20, copy=None, w_type=0, g_type=0, copy_type=0,
             lr_scale=1.0, weight_decay=0.0)
    d.update(kw)
    return _lib.AdamWTensor(**d)


def _tensor8(**kw):
    d = dict(numel=1000, W=1 << 20, G=2 << 20, M8=3 << 20, V8=4 << 20, MS=5 << 20, VS=6 << 20, copy=None, w_type=0,
             g_type=0, copy_type=0, lr_scale=1.0, weight_decay=0.0)
    d.update(kw)
    return _lib.AdamW8Tensor(**d)


def _step(lib, ctx, tensors, cfg=None, step=1):
    eight = isinstance(tensors[0], _lib.AdamW8Tensor)
    arr = (type(tensors[0]) * len(tensors))(*tensors)
    fn = lib.adamw8_step if eight else lib.adamw_step
    st = fn(ctx, arr, len(tensors), ctypes.byref(cfg or _cfg()), step, None)
    return st, lib.mo_last_error(ctx).decode()


@pytest.mark.parametrize("make", [_tensor, _tensor8])
@pytest.mark.parametrize("kw,word", [
    (dict(lr=-1.0), "lr"), (dict(lr=1e39), "lr"), (dict(lr=float("nan")), "lr"), (dict(eps=float("inf")), "eps"), (dict(beta1=1.0), "betas"),
    (dict(beta2=-0.1), "betas"), (dict(beta2=float("nan")), "betas"), (dict(lr_dev=18), "aligned"),
    (dict(step_dev=12), "aligned"), (dict(grad_scale=2), "aligned"), (dict(skip=1), "aligned")])
def test_bad_hyperparameters(lib, ctx, make, kw, word):
    st, msg = _step(lib, ctx, [make()], _cfg(**kw))
    assert st == BAD and word in msg and msg.startswith("adamw")


@pytest.mark.parametrize("make", [_tensor, _tensor8])
@pytest.mark.parametrize("kw,word", [
    (dict(numel=-1), "numel"), (dict(numel=(1 << 38) + 1), "numel"), (dict(W=None), "null W"), (dict(W=(1 << 20) + 2), "W must be aligned"),
    (dict(G=(2 << 20) + 1, g_type=1), "G must be aligned"), (dict(w_type=2), "w_type"), (dict(w_type=3), "w_type"),
    (dict(g_type=-1), "g_type"), (dict(lr_scale=-1.0), "lr_scale"), (dict(weight_decay=float("nan")), "weight_decay"),
    (dict(copy=7 << 20, copy_type=0), "copy"), (dict(copy=7 << 20, copy_type=1, w_type=1), "copy"),
    (dict(copy=(7 << 20) + 1, copy_type=1), "copy must be aligned"),
    (dict(G=(1 << 20) + 3996), "overlap"), (dict(copy=(1 << 20) + 2000, copy_type=1), "overlap")])
def test_bad_tensors(lib, ctx, make, kw, word):
    st, msg = _step(lib, ctx, [make(**kw)])
    assert st == BAD and word in msg
    # the same tensor behind a good one is named by its place
    st, msg = _step(lib, ctx, [make(W=8 << 20, **({"M": 9 << 20, "V": 10 << 20} if make is _tensor else
                                                 {"M8": 9 << 20, "V8": 10 << 20, "MS": 11 << 20, "VS": 12 << 20})),
                               make(**kw)])
    assert st == BAD and word in msg and ("overlap" in msg or "index 1" in msg)


@pytest.mark.parametrize("kw,word", [(dict(M=None), "null M"), (dict(V=None), "null V"), (dict(M=(3 << 20) + 2), "M must be aligned"),
                                     (dict(V=(3 << 20) + 4), "overlap"), (dict(M=1 << 20), "overlap")])
def test_bad_fp32_moments(lib, ctx, kw, word):
    st, msg = _step(lib, ctx, [_tensor(**kw)])
    assert st == BAD and word in msg


@pytest.mark.parametrize("kw,word", [(dict(M8=None), "null M8"), (dict(VS=None), "null VS"), (dict(V8=(3 << 20) + 999), "overlap"),
                                     (dict(MS=(3 << 20) + 999), "overlap"), (dict(VS=(5 << 20) + 3), "overlap")])
def test_bad_codes(lib, ctx, kw, word):
    st, msg = _step(lib, ctx, [_tensor8(**kw)])
    assert st == BAD and word in msg


def test_step_and_lists(lib, ctx):
    assert _step(lib, ctx, [_tensor()], step=0)[0] == BAD
    cfg = _cfg()
    assert lib.adamw_step(ctx, None, 1, ctypes.byref(cfg), 1, None) == BAD
    assert lib.adamw_step(ctx, None, -1, ctypes.byref(cfg), 1, None) == BAD
    assert lib.adamw_step(ctx, (_lib.AdamWTensor * 1)(_tensor()), 1, None, 1, None) == BAD
    assert lib.adamw_step(None, None, 0, ctypes.byref(cfg), 1, None) == BAD
    assert lib.adamw_step(ctx, None, 0, None, 1, None) == 0


def test_the_same_tensor_twice(lib, ctx):
    for make in (_tensor, _tensor8):
        st, msg = _step(lib, ctx, [make(), make()])
        assert st == BAD and "overlap" in msg
    # a gradient may serve two tensors
    other = dict(W=8 << 20, M=9 << 20, V=10 << 20)
    st, msg = _step(lib, ctx, [_tensor(), _tensor(**other, g_type=3)])
    assert st == BAD and "g_type" in msg                   # the next fault is found, not the gradient


def test_scalars_inside_written_buffers(lib, ctx):
    for make, first in ((_tensor, 3 << 20), (_tensor8, 5 << 20)):
        for kw in (dict(lr_dev=(1 << 20) + 3996), dict(step_dev=first), dict(grad_scale=4 << 20), dict(skip=1 << 20)):
            st, msg = _step(lib, ctx, [make()], _cfg(**kw))
            assert st == BAD and "overlap" in msg, kw


def test_moments(lib, ctx):
    def call(fn, cfg=None, **kw):
        d = dict(numel=1000, M8=3 << 20, V8=4 << 20, MS=5 << 20, VS=6 << 20, M=1 << 20, V=2 << 20, type=0)
        d.update(kw)
        arr = (_lib.AdamW8Moments * 1)(_lib.AdamW8Moments(**d))
        if fn == "pack":
            st = lib.adamw8_pack(ctx, arr, 1, ctypes.byref(cfg or _lib.PackCfg()), None)
        else:
            st = lib.adamw8_unpack(ctx, arr, 1, None)
        return st, lib.mo_last_error(ctx).decode()

    for fn in ("pack", "unpack"):
        for kw, word in ((dict(type=2), "type"), (dict(M=None), "null M"), (dict(MS=None), "null MS"),
                         (dict(V=(2 << 20) + 2), "aligned"), (dict(M8=1 << 20), "overlap"), (dict(numel=-5), "numel")):
            st, msg = call(fn, **kw)
            assert st == BAD and word in msg and msg.startswith("adamw8_" + fn), (fn, kw, msg)
    assert call("pack", V=1 << 20, type=3)[0] == BAD
    assert call("pack", _lib.PackCfg(step_dev=4))[0] == BAD
    assert lib.adamw8_pack(ctx, None, 1, ctypes.byref(_lib.PackCfg()), None) == BAD
    assert lib.adamw8_unpack(ctx, None, 1, None) == BAD
    assert lib.adamw8_unpack(ctx, None, 0, None) == 0


def test_clip_needs_a_workspace(lib, ctx):
    cfg = _lib.ClipCfg(1.0, 1, None, 16, 32, None)
    arr = (_lib.Grad * 1)(_lib.Grad(10, 1 << 20, None, 0, 0))
    assert lib.clip_grads(ctx, arr, 1, ctypes.byref(cfg), None) == _lib.MO_ERR_NO_WORKSPACE
    assert b"MO_CLIP_WORKSPACE_BYTES" in lib.mo_last_error(ctx)
    assert lib.clip_grads(ctx, arr, 1, None, None) == BAD
    assert lib.clip_grads(ctx, None, 1, ctypes.byref(cfg), None) == BAD
    assert lib.clip_grads(ctx, None, -1, ctypes.byref(cfg), None) == BAD


@pytest.mark.parametrize("cfg,grad,word", [
    (dict(max_norm=-1.0), {}, "max_norm"), (dict(max_norm=float("nan")), {}, "max_norm"), (dict(norm=None), {}, "null norm"),
    (dict(factor=None), {}, "null norm or factor"), (dict(scale=2), {}, "aligned"), (dict(factor=16), {}, "overlap"),
    (dict(scale=16), {}, "overlap"), (dict(nonfinite=32), {}, "overlap"), ({}, dict(g_type=3), "g_type"),
    ({}, dict(out=2 << 20, out_type=-1), "out_type"), ({}, dict(G=(1 << 20) + 2), "aligned"), ({}, dict(numel=-1), "numel"),
    ({}, dict(out=(1 << 20) + 4), "overlap"), ({}, dict(out=1 << 20, out_type=1), "in place"), ({}, dict(G=16), "overlap")])
def test_clip_refusals(lib, ctx, cfg, grad, word):
    c = dict(max_norm=1.0, apply=1, scale=None, norm=16, factor=32, nonfinite=None)
    c.update(cfg)
    g = dict(numel=10, G=1 << 20, out=None, g_type=0, out_type=0)
    g.update(grad)
    arr = (_lib.Grad * 1)(_lib.Grad(**g))
    cc = _lib.ClipCfg(**c)
    st = lib.clip_grads(ctx, arr, 1, ctypes.byref(cc), None)
    msg = lib.mo_last_error(ctx).decode()
    assert st == BAD and word in msg, msg


class _Dev:
    """Stands in for a CUDA tensor (no GPU here)."""

    place = 1 << 20

    def __init__(self, numel, dtype, device=0, contiguous=True, cuda=True):
        _Dev.place += 1 << 16                 # buffers of a list must not overlap
        self._at = _Dev.place
        self.is_cuda, self.dtype, self._n, self._c = cuda, dtype, numel, contiguous
        self.device = torch.device("cuda", device)

    def is_contiguous(self):
        return self._c

    def numel(self):
        return self._n

    def data_ptr(self):
        return self._at


def _context(device=0):
    return mo.Context(device)                 # host memory only


def _mat(**kw):
    f = torch.float32
    return dict(dict(W=_Dev(300, f), G=_Dev(300, torch.bfloat16), M=_Dev(300, f), V=_Dev(300, f)), **kw)


def _mat8(**kw):
    u = torch.uint8
    return dict(dict(W=_Dev(300, torch.float32), G=_Dev(300, torch.float16), M8=_Dev(300, u), V8=_Dev(300, u), MS=_Dev(2, u),
                     VS=_Dev(2, u)), **kw)


def test_binding_checks_lists(lib):
    c, f = _context(), torch.float32
    good = c.adamw_tensors([_mat(), _mat(G=None, copy=_Dev(300, torch.float16), lr_scale=0.5, weight_decay=0.1)])
    assert len(good) == 2 and good.handle
    with pytest.raises(mo.MoError, match="weight_decay"):
        c.adamw_tensors([_mat(weight_decay=-0.1)])
    twice = _mat()
    with pytest.raises(mo.MoError, match="overlap"):
        c.adamw_tensors([twice, twice])
    for bad in (_mat(W=_Dev(300, torch.float16)), _mat(W=_Dev(300, f, contiguous=False)), _mat(W=_Dev(300, f, cuda=False)),
                _mat(W=_Dev(300, f, device=1)), _mat(G=_Dev(299, f)), _mat(M=_Dev(300, torch.bfloat16)),
                _mat(V=_Dev(301, f)), _mat(copy=_Dev(300, f)), _mat(copy=_Dev(3, torch.bfloat16))):
        with pytest.raises(ValueError, match="tensor 1"):
            c.adamw_tensors([_mat(), bad])
    assert len(c.adamw8_tensors([_mat8()])) == 1
    for bad in (_mat8(M8=_Dev(299, torch.uint8)), _mat8(MS=_Dev(1, torch.uint8)), _mat8(VS=_Dev(3, torch.uint8)),
                _mat8(V8=_Dev(300, torch.int8)), _mat8(W=_Dev(256, f))):
        with pytest.raises(ValueError, match="tensor 0"):
            c.adamw8_tensors([bad])
    mom = {k: v for k, v in _mat8(M=_Dev(300, f), V=_Dev(300, f)).items() if k not in "WG"}
    assert len(c.adamw8_moments([mom])) == 1
    for k, v in (("M", _Dev(300, torch.float16)), ("V", _Dev(300, torch.bfloat16)), ("V", _Dev(3, f)), ("M8", _Dev(3, torch.uint8))):
        with pytest.raises(ValueError, match="tensor 0"):
            c.adamw8_moments([dict(mom, **{k: v})])
    assert len(c.clip_tensors([_Dev(5, f), None, dict(G=_Dev(4, torch.bfloat16), out=_Dev(4, f))])) == 3
    for bad in (_Dev(5, torch.float64), dict(G=_Dev(4, f), out=_Dev(5, f)), dict(G=_Dev(4, f), out=_Dev(4, torch.int32))):
        with pytest.raises(ValueError, match="tensor 0"):
            c.clip_tensors([bad])


def test_binding_refuses_a_list_of_another_kind(lib):
    c = _context()
    grads = c.clip_tensors([_Dev(5, torch.float32)])
    with pytest.raises(ValueError, match="'adamw'"):
        c._list("adamw", grads)
    with pytest.raises(ValueError, match="cuda:1"):
        _context(1)._list("grads", grads)


def test_prepared_lists(lib, ctx):
    """Lists refuse what the calls with arrays refuse, and the calls a list of another kind."""
    out = ctypes.c_void_p(5)
    arr = (_lib.AdamWTensor * 2)(_tensor(), _tensor())
    assert lib.mo_adamw_list(ctx, arr, 2, ctypes.byref(out)) == BAD and not out.value
    assert b"overlap" in lib.mo_last_error(ctx)
    assert lib.mo_adamw_list(ctx, None, 1, ctypes.byref(out)) == BAD and lib.mo_adamw_list(ctx, arr, -1, ctypes.byref(out)) == BAD
    assert lib.mo_adamw_list(ctx, arr, 1, None) == BAD
    assert lib.mo_adamw_list(ctx, arr, 1, ctypes.byref(out)) == 0 and out.value
    cfg, pack = _cfg(), _lib.PackCfg()
    clip = _lib.ClipCfg(1.0, 1, None, 16, 32, None)
    assert lib.adamw_step_list(ctx, out, ctypes.byref(_cfg(beta1=2.0)), 1, None) == BAD
    assert lib.adamw_step_list(ctx, out, None, 1, None) == BAD
    for st in (lib.adamw8_step_list(ctx, out, ctypes.byref(cfg), 1, None), lib.adamw8_pack_list(ctx, out, ctypes.byref(pack), None),
               lib.adamw8_unpack_list(ctx, out, None), lib.clip_grads_list(ctx, out, ctypes.byref(clip), None)):
        assert st == BAD and b"another call" in lib.mo_last_error(ctx)
    assert lib.adamw_step_list(ctx, None, ctypes.byref(cfg), 1, None) == BAD
    lib.mo_list_destroy(out)
    lib.mo_list_destroy(None)
    # scalars of a clip inside a gradient
    grads = (_lib.Grad * 1)(_lib.Grad(100, 1 << 20, None, 0, 0))
    assert lib.mo_grad_list(ctx, grads, 1, ctypes.byref(out)) == 0
    clip = _lib.ClipCfg(1.0, 1, None, (1 << 20) + 396, 32, None)
    assert lib.clip_grads_list(ctx, out, ctypes.byref(clip), None) == BAD and b"overlap" in lib.mo_last_error(ctx)
    lib.mo_list_destroy(out)


def test_scalars():
    from matrix_aware_optimizers_muon_b200 import _scalar
    assert _scalar(None, "x", 0, torch.float32) is None
    one = _Dev(1, torch.float32)
    assert _scalar(one, "x", 0, torch.float32) == one.data_ptr()
    for bad in (_Dev(2, torch.float32), _Dev(1, torch.float64), _Dev(1, torch.float32, cuda=False), _Dev(1, torch.float32, device=1)):
        with pytest.raises(ValueError, match="grad_scale"):
            _scalar(bad, "grad_scale", 0, torch.float32)
