"""Refusals and host-side rules of the AdamW, 8-bit-moment and clipping calls
that test_adamw_abi.py leaves open; none needs a GPU."""
import copy
import ctypes
import pickle

import pytest
from test_adamw_abi import BAD, _cfg, _context, _mat, _step, _tensor, _tensor8, ctx, lib  # noqa: F401

from matrix_aware_optimizers_muon_b200 import _lib

P = 64 << 20                                   # a place far from the tensors


@pytest.mark.parametrize("make,kw,scalar", [
    (_tensor, dict(W=P + 4), dict(step_dev=P)), (_tensor, dict(M=P + 4), dict(step_dev=P)),
    (_tensor, dict(V=P + 4), dict(step_dev=P)), (_tensor, dict(copy=P + 2, copy_type=1), dict(lr_dev=P)),
    (_tensor, dict(copy=P + 6, copy_type=2), dict(step_dev=P)),
    (_tensor, dict(W=P + 2, w_type=1), dict(lr_dev=P)), (_tensor, dict(W=P + 2, w_type=1), dict(grad_scale=P)),
    (_tensor, dict(W=P + 2, w_type=1), dict(skip=P)),
    (_tensor8, dict(M8=P + 1), dict(skip=P)), (_tensor8, dict(V8=P + 3), dict(grad_scale=P)),
    (_tensor8, dict(MS=P + 7), dict(step_dev=P)), (_tensor8, dict(VS=P + 3), dict(lr_dev=P)),
    # behind a written byte begins a gradient, inside the same scalar
    (_tensor8, dict(numel=1, MS=P + 1, G=P + 4), dict(step_dev=P))])
def test_scalars_that_begin_before_a_written_buffer(lib, ctx, make, kw, scalar):  # noqa: F811
    st, msg = _step(lib, ctx, [make(**kw)], _cfg(**scalar))
    assert st == BAD and "overlap" in msg


def test_scalar_of_packing_that_begins_before_a_buffer(lib, ctx):  # noqa: F811
    d = dict(numel=1000, M8=3 << 20, V8=4 << 20, MS=5 << 20, VS=6 << 20, M=1 << 20, V=2 << 20, type=0)
    for kw in (dict(M8=P + 1), dict(VS=P + 7), dict(M=P + 4), dict(V=P + 2, type=1, M=1 << 20)):
        arr = (_lib.AdamW8Moments * 1)(_lib.AdamW8Moments(**dict(d, **kw)))
        cfg = _lib.PackCfg(1, 0, 0, P)
        assert lib.adamw8_pack(ctx, arr, 1, ctypes.byref(cfg), None) == BAD, kw
        assert b"overlap" in lib.mo_last_error(ctx)


def test_a_list_belongs_to_its_contexts_device(lib, ctx):  # noqa: F811
    """Its addresses are those of one GPU: a context of another one refuses it (and one of the same takes it)."""
    other, same, out = ctypes.c_void_p(), ctypes.c_void_p(), ctypes.c_void_p()
    assert lib.mo_ctx_create(ctypes.byref(other), 1) == 0 and lib.mo_ctx_create(ctypes.byref(same), 0) == 0
    cfg, pack, clip = _cfg(), _lib.PackCfg(), _lib.ClipCfg(1.0, 1, None, 16, 32, None)
    mom = _lib.AdamW8Moments(numel=1000, M8=3 << 20, V8=4 << 20, MS=5 << 20, VS=6 << 20, M=1 << 20, V=2 << 20, type=0)
    lists = [(lib.mo_adamw_list, _tensor(), [lambda c, m: lib.adamw_step_list(c, m, ctypes.byref(cfg), 1, None)]),
             (lib.mo_adamw8_list, _tensor8(), [lambda c, m: lib.adamw8_step_list(c, m, ctypes.byref(cfg), 1, None)]),
             (lib.mo_moments_list, mom, [lambda c, m: lib.adamw8_pack_list(c, m, ctypes.byref(pack), None),
                                         lambda c, m: lib.adamw8_unpack_list(c, m, None)]),
             (lib.mo_grad_list, _lib.Grad(100, 1 << 20, None, 0, 0),
              [lambda c, m: lib.clip_grads_list(c, m, ctypes.byref(clip), None)])]
    for make, item, calls in lists:
        arr = (type(item) * 1)(item)
        assert make(ctx, arr, 1, ctypes.byref(out)) == 0
        for call in calls:
            assert call(other, out) == BAD and b"device" in lib.mo_last_error(other)
        lib.mo_list_destroy(out)
    # a list of no tensors, so that nothing is launched
    assert lib.mo_adamw_list(ctx, None, 0, ctypes.byref(out)) == 0
    assert lib.adamw_step_list(other, out, ctypes.byref(cfg), 1, None) == BAD
    assert lib.adamw_step_list(same, out, ctypes.byref(cfg), 1, None) in (0, _lib.MO_ERR_CUDA)   # no GPU here: not refused
    lib.mo_list_destroy(out)
    for c in (other, same):
        lib.mo_ctx_destroy(c)


@pytest.mark.parametrize("how", [copy.copy, copy.deepcopy, pickle.dumps])
def test_a_list_is_not_copied(lib, how):  # noqa: F811
    """Two owners of one handle would free it twice."""
    with pytest.raises(TypeError, match="not copied"):
        how(_context().adamw_tensors([_mat()]))
