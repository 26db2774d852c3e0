"""Refusals and host-side rules of the AdamW, 8-bit-moment and clipping calls
that test_adamw_abi.py leaves open; none needs a GPU."""
import ctypes

import pytest
from test_adamw_abi import BAD, _cfg, _step, _tensor, _tensor8, ctx, lib  # noqa: F401

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
