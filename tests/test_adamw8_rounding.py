"""Which rounding the 8-bit calls of the binding ask the library for (host only)."""
import pytest
from test_adamw_abi import _context, _mat8, lib  # noqa: F401

import matrix_aware_optimizers_muon_b200 as mo


@pytest.fixture
def calls(lib, monkeypatch):  # noqa: F811
    c, seen = _context(), []

    class Lib:
        def __getattr__(self, name):
            if name in ("adamw8_step_list", "adamw8_pack_list"):
                return lambda h, lst, cfg, *rest: seen.append((cfg.stochastic, cfg.seed)) or 0
            return getattr(lib, name)
    c.lib = Lib()
    monkeypatch.setattr(c, "_raw_stream", lambda s: None)
    monkeypatch.setattr(mo.Context, "_warned", False)
    return c, seen


def test_step(calls):
    c, seen = calls
    lst = c.adamw8_tensors([_mat8()])
    c.adamw8_step(lst, 1)
    c.adamw8_step(lst, 1, noise=7)
    c.adamw8_step(lst, 1, noise=None)
    c.adamw8_step(lst, 1, seed=None)
    with pytest.warns(UserWarning, match="noise="):
        c.adamw8_step(lst, 1, seed=0)
    c.adamw8_step(lst, 1, seed=7)
    assert seen == [(1, 0), (1, 7), (0, 0), (0, 0), (2, 0), (2, 7)]
    for kw in (dict(noise=1, seed=2), dict(noise=None, seed=2), dict(noise=1, seed=None)):
        with pytest.raises(ValueError, match="noise and seed"):
            c.adamw8_step(lst, 1, **kw)
    assert len(seen) == 6


def test_pack(calls):
    import torch
    from test_adamw_abi import _Dev
    c, seen = calls
    mom = {k: v for k, v in _mat8(M=_Dev(300, torch.float32), V=_Dev(300, torch.float32)).items() if k not in "WG"}
    lst = c.adamw8_moments([mom])
    c.adamw8_pack(lst)
    c.adamw8_pack(lst, noise=0)
    c.adamw8_pack(lst, seed=0)
    c.adamw8_pack(lst, noise=3)
    c.adamw8_pack(lst, seed=3)
    assert seen == [(0, 0), (1, 0), (2, 0), (1, 3), (2, 3)]
    with pytest.raises(ValueError, match="noise and seed"):
        c.adamw8_pack(lst, noise=1, seed=1)


def test_both_given(calls):
    """A noise of 0 that the caller wrote is not the default: with seed=None beside it the call would not know which is meant."""
    c, seen = calls
    lst = c.adamw8_tensors([_mat8()])
    for kw in (dict(noise=0, seed=None), dict(noise=0, seed=0), dict(noise=None, seed=None)):
        with pytest.raises(ValueError, match="noise and seed"):
            c.adamw8_step(lst, 1, **kw)
    assert not seen
