"""nucleus_project's host side: bad arguments are refused before anything is
launched (the addresses below are never dereferenced), and the binding's
checks of tensors."""
import ctypes

import pytest
import torch

EINVAL = -1
H, W, O = 1 << 40, 1 << 41, 1 << 42  # far apart: no operand meets another


@pytest.fixture(scope="module")
def L():
    import nucleus_sampling_amd as ns

    return ns.lib()


def _opt(**kw):
    import nucleus_sampling_amd as ns

    o = ns._ProjectOptions()
    for k, v in kw.items():
        setattr(o, k, v)
    return ctypes.byref(o)


def _call(L, h=H, w=W, M=3, N=8, K=16, out=O, opt=None):
    return L.nucleus_project(h, w, M, N, K, out, opt)


def test_host_side_argument_errors(L):
    for kw in (dict(h=None), dict(w=None), dict(out=None), dict(M=-1), dict(N=-1), dict(K=0), dict(K=-4),
               dict(M=1 << 31), dict(N=1 << 31), dict(K=1 << 31), dict(h=H + 2), dict(w=W + 1), dict(out=O + 2)):
        assert _call(L, **kw) == EINVAL, kw
    bad = (dict(dtype=3), dict(dtype=-1), dict(out_dtype=1), dict(dtype=1, out_dtype=2), dict(activation=5),
           dict(activation=-1), dict(activation=4), dict(activation=4, softcap=-1.0),
           dict(activation=4, softcap=float("inf")), dict(activation=4, softcap=float("nan")),
           dict(bias=1 << 43, bias_dtype=1), dict(bias=(1 << 43) + 2), dict(residual=1 << 43, residual_dtype=2),
           dict(residual=(1 << 43) + 1), dict(hidden_stride=15), dict(weight_stride=15), dict(out_stride=7),
           dict(residual_stride=7), dict(hidden_stride=-16), dict(hidden_stride=1 << 31), dict(out_stride=1 << 31))
    for kw in bad:
        assert _call(L, opt=_opt(**kw)) == EINVAL, kw


def test_overlapping_operands_are_refused(L):
    assert _call(L, out=H) == EINVAL
    assert _call(L, out=W + 4) == EINVAL
    assert _call(L, out=H + 4 * 16 * 3 - 4) == EINVAL       # the last element of hidden
    assert _call(L, opt=_opt(bias=O + 4)) == EINVAL
    assert _call(L, opt=_opt(residual=O + 32)) == EINVAL    # the residual, but not the same matrix
    assert _call(L, opt=_opt(residual=O, residual_stride=16)) == EINVAL
    assert _call(L, opt=_opt(dtype=1, residual=O, residual_dtype=1)) == EINVAL  # the same place in another type


def test_empty_products_launch_nothing(L):
    assert _call(L, M=0) == 0 and _call(L, N=0) == 0
    assert _call(L, M=0, h=None, w=None, out=None) == 0


def test_too_many_tiles_are_refused_before_the_device_is_touched(L):
    rc = _call(L, M=(1 << 31) - 1, N=(1 << 31) - 1, K=1, h=1 << 50, w=1 << 56, out=1 << 57)
    assert rc in (EINVAL, -4)  # (no usable device here)


def test_binding_refuses_what_it_cannot_take():
    import nucleus_sampling_amd as ns

    a, b = torch.zeros(2, 8), torch.zeros(4, 8)
    with pytest.raises(ns.NucleusError):
        ns.project(a, b)  # no CPU path
    with pytest.raises(ValueError):
        ns.project(a, b, activation="tanh")
    with pytest.raises(TypeError):
        ns.project(a.double(), b.double())
    with pytest.raises(TypeError):
        ns.project(a, b.half())
    with pytest.raises(ns.NucleusError, match="inference"):
        ns.project(a, b.requires_grad_())
