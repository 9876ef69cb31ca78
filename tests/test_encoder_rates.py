"""Rates of the optimiser and the norm's eps that are not numbers are refused by the C ABI before any device work (fake
pointers, never dereferenced)."""
import math

import numpy as np
import pytest

from late_interaction_retrieval_amd import binding as bd

SHAPE = 2
P = 0x10000


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("rate", ["lr", "weight_decay", "beta1", "beta2"])
def test_rates(rate, value):
    t = np.zeros(1, bd._TENSOR)
    for f in ("param", "grad", "m", "v"):
        t[f] = P
    t["n"] = 5
    a = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.0)
    a[rate] = value
    assert bd.lib().maxsim_adamw(t.ctypes.data, 1, bd.MAXSIM_F32, bd.MAXSIM_F32, bd.MAXSIM_F32, *a.values(), 1, None,
                                 None) == SHAPE


@pytest.mark.parametrize("value", [math.nan, -1.0, -math.inf])
def test_eps(value):
    t = np.zeros(1, bd._TENSOR)
    for f in ("param", "grad", "m", "v"):
        t[f] = P
    t["n"] = 5
    lib = bd.lib()
    assert lib.maxsim_adamw(t.ctypes.data, 1, 2, 2, 2, 1e-3, 0.9, 0.99, value, 0.0, 1, None, None) == SHAPE
    assert lib.maxsim_rmsnorm_fwd(P, 64, None, 0, None, 2, 3, 64, 2, value, 2, P, 64, None, None, 0, None, None) == SHAPE
