"""Host-only checks of the limits of the 8-bit activation, RMSNorm and embedding entry
points: what their documentation allows is accepted, what the kernels cannot take is
refused before anything is enqueued (fake device addresses, no device call)."""

import ctypes

import pytest
import torch

import backward_weight_gradient_amd as F

BASE = 0x7F0000000000
GAP = 1 << 38
S0 = 0   # the null stream: never reached by a refused call


def addr(i):
    return BASE + i * GAP


def mat(i, rows, cols, dt=F.FORGE_BF16, ld=None):
    return F.mat_raw(addr(i), dt, rows, cols, ld)


def rc(name, *args):
    conv = [ctypes.byref(a) if isinstance(a, ctypes.Structure) else a for a in args]
    return getattr(F.lib, name)(*conv)


# ---------------------------------------------------------------- RMSNorm
def norm(eps, rows=8):
    return rc("forge_rmsnorm", mat(0, rows, 100), None, mat(1, 1, 100), eps, None, mat(2, rows, 100), None, None, S0)


@pytest.mark.parametrize("eps", [3.5e38, 1e300, 1e-50, 5e-324, 2.0 ** -150])
def test_rmsnorm_eps_outside_fp32(eps):
    """The kernels add eps in fp32: infinite there it would make Y = 0, and a positive eps that
    becomes 0 would make a row of zeros NaN."""
    assert norm(eps) == F.FORGE_E_HYPER


@pytest.mark.parametrize("eps", [0.0, 2.0 ** -149, 1e-5, 1.0, 3.4e38])
def test_rmsnorm_eps_inside_fp32(eps):
    assert norm(eps, rows=0) == F.FORGE_OK
