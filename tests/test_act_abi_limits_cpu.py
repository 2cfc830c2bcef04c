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


# ---------------------------------------------------------------- the states' memory
def _on(index, t):
    """t as if it were on GPU `index`."""
    class Placed(torch.Tensor):
        def get_device(self):
            return index
    return t.as_subclass(Placed)


def _steps(m, v, h):
    """The two steps with every operand but the states given by address."""
    raw = mat(0, 4, 64, F.FORGE_F32)
    q = F.forge_act8(mat(1, 4, 64, F.FORGE_S8), addr(2), 64)
    yield lambda: F.forge_wgrad_step_act8(q, mat(3, 4, 4), raw, m, v, h, 1, 0, stream=S0)
    yield lambda: F.forge_embed_step(_on(0, torch.zeros(4, dtype=torch.int64)), raw, mat(4, 4, 64), m, v, h, 1, 0, stream=S0)


@pytest.mark.parametrize("host", ["m", "v", "codes"])
def test_states_on_the_host_are_refused(host):
    """A state's host address would be read and written by the kernel."""
    t, gpu = torch.zeros(4, 64), _on(0, torch.zeros(4, 64))
    if host == "codes":
        m = F.state(torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4, 1), 64)
        v = F.state(torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 1), 64)
    else:
        m, v = F.state(t if host == "m" else gpu), F.state(t if host == "v" else gpu)
    for call in _steps(m, v, F.hyper()):
        with pytest.raises(ValueError, match="expected a GPU"):
            call()


def test_states_on_another_gpu_are_refused():
    m, v = (F.state(_on(i, torch.zeros(4, 64))) for i in (0, 1))
    for call in _steps(m, v, F.hyper()):
        with pytest.raises(ValueError, match="cuda:0 and cuda:1"):
            call()


def test_a_state_keeps_its_tensors():
    q, s = torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4, 1)
    assert F.state(q, s, 64).tensors[0] is q and F.state(q, s, 64).tensors[1] is s
    assert F.state(s).tensors[0] is s


# ---------------------------------------------------------------- embedding
def embed_accumulate(T, V, K=8):
    return rc("forge_embed_accumulate", addr(0), 8, T, mat(1, T, K), 1.0, mat(2, V, K, F.FORGE_F32), 1, addr(7), 1 << 36, S0)


def test_embedding_gradient_token_limit():
    """2^24 tokens: the sort's launch, with its clearing workgroups, stays below 2^32 threads
    (checked where it is compiled) and its cost, quadratic in the end, below a second."""
    for V in (1, 1000, 2 ** 31 - 2):
        assert F.forge_embed_workspace_bytes(2 ** 24 - 1, V) > 0 and F.forge_embed_workspace_bytes(2 ** 24, V) == 0
        assert embed_accumulate(2 ** 24, V, 1) == F.FORGE_E_SHAPE
        assert embed_accumulate(2 ** 27 - 1, V, 1) == F.FORGE_E_SHAPE


# ---------------------------------------------------------------- launch sizes
@pytest.mark.parametrize("N,K", [(1, 2 ** 31 - 1), (2 ** 31 - 1, 2), (2, 2 ** 31 - 127)])
def test_layers_of_2_24_tiles_are_refused(N, K):
    """2^24 workgroups of 256 threads are 2^32, more than a launch takes."""
    X, X8 = mat(0, 4, K), F.forge_act8(mat(0, 4, K, F.FORGE_S8), addr(9), 32)
    dY, W, m, v = mat(1, 4, N), mat(2, N, K), *(F.forge_state(mat(i, N, K, F.FORGE_F32), None, 0) for i in (3, 4))
    assert F.forge_wgrad_check(X, dY, W, m, v, F.hyper(), 1) == F.FORGE_E_SHAPE
    assert F.forge_wgrad_check_act8(X8, dY, W, m, v, F.hyper(), 1) == F.FORGE_E_SHAPE
    acc = mat(5, N, K, F.FORGE_F32)
    assert rc("forge_wgrad_accumulate", X, dY, acc, 1, S0) == F.FORGE_E_SHAPE
    assert rc("forge_wgrad_accumulate_act8", X8, dY, acc, 1, S0) == F.FORGE_E_SHAPE


@pytest.mark.parametrize("N,K", [(1, 2 ** 31 - 128), (2 ** 31 - 128, 2), (2 ** 16 - 1, 2 ** 16)])
def test_layers_of_fewer_tiles_are_accepted(N, K):
    X, X8 = mat(0, 4, K), F.forge_act8(mat(0, 4, K, F.FORGE_S8), addr(9), 32)
    dY, W, m, v = mat(1, 4, N), mat(2, N, K), *(F.forge_state(mat(i, N, K, F.FORGE_F32), None, 0) for i in (3, 4))
    assert F.forge_wgrad_check(X, dY, W, m, v, F.hyper(), 1) == F.FORGE_OK
    assert F.forge_wgrad_check_act8(X8, dY, W, m, v, F.hyper(), 1) == F.FORGE_OK


def test_embedding_gradient_takes_every_vocabulary_below_2_31():
    V = 2 ** 31 - 1
    assert F.forge_embed_workspace_bytes(10, V) > 0 and F.forge_embed_workspace_bytes(10, V + 1) == 0
    assert embed_accumulate(10, V + 1, 1) == F.FORGE_E_SHAPE
    ws = F.forge_embed_workspace_bytes(10, V)
    small = rc("forge_embed_accumulate", addr(0), 8, 10, mat(1, 10, 1), 1.0, mat(2, V, 1, F.FORGE_F32), 1, addr(7) + 8, ws, S0)
    assert small == F.FORGE_E_ALIGN        # the sizes passed
