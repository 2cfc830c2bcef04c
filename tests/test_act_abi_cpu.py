"""Host-only checks of the 8-bit activation, RMSNorm and embedding entry points:
every refusal is made before anything is enqueued (fake device addresses, no
device call)."""

import ctypes

import pytest
import torch

import backward_weight_gradient_amd as F

BASE = 0x7F0000000000
GAP = 1 << 36
S0 = 0   # the null stream: never reached by a refused call


def addr(i):
    return BASE + i * GAP


def mat(i, rows, cols, dt=F.FORGE_BF16, ld=None):
    return F.mat_raw(addr(i), dt, rows, cols, ld)


def act(i, rows, cols, dt=F.FORGE_S8, block=64, ld=None):
    return F.forge_act8(F.mat_raw(addr(i), dt, rows, cols, ld), addr(i) + (1 << 35), block)


def rc(name, *args):
    fn = getattr(F.lib, name)
    conv = [ctypes.byref(a) if isinstance(a, ctypes.Structure) else a for a in args]
    return fn(*conv)


# ---------------------------------------------------------------- 8-bit copies
@pytest.mark.parametrize("name", ["forge_act_quantize", "forge_act_dequantize"])
def test_act_copy_refusals(name):
    def call(X, Q):
        return rc(name, X, Q, S0) if name == "forge_act_quantize" else rc(name, Q, X, S0)
    X, Q = mat(0, 8, 100), act(1, 8, 100)
    assert call(None, Q) == F.FORGE_E_NULL and call(X, None) == F.FORGE_E_NULL
    assert call(F.mat_raw(0, F.FORGE_BF16, 8, 100), Q) == F.FORGE_E_NULL
    assert call(X, F.forge_act8(mat(1, 8, 100, F.FORGE_S8), None, 64)) == F.FORGE_E_NULL
    assert call(X, act(1, 8, 99)) == F.FORGE_E_SHAPE and call(X, act(1, 7, 100)) == F.FORGE_E_SHAPE
    assert call(X, act(1, 8, 100, block=16)) == F.FORGE_E_SHAPE
    assert call(X, act(1, 8, 100, ld=99)) == F.FORGE_E_SHAPE
    assert call(mat(0, 1, 2 ** 31), act(1, 1, 2 ** 31)) == F.FORGE_E_SHAPE
    assert call(mat(0, 8, 100, F.FORGE_S8), Q) == F.FORGE_E_DTYPE
    assert call(X, act(1, 8, 100, F.FORGE_U8)) == F.FORGE_E_DTYPE
    assert call(X, act(1, 8, 100, F.FORGE_BF16)) == F.FORGE_E_DTYPE
    assert call(F.mat_raw(addr(0) + 1, F.FORGE_BF16, 8, 100), Q) == F.FORGE_E_ALIGN
    assert call(F.mat_raw(addr(1) + 100, F.FORGE_BF16, 8, 100), Q) == F.FORGE_E_ALIAS
    over = act(1, 8, 100)
    over.scale = addr(0) + 4
    assert call(X, over) == F.FORGE_E_ALIAS
    # empty: a no-op, nothing to launch
    assert call(mat(0, 0, 100), act(1, 0, 100)) == F.FORGE_OK
    assert call(mat(0, 8, 0), act(1, 8, 0)) == F.FORGE_OK


# ---------------------------------------------------------------- weight gradient
def step_args(BT=64, N=256, K=200, m_dt=F.FORGE_F32, v_dt=F.FORGE_F32, x_dt=F.FORGE_E4M3, block=64):
    X = act(0, BT, K, x_dt, block)
    dY, W = mat(1, BT, N), mat(2, N, K)
    m = F.forge_state(mat(3, N, K, m_dt), None, 0)
    v = F.forge_state(mat(4, N, K, v_dt), None, 0) if v_dt is not None else None
    return [X, dY, W, m, v, F.hyper(), 10]


def test_step_act8_accepts():
    assert F.forge_wgrad_check_act8(*step_args()) == F.FORGE_OK
    assert F.forge_wgrad_check_act8(*step_args(x_dt=F.FORGE_S8, block=128, K=131, N=7)) == F.FORGE_OK
    assert F.forge_wgrad_check_act8(*step_args(m_dt=F.FORGE_BF16, v_dt=F.FORGE_BF16)) == F.FORGE_OK
    a = step_args(v_dt=None)
    for opt in ("lion", "sgdm"):
        a[5] = F.hyper(opt)
        assert F.forge_wgrad_check_act8(*a) == F.FORGE_OK
    # X's block need not be the states'
    a = step_args(K=256, block=32)
    a[3] = F.forge_state(mat(3, 256, 256, F.FORGE_S8), addr(5), 128)
    a[4] = F.forge_state(mat(4, 256, 256, F.FORGE_U8), addr(6), 128)
    assert F.forge_wgrad_check_act8(*a) == F.FORGE_OK


def test_step_act8_refusals():
    def check(i, val, want):
        a = step_args()
        a[i] = val
        assert F.forge_wgrad_check_act8(*a) == want, (i, want)
    check(0, None, F.FORGE_E_NULL)
    check(1, None, F.FORGE_E_NULL)
    check(3, None, F.FORGE_E_NULL)
    check(0, act(0, 63, 200), F.FORGE_E_SHAPE)
    check(0, act(0, 64, 199), F.FORGE_E_SHAPE)
    check(0, act(0, 64, 200, block=48), F.FORGE_E_SHAPE)
    check(0, act(0, 64, 200, F.FORGE_U8), F.FORGE_E_DTYPE)
    check(0, F.forge_act8(mat(0, 64, 200, F.FORGE_S8), None, 64), F.FORGE_E_NULL)
    check(1, mat(1, 64, 256, F.FORGE_F32), F.FORGE_E_DTYPE)
    check(2, mat(2, 256, 200, F.FORGE_E4M3), F.FORGE_E_DTYPE)
    check(5, F.hyper("nadam"), F.FORGE_E_UNSUPPORTED)
    check(5, F.hyper("lion"), F.FORGE_E_UNSUPPORTED)      # v given, Lion keeps none
    check(6, 0, F.FORGE_E_STEP)
    check(2, F.mat_raw(addr(0) + 100, F.FORGE_BF16, 256, 200), F.FORGE_E_ALIAS)          # W over the codes
    check(2, F.mat_raw(addr(0) + (1 << 35), F.FORGE_BF16, 256, 200), F.FORGE_E_ALIAS)    # W over X's scales
    check(3, F.forge_state(mat(2, 256, 200, F.FORGE_F32), None, 0), F.FORGE_E_ALIAS)


def test_accumulate_act8_refusals():
    X, dY, acc = act(0, 64, 200), mat(1, 64, 256), mat(2, 256, 200, F.FORGE_F32)
    f = lambda *a: rc("forge_wgrad_accumulate_act8", *a, 1, S0)
    assert f(None, dY, acc) == F.FORGE_E_NULL and f(X, None, acc) == F.FORGE_E_NULL and f(X, dY, None) == F.FORGE_E_NULL
    assert f(X, mat(1, 64, 256, F.FORGE_F32), acc) == F.FORGE_E_DTYPE
    assert f(X, dY, mat(2, 256, 200)) == F.FORGE_E_DTYPE
    assert f(X, dY, mat(2, 255, 200, F.FORGE_F32)) == F.FORGE_E_SHAPE
    assert f(X, dY, F.mat_raw(addr(0) + (1 << 35), F.FORGE_F32, 256, 200)) == F.FORGE_E_ALIAS
    assert f(act(0, 64, 0), dY, mat(2, 256, 0, F.FORGE_F32)) == F.FORGE_OK


# ---------------------------------------------------------------- RMSNorm
def norm_args(**kw):
    a = dict(X=mat(0, 8, 100), R=mat(1, 8, 100), gamma=mat(2, 1, 100, F.FORGE_F32), eps=1e-5, H=mat(3, 8, 100),
             Y=mat(4, 8, 100), Q=act(5, 8, 100), rstd=addr(6))
    a.update(kw)
    return rc("forge_rmsnorm", *a.values(), S0)


def test_rmsnorm_refusals():
    assert norm_args(X=None) == F.FORGE_E_NULL and norm_args(gamma=None) == F.FORGE_E_NULL
    assert norm_args(R=None) == F.FORGE_E_NULL and norm_args(H=None) == F.FORGE_E_NULL
    assert norm_args(R=None, H=None, Y=None, Q=None, rstd=None) == F.FORGE_E_NULL
    assert norm_args(gamma=mat(2, 1, 99)) == F.FORGE_E_SHAPE and norm_args(gamma=mat(2, 8, 100)) == F.FORGE_E_SHAPE
    assert norm_args(Y=mat(4, 7, 100)) == F.FORGE_E_SHAPE and norm_args(Q=act(5, 8, 99)) == F.FORGE_E_SHAPE
    assert norm_args(X=mat(0, 8, 100, F.FORGE_E4M3)) == F.FORGE_E_DTYPE
    assert norm_args(H=mat(3, 8, 100, F.FORGE_F32)) == F.FORGE_E_DTYPE       # H is stored as R is
    assert norm_args(Y=mat(4, 8, 100, F.FORGE_S8)) == F.FORGE_E_DTYPE
    for eps in (-1e-6, float("nan"), float("inf")):
        assert norm_args(eps=eps) == F.FORGE_E_HYPER
    assert norm_args(rstd=addr(6) + 2) == F.FORGE_E_ALIGN
    assert norm_args(Y=mat(0, 8, 100)) == F.FORGE_E_ALIAS                     # Y is not written in place
    assert norm_args(H=F.mat_raw(addr(1) + 2, F.FORGE_BF16, 8, 100)) == F.FORGE_E_ALIAS
    assert norm_args(H=mat(1, 8, 100, ld=101)) == F.FORGE_E_ALIAS             # R's place, another pitch
    assert norm_args(H=mat(2, 8, 100)) == F.FORGE_E_ALIAS
    assert norm_args(rstd=addr(4)) == F.FORGE_E_ALIAS
    empty = dict(X=mat(0, 0, 100), R=mat(1, 0, 100), H=mat(1, 0, 100), Y=mat(4, 0, 100), Q=act(5, 0, 100))
    assert norm_args(**empty) == F.FORGE_OK


def norm_bwd(**kw):
    a = dict(dY=mat(0, 8, 100), H=mat(1, 8, 100), gamma=mat(2, 1, 100), rstd=addr(3), dR=mat(4, 8, 100), dX=mat(5, 8, 100),
             dgamma=addr(6), first=1, ws=addr(7), bytes=F.forge_rmsnorm_workspace_bytes(8, 100))
    a.update(kw)
    return rc("forge_rmsnorm_backward", *a.values(), S0)


def test_rmsnorm_backward_refusals():
    assert F.forge_rmsnorm_workspace_bytes(8, 100) > 0
    assert F.forge_rmsnorm_workspace_bytes(0, 100) == 0 and F.forge_rmsnorm_workspace_bytes(-1, 4) == 0
    for name in ("dY", "H", "gamma", "rstd"):
        assert norm_bwd(**{name: None}) == F.FORGE_E_NULL
    assert norm_bwd(dX=None, dgamma=None, dR=None) == F.FORGE_E_NULL
    assert norm_bwd(dX=None) == F.FORGE_E_NULL                                # dR without dX
    assert norm_bwd(ws=None) == F.FORGE_E_NULL
    assert norm_bwd(bytes=F.forge_rmsnorm_workspace_bytes(8, 100) - 1) == F.FORGE_E_SHAPE
    assert norm_bwd(bytes=-1) == F.FORGE_E_SHAPE
    assert norm_bwd(ws=addr(7) + 4) == F.FORGE_E_ALIGN and norm_bwd(dgamma=addr(6) + 1) == F.FORGE_E_ALIGN
    assert norm_bwd(dY=mat(0, 8, 99)) == F.FORGE_E_SHAPE and norm_bwd(gamma=mat(2, 1, 101)) == F.FORGE_E_SHAPE
    assert norm_bwd(dR=mat(4, 8, 100, F.FORGE_F32)) == F.FORGE_E_DTYPE        # dX's dtype
    assert norm_bwd(H=mat(1, 8, 100, F.FORGE_S8)) == F.FORGE_E_DTYPE
    assert norm_bwd(dX=mat(1, 8, 100)) == F.FORGE_E_ALIAS                     # H is read again
    assert norm_bwd(dX=F.mat_raw(addr(4) + 2, F.FORGE_BF16, 8, 100)) == F.FORGE_E_ALIAS
    assert norm_bwd(ws=addr(5)) == F.FORGE_E_ALIAS and norm_bwd(dgamma=addr(3)) == F.FORGE_E_ALIAS


# ---------------------------------------------------------------- embedding
def test_embed_refusals():
    def call(ids=addr(0), width=8, T=10, W=mat(1, 50, 100), scale=1.0, Y=mat(2, 10, 100)):
        return rc("forge_embed", ids, width, T, W, scale, Y, S0)
    assert call(ids=None) == F.FORGE_E_NULL and call(W=None) == F.FORGE_E_NULL and call(Y=None) == F.FORGE_E_NULL
    assert call(width=2) == F.FORGE_E_SHAPE and call(T=-1) == F.FORGE_E_SHAPE and call(T=2 ** 31) == F.FORGE_E_SHAPE
    assert call(Y=mat(2, 11, 100)) == F.FORGE_E_SHAPE and call(Y=mat(2, 10, 99)) == F.FORGE_E_SHAPE
    assert call(W=mat(1, 50, 100, F.FORGE_E4M3)) == F.FORGE_E_DTYPE
    assert call(ids=addr(0) + 4) == F.FORGE_E_ALIGN
    for s in (float("nan"), float("inf"), 1e300):
        assert call(scale=s) == F.FORGE_E_HYPER
    assert call(Y=F.mat_raw(addr(1) + 2, F.FORGE_BF16, 10, 100)) == F.FORGE_E_ALIAS
    assert call(ids=addr(2)) == F.FORGE_E_ALIAS
    assert call(T=0, ids=None, Y=mat(2, 0, 100)) == F.FORGE_OK


def embed_grad(name, **kw):
    a = dict(ids=addr(0), width=4, T=10, dY=mat(1, 10, 128), scale=1.0)
    if name == "forge_embed_accumulate":
        a.update(acc=mat(2, 50, 128, F.FORGE_F32), first=0)
    else:
        a.update(W=mat(2, 50, 128), m=F.forge_state(mat(3, 50, 128, F.FORGE_F32), None, 0),
                 v=F.forge_state(mat(4, 50, 128, F.FORGE_F32), None, 0), h=F.hyper(), step=3, seed=1)
    a.update(ws=addr(7), bytes=F.forge_embed_workspace_bytes(10, 50))
    a.update(kw)
    return rc(name, *a.values(), S0)


@pytest.mark.parametrize("name", ["forge_embed_accumulate", "forge_embed_step"])
def test_embed_gradient_refusals(name):
    f = lambda **kw: embed_grad(name, **kw)
    assert f(ids=None) == F.FORGE_E_NULL and f(dY=None) == F.FORGE_E_NULL and f(ws=None) == F.FORGE_E_NULL
    assert f(width=3) == F.FORGE_E_SHAPE and f(T=9) == F.FORGE_E_SHAPE
    assert f(bytes=F.forge_embed_workspace_bytes(10, 50) - 1) == F.FORGE_E_SHAPE
    assert f(dY=mat(1, 10, 127)) == F.FORGE_E_SHAPE
    assert f(T=2 ** 27, dY=mat(1, 2 ** 27, 128), bytes=1 << 34) == F.FORGE_E_SHAPE
    assert f(dY=mat(1, 10, 128, F.FORGE_S8)) == F.FORGE_E_DTYPE
    assert f(ws=addr(7) + 8) == F.FORGE_E_ALIGN and f(ids=addr(0) + 2) == F.FORGE_E_ALIGN
    assert f(scale=float("inf")) == F.FORGE_E_HYPER
    assert f(ws=addr(2)) == F.FORGE_E_ALIAS and f(ws=addr(0)) == F.FORGE_E_ALIAS and f(dY=mat(2, 10, 128)) == F.FORGE_E_ALIAS
    if name == "forge_embed_accumulate":
        assert f(acc=None) == F.FORGE_E_NULL and f(acc=mat(2, 50, 128)) == F.FORGE_E_DTYPE
        assert f(acc=mat(2, 0, 128, F.FORGE_F32), ws=None, bytes=0) == F.FORGE_OK
    else:
        assert f(W=None) == F.FORGE_E_NULL and f(m=None) == F.FORGE_E_NULL and f(h=None) == F.FORGE_E_NULL
        assert f(step=0) == F.FORGE_E_STEP
        V = 2 ** 28 - 15     # ceil(V / 16) = 2^24 tiles: one too many
        big = lambda i, dt=F.FORGE_BF16: mat(i, V, 8, dt)
        assert f(dY=mat(1, 10, 8), W=big(2), m=F.forge_state(big(3), None, 0), v=F.forge_state(big(4), None, 0),
                 bytes=1 << 34) == F.FORGE_E_SHAPE
        assert f(W=mat(2, 50, 128, F.FORGE_E4M3)) == F.FORGE_E_DTYPE
        assert f(m=F.forge_state(mat(3, 50, 127, F.FORGE_F32), None, 0)) == F.FORGE_E_SHAPE
        assert f(h=F.hyper("lion")) == F.FORGE_E_UNSUPPORTED
        assert f(m=F.forge_state(mat(2, 50, 128, F.FORGE_F32), None, 0)) == F.FORGE_E_ALIAS


def test_embed_workspace_bytes():
    b = F.forge_embed_workspace_bytes
    assert b(10, 0) == 0 and b(-1, 5) == 0 and b(2 ** 27, 5) == 0
    assert b(0, 5) > 0 and b(1000, 5) > b(10, 5) and b(10, 128256) > b(10, 5)


# ---------------------------------------------------------------- binding
def test_binding_checks_its_tensors():
    codes, scale = torch.zeros(4, 100, dtype=torch.int8), torch.zeros(4, 2, dtype=torch.uint8)
    assert F.act8(codes, scale, 64).block == 64
    for args in ((codes, scale, 32), (codes, scale, 48), (codes, scale.int(), 64), (codes, torch.zeros(2, 4, dtype=torch.uint8).t(), 64)):
        with pytest.raises(ValueError):
            F.act8(*args)
    x, g = torch.zeros(4, 100), torch.zeros(100)
    with pytest.raises(ValueError):
        F.forge_rmsnorm(x, g, x.clone(), rstd=torch.zeros(3), stream=0)
    with pytest.raises(ValueError):
        F.forge_rmsnorm(x, torch.zeros(200)[::2], x.clone(), stream=0)
    with pytest.raises(ValueError):
        F.forge_rmsnorm_backward(x, x, g, torch.zeros(4), x.clone(), dgamma=torch.zeros(99), stream=0)
    with pytest.raises(ValueError):
        F.forge_embed(torch.zeros(4, dtype=torch.int16), x, x.clone(), stream=0)
    with pytest.raises(ValueError):
        F.forge_embed(torch.zeros(8, dtype=torch.int64)[::2], x, x.clone(), stream=0)
    with pytest.raises(ValueError):   # two devices in one call
        F.forge_rmsnorm(x, g.to("meta"), x.clone(), stream=0)
    with pytest.raises(F.ForgeError):
        F.forge_act_quantize(mat(0, 3, 100), act(1, 4, 100), stream=0)


def test_binding_refuses_host_tensors():
    """An address of host memory would fault in a kernel: tensors that are not on a GPU are refused before the call."""
    x, g, ids = torch.zeros(4, 64), torch.ones(64), torch.zeros(4, dtype=torch.int64)
    q = F.act8(torch.zeros((4, 64), dtype=torch.int8), torch.zeros((4, 1), dtype=torch.uint8), 64)
    st, h = F.state(torch.zeros(4, 64)), F.hyper("sgdm")
    ws = torch.zeros(F.forge_embed_workspace_bytes(4, 4), dtype=torch.uint8)
    raw = mat(0, 4, 64, F.FORGE_F32)
    for call in (lambda: F.forge_act_quantize(x, q), lambda: F.forge_act_dequantize(q, raw),
                 lambda: F.forge_wgrad_step_act8(q, raw, raw, st, None, h, 1, 0),
                 lambda: F.forge_wgrad_accumulate_act8(q, raw, raw, True), lambda: F.forge_rmsnorm(x, g, torch.empty_like(x)),
                 lambda: F.forge_rmsnorm(raw, mat(1, 1, 64), Q=q), lambda: F.forge_embed(ids, raw, raw),
                 lambda: F.forge_rmsnorm_backward(x, x, g, torch.ones(4), torch.empty_like(x)),
                 lambda: F.forge_embed_accumulate(ids, raw, raw, True, workspace=ws),
                 lambda: F.forge_embed_step(ids, raw, raw, st, None, h, 1, 0, workspace=ws)):
        with pytest.raises(ValueError, match="expected a GPU"):
            call()
