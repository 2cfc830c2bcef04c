"""GPU: the activation-copy, norm and embedding operators as a training step uses them
together, on streams of their own, in two calls at once, and past 2^31 elements.

Tolerances of the whole step (test_training_step).  All values are compared with the
step in fp64 from the same inputs, u = 2^-24 and b = 2^-8 (half a bf16 step):
* H = rn(x + r) is off by b, so s = rstd is off by b and n = h s by 2 b.
* dN = forge_dgrad's bf16 output is off by b of itself and by N u of the sum of
  absolute values.
* dX = s (g - n mean(g n)) + dr: its first product is off by s and g, 2 b; its second
  by s, n, g, n, 6 b; the bf16 store by b: within 7 b of the sum of absolute values,
  7.2 b with the second-order terms and fp32 arithmetic (under 100 u).
* dgamma = sum dN n: 3 b, 3.1 b so.
* the 8-bit copy of y: off by 2^-4 of y, or by half the smallest code 2^-10 2^e with
  2^e < a / 224 for the block's absmax a, and y itself by 2 b.
"""

import numpy as np
import pytest
import torch

import backward_weight_gradient_amd as F
import oracle as O

pytestmark = pytest.mark.gpu
U, B = 2.0 ** -24, 2.0 ** -8


def _say(*a):
    print(*a, flush=True)


def _rand(shape, seed, std, dtype):
    g = torch.Generator()
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype).cuda()


def _np(t):
    return t.cpu().double().numpy()


def _bytes(n):
    return torch.full((n,), 0xEE, dtype=torch.uint8, device="cuda")


class Step:
    """embedding -> residual and norm, kept in 8 bits -> linear layer; then all gradients.
    SGD with momentum from zero, without decay: the new momentum is the gradient."""

    def __init__(self, T, V, K, N, seed):
        g = torch.Generator()
        g.manual_seed(seed)
        self.ids = torch.randint(-1, V, (T,), generator=g).cuda()
        self.E = _rand((V, K), seed + 1, 1.0, torch.bfloat16)
        self.R = _rand((T, K), seed + 2, 1.0, torch.bfloat16)
        self.gamma = 1 + _rand((K,), seed + 3, 0.2, torch.float32)
        self.W = _rand((N, K), seed + 4, 0.05, torch.bfloat16)
        self.dz = _rand((T, N), seed + 5, 1e-2, torch.bfloat16)
        self.dR = _rand((T, K), seed + 6, 1e-2, torch.bfloat16)
        self.h = F.hyper("sgdm", lr=1e-3, beta1=0.9, weight_decay=0.0)
        bf = dict(device="cuda", dtype=torch.bfloat16)
        self.x, self.H, self.Y, self.dN, self.dX = (torch.empty((T, K), **bf) for _ in range(5))
        self.codes = torch.empty((T, K), device="cuda", dtype=torch.float8_e4m3fn)
        self.scale = torch.empty((T, -(-K // 64)), device="cuda", dtype=torch.uint8)
        self.rstd, self.dgamma = torch.empty(T, device="cuda"), torch.empty(K, device="cuda")
        self.mW, self.mE = torch.zeros((N, K), device="cuda"), torch.zeros((V, K), device="cuda")
        self.wn = _bytes(F.forge_rmsnorm_workspace_bytes(T, K))
        self.we = _bytes(F.forge_embed_workspace_bytes(T, V))
        self.start = [t.clone() for t in (self.E, self.W)]

    def reset(self):
        self.E.copy_(self.start[0])
        self.W.copy_(self.start[1])
        self.mW.zero_()
        self.mE.zero_()

    def run(self):
        q = F.act8(self.codes, self.scale, 64)
        F.forge_embed(self.ids, self.E, self.x)
        F.forge_rmsnorm(self.x, self.gamma, self.Y, eps=1e-5, R=self.R, H=self.H, Q=q, rstd=self.rstd)
        F.forge_dgrad(self.dz, self.W, self.dN)
        F.forge_wgrad_step_act8(q, self.dz, self.W, F.state(self.mW), None, self.h, 1, 7)
        F.forge_rmsnorm_backward(self.dN, self.H, self.gamma, self.rstd, self.dX, dR=self.dR, dgamma=self.dgamma,
                                 workspace=self.wn)
        F.forge_embed_step(self.ids, self.dX, self.E, F.state(self.mE), None, self.h, 1, 8, workspace=self.we)

    def results(self):
        return [self.Y, self.scale, self.codes.view(torch.uint8), self.mW, self.dgamma, self.dX, self.mE, self.E, self.W]


@pytest.mark.parametrize("T,V,K,N", [(96, 50, 256, 192), (37, 300, 129, 71), (1, 3, 64, 8), (700, 40, 1024, 520)])
def test_training_step(T, V, K, N):
    _say(f"case: training step {T} tokens, {V} rows, {K} -> {N}")
    s = Step(T, V, K, N, 100)
    s.run()
    ids, E, W = s.ids.cpu().numpy(), _np(s.start[0]), _np(s.start[1])
    R, gamma, dz, dR = _np(s.R), _np(s.gamma), _np(s.dz), _np(s.dR)
    h = O.embed(ids, E, 1.0) + R
    y, rstd = O.rmsnorm(h, gamma, 1e-5)
    dN, dN_abs = dz @ W, np.abs(dz) @ np.abs(W)
    dx, dgamma, dx_abs, dg_abs = O.rmsnorm_backward(dN, h, gamma, rstd, dR)
    # dgrad's fp32 sums enter like an error of g
    more = O.rmsnorm_backward(dN_abs, h, gamma, rstd)
    dx_tol = 7.2 * B * dx_abs + N * U * np.abs(more[2])
    assert np.all(np.abs(_np(s.dX) - dx) <= dx_tol)
    assert np.all(np.abs(_np(s.dgamma) - dgamma) <= 3.1 * B * dg_abs + (N + T) * U * more[3])
    GE, _, cnt = O.embed_grad(ids, dx, V, 1.0)
    tol, _, _ = O.embed_grad(ids, dx_tol, V, 1.0)
    amt, _, _ = O.embed_grad(ids, np.abs(dx) + dx_tol, V, 1.0)
    assert np.all(np.abs(_np(s.mE) - GE) <= tol + (cnt[:, None] + 3) * U * amt)
    blk = np.abs(np.pad(y, ((0, 0), (0, -K % 64))).reshape(T, -1, 64)).max(axis=2)
    a = np.repeat(blk, 64, axis=1)[:, :K] * (1 + 3 * B)
    q_tol = np.abs(y) * ((1 + 2.0 ** -4) * (1 + 2.1 * B) - 1) + 2.0 ** -10 * a / 224
    GW, W_tol = dz.T @ y, np.abs(dz).T @ q_tol
    assert np.all(np.abs(_np(s.mW) - GW) <= W_tol + (T + 2) * U * (np.abs(dz).T @ (np.abs(y) + q_tol)))
    # the steps themselves: w - lr m, rounded once to bf16 (stochastically: less than one step, 2 B)
    for w, m, w0 in ((s.W, s.mW, W), (s.E, s.mE, E)):
        want = w0 - 1e-3 * _np(m)
        assert np.all(np.abs(_np(w) - want) <= 2 * B * np.abs(want) + 2 * U * (np.abs(w0) + np.abs(want)) + 1e-38)


def test_gradients_against_differences_of_the_loss():
    """Along a random direction of (E, gamma, W) the loss sum(z dz) + sum(h dR) changes as the
    gradients say: fp64 central differences (error below 1e-6 of the terms), and the step's
    gradients within the bounds of test_training_step."""
    T, V, K, N = 96, 50, 256, 192
    s = Step(T, V, K, N, 100)
    s.run()
    ids, E, W = s.ids.cpu().numpy(), _np(s.start[0]), _np(s.start[1])
    R, gamma, dz, dR = _np(s.R), _np(s.gamma), _np(s.dz), _np(s.dR)
    rng = np.random.default_rng(5)
    dE, dg, dW = (rng.standard_normal(t.shape) for t in (E, gamma, W))

    def loss(t):
        h = O.embed(ids, E + t * dE, 1.0) + R
        y, _ = O.rmsnorm(h, gamma + t * dg, 1e-5)
        return np.sum((y @ (W + t * dW).T) * dz) + np.sum(h * dR)

    h = O.embed(ids, E, 1.0) + R
    y, rstd = O.rmsnorm(h, gamma, 1e-5)
    dx, dgamma, dx_abs, dg_abs = O.rmsnorm_backward(dz @ W, h, gamma, rstd, dR)
    GE, _, _ = O.embed_grad(ids, dx, V, 1.0)
    GW = dz.T @ y
    exact = np.sum(GE * dE) + np.sum(dgamma * dg) + np.sum(GW * dW)
    size = np.sum(np.abs(GE * dE)) + np.sum(np.abs(dgamma * dg)) + np.sum(np.abs(GW * dW))
    t = 1e-4
    assert abs((loss(t) - loss(-t)) / (2 * t) - exact) <= 1e-6 * size
    more = O.rmsnorm_backward(np.abs(dz) @ np.abs(W), h, gamma, rstd)
    dx_tol = 7.2 * B * dx_abs + N * U * more[2]
    tE, _, cnt = O.embed_grad(ids, dx_tol, V, 1.0)
    a, _, _ = O.embed_grad(ids, np.abs(dx) + dx_tol, V, 1.0)
    tol = np.sum((tE + (cnt[:, None] + 3) * U * a) * np.abs(dE))
    tol += np.sum((3.1 * B * dg_abs + (N + T) * U * more[3]) * np.abs(dg))
    blk = np.repeat(np.abs(y).reshape(T, -1, 64).max(axis=2), 64, axis=1) * (1 + 3 * B)
    q_tol = np.abs(y) * ((1 + 2.0 ** -4) * (1 + 2.1 * B) - 1) + 2.0 ** -10 * blk / 224
    tol += np.sum((np.abs(dz).T @ (q_tol + (T + 2) * U * (np.abs(y) + q_tol))) * np.abs(dW))
    ours = np.sum(_np(s.mE) * dE) + np.sum(_np(s.dgamma) * dg) + np.sum(_np(s.mW) * dW)
    assert abs(ours - exact) <= tol


def test_captured_step_with_two_graphs():
    """Two captured steps with workspaces of their own, replayed in turn and on two streams
    at once, with eager work between: every replay gives the eager bits."""
    a, b = Step(300, 90, 512, 256, 200), Step(300, 90, 512, 256, 300)
    want = []
    for s in (a, b):
        s.run()
        torch.cuda.synchronize()
        want.append([t.clone() for t in s.results()])
    graphs = []
    for s in (a, b):
        s.reset()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.run()
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i in range(4):
        for s in (a, b):
            s.reset()
            for t in s.results()[:6]:
                t.zero_()
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st if i & 1 else torch.cuda.current_stream()):
                g.replay()
        torch.cuda.synchronize()
        for s, w in zip((a, b), want):
            for x, y in zip(s.results(), w):
                assert torch.equal(x, y), i


def test_two_streams_at_once():
    """Eager steps enqueued on two streams without waiting in between: each as if alone."""
    a, b = Step(2000, 500, 1024, 512, 400), Step(1999, 501, 1000, 500, 500)
    want = []
    for s in (a, b):
        s.run()
        torch.cuda.synchronize()
        want.append([t.clone() for t in s.results()])
        s.reset()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for s, st in zip((a, b), streams):
            with torch.cuda.stream(st):
                s.reset()
                s.run()
    torch.cuda.synchronize()
    for s, w in zip((a, b), want):
        for x, y in zip(s.results(), w):
            assert torch.equal(x, y)


# ---------------------------------------------------------------------------
# Offsets past 32 bits.  Buffers are wide or long, the work in them small.
# ---------------------------------------------------------------------------
def test_rows_past_2_31_elements():
    """Matrices whose pitch puts the last rows past 2^31 elements: the same bits as dense ones."""
    T, K, N, pitch = 40, 320, 130, 2 ** 31 // 38 // 8 * 8
    x = _rand((T, K), 1, 1.0, torch.bfloat16)
    far = torch.empty(T * pitch, dtype=torch.bfloat16, device="cuda").view(T, pitch)[:, 64:64 + K]
    far.copy_(x)
    assert (T - 1) * pitch > 2 ** 31
    gamma = torch.ones(K, device="cuda")
    outs = []
    for v in (x, far):
        y, rstd = torch.empty_like(x), torch.empty(T, device="cuda")
        F.forge_rmsnorm(v, gamma, y, rstd=rstd)
        dx, dg = torch.empty_like(x), torch.empty(K, device="cuda")
        F.forge_rmsnorm_backward(v, v, gamma, rstd, dx, dgamma=dg, workspace=_bytes(F.forge_rmsnorm_workspace_bytes(T, K)))
        codes, scale = torch.empty((T, K), dtype=torch.int8, device="cuda"), torch.empty((T, 5), dtype=torch.uint8, device="cuda")
        F.forge_act_quantize(v, F.act8(codes, scale, 64))
        ids = torch.arange(T, device="cuda") // 3
        acc = torch.empty((20, K), device="cuda")
        F.forge_embed_accumulate(ids, v, acc, True, workspace=_bytes(F.forge_embed_workspace_bytes(T, 20)))
        e = torch.empty_like(x)
        F.forge_embed(torch.arange(T - 1, -1, -1, device="cuda"), v, e)
        outs.append((y, rstd, dx, dg, codes, scale, acc, e))
    for p, q in zip(*outs):
        assert torch.equal(p, q)
    codes, scale = outs[0][4], outs[0][5]
    wide = torch.empty(T * pitch, dtype=torch.int8, device="cuda").view(T, pitch)[:, 64:64 + K]
    wide.copy_(codes)
    dY = _rand((T, N), 2, 1e-2, torch.bfloat16)
    accs = []
    for c in (codes, wide):
        q = F.act8(c, scale, 64)
        back, acc = torch.empty_like(x), torch.empty((N, K), device="cuda")
        F.forge_act_dequantize(q, back)
        F.forge_wgrad_accumulate_act8(q, dY, acc, True)
        accs.append((back, acc))
    assert torch.equal(accs[0][0], accs[1][0])
    d, v = _np(dY), _np(accs[0][0])
    for _, acc in accs:
        assert np.all(np.abs(_np(acc) - d.T @ v) <= (T + 2) * U * (np.abs(d).T @ np.abs(v)))


def test_vocabulary_past_2_31_elements():
    """Rows past 2^31 elements of W and of the accumulator."""
    V, K, T = 2 ** 20 + 77, 2056, 200
    W = torch.empty((V, K), dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([V - 1, 0, V - 2, 2 ** 20, V, -1, V - 1] + list(range(V - 193, V)), device="cuda")
    assert ids.numel() == T and (V - 1) * K > 2 ** 31
    rows = _rand((T, K), 3, 1.0, torch.bfloat16)
    ok = (ids >= 0) & (ids < V)
    W[ids[ok]] = rows[ok]
    y = torch.full((T, K), 9.0, dtype=torch.bfloat16, device="cuda")
    F.forge_embed(ids, W, y)
    assert torch.equal(y[ok], W[ids[ok]]) and not bool(y[~ok].any())
    acc = torch.empty((V, K), device="cuda")
    F.forge_embed_accumulate(ids, rows, acc, True, workspace=_bytes(F.forge_embed_workspace_bytes(T, V)))
    want = torch.zeros((T, K), dtype=torch.float64, device="cuda")
    eq = (ids[:, None] == ids[None, :]).double()
    want = eq @ rows.double()
    bound = 4 * U * (eq @ rows.double().abs())
    assert bool(((acc[ids[ok]].double() - want[ok]).abs() <= bound[ok]).all())
    touched = torch.zeros(V, dtype=torch.bool, device="cuda")
    touched[ids[ok]] = True
    assert not bool(acc[~touched][::4099].any())


# ---------------------------------------------------------------------------
# The embedding step's variants: tiles of 16 and 128 rows, whole lines and others
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("V,K", [(40000, 192), (40000, 200), (33000, 257), (70000, 7), (500, 320), (501, 96), (17, 6), (129, 1000)])
@pytest.mark.parametrize("T,d_ty", [(3000, torch.bfloat16), (9000, torch.float32)])
def test_embedding_step_gradient(V, K, T, d_ty):
    """Momentum from zero without decay is the gradient: against fp64, over every row; tokens
    of one and of two sorted parts, half of them one id."""
    _say(f"case: embedding step {T} tokens of {V}x{K}")
    g = torch.Generator()
    g.manual_seed(T)
    ids = torch.randint(-2, V + 2, (T,), generator=g)
    ids[torch.rand(T, generator=g) < 0.5] = V - 1
    ids, dY = ids.cuda(), _rand((T, K), 4, 1e-2, d_ty)
    m, W = torch.zeros((V, K), device="cuda"), _rand((V, K), 5, 1.0, torch.float32)
    w0, h = W.clone(), F.hyper("sgdm", lr=0.5, beta1=0.9, weight_decay=0.0)
    F.forge_embed_step(ids, dY, W, F.state(m), None, h, 1, 0, scale=2.0, workspace=_bytes(F.forge_embed_workspace_bytes(T, V)))
    ok = (ids >= 0) & (ids < V)
    G, A = (torch.zeros((V, K), dtype=torch.float64, device="cuda") for _ in range(2))
    G.index_add_(0, ids[ok], 2 * dY[ok].double())
    A.index_add_(0, ids[ok], 2 * dY[ok].double().abs())
    n = torch.zeros(V, device="cuda", dtype=torch.float64).index_add_(0, ids[ok], torch.ones_like(ids[ok], dtype=torch.float64))
    assert bool(((m.double() - G).abs() <= (n[:, None] + 3) * U * A).all())
    assert bool(((W.double() - (w0.double() - 0.5 * m.double())).abs() <= 2 * U * (w0.abs() + m.abs())).all())


@pytest.mark.parametrize("V,K,block", [(300, 96, 32), (36000, 224, 32), (129, 160, 32), (200, 192, 64)])
@pytest.mark.parametrize("state", ["int8", "e4m3"])
def test_embedding_step_8_bit_states_as_the_linear_step(V, K, block, state):
    """No token at all: the rows decay bit for bit as in forge_wgrad_step with no tokens."""
    m = torch.randint(1, 120, (V, K), device="cuda", dtype=torch.int8)
    v = torch.randint(1, 120, (V, K), device="cuda", dtype=torch.uint8)
    if state == "e4m3":
        m, v = m.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn)
    sm, sv = (torch.rand((V, K // block), device="cuda") * 1e-4 + 1e-6 for _ in range(2))
    W = _rand((V, K), 6, 1.0, torch.bfloat16)
    h, none = F.hyper("adamw"), torch.full((5,), -1, dtype=torch.int32, device="cuda")
    outs = []
    for use in (0, 1):
        w, a, b, c, d = W.clone(), m.clone(), v.clone(), sm.clone(), sv.clone()
        if use:
            F.forge_embed_step(none, torch.zeros((5, K), device="cuda"), w, F.state(a, c, block), F.state(b, d, block), h, 9, 4,
                               workspace=_bytes(F.forge_embed_workspace_bytes(5, V)))
        else:
            F.forge_wgrad_step(torch.zeros((0, K), dtype=torch.bfloat16, device="cuda"),
                               torch.zeros((0, V), dtype=torch.bfloat16, device="cuda"), w, F.state(a, c, block),
                               F.state(b, d, block), h, 9, 4)
        outs.append([t.view(torch.uint8) for t in (w, a, b, c, d)])
    for x, y in zip(*outs):
        assert torch.equal(x, y)
