"""GPU: the embedding's lookup, its gradient by sorted tokens and its fused step.

The lookup is one fp32 product and one rounding: bit for bit the oracle's.  The
gradient of a row with n tokens is n fp32 additions and one product: within
(n + 2) 2^-24 of the sum of absolute values.  The step is checked like the linear
layer's: with one-hot rows in dY's place and the token gradients in X's, G = dY^T X
is the embedding's gradient, so the same oracle and tolerances apply.
"""

import numpy as np
import pytest
import torch

import backward_weight_gradient_amd as F
import oracle as O
import synth
from forge_testlib import Layer, assert_ok, check_against_oracle, make_layer, snapshot

pytestmark = pytest.mark.gpu
T = {"f32": torch.float32, "bf16": torch.bfloat16}


def _say(*a):
    print(*a, flush=True)


def _ids(n, V, seed, kind="mixed", dtype=torch.int64):
    """Token ids: uniform, padding among them; 'hot': half of them one id; 'one': all the same."""
    g = torch.Generator()
    g.manual_seed(seed)
    ids = torch.randint(0, V, (n,), generator=g, dtype=torch.int64)
    if kind == "hot":
        ids[torch.rand(n, generator=g) < 0.5] = V // 2
    if kind == "one":
        ids[:] = V - 1
    if kind != "one":
        ids[torch.rand(n, generator=g) < 0.1] = -1
        ids[torch.rand(n, generator=g) < 0.05] = V
        if n > 3:
            ids[3] = 2 ** 31 - 1 if dtype == torch.int32 else 2 ** 40 + 1
    return ids.to(dtype)


def _rand(shape, seed, std, ty):
    g = torch.Generator()
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(T[ty])


def _ws(n, V):
    return torch.full((F.forge_embed_workspace_bytes(n, V),), 0xEE, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("w_ty,y_ty,dtype", [("bf16", "bf16", torch.int64), ("f32", "bf16", torch.int32),
                                             ("bf16", "f32", torch.int32), ("f32", "f32", torch.int64)])
@pytest.mark.parametrize("n,V,K,pad", [(1, 1, 1, 0), (1, 1000, 4096, 0), (37, 50, 129, 1), (300, 7, 8, 0), (5, 9, 5000, 3),
                                       (1025, 300, 256, 2)])
def test_lookup_is_exact(w_ty, y_ty, dtype, n, V, K, pad):
    _say(f"case: embed {n} of {V}x{K} {w_ty} {y_ty}")
    W = _rand((V, K), 1, 0.05, w_ty)
    ids = _ids(n, V, 2, dtype=dtype)
    wide = torch.full((n, K + pad), 9.0, dtype=T[y_ty], device="cuda")
    scale = 1.7
    wv = torch.zeros((V, K + pad), dtype=T[w_ty], device="cuda")
    wv[:, :K] = W.cuda()
    F.forge_embed(ids.cuda(), wv[:, :K], wide[:, :K], scale=scale)
    i = ids.long()
    ok = (i >= 0) & (i < V)
    want = torch.where(ok[:, None], W[i.clamp(0, V - 1)].float() * torch.tensor(scale, dtype=torch.float32),
                       torch.zeros(())).to(T[y_ty])
    assert torch.equal(wide[:, :K].cpu(), want)
    assert bool((wide[:, K:] == 9).all())


@pytest.mark.parametrize("n,V,K,kind", [(0, 5, 8, "mixed"), (1, 1, 1, "one"), (37, 50, 129, "mixed"), (64, 3, 130, "mixed"),
                                        (2047, 100, 64, "hot"), (2049, 5000, 33, "mixed"), (5000, 1000, 257, "hot"),
                                        (20000, 40000, 16, "mixed"), (300, 17, 512, "one"), (16385, 3, 8, "hot")])
@pytest.mark.parametrize("d_ty,dtype", [("bf16", torch.int64), ("f32", torch.int32)])
def test_gradient(n, V, K, kind, d_ty, dtype):
    _say(f"case: embed gradient {n} {V}x{K} {kind} {d_ty}")
    ids, dY = _ids(n, V, 3, kind, dtype), _rand((n, K), 4, 1e-3, d_ty)
    scale = 1.5
    G, A, cnt = O.embed_grad(ids.long().numpy(), dY.double().numpy(), V, scale)
    tol = A * (cnt[:, None] + 3) * 2.0 ** -24 + 1e-38
    acc = torch.full((V, K + 3), 7.0, device="cuda")
    view = acc[:, :K]
    a, d = ids.cuda(), dY.cuda()
    F.forge_embed_accumulate(a, d, view, True, scale=scale, workspace=_ws(n, V))
    first = view.clone()
    assert np.all(np.abs(first.cpu().double().numpy() - G) <= tol)
    # a second micro-batch: one fp32 addition on the rows that occur, the others untouched
    view.copy_(torch.where((torch.from_numpy(cnt) > 0)[:, None].cuda(), view, torch.full_like(view, float("inf"))))
    F.forge_embed_accumulate(a, d, view, False, scale=scale, workspace=_ws(n, V))
    hit = (torch.from_numpy(cnt) > 0).cuda()
    assert torch.equal(view[hit], first[hit] + first[hit])
    assert bool((view[~hit] == float("inf")).all()) and bool((acc[:, K:] == 7).all())
    # the same call twice gives the same bits
    again = torch.empty_like(first)
    F.forge_embed_accumulate(a, d, again, True, scale=scale, workspace=_ws(n, V))
    assert torch.equal(again, first)


def test_strided_gradient_rows():
    ids = _ids(500, 40, 5).cuda()
    wide = _rand((500, 300), 6, 1.0, "bf16").cuda()
    a, b = torch.empty((40, 111), device="cuda"), torch.empty((40, 111), device="cuda")
    F.forge_embed_accumulate(ids, wide[:, 7:118], a, True, workspace=_ws(500, 40))
    F.forge_embed_accumulate(ids, wide[:, 7:118].contiguous(), b, True, workspace=_ws(500, 40))
    assert torch.equal(a, b)


# ---------------------------------------------------------------------------
# The fused step
# ---------------------------------------------------------------------------
def _embed_layer(V, K, n, spec, ids, dY, scale):
    """The linear layer whose weight gradient is the embedding's: dY one-hot [n, V], X = scale dY."""
    L = make_layer(80, V, K, 1, 5, spec)
    one = torch.zeros((n, V), dtype=torch.float32)
    i = ids.long()
    ok = (i >= 0) & (i < V)
    one[torch.arange(n)[ok], i[ok]] = 1
    L.X, L.dY, L.BT = (dY.float() * scale).cuda(), one.cuda(), n
    return L


def _spec(opt, state, w):
    m = None if opt not in F.KEEPS_M else ("s8" if state == "int8" else state)
    v = None if opt not in F.KEEPS_V else ("u8" if state == "int8" else state)
    return synth.LayerSpec("f32", w, m, v, block=64)


@pytest.mark.parametrize("opt,state,w", [("adamw", "f32", "bf16"), ("adamw", "bf16", "f32"), ("adamw", "int8", "bf16"),
                                         ("adamw", "e4m3", "bf16"), ("lion", "bf16", "bf16"), ("sgdm", "f32", "f32"),
                                         ("nadam", "f32", "bf16"), ("radam", "bf16", "bf16"), ("rmsprop", "f32", "bf16"),
                                         ("adagrad", "bf16", "f32"), ("sgd", None, "bf16")])
@pytest.mark.parametrize("n,V,K,kind", [(100, 300, 192, "mixed"), (700, 129, 64, "hot")])
def test_step_matches_the_oracle(opt, state, w, n, V, K, kind):
    _say(f"case: embed step {opt} {state} {w} {n} {V}x{K} {kind}")
    ids, dY = _ids(n, V, 7, kind), _rand((n, K), 8, 1e-3, "bf16")
    scale = 2.0     # a power of two: scale * dY is exact, so the oracle's G has the same terms
    L = _embed_layer(V, K, n, _spec(opt, state, w), ids, dY, scale)
    h = F.hyper(opt, lr=1e-4) if opt == "lion" else F.hyper(opt)
    snap = snapshot(L)
    F.forge_embed_step(ids.cuda(), dY.cuda(), L.W, L.forge_m(), L.forge_v(), h, 5, 99, scale=scale, workspace=_ws(n, V))
    assert_ok(check_against_oracle(snap, L, h, 5, 99))


@pytest.mark.parametrize("n,V,K,d_ty", [(0, 70, 40, "bf16"), (1, 1, 1, "f32"), (50, 130, 131, "bf16"), (2100, 1, 257, "f32"),
                                        (333, 1000, 33, "f32")])
def test_step_ragged(n, V, K, d_ty):
    _say(f"case: embed step ragged {n} {V}x{K} {d_ty}")
    ids, dY = _ids(n, V, 9, dtype=torch.int32), _rand((n, K), 10, 1e-3, d_ty)
    L = _embed_layer(V, K, n, synth.LayerSpec("f32", "bf16", "f32", "f32"), ids, dY, 0.5)
    snap, h = snapshot(L), F.hyper("adamw")
    F.forge_embed_step(ids.cuda(), dY.cuda(), L.W, L.forge_m(), L.forge_v(), h, 5, 99, scale=0.5, workspace=_ws(n, V))
    assert_ok(check_against_oracle(snap, L, h, 5, 99))


def test_step_equals_the_linear_step_without_tokens():
    """No tokens: every row still decays, bit for bit as forge_wgrad_step with BT = 0."""
    L = make_layer(81, 300, 256, 0, 5, synth.LayerSpec("bf16", "bf16", "s8", "u8"))
    P, h = L.clone(), F.hyper("adamw")
    ids = torch.full((40,), -1, dtype=torch.int64, device="cuda")       # padding only
    F.forge_embed_step(ids, torch.full((40, 256), float("nan"), device="cuda"), L.W, L.forge_m(), L.forge_v(), h, 5, 3,
                       workspace=_ws(40, 300))
    F.forge_wgrad_step(P.X, P.dY, P.W, P.forge_m(), P.forge_v(), h, 5, 3)
    for a, b in ((L.W, P.W), (L.m, P.m), (L.v, P.v), (L.ms, P.ms), (L.vs, P.vs)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_tied_embedding_through_the_accumulator():
    """forge_embed_accumulate, then the output layer's step with that accumulator: G is the sum of both uses."""
    V, K, n = 300, 128, 90
    L = make_layer(82, V, K, n, 5, synth.LayerSpec("bf16", "bf16", "f32", "f32"))
    ids, dE = _ids(n, V, 11), _rand((n, K), 12, 1e-3, "bf16")
    acc = torch.empty((V, K), device="cuda")
    F.forge_embed_accumulate(ids.cuda(), dE.cuda(), acc, True, scale=2.0, workspace=_ws(n, V))
    G, _, _ = O.embed_grad(ids.numpy(), dE.double().numpy(), V, 2.0)
    G = G + L.dY.cpu().double().numpy().T @ L.X.cpu().double().numpy()
    h = F.hyper("adamw")
    m0, v0 = L.m.cpu().double().numpy(), L.v.cpu().double().numpy()
    F.forge_wgrad_step_accumulated(L.X, L.dY, acc, L.W, L.forge_m(), L.forge_v(), h, 5, 1)
    bound = 0.1 * 2.0 ** -23 * 200 * (np.abs(L.dY.cpu().double().numpy()).T @ np.abs(L.X.cpu().double().numpy())
                                      + np.abs(G) + 1e-2)
    assert np.all(np.abs(L.m.cpu().double().numpy() - (0.9 * m0 + 0.1 * G)) <= bound)


def test_captured_step_replays_with_new_tokens():
    V, K, n = 500, 128, 300
    L = make_layer(83, V, K, 1, 5, synth.LayerSpec("bf16", "bf16", "f32", "f32"))
    P, h = L.clone(), F.hyper("adamw")
    ids, dY = _ids(n, V, 13).cuda(), _rand((n, K), 14, 1e-3, "bf16").cuda()
    y0, y1 = (torch.empty((n, K), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    w0, w1 = _ws(n, V), _ws(n, V)

    def go(M, y, ws):
        F.forge_embed(ids, M.W, y, scale=3.0)
        F.forge_embed_step(ids, dY, M.W, M.forge_m(), M.forge_v(), h, 5, 2, scale=3.0, workspace=ws)

    warm = P.clone()
    go(warm, y1, w1)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go(L, y0, w0)
    for i in range(4):
        ids.copy_(_ids(n, V, 20 + i, "hot" if i & 1 else "mixed"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        go(P, y1, w1)
        torch.cuda.synchronize()
        assert torch.equal(y0, y1)
        for a, b in ((L.W, P.W), (L.m, P.m), (L.v, P.v)):
            assert torch.equal(a, b), i
