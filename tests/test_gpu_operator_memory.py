"""GPU: the memory the norm and embedding calls may touch: operands as columns of wider
buffers, workspaces between guard bytes, and captured calls with workspaces of their own."""

import pytest
import torch

import backward_weight_gradient_amd as F

pytestmark = pytest.mark.gpu


def _say(*a):
    print(*a, flush=True)


def _rand(shape, seed, std, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _ids(n, V, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randint(-1, V + 1, (n,), generator=g, device="cuda")


def _guarded(nbytes):
    buf = torch.full((nbytes + 256,), 0xA5, dtype=torch.uint8, device="cuda")
    return buf, buf[128:128 + nbytes]


def _intact(buf, nbytes):
    return bool((buf[:128] == 0xA5).all()) and bool((buf[128 + nbytes:] == 0xA5).all())


@pytest.mark.parametrize("T", [0, 1, 33, 5000, 8192, 8193, 20000])
@pytest.mark.parametrize("V", [1, 15, 16, 17, 1000])
def test_embedding_workspace(T, V):
    _say(f"case: embedding workspace {T} of {V}")
    K = 24
    ids, dY, nb = _ids(T, V, 1), _rand((T, K), 2, 1.0, torch.bfloat16), F.forge_embed_workspace_bytes(T, V)
    h, W, m = F.hyper("sgdm"), _rand((V, K), 3, 1.0, torch.float32), torch.zeros((V, K), device="cuda")
    buf, ws = _guarded(nb)
    F.forge_embed_accumulate(ids, dY, torch.empty((V, K), device="cuda"), True, workspace=ws)
    assert _intact(buf, nb)
    buf, ws = _guarded(nb)
    F.forge_embed_step(ids, dY, W, F.state(m), None, h, 1, 0, workspace=ws)
    assert _intact(buf, nb)


@pytest.mark.parametrize("rows,cols", [(1, 1), (5, 7), (300, 41), (300, 129), (257, 1001), (1025, 2049), (300, 5003), (300, 16391)])
def test_norm_workspace(rows, cols):
    _say(f"case: norm workspace {rows}x{cols}")
    x, nb = _rand((rows, cols), 4, 1.0, torch.bfloat16), F.forge_rmsnorm_workspace_bytes(rows, cols)
    buf, ws = _guarded(nb)
    gbuf = torch.full((cols + 8,), -3.0, device="cuda")
    rbuf = torch.full((rows + 8,), -3.0, device="cuda")
    one, y = torch.ones(cols, device="cuda"), torch.empty_like(x)
    F.forge_rmsnorm(x, one, y, rstd=rbuf[4:4 + rows])
    F.forge_rmsnorm_backward(y, x, one, rbuf[4:4 + rows], dgamma=gbuf[4:4 + cols], workspace=ws)
    assert _intact(buf, nb)
    for b in (gbuf, rbuf):
        assert bool((b[:4] == -3).all()) and bool((b[-4:] == -3).all()) and bool((b[4:-4] != -3).all())


@pytest.mark.parametrize("state", ["f32", "bf16", "int8"])
@pytest.mark.parametrize("V,K,T", [(130, 131, 200), (300, 256, 9000), (40, 8, 50), (19, 5, 30), (130, 192, 100)])
def test_embedding_step_on_columns_of_wider_buffers(V, K, T, state):
    """W, the moments and dY at odd offsets of buffers full of NaN: the bits of dense operands, and nothing
    beside them is written."""
    if state == "int8" and K % 64:
        K = 128
    _say(f"case: embedding step {T} of {V}x{K} strided {state}")
    ids, dY, W = _ids(T, V, 5), _rand((T, K), 6, 1e-2, torch.bfloat16), _rand((V, K), 7, 1.0, torch.bfloat16)
    if state == "int8":
        g = torch.Generator(device="cuda")
        g.manual_seed(8)
        m = torch.randint(-120, 120, (V, K), generator=g, device="cuda", dtype=torch.int8)
        v = torch.randint(1, 250, (V, K), generator=g, device="cuda", dtype=torch.uint8)
        ms, vs = (torch.rand((V, K // 64), generator=g, device="cuda") * 1e-4 + 1e-6 for _ in range(2))
    else:
        dt = torch.float32 if state == "f32" else torch.bfloat16
        m, v, ms, vs = _rand((V, K), 8, 1e-2, dt), _rand((V, K), 9, 1e-2, torch.float32).square().to(dt), None, None

    def wide(t, off):
        w = torch.full((t.shape[0], t.shape[1] + 11), 77 if not t.is_floating_point() else float("nan"), dtype=t.dtype, device="cuda")
        w[:, off:off + t.shape[1]] = t
        return w, w[:, off:off + t.shape[1]]

    def run(dy, w, a, b):
        sa, sb = (t.clone() if t is not None else None for t in (ms, vs))
        F.forge_embed_step(ids, dy, w, F.state(a, sa, 64 if sa is not None else 0), F.state(b, sb, 64 if sb is not None else 0),
                           F.hyper("adamw"), 3, 11, workspace=torch.empty(F.forge_embed_workspace_bytes(T, V), dtype=torch.uint8,
                                                                         device="cuda"))
        return [t for t in (w, a, b, sa, sb) if t is not None]

    wides = [wide(t, off) for t, off in ((dY, 3), (W, 5), (m, 1), (v, 7))]
    got = run(*(w[1] for w in wides))
    want = run(dY, W.clone(), m.clone(), v.clone())
    for a, b in zip(got, want):
        assert torch.equal(a, b) and not bool(a.float().isnan().any())
    for (buf, _), off in zip(wides[1:], (5, 1, 7)):
        side = torch.cat([buf[:, :off], buf[:, off + K:]], 1)
        assert bool(side.isnan().all()) if buf.is_floating_point() else bool((side == 77).all())


def test_captured_gradients_of_several_parts():
    """Two captured micro-steps (the second adds) of 20000 tokens, their own workspace each, replayed with new
    tokens and eager calls between: every replay gives the eager bits."""
    T, V, K = 20000, 300, 200
    ids, dY = _ids(T, V, 20), _rand((T, K), 21, 1.0, torch.bfloat16)
    acc = [torch.empty((V, K), device="cuda") for _ in range(2)]
    ws = [[torch.empty(F.forge_embed_workspace_bytes(T, V), dtype=torch.uint8, device="cuda") for _ in range(2)] for _ in range(2)]

    def go(a, w):
        F.forge_embed_accumulate(ids, dY, a, True, workspace=w[0])
        F.forge_embed_accumulate(ids, dY, a, False, scale=0.5, workspace=w[1])

    go(acc[1], ws[1])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go(acc[0], ws[0])
    for i in range(4):
        ids.copy_(_ids(T, V if i & 1 else 4, 30 + i))
        dY.mul_(-1.5)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        go(acc[1], ws[1])
        torch.cuda.synchronize()
        assert torch.equal(acc[0], acc[1]), i
