"""GPU: RMSNorm with the residual's addition and 8-bit output, and its backward
pass, against the oracle in fp64.

Tolerances.  u = 2^-24.  A row's sum of squares is a sum of d <= 80 + K / 1024
sequential fp32 additions per path (a lane's values, then the lanes; rows past
16384 columns K / 1024 per lane), all terms positive, so its relative error is at
most (d + 1) u; s = 1 / sqrt(that / K + eps) halves it and adds a division, an
addition, a root and a reciprocal, 4 u.  y adds two multiplications.  A bf16
store adds 2^-8 of the value.  dx and dgamma are sums with signs: the same counts
against the sums of absolute values.
"""

import numpy as np
import pytest
import torch

import backward_weight_gradient_amd as F
import oracle as O

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
T = {"f32": torch.float32, "bf16": torch.bfloat16}
CODE = {"s8": torch.int8, "e4m3": torch.float8_e4m3fn}


def _say(*a):
    print(*a, flush=True)


def _d(K):
    return 80 + K / 1024


def _half(t):
    return {"f32": 0.0, "bf16": 2.0 ** -8}[t]     # fp32 results: counted in the arithmetic


def _rand(shape, seed, std, ty):
    g = torch.Generator()
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(T[ty])


def _wide(t, pad):
    """t as the columns of a wider buffer (filled with -3), at an odd offset when pad is odd."""
    w = torch.full((t.shape[0], t.shape[1] + 2 * pad), -3.0, dtype=t.dtype, device="cuda")
    v = w[:, pad:pad + t.shape[1]]
    v.copy_(t)
    return w, v


SHAPES = [(1, 1), (1, 4096), (3, 8), (70, 128), (5, 129), (33, 512), (9, 1000), (6, 1024), (4, 2048), (1030, 96),
          (2100, 256), (5, 4097), (3, 8192), (2, 8200), (3, 16384), (2, 16391), (2, 40000)]


@pytest.mark.parametrize("x_ty,r_ty,y_ty,g_ty", [("bf16", None, "bf16", "f32"), ("f32", None, "f32", "bf16"),
                                                 ("bf16", "bf16", "bf16", "bf16"), ("bf16", "f32", "f32", "f32"),
                                                 ("f32", "bf16", "bf16", "f32"), ("f32", "f32", "f32", "f32")])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward(rows, cols, x_ty, r_ty, y_ty, g_ty):
    _say(f"case: rmsnorm {rows}x{cols} {x_ty} {r_ty} {y_ty} {g_ty}")
    pad = (rows + cols) % 3
    eps = 1e-5
    x, gamma = _rand((rows, cols), 1, 1.5, x_ty), 1 + _rand((cols,), 2, 0.2, g_ty)
    gamma = gamma.to(T[g_ty])
    _, xv = _wide(x, pad)
    yw, yv = _wide(torch.zeros((rows, cols), dtype=T[y_ty]), pad)
    rstd = torch.empty(rows, device="cuda")
    if r_ty:
        r = _rand((rows, cols), 3, 2.0, r_ty)
        _, rv = _wide(r, pad)
        hw, hv = _wide(torch.zeros((rows, cols), dtype=T[r_ty]), pad)
        h = (x.float() + r.float()).to(T[r_ty])       # fp32 sum, one rounding
    else:
        rv = hv = hw = None
        h = x
    F.forge_rmsnorm(xv, gamma.cuda(), yv, eps=eps, R=rv, H=hv, rstd=rstd)
    if r_ty:
        assert torch.equal(hv.cpu(), h)
        assert bool((hw[:, :pad] == -3).all()) and bool((hw[:, pad + cols:] == -3).all())
    y, s = O.rmsnorm(h.double().numpy(), gamma.double().numpy(), eps)
    tol = (0.5 * (_d(cols) + 1) + 4) * U
    assert np.all(np.abs(rstd.cpu().double().numpy() - s) <= s * tol)
    got = yv.cpu().double().numpy()
    assert np.all(np.abs(got - y) <= np.abs(y) * ((tol + 2 * U) * (1 + 2.0 ** -7) + _half(y_ty)) + 1e-38)
    assert bool((yw[:, :pad] == -3).all()) and bool((yw[:, pad + cols:] == -3).all())


@pytest.mark.parametrize("fmt", ["s8", "e4m3"])
@pytest.mark.parametrize("block", [32, 64, 128])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 8), (70, 128), (5, 130), (9, 1000), (4, 2048), (7, 4096), (5, 4097),
                                       (2, 9000), (2, 16391)])
def test_eight_bit_output(fmt, block, rows, cols):
    """Q is the copy of the fp32 output: bit for bit that of Y when Y is fp32, and
    the same Q when Y is bf16 or absent."""
    _say(f"case: rmsnorm 8-bit {fmt} {block} {rows}x{cols}")
    x, gamma = _rand((rows, cols), 4, 1.0, "bf16").cuda(), 1 + _rand((cols,), 5, 0.5, "f32").cuda()
    x[0] = 0
    outs = []
    for y_ty in ("f32", "bf16", None):
        y = torch.empty((rows, cols), dtype=T[y_ty], device="cuda") if y_ty else None
        codes = torch.zeros((rows, cols + 3), dtype=torch.uint8, device="cuda")
        scale = torch.zeros((rows, -(-cols // block)), dtype=torch.uint8, device="cuda")
        F.forge_rmsnorm(x, gamma, y, Q=F.act8(codes[:, :cols].view(CODE[fmt]), scale, block))
        assert not bool(codes[:, cols:].any())
        outs.append((y, codes[:, :cols].cpu().contiguous(), scale.cpu()))
    ref_c, ref_s = O.act8_encode(outs[0][0].cpu().numpy(), fmt, block)
    np.testing.assert_array_equal(outs[0][2].numpy(), ref_s)
    np.testing.assert_array_equal(outs[0][1].view(torch.int8).numpy().view(ref_c.dtype), ref_c)
    for _, c, s in outs[1:]:
        assert torch.equal(c, outs[0][1]) and torch.equal(s, outs[0][2])


def test_non_finite_rows_stay_in_their_rows():
    x = _rand((6, 200), 6, 1.0, "f32").cuda()
    x[1, 7], x[3, 199], x[4] = float("nan"), float("inf"), 0.0
    y = torch.empty_like(x)
    codes, scale = torch.empty((6, 200), dtype=torch.int8, device="cuda"), torch.empty((6, 4), dtype=torch.uint8, device="cuda")
    F.forge_rmsnorm(x, torch.ones(200, device="cuda"), y, Q=F.act8(codes, scale, 64))
    assert bool(y[1].isnan().all()) and bool((scale[1] == 255).all())
    # an infinity: s = 0, so finite values become 0 and the infinity itself NaN, as the formula gives
    assert bool(y[3, 199].isnan()) and bool((y[3, :199] == 0).all()) and scale[3].tolist() == [7, 7, 7, 255]
    assert bool((y[4] == 0).all())
    for r in (0, 2, 5):
        assert bool(y[r].isfinite().all())


def test_forward_in_place_and_partial_outputs():
    """H in R's or X's place; H alone; rstd alone."""
    x, r, gamma = _rand((37, 768), 7, 1.0, "bf16").cuda(), _rand((37, 768), 8, 1.0, "bf16").cuda(), \
        torch.ones(768, device="cuda")
    want_h, y0, y1 = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    rstd = torch.empty(37, device="cuda")
    F.forge_rmsnorm(x, gamma, y0, R=r, H=want_h, rstd=rstd)
    h = r.clone()
    F.forge_rmsnorm(x, gamma, y1, R=h, H=h)
    assert torch.equal(h, want_h) and torch.equal(y0, y1)
    h = x.clone()
    F.forge_rmsnorm(h, gamma, y1, R=r, H=h)
    assert torch.equal(h, want_h) and torch.equal(y0, y1)
    h, s = torch.empty_like(x), torch.empty_like(rstd)
    F.forge_rmsnorm(x, gamma, None, R=r, H=h, rstd=s)
    assert torch.equal(h, want_h) and torch.equal(s, rstd)
    xl = _rand((3, 20000), 9, 1.0, "f32").cuda()
    gl, hl, yl = torch.ones(20000, device="cuda"), torch.empty_like(xl), torch.empty_like(xl)
    F.forge_rmsnorm(xl, gl, yl, R=xl.clone(), H=hl)
    xx, y2 = xl.clone(), torch.empty_like(xl)
    F.forge_rmsnorm(xx, gl, y2, R=xl.clone(), H=xx)
    assert torch.equal(xx, hl) and torch.equal(y2, yl)


@pytest.mark.parametrize("h_ty,d_ty,g_ty,res", [("bf16", "bf16", "f32", True), ("f32", "bf16", "bf16", False),
                                                ("f32", "f32", "f32", True), ("bf16", "f32", "bf16", False)])
@pytest.mark.parametrize("rows,cols", SHAPES + [(3000, 64), (700, 1000)])
def test_backward(rows, cols, h_ty, d_ty, g_ty, res):
    _say(f"case: rmsnorm backward {rows}x{cols} {h_ty} {d_ty} {g_ty} {res}")
    pad = (rows + cols) % 3
    h, dy = _rand((rows, cols), 10, 1.5, h_ty), _rand((rows, cols), 11, 1e-3, d_ty)
    gamma = (1 + _rand((cols,), 12, 0.2, "f32")).to(T[g_ty])
    rstd = (1.0 / torch.sqrt(h.double().square().mean(1) + 1e-5)).float()
    dr = _rand((rows, cols), 13, 1e-3, h_ty) if res else None
    hv, dyv = _wide(h, pad)[1], _wide(dy, pad)[1]
    drv = _wide(dr, pad)[1] if res else None
    dxw, dxv = _wide(torch.zeros((rows, cols), dtype=T[h_ty]), pad)
    dg = torch.full((cols,), float("nan"), device="cuda")
    ws = torch.full((F.forge_rmsnorm_workspace_bytes(rows, cols),), 0xFF, dtype=torch.uint8, device="cuda")
    F.forge_rmsnorm_backward(dyv, hv, gamma.cuda(), rstd.cuda(), dxv, dR=drv, dgamma=dg, workspace=ws)
    f64 = lambda t: None if t is None else t.double().numpy()
    dx, dgm, dx_abs, dg_abs = O.rmsnorm_backward(f64(dy), f64(h), f64(gamma), f64(rstd), f64(dr))
    # dx: the mean's sum (d additions, 3 multiplications a term), then 6 operations
    assert np.all(np.abs(dxv.cpu().double().numpy() - dx) <= dx_abs * (_d(cols) + 12) * U + np.abs(dx) * _half(h_ty) + 1e-38)
    # dgamma: rows in a workgroup's order (at most rows / 256 of one lane), row groups, 512 parts by 32
    d = rows / 256 + 1 + 64 + 32 + 16 + 3
    assert np.all(np.abs(dg.cpu().double().numpy() - dgm) <= dg_abs * d * U + 1e-38)
    assert bool((dxw[:, :pad] == -3).all()) and bool((dxw[:, pad + cols:] == -3).all())
    # a second micro-batch is added
    ws.fill_(0xFF)
    once = dg.clone()
    F.forge_rmsnorm_backward(dyv, hv, gamma.cuda(), rstd.cuda(), None, dgamma=dg, first=False, workspace=ws)
    assert torch.equal(dg, once + once)
    # without dgamma no workspace is needed and dx is the same
    dx2 = torch.empty((rows, cols), dtype=T[h_ty], device="cuda")
    F.forge_rmsnorm_backward(dyv, hv, gamma.cuda(), rstd.cuda(), dx2, dR=drv)
    assert torch.equal(dx2, dxv)


def test_backward_in_place_and_empty():
    h, dy, dr = (_rand((50, 640), s, 1.0, "bf16").cuda() for s in (14, 15, 16))
    gamma, rstd = torch.ones(640, device="cuda"), (h.float().square().mean(1) + 1e-5).rsqrt()
    dx = torch.empty_like(h)
    F.forge_rmsnorm_backward(dy, h, gamma, rstd, dx, dR=dr)
    for target in ("dy", "dr"):
        a, b = dy.clone(), dr.clone()
        out = a if target == "dy" else b
        F.forge_rmsnorm_backward(a, h, gamma, rstd, out, dR=b)
        assert torch.equal(out, dx)
    dg = torch.full((640,), 5.0, device="cuda")
    e = h[:0]
    F.forge_rmsnorm_backward(e, e, gamma, rstd[:0], e.clone(), dgamma=dg, first=False)
    assert bool((dg == 5).all())
    F.forge_rmsnorm_backward(e, e, gamma, rstd[:0], e.clone(), dgamma=dg, first=True)
    assert bool((dg == 0).all())


def test_gradient_against_differences():
    """The forward kernel's own differences (fp32, a step that leaves 1e-3) against the backward kernel."""
    rows, cols, eps = 3, 24, 1e-3
    x, gamma, dy = (_rand(s, k, 1.0, "f32").cuda() for s, k in (((rows, cols), 17), ((cols,), 18), ((rows, cols), 19)))
    y, rstd, dx, dg = torch.empty_like(x), torch.empty(rows, device="cuda"), torch.empty_like(x), torch.empty_like(gamma)
    ws = torch.empty(F.forge_rmsnorm_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")

    def f(xx, gg):
        F.forge_rmsnorm(xx, gg, y, eps=eps, rstd=rstd)
        return (y.double() * dy.double()).sum().item()

    f(x, gamma)
    F.forge_rmsnorm_backward(dy, x, gamma, rstd, dx, dgamma=dg, workspace=ws)
    d = 2.0 ** -7
    # truncation d^2 f''' / 6 (|f'''| under 30 for these O(1) rows) and fp32 noise 24 terms x 2^-23 / d
    tol = d * d * 5 + 24 * 4 * 2.0 ** -23 / d
    for r, c in ((0, 0), (1, 13), (2, 23)):
        up, dn = x.clone(), x.clone()
        up[r, c] += d
        dn[r, c] -= d
        assert abs((f(up, gamma) - f(dn, gamma)) / (2 * d) - dx[r, c].item()) < tol
    for c in (0, 11, 23):
        up, dn = gamma.clone(), gamma.clone()
        up[c] += d
        dn[c] -= d
        assert abs((f(x, up) - f(x, dn)) / (2 * d) - dg[c].item()) < tol


def test_captured_norm_replays():
    rows, cols = 600, 1024
    x, r, dy = (_rand((rows, cols), s, 1.0, "bf16").cuda() for s in (20, 21, 22))
    gamma = torch.ones(cols, device="cuda")
    bufs = []
    for _ in range(2):
        b = dict(h=torch.empty_like(x), y=torch.empty_like(x), s=torch.empty(rows, device="cuda"), dx=torch.empty_like(x),
                 dg=torch.empty(cols, device="cuda"),
                 ws=torch.empty(F.forge_rmsnorm_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda"))
        bufs.append(b)

    def go(b):
        F.forge_rmsnorm(x, gamma, b["y"], R=r, H=b["h"], rstd=b["s"])
        F.forge_rmsnorm_backward(dy, b["h"], gamma, b["s"], b["dx"], dgamma=b["dg"], workspace=b["ws"])

    go(bufs[1])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go(bufs[0])
    for i in range(4):
        x.add_(0.5)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        go(bufs[1])
        torch.cuda.synchronize()
        for k in ("h", "y", "s", "dx", "dg"):
            assert torch.equal(bufs[0][k], bufs[1][k]), (i, k)
