"""GPU: the loops that the norm, embedding and copy kernels take when there is more work than
workgroups, each with a remainder: several rows per workgroup in the norm's forms (the row
requested ahead, the alternating LDS buffers, the sums of dgamma over rows), several units in
the embedding's long rows, in the lookup, in the copies and in what clears memory.

Rows differ in magnitude by powers of two, so that a sum that reaches the wrong row is far off.

Tolerances, u = 2^-24.  A row's sum: a lane adds at most 16 terms (K / 1024 past 16384
columns), then 6 steps over a wave's lanes and 16 over its waves: d = 40 + K / 1024
additions of positive terms, (d + 1) u; s = 1 / sqrt(sum / K + eps) halves that and adds
4 u; y two products more.  dx: the mean's sum with 3 products a term and 6 operations,
against the sum of absolute values.  dgamma: two products a term; a lane's rows one after
another, then at most 2 + 16 row groups, 16 of the 256 parts in order, 16 sums of those and
the old value.  A bf16 store adds 2^-8.
"""

import numpy as np
import pytest
import torch

import backward_weight_gradient_amd as F
import oracle as O

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
T = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-5

# Forward: 2048 workgroups of 16, 4 or 1 rows, 512 of one row above 4096 columns.  Backward: 256
# of 64, 16, 4 or 1.  Every (lanes per row, vectors per lane), whole vectors and others, and the
# rows read twice (below 8 and above 16384 columns).
SHAPES = [(40001, 40), (33001, 128), (8501, 300), (8501, 512), (8501, 1000), (8209, 1024), (4501, 1500), (2600, 2048),
          (4100, 4096), (2051, 4001), (1100, 5001), (1025, 8192), (600, 16384), (1100, 12345), (1100, 16391), (1100, 5)]


def _say(*a):
    print(*a, flush=True)


def _rand(shape, seed, std, ty):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(T[ty])


def _rows(shape, seed, std, ty):
    """Row r times 2^(5 r mod 13 - 6)."""
    f = torch.exp2((torch.arange(shape[0], device="cuda") * 5 % 13 - 6).float())
    return (_rand(shape, seed, std, "f32") * f[:, None]).to(T[ty])


def _half(ty):
    return 2.0 ** -8 if ty == "bf16" else 0.0


@pytest.mark.parametrize("x_ty,r_ty", [("bf16", "bf16"), ("f32", None), ("bf16", "f32")])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_norm_forward(rows, cols, x_ty, r_ty):
    _say(f"case: norm loop {rows}x{cols} {x_ty} {r_ty}")
    x, gamma = _rows((rows, cols), 1, 1.0, x_ty), 1 + _rand((cols,), 2, 0.2, "f32")
    y, rstd = torch.empty((rows, cols), device="cuda"), torch.empty(rows, device="cuda")
    codes = torch.empty((rows, cols), dtype=torch.int8, device="cuda")
    scale = torch.empty((rows, -(-cols // 64)), dtype=torch.uint8, device="cuda")
    h = x
    if r_ty:
        r = _rows((rows, cols), 3, 0.5, r_ty)
        want = (x.float() + r.float()).to(T[r_ty])
        h = r                                       # the sum in the residual's place
    F.forge_rmsnorm(x, gamma, y, eps=EPS, R=h if r_ty else None, H=h if r_ty else None, Q=F.act8(codes, scale, 64), rstd=rstd)
    if r_ty:
        assert torch.equal(h, want)
    hd = h.double()
    s = 1 / (hd.square().mean(1) + EPS).sqrt()
    tol = (0.5 * (40 + cols / 1024 + 1) + 4) * U
    assert bool(((rstd.double() - s).abs() <= s * tol).all())
    yd = hd * s[:, None] * gamma.double()
    assert bool(((y.double() - yd).abs() <= yd.abs() * ((tol + 2 * U) * (1 + 2.0 ** -20)) + 1e-38).all())
    c2, s2 = torch.empty_like(codes), torch.empty_like(scale)
    F.forge_act_quantize(y, F.act8(c2, s2, 64))
    assert torch.equal(codes, c2) and torch.equal(scale, s2)
    # Y in bf16 and no other output: the same values, rounded
    yb = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
    F.forge_rmsnorm(h, gamma, yb, eps=EPS)
    assert torch.equal(yb, y.bfloat16())


@pytest.mark.parametrize("h_ty,d_ty,place", [("bf16", "bf16", "dr"), ("f32", "bf16", None), ("f32", "f32", "dy"), ("bf16", "f32", None)])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_norm_backward(rows, cols, h_ty, d_ty, place):
    """place: dX takes dR's or dY's memory, with a residual gradient; None: neither."""
    _say(f"case: norm gradient loop {rows}x{cols} {h_ty} {d_ty} {place}")
    h, dy = _rows((rows, cols), 10, 1.0, h_ty), _rows((rows, cols), 11, 1e-3, d_ty).flip(0).contiguous()
    gamma = 1 + _rand((cols,), 12, 0.2, "f32")
    rstd = (1 / (h.double().square().mean(1) + EPS).sqrt()).float()
    dr = _rand((rows, cols), 13, 1e-3, h_ty) if place else None
    hd, dyd, s = h.double(), dy.double(), rstd.double()[:, None]
    g, n = dyd * gamma.double(), hd * s
    dx = s * (g - n * (g * n).mean(1, keepdim=True))
    dx_abs = s * (g.abs() + n.abs() * (g * n).abs().mean(1, keepdim=True))
    if place:
        dx, dx_abs = dx + dr.double(), dx_abs + dr.double().abs()
    dg64, dg_abs = (dyd * n).sum(0), (dyd * n).abs().sum(0)
    del g, n, hd, dyd
    dy0, dr0 = dy.clone(), dr.clone() if place else None
    out = {"dr": dr, "dy": dy, None: torch.empty_like(h)}[place]
    dg = torch.full((cols,), float("nan"), device="cuda")
    ws = torch.full((F.forge_rmsnorm_workspace_bytes(rows, cols),), 0xFF, dtype=torch.uint8, device="cuda")
    F.forge_rmsnorm_backward(dy, h, gamma, rstd, out, dR=dr, dgamma=dg, workspace=ws)
    d = 40 + cols / 1024 + 12
    assert bool(((out.double() - dx).abs() <= dx_abs * d * U + dx.abs() * _half(h_ty) + 1e-38).all())
    per = 1 if cols < 8 or cols > 4096 else 4 if cols > 1024 else 16 if cols > 128 else 64
    d = -(-rows // (256 * per)) + 2 + 18 + 16 + 16 + 1
    assert bool(((dg.double() - dg64).abs() <= dg_abs * d * U + 1e-38).all())
    # added to what is there, without dX: the same sums
    ws.fill_(0xFF)
    more = torch.arange(cols, device="cuda").float()
    want = more + dg
    F.forge_rmsnorm_backward(dy0, h, gamma, rstd, None, dgamma=more, first=False, workspace=ws)
    assert torch.equal(more, want)
    # dX alone, into memory of its own: the same bits
    alone = torch.empty_like(h)
    F.forge_rmsnorm_backward(dy0, h, gamma, rstd, alone, dR=dr0)
    assert torch.equal(alone, out)


def test_norm_gradient_of_very_long_rows():
    """More columns than 2^20 workgroups of 64 take at once in dgamma's last sum."""
    rows, cols = 2, 2 ** 26 + 77
    _say(f"case: norm gradient {rows}x{cols}")
    h, dy = _rand((rows, cols), 14, 1.0, "bf16"), _rand((rows, cols), 15, 1.0, "bf16")
    gamma, rstd = torch.ones(cols, device="cuda"), torch.tensor([0.75, 1.25], device="cuda")
    dg = torch.full((cols,), float("nan"), device="cuda")
    ws = torch.empty(F.forge_rmsnorm_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    F.forge_rmsnorm_backward(dy, h, gamma, rstd, None, dgamma=dg, workspace=ws)
    t = dy.double() * h.double() * rstd.double()[:, None]
    # n = h s is one product, rounded; its product with dy and the sum over two rows
    assert bool(((dg.double() - t.sum(0)).abs() <= 4 * U * t.abs().sum(0)).all())


@pytest.mark.parametrize("d_ty", ["bf16", "f32"])
@pytest.mark.parametrize("n,V,K", [(8192, 100, 4096), (8229, 97, 4100), (20000, 300, 1001), (6000, 40, 1500)])
@pytest.mark.parametrize("first", [True, False])
def test_embedding_gradient_of_many_long_rows(n, V, K, d_ty, first):
    """More units of long rows (32 tokens by 64 columns) than the 2048 workgroups that take them; a row of each
    length, short ones between.  Small integers: the sums are exact."""
    _say(f"case: embedding gradient, long rows, {n} of {V}x{K} {d_ty} {first}")
    assert -(-n // 32) * -(-K // 64) > 2 * 2048
    g = torch.Generator(device="cuda")
    g.manual_seed(16)
    ids = (torch.rand(n, generator=g, device="cuda") ** 3 * V).long().clamp(max=V - 1)
    ids[::101] = -1
    ids[7:40] = 0
    dY = torch.randint(-8, 9, (n, K), generator=g, device="cuda").to(T[d_ty])
    acc = torch.full((V + 2, K + 3), 5.0, device="cuda")
    view = acc[:V, :K]
    ws = torch.full((F.forge_embed_workspace_bytes(n, V),), 0xEE, dtype=torch.uint8, device="cuda")
    F.forge_embed_accumulate(ids, dY, view, first, scale=2.0, workspace=ws)
    ok = ids >= 0
    want = torch.full((V, K), 0.0 if first else 5.0, dtype=torch.float64, device="cuda")
    want.index_add_(0, ids[ok], 2 * dY[ok].double())
    assert torch.equal(view.double(), want)
    assert bool((acc[V:] == 5).all()) and bool((acc[:, K:] == 5).all())


def test_copies_of_more_units_than_workgroups():
    """2^22 workgroups of 64 rows, and a few rows more."""
    rows = 2 ** 28 + 131
    _say(f"case: act8 {rows}x1")
    x = (torch.arange(rows, device="cuda") % 251 - 125).to(torch.bfloat16)[:, None]
    codes = torch.empty((rows, 1), dtype=torch.int8, device="cuda")
    scale = torch.empty((rows, 1), dtype=torch.uint8, device="cuda")
    back = torch.full((rows, 1), float("nan"), dtype=torch.bfloat16, device="cuda")
    q = F.act8(codes, scale, 32)
    F.forge_act_quantize(x, q)
    F.forge_act_dequantize(q, back)
    assert torch.equal(back, x)            # one element a block, 8 bits of significand: exact


def test_lookup_of_more_units_than_workgroups():
    """2^22 workgroups of 4 tokens, and a few tokens more."""
    n, V, K = 2 ** 24 + 5, 3, 1025
    _say(f"case: embed {n} of {V}x{K}")
    W = _rand((V, K), 17, 1.0, "bf16")
    ids = torch.arange(n, device="cuda", dtype=torch.int32) % 5 - 1          # -1, 0, 1, 2, 3
    y = torch.full((n, K), 9.0, dtype=torch.bfloat16, device="cuda")
    F.forge_embed(ids, W, y, scale=0.5)
    z = torch.zeros((1, K), dtype=torch.bfloat16, device="cuda")
    five = torch.cat([z, W * 0.5, z]).repeat(20000, 1)
    for t in range(0, n, five.shape[0]):
        assert torch.equal(y[t:t + five.shape[0]], five[:n - t]), t
    del y
    torch.cuda.empty_cache()


def test_lookup_in_an_empty_vocabulary():
    """Nothing but padding: zeros, of more rows than 2^20 workgroups of 256 clear at once."""
    n = 2 ** 28 + 77
    _say(f"case: embed {n} of 0x1")
    ids = torch.zeros(n, dtype=torch.int32, device="cuda")
    y = torch.full((n, 2), float("nan"), dtype=torch.bfloat16, device="cuda")
    F.forge_embed(ids, torch.empty((0, 1), dtype=torch.bfloat16, device="cuda"), y[:, :1])
    assert not bool(y[:, 0].any()) and bool(y[:, 1].isnan().all())
