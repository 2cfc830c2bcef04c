"""GPU: activations in 8 bits and the weight-gradient step that reads them.

The copies are exact functions of their inputs (a power-of-two scale, one
rounding), so codes, scales and decoded values must equal the oracle's bit for
bit.  The step must agree with the oracle within the tolerances of the other
parity tests everywhere, and equal forge_wgrad_step on the decoded bf16 X bit for
bit in the kernels of aligned layers that fill the chip, whose sums have the same
order (256 tiles of 128 x 128 and more, or fewer than 128 tokens).
"""

import numpy as np
import pytest
import torch

import backward_weight_gradient_amd as F
import oracle as O
import synth
from forge_testlib import Layer, assert_ok, check_against_oracle, make_layer, oracle_hyper, snapshot

pytestmark = pytest.mark.gpu
FMTS = ["s8", "e4m3"]
CODE = {"s8": torch.int8, "e4m3": torch.float8_e4m3fn}


def _say(*a):
    print(*a, flush=True)


def _gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def _act(rows, cols, fmt, block, ld=None, guard=0x5A):
    """An empty 8-bit matrix (codes with pitch ld) whose memory is filled with `guard`."""
    ld = ld or cols
    buf = torch.full((max(1, rows) * ld + 64,), guard, dtype=torch.uint8, device="cuda")
    codes = buf[:rows * ld].view(rows, ld)[:, :cols].view(CODE[fmt])
    scale = torch.full((rows, -(-cols // block)), guard, dtype=torch.uint8, device="cuda")
    return buf, codes, scale, F.act8(codes, scale, block)


def _host_codes(codes, fmt):
    return codes.cpu().contiguous().view(torch.int8 if fmt == "s8" else torch.uint8).numpy()


def _values(rows, cols, seed, dtype):
    """Values over many magnitudes, with exact ties, zero blocks, subnormals, the largest values,
    infinities and NaNs."""
    g = _gen(seed)
    x = torch.randn((rows, cols), generator=g) * torch.exp2(torch.randint(-20, 20, (rows, 1), generator=g).float())
    if rows > 7:
        x[0] = 0
        x[1] = torch.round(x[1] * 64) / 2                       # ties of the S8 grid
        x[2] = x[2] * 2.0 ** -130
        x[3, ::3] = 3.0e38
        x[4, min(5, cols - 1)] = float("inf")
        x[5, -1] = float("nan")
        x[6, 0] = -float("inf")
        x[7] = 2.0 ** -149
    return x.to(dtype)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("block", [32, 64, 128])
@pytest.mark.parametrize("rows,cols,dtype", [(1, 1, "f32"), (1, 4096, "bf16"), (9, 128, "bf16"), (33, 130, "f32"),
                                             (17, 1000, "bf16"), (70, 2049, "bf16"), (5, 8200, "f32"), (300, 31, "bf16")])
def test_copies_are_exact(fmt, block, rows, cols, dtype):
    _say(f"case: act8 {fmt} block {block} {rows}x{cols} {dtype}")
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    x = _values(rows, cols, rows * 131 + cols, dt)
    buf, codes, scale, q = _act(rows, cols, fmt, block, ld=cols + 3)
    F.forge_act_quantize(x.cuda(), q)
    ref_c, ref_s = O.act8_encode(x.float().numpy(), fmt, block)
    np.testing.assert_array_equal(scale.cpu().numpy(), ref_s)
    np.testing.assert_array_equal(_host_codes(codes, fmt), ref_c)
    pad = buf[:rows * (cols + 3)].view(rows, cols + 3)[:, cols:]
    assert bool((pad == 0x5A).all()) and bool((buf[rows * (cols + 3):] == 0x5A).all())
    val = O.act8_decode(ref_c, ref_s, fmt, block)
    for out_t in (torch.float32, torch.bfloat16):
        y = torch.full((rows, cols + 5), -7.0, dtype=out_t, device="cuda")
        F.forge_act_dequantize(q, y[:, :cols])
        with np.errstate(over="ignore"):
            want = torch.from_numpy(val.astype(np.float32)).to(out_t)
        got = y[:, :cols].cpu()
        same = (got == want) | (got.isnan() & want.isnan())
        assert bool(same.all()), (got[~same][:4], want[~same][:4])
        assert bool((y[:, cols:] == -7.0).all())


def test_copies_of_strided_and_offset_views():
    """Rows at odd element offsets: no alignment beyond the element's is assumed."""
    base = _values(40, 999, 3, torch.bfloat16).cuda()
    x = base[3:, 1:514]
    _, codes, scale, q = _act(37, 513, "e4m3", 64, ld=515)
    F.forge_act_quantize(x, q)
    ref_c, ref_s = O.act8_encode(x.float().cpu().numpy(), "e4m3", 64)
    np.testing.assert_array_equal(_host_codes(codes, "e4m3"), ref_c)
    np.testing.assert_array_equal(scale.cpu().numpy(), ref_s)
    out = torch.zeros((37, 1025), dtype=torch.bfloat16, device="cuda")[:, 3:516]
    F.forge_act_dequantize(q, out)
    want = torch.from_numpy(O.act8_decode(ref_c, ref_s, "e4m3", 64).astype(np.float32)).to(torch.bfloat16)
    assert bool(((out.cpu() == want) | want.isnan()).all())


# ---------------------------------------------------------------------------
# The step
# ---------------------------------------------------------------------------
def _spec(opt, state, w="bf16", block=128):
    m = "s8" if state == "int8" else state
    v = None if opt != "adamw" else ("u8" if state == "int8" else state)
    return synth.LayerSpec("bf16", w, m, v, block=block)


def _layer8(cfg, N, K, BT, spec, fmt, xblock, **kw):
    """A layer whose X is what an 8-bit copy decodes to, and that copy."""
    L = make_layer(cfg, N, K, BT, 10, spec, **kw)
    codes = torch.empty((BT, K), dtype=CODE[fmt], device="cuda")
    scale = torch.empty((BT, -(-K // xblock)), dtype=torch.uint8, device="cuda")
    q = F.act8(codes, scale, xblock)
    F.forge_act_quantize(L.X, q)
    F.forge_act_dequantize(q, L.X)
    return L, q, (codes, scale)


def _hyper(opt, round_="sr"):
    return F.hyper("lion", lr=1e-4, beta2=0.99, round=round_) if opt == "lion" else F.hyper(opt, round=round_)


def _same(a: Layer, b: Layer):
    for n in ("W", "m", "v", "ms", "vs"):
        x, y = getattr(a, n), getattr(b, n)
        if x is not None:
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), n


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("opt,state,w,round_", [("adamw", "f32", "bf16", "sr"), ("adamw", "bf16", "bf16", "sr"),
                                                ("adamw", "int8", "bf16", "rne"), ("adamw", "e4m3", "f32", "sr"),
                                                ("lion", "f32", "f32", "sr"), ("lion", "bf16", "bf16", "rne"),
                                                ("sgdm", "f32", "bf16", "rne"), ("sgdm", "bf16", "f32", "sr")])
@pytest.mark.parametrize("N,K,BT", [(256, 384, 96), (200, 256, 333)])
def test_step_matches_the_oracle(fmt, opt, state, w, round_, N, K, BT):
    _say(f"case: step act8 {fmt} {opt} {state} {w} {round_} {N}x{K} BT {BT}")
    L, q, _keep = _layer8(70, N, K, BT, _spec(opt, state, w), fmt, 64)
    P, snap, h = L.clone(), snapshot(L), _hyper(opt, round_)
    F.forge_wgrad_step_act8(q, L.dY, L.W, L.forge_m(), L.forge_v(), h, 10, 1337)
    assert_ok(check_against_oracle(snap, L, h, 10, 1337))
    if BT < 128:
        F.forge_wgrad_step(P.X, P.dY, P.W, P.forge_m(), P.forge_v(), h, 10, 1337)
        _same(L, P)


@pytest.mark.parametrize("fmt,xblock,N,K,BT", [("s8", 32, 1, 1, 1), ("e4m3", 128, 129, 131, 65), ("s8", 128, 77, 1003, 40),
                                               ("e4m3", 64, 1001, 63, 7), ("s8", 64, 130, 260, 2), ("e4m3", 32, 40, 33, 0),
                                               ("s8", 128, 264, 136, 129), ("e4m3", 32, 128, 128, 63),
                                               ("s8", 32, 8, 16, 300), ("e4m3", 64, 9, 17, 257), ("s8", 64, 7, 200, 90),
                                               ("e4m3", 32, 200, 15, 90), ("s8", 64, 71, 145, 1000), ("e4m3", 128, 65, 129, 33),
                                               ("s8", 32, 300, 47, 256), ("e4m3", 64, 64, 128, 128)])
def test_step_ragged(fmt, xblock, N, K, BT):
    _say(f"case: step act8 ragged {fmt} block {xblock} {N}x{K} BT {BT}")
    L, q, _keep = _layer8(71, N, K, BT, _spec("adamw", "f32"), fmt, xblock)
    snap, h = snapshot(L), _hyper("adamw")
    F.forge_wgrad_step_act8(q, L.dY, L.W, L.forge_m(), L.forge_v(), h, 10, 1337)
    assert_ok(check_against_oracle(snap, L, h, 10, 1337))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("opt,state,w", [("adamw", "f32", "bf16"), ("adamw", "bf16", "bf16"), ("adamw", "int8", "bf16"),
                                         ("adamw", "e4m3", "f32"), ("lion", "bf16", "bf16"), ("sgdm", "f32", "f32")])
@pytest.mark.parametrize("BT,N,K", [(2048, 512, 256), (2049, 264, 640), (4100, 250, 513)])
def test_step_long_token_axis(fmt, opt, state, w, BT, N, K):
    _say(f"case: step act8 long {fmt} {opt} {state} {w} {N}x{K} BT {BT}")
    if K % 128 and state in ("int8", "e4m3"):
        K = 512          # 8-bit states: whole blocks
    L, q, _keep = _layer8(72, N, K, BT, _spec(opt, state, w), fmt, 128)
    snap, h = snapshot(L), _hyper(opt)
    F.forge_wgrad_step_act8(q, L.dY, L.W, L.forge_m(), L.forge_v(), h, 10, 1337)
    assert_ok(check_against_oracle(snap, L, h, 10, 1337))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("opt,state,w", [("adamw", "f32", "bf16"), ("adamw", "bf16", "f32"), ("adamw", "int8", "bf16"),
                                         ("adamw", "e4m3", "f32"), ("lion", "f32", "bf16"), ("sgdm", "bf16", "f32")])
@pytest.mark.parametrize("BT,N,K", [(300, 2600, 512), (129, 2605, 515), (31, 1001, 1503)])
def test_step_more_tiles_than_cus(fmt, opt, state, w, BT, N, K):
    """Over 256 tiles of 32 x 128, under 256 of 128 x 128 or unaligned; sampled rows."""
    _say(f"case: step act8 tiles {fmt} {opt} {state} {w} {N}x{K} BT {BT}")
    if K % 128 and state in ("int8", "e4m3"):
        K = K // 128 * 128
    L, q, _keep = _layer8(79, N, K, BT, _spec(opt, state, w), fmt, 32)
    snap, h = snapshot(L, np.array([0, 31, 63, 64, 500, N - 64, N - 1])), _hyper(opt)
    F.forge_wgrad_step_act8(q, L.dY, L.W, L.forge_m(), L.forge_v(), h, 10, 1337)
    assert_ok(check_against_oracle(snap, L, h, 10, 1337))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("opt,state,w", [("adamw", "f32", "bf16"), ("adamw", "bf16", "bf16"), ("adamw", "int8", "bf16"),
                                         ("adamw", "e4m3", "f32"), ("lion", "f32", "f32"), ("lion", "bf16", "bf16"),
                                         ("sgdm", "f32", "bf16"), ("sgdm", "bf16", "f32")])
@pytest.mark.parametrize("BT,N,K", [(0, 2048, 2048), (1, 2048, 2048), (200, 2048, 2048), (513, 2056, 2064), (2100, 2048, 2048),
                                    (2048, 4096, 3584), (2049, 3592, 4112)])
def test_step_equals_the_decoded_step(fmt, opt, state, w, BT, N, K):
    """Layers that fill the chip: bit for bit forge_wgrad_step on the decoded X, and the oracle on sampled rows."""
    _say(f"case: step act8 ring {fmt} {opt} {state} {w} {N}x{K} BT {BT}")
    block = 128 if K % 128 == 0 else 16
    if block == 16 and state in ("int8", "e4m3"):
        K = K // 128 * 128
    L, q, _keep = _layer8(78, N, K, BT, _spec(opt, state, w), fmt, 64, gen_device="cuda")
    rows = np.array([0, 63, 64, 1000, N - 1])
    P, snap, h = L.clone(), snapshot(L, rows), _hyper(opt)
    F.forge_wgrad_step_act8(q, L.dY, L.W, L.forge_m(), L.forge_v(), h, 10, 1337)
    F.forge_wgrad_step(P.X, P.dY, P.W, P.forge_m(), P.forge_v(), h, 10, 1337)
    _same(L, P)
    assert_ok(check_against_oracle(snap, L, h, 10, 1337))


@pytest.mark.parametrize("N,K,BT", [(264, 272, 300), (264, 272, 2500), (264, 272, 60), (2056, 2064, 300), (3, 40, 70), (40, 9, 70)])
@pytest.mark.parametrize("off,doff", [(16, 8), (3, 1), (20, 8)])
def test_step_strided_operands(N, K, BT, off, doff):
    """Codes, dY and W as columns of wider buffers filled with poison (NaN where the
    type has one), at aligned and at odd offsets: the same bits as dense operands of the
    same kernel, or the oracle's where alignment picks another."""
    L, q, (codes, scale) = _layer8(73, N, K, BT, _spec("adamw", "f32"), "e4m3", 64, gen_device="cuda")
    wide = torch.full((BT, K + 32), 0x7F, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)   # NaN codes
    wide[:, off:off + K] = codes
    dwide = torch.full((BT, N + 24), float("nan"), device="cuda", dtype=torch.bfloat16)
    dwide[:, doff:doff + N] = L.dY
    ww = torch.full((N, K + 16), float("nan"), device="cuda", dtype=torch.bfloat16)
    wv = ww[:, 5:5 + K]
    wv.copy_(L.W)
    rows = np.unique(np.array([0, N // 2, N - 1]))
    snap, h = snapshot(L, rows), _hyper("adamw")
    F.forge_wgrad_step_act8(F.act8(wide[:, off:off + K], scale, 64), dwide[:, doff:doff + N], wv, L.forge_m(), L.forge_v(), h,
                            10, 1)
    L.W = wv.contiguous()
    assert_ok(check_against_oracle(snap, L, h, 10, 1))
    assert bool(ww[:, :5].isnan().all()) and bool(ww[:, 5 + K:].isnan().all())


@pytest.mark.parametrize("BT", [64, 2048])
def test_a_poisoned_block_reaches_the_gradient(BT):
    """A NaN in X: every element of G in the block's columns is NaN, no other is."""
    N, K = 128, 256
    x = synth.normal((BT, K), 1.0, "cuda", 74, 1, synth.T_X).to(torch.bfloat16)
    x[5, 70] = float("nan")
    dY = synth.normal((BT, N), 1e-3, "cuda", 74, 1, synth.T_DY).to(torch.bfloat16)
    for fmt in FMTS:
        codes = torch.empty((BT, K), dtype=CODE[fmt], device="cuda")
        scale = torch.empty((BT, 4), dtype=torch.uint8, device="cuda")
        q = F.act8(codes, scale, 64)
        F.forge_act_quantize(x, q)
        acc = torch.empty((N, K), device="cuda")
        F.forge_wgrad_accumulate_act8(q, dY, acc, True)
        bad = acc.isnan().cpu()
        assert bool(bad[:, 64:128].all()) and not bool(bad[:, :64].any()) and not bool(bad[:, 128:].any())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("N,K,BT", [(256, 384, 96), (77, 130, 65), (256, 256, 2050), (16, 8, 0), (2048, 2048, 130), (5, 5, 40), (2605, 515, 150),
                                    (100, 64, 200)])
def test_accumulate(fmt, N, K, BT):
    """acc = G within the bound of an fp32 sum in any order; then one fp32 addition of G."""
    _say(f"case: accumulate act8 {fmt} {N}x{K} BT {BT}")
    L, q, _keep = _layer8(75, N, K, BT, _spec("adamw", "f32"), fmt, 32)
    a = torch.full((N, K + 5), 3.0, device="cuda")
    v = a[:, 1:1 + K]
    F.forge_wgrad_accumulate_act8(q, L.dY, v, True)
    x, dy = synth.host(L.X), synth.host(L.dY)
    rows = np.unique(np.linspace(0, N - 1, 64).astype(int))
    got = v.cpu().double().numpy()[rows]
    assert np.all(np.abs(got - O.weight_grad(x, dy, rows)) <= O.grad_error_bound(x, dy, rows) + 1e-38)
    G = v.clone()
    for _ in range(2):
        old = v.clone()
        F.forge_wgrad_accumulate_act8(q, L.dY, v, False)
        assert torch.equal(v, old + G)
    assert bool((a[:, 0] == 3.0).all()) and bool((a[:, 1 + K:] == 3.0).all())
    # and the documented route to any other optimizer: accumulate, then the step with no tokens
    G = torch.empty((N, K), device="cuda")
    F.forge_wgrad_accumulate_act8(q, L.dY, G, True)
    W = L.W.clone()
    v = torch.zeros((N, K), device="cuda")
    empty = lambda c: torch.empty((0, c), dtype=torch.bfloat16, device="cuda")
    F.forge_wgrad_step_accumulated(empty(K), empty(N), G.clone(), W, None, F.state(v), F.hyper("rmsprop", round="rne"), 1, 0)
    gg = G.double() + 0.01 * L.W.double()
    want = 0.01 * gg * gg
    assert bool(((v.double() - want).abs() <= want * 8 * 2.0 ** -24 + 2.0 ** -24 * G.abs().double() * 0.02 + 1e-38).all())


def test_full_size_gate_proj_sampled_rows():
    N, K = synth.LLAMA8B_LAYERS["gate_proj"]
    L, q, _keep = _layer8(76, N, K, 512, _spec("adamw", "f32"), "e4m3", 128, gen_device="cuda")
    rows = np.array([0, 127, 128, 5000, N - 1])
    snap, h = snapshot(L, rows), _hyper("adamw")
    F.forge_wgrad_step_act8(q, L.dY, L.W, L.forge_m(), L.forge_v(), h, 10, 1337)
    assert_ok(check_against_oracle(snap, L, h, 10, 1337))


def test_captured_step_replays():
    """Quantise and step captured into a graph: every replay equals the eager calls."""
    L, q, (codes, scale) = _layer8(77, 256, 256, 200, _spec("adamw", "f32"), "s8", 64)
    P, h = L.clone(), _hyper("adamw")
    codes2, scale2 = torch.empty_like(codes), torch.empty_like(scale)
    q2 = F.act8(codes2, scale2, 64)
    x = L.X.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        F.forge_act_quantize(x, q2)      # warm-up: kernels loaded
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        F.forge_act_quantize(x, q2)
        F.forge_wgrad_step_act8(q2, L.dY, L.W, L.forge_m(), L.forge_v(), h, 10, 7)
    for i in range(4):
        x.copy_(P.X * (i + 1))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        F.forge_act_quantize(x, q)
        F.forge_wgrad_step_act8(q, P.dY, P.W, P.forge_m(), P.forge_v(), h, 10, 7)
        torch.cuda.synchronize()
        _same(L, P)
