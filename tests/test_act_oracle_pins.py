"""Pins of the oracle's 8-bit activations, RMSNorm and embedding: hand-worked
values, brute force over the definitions, torch's autograd in float64 and
central differences.  CPU only."""

import math

import numpy as np
import pytest
import torch

import oracle as O


def test_act8_exponent_by_hand():
    # S8: 127 2^e; E4M3: 448 2^e
    for a, s8, e4 in ((127.0, 0, -1), (127.00001, 1, -1), (448.0, 2, 0), (448.1, 2, 1), (1.0, -6, -8), (0.0, -120, -120),
                      (254.0, 1, 0), (2.0 ** -130, -120, -120), (3.4e38, 122, 120)):
        assert O.act8_exponent(a, "s8") == s8 and O.act8_exponent(a, "e4m3") == e4, a


@pytest.mark.parametrize("fmt", ["s8", "e4m3"])
def test_act8_encode_follows_the_definition(fmt):
    rng = np.random.default_rng(5)
    x = (rng.standard_normal((64, 70)) * 10.0 ** rng.uniform(-38, 38, (64, 1))).astype(np.float32)
    x[3, :32] = 0
    x[4, 33] = np.inf
    x[5, 65] = np.nan
    codes, scale = O.act8_encode(x, fmt, 32)
    val = O.act8_decode(codes, scale, fmt, 32)
    assert scale.shape == (64, 3)
    for r in range(64):
        for b in range(3):
            part = x[r, 32 * b:32 * b + 32].astype(np.float64)
            got = val[r, 32 * b:32 * b + 32]
            if not np.isfinite(part).all():
                assert scale[r, b] == 255 and np.isnan(got).all() and not codes[r, 32 * b:32 * b + 32].any()
                continue
            e = O.act8_exponent(np.abs(part).max(), fmt)
            assert scale[r, b] == e + 127
            # nearest: no representable value lies closer
            step = math.ldexp(1.0, e)
            grid = np.arange(-127, 128) if fmt == "s8" else np.concatenate([-O.e4m3_to_f64(np.arange(127)),
                                                                           O.e4m3_to_f64(np.arange(127))])
            best = np.min(np.abs(part[:, None] - grid[None, :] * step), axis=1)
            np.testing.assert_array_equal(np.abs(got - part), best)


def test_act8_values_are_exact_in_bf16():
    for fmt in ("s8", "e4m3"):
        codes = np.arange(256).astype(np.uint8)
        codes = codes[(codes & 0x7F) != 0x7F] if fmt == "e4m3" else codes.astype(np.int8)
        for e in (-120, -7, 0, 100):
            v = O.act8_decode(codes[None, :], np.full((1, -(-codes.size // 128)), e + 127, np.uint8), fmt, 128)
            assert np.array_equal(torch.from_numpy(v).to(torch.bfloat16).double().numpy(), v)


def test_act8_ties_go_to_even():
    x = np.float32([[127, 0.5, 1.5, 2.5, -0.5, -1.5] + [0] * 26])
    np.testing.assert_array_equal(O.act8_encode(x, "s8", 32)[0][0, :6], [127, 0, 2, 2, 0, -2])
    x = np.float32([[448, 17, 19, 2.0 ** -10, 3 * 2.0 ** -10] + [0] * 27])
    codes, scale = O.act8_encode(x, "e4m3", 32)
    np.testing.assert_array_equal(O.act8_decode(codes, scale, "e4m3", 32)[0, :5], [448, 16, 20, 0, 2.0 ** -8])


def test_rmsnorm_against_autograd_and_differences():
    rng = np.random.default_rng(6)
    h, gamma, dy, dr = rng.standard_normal((5, 37)), rng.standard_normal(37), rng.standard_normal((5, 37)), \
        rng.standard_normal((5, 37))
    eps = 1e-3
    y, s = O.rmsnorm(h, gamma, eps)
    H, Ga = torch.tensor(h, requires_grad=True), torch.tensor(gamma, requires_grad=True)
    Y = H * torch.rsqrt((H * H).mean(1, keepdim=True) + eps) * Ga
    np.testing.assert_allclose(y, Y.detach().numpy(), rtol=1e-13)
    (Y * torch.tensor(dy) + H * torch.tensor(dr)).sum().backward()
    dx, dg, _, _ = O.rmsnorm_backward(dy, h, gamma, s, dr)
    np.testing.assert_allclose(dx, H.grad.numpy(), rtol=1e-11, atol=1e-12)
    np.testing.assert_allclose(dg, Ga.grad.numpy(), rtol=1e-11, atol=1e-12)
    for r, c in ((0, 0), (2, 17), (4, 36)):
        d = 1e-6
        up, dn = h.copy(), h.copy()
        up[r, c] += d
        dn[r, c] -= d
        f = lambda z: (O.rmsnorm(z, gamma, eps)[0] * dy + z * dr).sum()
        assert abs((f(up) - f(dn)) / (2 * d) - dx[r, c]) < 1e-7


def test_embedding_against_torch():
    rng = np.random.default_rng(7)
    W, dy = rng.standard_normal((11, 6)), rng.standard_normal((9, 6))
    ids = np.array([3, -1, 3, 0, 10, 11, 3, 10, 2 ** 40])
    keep = (ids >= 0) & (ids < 11)
    Wt = torch.tensor(W, requires_grad=True)
    Y = torch.nn.functional.embedding(torch.tensor(ids[keep]), Wt) * 2.5
    y = O.embed(ids, W, 2.5)
    np.testing.assert_allclose(y[keep], Y.detach().numpy(), rtol=1e-15)
    assert not y[~keep].any()
    (Y * torch.tensor(dy[keep])).sum().backward()
    G, _, n = O.embed_grad(ids, dy, 11, 2.5)
    np.testing.assert_allclose(G, Wt.grad.numpy(), rtol=1e-13)
    assert n.tolist() == [1, 0, 0, 3, 0, 0, 0, 0, 0, 0, 2]
