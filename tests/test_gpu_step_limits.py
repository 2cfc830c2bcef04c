"""GPU: the step from 8-bit X at the ends of its documented sizes."""

import pytest
import torch

import backward_weight_gradient_amd as F

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("BT", [2 ** 31 - 1])
def test_token_counts_up_to_2_31(BT):
    """The longest token axis: all tokens but a few are zeros, the last one among the others.
    Every product and sum is a small integer, so G is exact."""
    print(f"case: accumulate act8 8x16 BT {BT}", flush=True)
    N, K = 8, 16
    dY = torch.zeros((BT, N), dtype=torch.bfloat16, device="cuda")
    codes = torch.zeros((BT, K), dtype=torch.int8, device="cuda")
    scale = torch.full((BT, 1), 127, dtype=torch.uint8, device="cuda")      # 2^0
    at = torch.tensor([0, 1, 2 ** 30 + 5, BT - 70, BT - 33, BT - 32, BT - 31, BT - 2, BT - 1], device="cuda")
    g = torch.Generator()
    g.manual_seed(1)
    d = torch.randint(-8, 9, (len(at), N), generator=g).cuda()
    x = torch.randint(-100, 101, (len(at), K), generator=g).cuda()
    dY[at] = d.to(torch.bfloat16)
    codes[at] = x.to(torch.int8)
    acc = torch.full((N, K), float("nan"), device="cuda")
    F.forge_wgrad_accumulate_act8(F.act8(codes, scale, 32), dY, acc, True)
    assert torch.equal(acc.double().cpu(), d.double().cpu().t() @ x.double().cpu())
    del dY, codes, scale
    torch.cuda.empty_cache()


@pytest.mark.parametrize("T", [2 ** 24 - 1])
def test_embedding_gradient_of_the_most_tokens(T):
    """The sort's largest launch.  Values are small integers: G is exact."""
    V, K = 100003, 8
    print(f"case: embedding gradient {T} of {V}x{K}", flush=True)
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    ids = torch.randint(-1, V + 1, (T,), generator=g, device="cuda")
    dY = torch.randint(-8, 9, (T, K), generator=g, device="cuda").to(torch.bfloat16)
    acc = torch.full((V, K), float("nan"), device="cuda")
    ws = torch.empty(F.forge_embed_workspace_bytes(T, V), dtype=torch.uint8, device="cuda")
    F.forge_embed_accumulate(ids, dY, acc, True, workspace=ws)
    ok = (ids >= 0) & (ids < V)
    want = torch.zeros((V, K), dtype=torch.float64, device="cuda").index_add_(0, ids[ok], dY[ok].double())
    assert torch.equal(acc.double(), want)


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_embedding_gradient_of_the_largest_vocabulary(dtype):
    """2^31 - 1 rows of one column; the id 2^31 - 1 is padding."""
    V = 2 ** 31 - 1
    print(f"case: embedding gradient of {V} rows, {dtype}", flush=True)
    ids = torch.tensor([V - 1, V, -1, 0, V - 1, 2 ** 30, V, V - 2, 0, 7], device="cuda").to(dtype)
    dY = torch.tensor([1.0, 100, 200, 3, 4, 5, 300, 6, 7, 8], device="cuda")[:, None].contiguous()
    acc = torch.full((V, 1), float("nan"), device="cuda")
    ws = torch.empty(F.forge_embed_workspace_bytes(10, V), dtype=torch.uint8, device="cuda")
    F.forge_embed_accumulate(ids, dY, acc, True, workspace=ws)
    for row, g in ((V - 1, 5.0), (V - 2, 6.0), (2 ** 30, 5.0), (0, 10.0), (7, 8.0)):
        assert acc[row].item() == g
        acc[row] = 0
    assert not bool(acc.any())
    del acc
    torch.cuda.empty_cache()


def test_longest_rows():
    """One row (two for the lookup) of 2^31 - 1 columns through the copies, the norm, and the embedding."""
    K = 2 ** 31 - 1
    print(f"case: rows of {K} columns", flush=True)
    x = torch.empty((1, K), dtype=torch.bfloat16, device="cuda")
    x[0] = (torch.arange(K, device="cuda", dtype=torch.int32) % 127 - 63).to(torch.bfloat16)
    x[0, K - 2] = 126
    codes, scale = torch.empty((1, K), dtype=torch.int8, device="cuda"), torch.empty((1, 2 ** 24), dtype=torch.uint8, device="cuda")
    back = torch.empty_like(x)
    q = F.act8(codes, scale, 128)
    F.forge_act_quantize(x, q)
    F.forge_act_dequantize(q, back)
    # |x| <= 63: 2^-1 resolves halves; the last block, of 127 columns up to 126, has 2^0
    assert torch.equal(back, x) and scale[0, -1].item() == 127 and bool((scale[0, :-1] == 126).all())
    # the same row as a gradient and as a weight
    acc = torch.full((1, K), float("nan"), device="cuda")
    ids = torch.tensor([0, 0], device="cuda")
    F.forge_embed_accumulate(ids, x.expand(2, K).contiguous(), acc, True, workspace=torch.empty(
        F.forge_embed_workspace_bytes(2, 1), dtype=torch.uint8, device="cuda"))
    assert torch.equal(acc.bfloat16(), x + x) and acc[0, K - 1].item() == 2 * x[0, K - 1].item()
    del acc
    y = torch.full((2, K), 9.0, dtype=torch.bfloat16, device="cuda")
    F.forge_embed(torch.tensor([1, 0], device="cuda"), x, y, scale=2.0)
    assert not bool(y[0].any()) and torch.equal(y[1], (x + x)[0])
    del y
    # the norm of a row of ones but for its last columns: powers of two, exact products; the sum of squares,
    # 2^21 terms a thread and 16 lanes and waves after them, is within (2^21 + 40) 2^-24 of K
    x.fill_(1.0)
    rstd, one, h = torch.empty(1, device="cuda"), torch.ones(K, dtype=torch.bfloat16, device="cuda"), torch.empty_like(x)
    F.forge_rmsnorm(x, one, back, rstd=rstd)
    assert abs(rstd.item() - 1) <= 0.5 * (2 ** 21 + 40) * 2.0 ** -24 + 1e-5
    assert torch.equal(back, (x * rstd).bfloat16())
    F.forge_rmsnorm_backward(x, x, one, torch.ones(1, device="cuda"), h)
    # dX = g - n mean(g n) = 1 - mean: the mean's sum as above
    assert float(h.abs().max()) <= (2 ** 21 + 40) * 2.0 ** -24 and bool((h == h[0, 0]).all())
    torch.cuda.empty_cache()
