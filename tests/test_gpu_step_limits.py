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
