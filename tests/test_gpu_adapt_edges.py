"""GPU tests at the edges of the layer norm, the adapters, the AdamW step and what is built on them."""
import pytest
import torch

pytestmark = pytest.mark.gpu

rtl = pytest.importorskip("activation_sparse_gemm_amd")

BF = torch.bfloat16


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def digits(seed, M):
    """[M, 3] in bf16: a value of 24 digits, eight in each."""
    eight = torch.randint(128, 256, (M, 3), generator=torch.Generator().manual_seed(seed)) / 128
    return (eight * torch.tensor([1.0, 2.0 ** -8, 2.0 ** -16])).to(BF).cuda()


@pytest.mark.parametrize("M", (1, 12, 40, 200))  # joined in up's own launch, a block of rows, a tile, several
@pytest.mark.parametrize("R", (8, 40, 72, 128))
def test_every_digit_of_the_inner_product(M, R):
    """T = (h + m + l, -(h + m)) with 8 digits in each of h, m and l, added up: l to the bit.  All sums on the
    way are whole multiples of 2^-23 below 4, exact in fp32; T in two bf16 parts has 17 digits, which leave none of l."""
    K, N = 72, 136
    v = digits(M + R, M)
    plan = rtl.rtl_adapters_plan(torch.zeros(M, dtype=torch.int32, device="cuda"), 1)
    # forward: three channels of X through two ranks into every column
    X = torch.zeros(M, K, dtype=BF, device="cuda")
    X[:, :3] = v
    LB, LA = torch.zeros(1, R, K, dtype=BF, device="cuda"), torch.zeros(1, N, R, dtype=BF, device="cuda")
    LB[0, 0, :3], LB[0, R - 1, :2], LA[0, :, 0], LA[0, :, R - 1] = 1.0, -1.0, 1.0, 1.0
    assert torch.equal(rtl.rtl_adapters(X, LA, LB, plan), v[:, 2:].expand(M, N))
    # back: three channels of dY through two ranks into every channel of dX
    dY = torch.zeros(M, N, dtype=BF, device="cuda")
    dY[:, :3] = v
    LB, LA = torch.zeros_like(LB), torch.zeros_like(LA)
    LA[0, :3, 0], LA[0, :2, R - 1], LB[0, 0], LB[0, R - 1] = 1.0, -1.0, 1.0, 1.0
    dX = rtl.rtl_adapters_backward(X, LA, LB, plan, None, dY, need_dw=False)[0]
    assert torch.equal(dX, v[:, 2:].expand(M, K))
