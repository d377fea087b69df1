"""The few-token layer over bf16 weights where H comes near fp32's largest value."""
import pytest
import torch

from dropless_mixture_experts_dmoe_b200 import binding as B

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 40])
def test_h_between_bf16s_largest_and_fp32s(T):
    """H = 2^64 (2^64 - 2^54) = 2^128 (1 - 2^-10) is finite in fp32 and rounds to an inf in bf16; with
    w2 = 2^-100, y is 2^28 (1 - 2^-10), which bf16 rounds to 2^28 (its step there is 2^20).  An H
    of 2^128 is an inf, and a NaN stays one."""
    h, f, E, k = 128, 128, 4, 1
    bf = dict(dtype=torch.bfloat16, device="cuda")
    w1, w3, w2 = torch.zeros(E, f, h, **bf), torch.zeros(E, f, h, **bf), torch.zeros(E, h, f, **bf)
    w1[:, 5, 0] = 2.0 ** 64
    w3[0, 5, 0], w3[0, 5, 1] = 2.0 ** 64, -2.0 ** 54
    w3[1, 5, 0], w3[1, 5, 1] = -2.0 ** 64, 2.0 ** 54
    w3[2, 5, 0] = 2.0 ** 64
    w3[3, 5, 0] = float("nan")
    w2[:, :, 5] = 2.0 ** -100
    x = torch.zeros(T, h, **bf)
    x[:, :2] = 1.0
    d = B.make_dims(T, h, f, E, k)
    for e, want in ((0, 2.0 ** 28), (1, -2.0 ** 28), (2, float("inf")), (3, float("nan"))):
        bufs = B.FewBuffers(d)
        bufs.top_experts.fill_(e)
        bufs.weights.fill_(1.0)
        y = torch.empty_like(x)
        B.dmoe_forward_few(d, x, None, w1, w3, w2, bufs, y)
        torch.cuda.synchronize()
        right = y.isnan() if want != want else y == want
        assert bool(right.all()), (e, y[0, 0].item())
