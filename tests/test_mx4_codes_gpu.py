"""Code bytes of the microscaled 4-bit format, the sign of zero included: comparing values cannot
tell the elements 0 and -0 apart."""
import numpy as np
import pytest
import torch

from dropless_mixture_experts_dmoe_b200 import binding as B

import serving_ref as R

pytestmark = pytest.mark.gpu


def expected_codes(x: torch.Tensor) -> torch.Tensor:
    """[rows, cols / 2] bytes from the definition: the magnitude's place on the grid and x's own sign
    bit; zero bytes in a block with an inf or NaN."""
    v = x.double().cpu().numpy()
    q, e = R.mx4_blocks(v)
    code = np.searchsorted(R.E2M1, np.abs(q)).reshape(v.shape) + 8 * np.signbit(v)
    code = np.where(np.repeat(np.isnan(e), 32, axis=1), 0, code)
    return torch.from_numpy((code[:, 0::2] | code[:, 1::2] << 4).astype(np.uint8)).cuda()


def test_codes_of_every_bf16_value():
    """All 65536 bit patterns as a column of a block whose other values put it anywhere on the grid."""
    val = torch.arange(65536, dtype=torch.int32, device="cuda").to(torch.int16).view(torch.bfloat16)
    rows = []
    for lead in (0.0, -0.0, 1.0, 6.0, 2.0 ** -120, 2.0 ** -133, 3e38):
        blk = torch.full((65536, 32), lead, dtype=torch.bfloat16, device="cuda")
        blk[:, 3] = val
        blk[:, 5] = -lead
        rows.append(blk.reshape(-1, 128))
    x = torch.cat(rows)
    q = B.Mx4.empty(*x.shape)
    q.codes.fill_(0xAA)
    B.dmoe_mx4_quantize(x, q)
    torch.cuda.synchronize()
    want = expected_codes(x)
    # the input holds zeros of both signs and negative values that round to zero
    assert all(bool(((want & 15) == z).any()) for z in (0, 8))
    assert torch.equal(q.codes, want)


def test_dequantize_keeps_the_sign_of_zero():
    """Every pair of elements under every scale but NaN, bit for bit: element times scale, rounded
    once to bf16 (exact, or an inf)."""
    s = torch.arange(255, dtype=torch.uint8, device="cuda")
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").reshape(1, -1).repeat(255, 1)
    scales = torch.zeros(B.Mx4.scales_shape(255, 512), dtype=torch.uint8, device="cuda")
    r = torch.arange(255, device="cuda")
    for b in range(16):
        scales[r // 128, b // 4, r % 32, r % 128 // 32, b % 4] = s
    out = torch.empty((255, 512), dtype=torch.bfloat16, device="cuda")
    B.dmoe_mx4_dequantize(B.Mx4(codes.contiguous(), scales), out)
    el = torch.stack((codes & 15, codes >> 4), -1).reshape(255, 512)
    mag = torch.from_numpy(R.E2M1).cuda()[(el & 7).long()]
    val = torch.where(el >= 8, -mag, mag) * torch.exp2(s.double() - 127)[:, None]
    want = val.float().bfloat16()
    assert bool((torch.signbit(want) & (want == 0)).any())
    assert torch.equal(out.view(torch.int16), want.view(torch.int16))
