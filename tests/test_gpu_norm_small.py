"""Codes of norm rows so small that a step size of their own has no reciprocal in 32 bits."""
import pytest
import torch

import attention_reference as aref
import block_reference as ref
from gpu_harness import log, tile_for

pytestmark = pytest.mark.gpu
INT, E2M3 = 0, 1


@pytest.fixture(scope="module")
def rudder():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    from w4a4_quantized_gemm_rudder_amd import rudder as r
    r.load_library()
    return r


@pytest.mark.parametrize("bits,codes", [(8, INT), (4, INT), (4, E2M3)])
@pytest.mark.parametrize("M,K", [(40, 128), (40, 4160), (600, 128), (600, 2112), (40, 8256)])
def test_small_rows(rudder, M, K, bits, codes):
    """Rows of 2^-112 down to the smallest numbers, zeros among them: step sizes up to 2^-128, whose
    reciprocals pass 32 bits, count as 0, and so do the row's codes; above it codes are the rule's.  No
    element is further from its value than half a step, or Qa 2^-128."""
    log(f"case norm small rows M={M} K={K} bits={bits} codes={codes}")
    g = torch.Generator().manual_seed(M + K)
    x = torch.randn(M, K, generator=g)
    x[:, ::3] = 0
    x = (x.double() * 2.0 ** (-112.0 - torch.arange(M) % 24)[:, None]).to(torch.bfloat16)
    gamma, smooth = torch.ones(K), torch.rand(K, generator=g) + 0.5
    y, _ = ref.norm(x, gamma, 1.0)
    u, q = y.float() * smooth, ref.QMAX[bits]
    s = (u.abs().amax(1).double() / q).float()
    s = torch.where(s <= 2.0 ** -128, 0.0, s)
    assert (s == 0).any() and (s > 0).any() and (u[s == 0] != 0).any()
    c = torch.round(torch.clamp(u * aref.recip(s)[:, None], -q, q)).to(torch.int8)
    xq, rs = rudder.norm_quant(x.cuda(), gamma.cuda(), smooth.cuda(), 1.0, bits, codes)
    assert torch.equal(rs.cpu(), s)
    assert torch.equal(xq.cpu(), torch.from_numpy(tile_for(codes, c.numpy(), bits)))
    values = rudder.dequant_act(xq, rs, M, K, bits, codes).cpu().double()
    assert (values[u == 0] == 0).all()
    # beside half a step: rounding of the step (2^-22 of it down there) and of the value, times Qa
    far = torch.where(s > 0, s.double() * (0.5 + q * 2.0 ** -20), q * 2.0 ** -128)
    assert ((values - u.double()).abs() <= far[:, None]).all()
