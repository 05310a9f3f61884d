"""Few-row products with group-scaled 4-bit weights: preparation bit for bit,
outputs against the 64-bit form and, on data whose sums are exact, bit for
bit."""
import pytest
import torch

import attention_reference as ref
from gpu_harness import log

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rudder():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    from w4a4_quantized_gemm_rudder_amd import rudder as r
    r.load_library()
    return r


def _case(M, K, N, group, seed, S=3):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g)
    x[:, torch.randperm(K, generator=g)[:max(1, K // 50)]] *= 30.0
    W = torch.randn(K, N, generator=g) * 0.02
    W[:group, N // 2] = 0.0                                  # a group of zeros
    sid = torch.randint(0, S, (M,), generator=g).to(torch.uint8)
    a = torch.rand(S, N, generator=g) * 0.2 + 0.9
    b = torch.randn(S, N, generator=g) * 0.01
    return x.to(torch.bfloat16), W.to(torch.bfloat16), sid, a, b


@pytest.mark.parametrize("K,N,group", [(32, 1, 32), (96, 17, 32), (320, 33, 64), (384, 40, 128),
                                       (128, 16, 128)])
def test_preparation_bit_exact(rudder, K, N, group):
    log(f"case prepare K={K} N={N} group={group}")
    _, W, _, _, _ = _case(1, K, N, group, 1)
    q, s = ref.group_codes(W, group)
    want, ws = ref.pack_grouped(q, s)
    Wq, gs = rudder.quantize_weights_grouped(W.cuda(), group)
    assert torch.equal(Wq.cpu(), want)
    assert torch.equal(gs.cpu().view(torch.int16).view(ws.shape), ws.view(torch.int16))


@pytest.mark.parametrize("comp", [False, True])
@pytest.mark.parametrize("M,K,N,group", [
    (1, 32, 1, 32), (1, 2048, 256, 128), (2, 96, 33, 32), (5, 320, 17, 64), (16, 1024, 100, 32),
    (17, 640, 48, 128), (40, 4096, 16, 64), (3, 8192, 31, 128), (1, 16384, 20, 32),
    (33, 256, 2050, 64),
    # two and four channel tiles a workgroup, the last one not full
    (1, 96, 24590, 32), (6, 128, 24577, 128), (9, 192, 6150, 64), (16, 96, 12300, 32),
    (13, 384, 12289, 128), (30, 64, 12340, 64), (21, 160, 6177, 32),
])
def test_product(rudder, M, K, N, group, comp):
    log(f"case matvec M={M} K={K} N={N} group={group} comp={comp}")
    x, W, sid, a, b = _case(M, K, N, group, 2)
    q, s = ref.group_codes(W, group)
    Wq, gs = rudder.quantize_weights_grouped(W.cuda(), group)
    if comp:
        want, bound = ref.matvec(x, q, s, group, sid, a, b)
        y = rudder.matvec_w4(x.cuda(), Wq, gs, N, group, sid.cuda(), a.cuda(), b.cuda())
    else:
        want, bound = ref.matvec(x, q, s, group)
        y = rudder.matvec_w4(x.cuda(), Wq, gs, N, group)
    ref.assert_within("Y", y, want, bound)


@pytest.mark.parametrize("M,K,N,group", [(1, 2048, 48, 128), (7, 416, 33, 32), (20, 8192, 17, 64)])
def test_exact_sums_bit_exact(rudder, M, K, N, group):
    """Integer activations and weights on a grid of 1/8 whose every group has an element of
    7/8: the scales are 1/8, every sum is exact in 32 bits, the output is its rounding."""
    log(f"case exact M={M} K={K} N={N} group={group}")
    g = torch.Generator().manual_seed(3)
    x = torch.randint(-8, 9, (M, K), generator=g).to(torch.bfloat16)
    W = torch.randint(-7, 8, (K, N), generator=g).double() / 8
    W[::group] = 7 / 8
    W = W.to(torch.bfloat16)
    Wq, gs = rudder.quantize_weights_grouped(W.cuda(), group)
    y = rudder.matvec_w4(x.cuda(), Wq, gs, N, group)
    assert torch.equal(y.cpu(), (x.double() @ W.double()).to(torch.bfloat16))


def test_rows_are_independent_and_nothing_else_is_written(rudder):
    """A row of NaN and one of infinities stay in their rows; what lies behind Y stays."""
    M, K, N, group = 6, 256, 40, 64
    log("case matvec non-finite rows")
    x, W, _, _, _ = _case(M, K, N, group, 4)
    Wq, gs = rudder.quantize_weights_grouped(W.cuda(), group)
    clean = rudder.matvec_w4(x.cuda(), Wq, gs, N, group)
    x[2], x[4, 7] = float("nan"), float("inf")
    buf = torch.full((M * N + 64,), -3.0, dtype=torch.bfloat16, device="cuda")
    rudder.rudder_matvec_w4(x.cuda(), None, Wq, gs, None, None, M, N, K, group, 1, buf)
    got = buf[:M * N].view(M, N)
    keep = [0, 1, 3, 5]
    assert torch.equal(got[keep], clean[keep])
    assert torch.isnan(got[2]).all()
    assert (buf[M * N:] == -3.0).all()


def test_codes_far_apart(rudder):
    """More than 4 GiB of codes: offsets pass 32 bits in preparation and product."""
    K, N, group, last = 16384, 530011, 128, 100
    log(f"case matvec far apart K={K} N={N}")
    g = torch.Generator().manual_seed(6)
    x = torch.randn(2, K, generator=g).to(torch.bfloat16)
    end = (torch.randn(K, last, generator=g) * 0.02).to(torch.bfloat16)
    W = torch.zeros(K, N, dtype=torch.bfloat16, device="cuda")
    W[:, -last:] = end.cuda()
    Wq, gs = rudder.quantize_weights_grouped(W, group)
    assert Wq.numel() > 1 << 32
    want, bound = ref.matvec(x, *ref.group_codes(end, group), group)
    y = rudder.matvec_w4(x.cuda(), Wq, gs, N, group)
    ref.assert_within("Y", y[:, -last:], want, bound)
    assert not y[:, :-last].any()


@pytest.mark.parametrize("M,K,N,group", [(1, 2048, 40, 128), (9, 512, 64, 32), (4, 1024, 48, 64)])
def test_activations_of_one_sign(rudder, M, K, N, group):
    """Activations of one sign (after a GELU) and in each group one of 2^18 under a code of 0: what
    the codes' offset adds to the sums and takes away again is far larger than the result.  A code
    with its offset is at most 31, so that every sum stays below 31 * (2^18 + 2 * 127) < 2^24 and
    is exact in 32 bits, whatever the order."""
    log(f"case one sign M={M} K={K} N={N} group={group}")
    g = torch.Generator().manual_seed(5)
    x = torch.randint(1, 3, (M, K), generator=g).to(torch.bfloat16)
    x[:, 7::group] = 2.0 ** 18
    W = torch.randint(-7, 8, (K, N), generator=g).float() / 8
    W[::group] = 7 / 8
    W[7::group] = 0.0
    W = W.to(torch.bfloat16)
    Wq, gs = rudder.quantize_weights_grouped(W.cuda(), group)
    y = rudder.matvec_w4(x.cuda(), Wq, gs, N, group)
    assert torch.equal(y.cpu(), (x.double() @ W.double()).to(torch.bfloat16))
