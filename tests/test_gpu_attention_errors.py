"""How far the outputs are off as a whole.  The bounds of single elements count every rounding at
its worst and all of them in step, many times what long sums of them make in earnest; a mistake
that costs a few percent of an output can stay inside.  Here the norm of the difference over a
sequence and head (a product's row) is held to the roundings' own size."""
import math

import pytest
import torch

import attention_reference as ref
from gpu_harness import log
from test_gpu_attention import (CACHE_CASES, CROSS_CASES, LARGE_CASES, _cache, _run_cache,
                                _starts)
from test_gpu_matvec import _case

pytestmark = pytest.mark.gpu

# Relative to the norm: the outputs' rounding at most 2^-8 (every element at half a step), and once
# more half of that for what stands before it: weights' roundings of 2^-11 and below and those of
# the query (2^-15 of its largest element, which in a score of 128 products of N(0, 1) queries
# and keys is 2^-13), independent of each other and weighted like the outputs themselves.
TOLERANCE = 1.5 * ref.BF16


@pytest.fixture(scope="module")
def rudder():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    from w4a4_quantized_gemm_rudder_amd import rudder as r
    r.load_library()
    return r


def _assert_close(name, got, want):
    got = got.double().cpu()
    assert torch.isfinite(got).all(), name
    off, size = float((got - want).norm()), float(want.norm())
    assert off <= TOLERANCE * size, f"{name}: off by {off / max(size, 1e-300):.5f} of the norm"


@pytest.mark.parametrize("counts,lens,Hq,Hkv,D,causal,heads",
                         [(*c, None) for c in CACHE_CASES] + LARGE_CASES)
def test_cache_attention(rudder, counts, lens, Hq, Hkv, D, causal, heads):
    log(f"case cache norms {counts} {lens} Hq={Hq} Hkv={Hkv} D={D} causal={causal}")
    g = torch.Generator().manual_seed(101)
    codes, scales, table = _cache(g, lens, Hkv, D)
    starts = _starts(counts)
    q = torch.randn(int(starts[-1]), Hq, D, generator=g).to(torch.bfloat16)
    sm = 1 / math.sqrt(D)
    want, _ = ref.cache_attention(q, starts, lens, table, codes, scales, sm, causal, heads)
    got = _run_cache(rudder, q, starts, lens, table, codes, scales, sm, causal)
    for b in range(len(lens)):
        for h in range(Hq) if heads is None else heads:
            at = slice(int(starts[b]), int(starts[b + 1]))
            _assert_close(f"{b} {h}", got[at, h], want[at, h])


@pytest.mark.parametrize("counts,lens,Hq,Hkv,D", CROSS_CASES + [
    ([300, 41], [1100, 1030], 4, 2, 128), ([600], [2000], 2, 2, 64)])
def test_cross_attention(rudder, counts, lens, Hq, Hkv, D):
    log(f"case cross norms {counts} {lens} Hq={Hq} Hkv={Hkv} D={D}")
    g = torch.Generator().manual_seed(102)
    starts, kv_start = _starts(counts), _starts(lens)[:-1]
    q = torch.randn(int(starts[-1]), Hq, D, generator=g).to(torch.bfloat16)
    kv = torch.randn(sum(lens), 2 * Hkv, D, generator=g).to(torch.bfloat16)
    sm = 1 / math.sqrt(D)
    want, _ = ref.cross_attention(q, kv[:, :Hkv], kv[:, Hkv:], starts, kv_start, lens, sm)
    dev = kv.cuda()
    got = rudder.cross_attention(q.cuda(), dev[:, :Hkv], dev[:, Hkv:], starts.cuda(),
                                 kv_start.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                                 max(counts), max(lens), sm)
    for b in range(len(lens)):
        for h in range(Hq):
            at = slice(int(starts[b]), int(starts[b + 1]))
            _assert_close(f"{b} {h}", got[at, h], want[at, h])


# rows of one, two and four channel tiles a workgroup, whole and split K loops
MATVEC = [(1, 2048, 48, 128), (3, 8192, 93, 128), (1, 16384, 40, 32), (7, 8320, 64, 64),
          (20, 8192, 100, 64), (1, 96, 24590, 32), (6, 640, 24577, 128), (9, 192, 6150, 64),
          (16, 4096, 12300, 32), (13, 4224, 6177, 32)]


@pytest.mark.parametrize("M,K,N,group", MATVEC)
def test_product(rudder, M, K, N, group):
    log(f"case matvec norms M={M} K={K} N={N} group={group}")
    x, W, _, _, _ = _case(M, K, N, group, 103)
    q, s = ref.group_codes(W, group)
    want, _ = ref.matvec(x, q, s, group)
    Wq, gs = rudder.quantize_weights_grouped(W.cuda(), group)
    y = rudder.matvec_w4(x.cuda(), Wq, gs, N, group)
    for m in range(M):
        _assert_close(f"row {m}", y[m], want[m])


@pytest.mark.parametrize("M,K,N,group", MATVEC)
def test_exact_products(rudder, M, K, N, group):
    """Integer activations, weights on a grid of 1/8 whose every group has an element of 7/8: the
    scales are 1/8 and every sum is exact in 32 bits, in every variant; a missing or repeated
    input channel shows."""
    log(f"case matvec exact M={M} K={K} N={N} group={group}")
    g = torch.Generator().manual_seed(104)
    x = torch.randint(1, 3, (M, K), generator=g) * (torch.randint(0, 2, (M, K), generator=g) * 2
                                                    - 1)
    x = x.to(torch.bfloat16)
    W = torch.randint(-7, 8, (K, N), generator=g).float() / 8
    W[::group] = 7 / 8
    W = W.to(torch.bfloat16)
    Wq, gs = rudder.quantize_weights_grouped(W.cuda(), group)
    y = rudder.matvec_w4(x.cuda(), Wq, gs, N, group)
    assert torch.equal(y.cpu(), (x.double() @ W.double()).to(torch.bfloat16))
