"""The paged 8-bit cache: codes and scales of appends bit for bit against the
rule applied page by page, values read back exactly."""
import pytest
import torch

import attention_reference as ref
from gpu_harness import log

pytestmark = pytest.mark.gpu
PAGE = 64


@pytest.fixture(scope="module")
def rudder():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    from w4a4_quantized_gemm_rudder_amd import rudder as r
    r.load_library()
    return r


def _pool(g, B, width, H, D, extra=2):
    P = B * width + extra
    codes = torch.randint(-127, 128, (P, H, 2, PAGE * D), generator=g).to(torch.int8)
    scales = torch.rand(P, H, 2, generator=g) * 0.03
    table = torch.randperm(P, generator=g)[:B * width].view(B, width).to(torch.int32)
    return codes, scales, table


def _rows(g, T, H, D):
    """K and V as they lie in a wider buffer, magnitudes that differ from row to row."""
    buf = torch.randn(T, 3 * H + 1, D, generator=g) * (4.0 ** torch.randn(T, 1, 1, generator=g))
    buf = buf.to(torch.bfloat16)
    return buf[:, :H], buf[:, 2 * H:3 * H], buf


def _append(rudder, K, V, buf, starts, pos, table, codes, scales, H, D, max_rows):
    dev = buf.cuda()
    dc, ds = codes.cuda(), scales.cuda()
    k, v = dev[:, :H], dev[:, 2 * H:3 * H]
    rudder.cache_append(k, v, starts.cuda(), pos.cuda(), table.cuda(), max_rows, dc, ds)
    return dc, ds


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,counts,pos", [
    (1, [1], [0]),
    (2, [1, 1, 1], [63, 64, 5]),
    (3, [64, 0, 130], [0, 10, 1]),
    (2, [200, 3], [61, 190]),
    (1, [63, 65, 1], [1, 63, 0]),
])
def test_append_bit_exact(rudder, D, H, counts, pos):
    log(f"case append D={D} H={H} counts={counts} pos={pos}")
    g = torch.Generator().manual_seed(11)
    B = len(counts)
    width = max((p + n + PAGE - 1) // PAGE for p, n in zip(pos, counts)) + 1
    codes, scales, table = _pool(g, B, width, H, D)
    starts = torch.tensor([0] + counts).cumsum(0).to(torch.int32)
    T = int(starts[-1]) + 2                                  # rows behind the last sequence
    K, V, buf = _rows(g, T, H, D)
    pos = torch.tensor(pos, dtype=torch.int32)
    dc, ds = _append(rudder, K, V, buf, starts, pos, table, codes, scales, H, D, max(counts))
    ref.append(K, V, starts, pos, table, codes, scales)
    assert torch.equal(ds.cpu(), scales)
    assert torch.equal(dc.cpu(), codes)


@pytest.mark.parametrize("D", [64, 128])
def test_append_one_by_one(rudder, D):
    """A page filled token by token, its scale growing on the way; the same token again changes
    nothing; zeros in front give scale 0."""
    log(f"case append one by one D={D}")
    g = torch.Generator().manual_seed(12)
    H = 2
    codes, scales, table = _pool(g, 1, 2, H, D)
    dc, ds = codes.cuda(), scales.cuda()
    starts = torch.tensor([0, 1], dtype=torch.int32)
    for t in range(70):
        K, V, buf = _rows(g, 1, H, D)
        if t < 2:
            buf.zero_()
        pos = torch.tensor([t], dtype=torch.int32)
        for _ in range(2):
            dev = buf.cuda()
            rudder.cache_append(dev[:, :H], dev[:, 2 * H:3 * H], starts.cuda(), pos.cuda(),
                                table.cuda(), 1, dc, ds)
        ref.append(buf[:, :H], buf[:, 2 * H:3 * H], starts, pos, table, codes, scales)
        assert torch.equal(ds.cpu(), scales), t
        assert torch.equal(dc.cpu(), codes), t


def test_append_keeps_out_of_absent_pages(rudder):
    """Pages outside the pool, positions behind the table, negative positions and rows beyond
    max_rows are not written; their neighbours are."""
    log("case append absent pages")
    g = torch.Generator().manual_seed(13)
    H, D, P = 2, 64, 6
    codes, scales, _ = _pool(g, 1, P, H, D, extra=0)
    codes, scales = codes[:P], scales[:P]
    table = torch.tensor([[0, -1, 1], [P, 2, 3], [4, 5, -7], [2 ** 31 - 1, 4, 5]],
                         dtype=torch.int32)
    counts = [180, 100, 30, 40]
    starts = torch.tensor([0] + counts).cumsum(0).to(torch.int32)
    K, V, buf = _rows(g, int(starts[-1]), H, D)
    pos = torch.tensor([10, 40, -1, 2 ** 31 - 20], dtype=torch.int32)
    dc, ds = _append(rudder, K, V, buf, starts, pos, table, codes, scales, H, D, 170)
    cut = starts.clone()
    # the first sequence's rows beyond 170 are not processed: the rule on its first 170
    for b, (n, p) in enumerate(zip(counts, pos.tolist())):
        if p < 0 or p > 10 ** 6:
            continue
        n = min(n, 170)
        two = torch.tensor([int(cut[b]), int(cut[b]) + n], dtype=torch.int32)
        ref.append(K, V, two, pos[b:b + 1], table[b:b + 1], codes, scales)
    assert torch.equal(ds.cpu(), scales)
    assert torch.equal(dc.cpu(), codes)


@pytest.mark.parametrize("D", [64, 128])
def test_dequant(rudder, D):
    log(f"case dequant D={D}")
    g = torch.Generator().manual_seed(14)
    codes, scales, _ = _pool(g, 1, 7, 3, D)
    P = len(codes)
    pages = torch.tensor([3, 0, 3, P - 1], dtype=torch.int32)     # one of them twice
    k, v = rudder.cache_dequant(codes.cuda(), scales.cuda(), pages.cuda())
    wk, wv = ref.values(codes, scales, pages)
    assert torch.equal(k.cpu(), wk.float()) and torch.equal(v.cpu(), wv.float())
    bad = torch.tensor([-1, 1, P], dtype=torch.int32)
    k, v = rudder.cache_dequant(codes.cuda(), scales.cuda(), bad.cuda())
    wk, wv = ref.values(codes, scales, bad.clamp(1, 1))
    for got, want in ((k.cpu(), wk), (v.cpu(), wv)):
        assert not got[0].any() and not got[2].any()
        assert torch.equal(got[1], want[1].float())
    k, v = rudder.cache_dequant(codes.cuda(), scales.cuda(), pages[:0].cuda())
    assert k.shape == (0, 3, PAGE, D)
