"""Attention over the 8-bit cache and cross attention against the 64-bit form,
within bounds that count the kernels' roundings."""
import math

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


def _cache(g, lens, H, D, spread=0.0):
    """Codes (garbage behind each length), scales and a table with absent pages behind."""
    need = [(n + PAGE - 1) // PAGE for n in lens]
    width = max(max(need), 1) + 1
    P = sum(need) + 2
    codes = torch.randint(-128, 128, (P, H, 2, PAGE * D), generator=g).to(torch.int8)
    scales = (torch.rand(P, H, 2, generator=g) + 0.5) * 0.01
    scales = scales * 2.0 ** (spread * (torch.rand(P, H, 2, generator=g) - 0.5))
    order = torch.randperm(P, generator=g)
    table = torch.full((len(lens), width), -5, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n].to(torch.int32)
        at += n
    return codes, scales, table


def _starts(counts):
    return torch.tensor([0] + counts).cumsum(0).to(torch.int32)


def _run_cache(rudder, q, starts, lens, table, codes, scales, sm, causal, max_rows=None,
               max_kv=None):
    counts = (starts[1:] - starts[:-1]).tolist()
    return rudder.cache_attention(
        q.cuda(), starts.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), table.cuda(),
        codes.cuda(), scales.cuda(), max(counts) if max_rows is None else max_rows,
        max(lens) if max_kv is None else max_kv, sm, causal)


CACHE_CASES = [
    # counts, lens, Hq, Hkv, D, causal
    ([1], [1], 1, 1, 64, True),
    ([1], [0], 2, 2, 128, True),                       # an empty cache
    ([1, 1, 1, 1], [1, 64, 65, 777], 4, 4, 128, True),
    ([1, 1], [2000, 63], 8, 2, 64, True),              # grouped heads
    ([1, 1], [300, 129], 6, 2, 128, False),            # a group of three
    ([1], [9000], 2, 1, 128, True),                    # split over the tokens
    ([5, 0, 2], [40, 100, 2], 3, 1, 64, True),         # an empty sequence
    ([7, 3], [4, 0], 2, 2, 64, True),                  # rows in front of the first token
    ([33, 129], [200, 129], 4, 2, 128, True),
    ([200], [200], 2, 2, 64, True),
    ([96, 96], [4100, 4100], 2, 2, 128, False),
    ([130, 40], [700, 650], 12, 4, 64, False),
    ([64, 16], [128, 500], 16, 1, 128, True),          # one cached head
    ([300], [2500], 1, 1, 128, True),
    ([20], [3000], 4, 4, 64, True),
]


@pytest.mark.parametrize("counts,lens,Hq,Hkv,D,causal", CACHE_CASES)
def test_cache_attention(rudder, counts, lens, Hq, Hkv, D, causal):
    log(f"case cache {counts} {lens} Hq={Hq} Hkv={Hkv} D={D} causal={causal}")
    g = torch.Generator().manual_seed(21)
    codes, scales, table = _cache(g, lens, Hkv, D)
    starts = _starts(counts)
    T = int(starts[-1])
    q = (torch.randn(T, Hq, D, generator=g) * 2).to(torch.bfloat16)
    sm = 1 / math.sqrt(D)
    want, bound = ref.cache_attention(q, starts, lens, table, codes, scales, sm, causal)
    got = _run_cache(rudder, q, starts, lens, table, codes, scales, sm, causal)
    ref.assert_within("O", got, want, bound)


# Row tiles left over after whole rounds of workgroups are split over the tokens, rows of 256 go
# to a workgroup where all see long stretches: every head takes part, a few are compared.
LARGE_CASES = [
    # counts, lens, Hq, Hkv, D, causal, heads
    ([300, 41], [1100, 1030], 4, 2, 128, False, [0, 3]),       # 256 rows a workgroup
    ([300, 130, 200], [1100, 0, 63], 2, 2, 128, False, [0, 1]),
    ([260, 300], [64, 1200], 1, 1, 128, False, [0]),
    ([1100, 700], [1025, 1500], 32, 32, 128, False, [0, 17, 31]),
    ([700], [1400], 96, 96, 64, True, [0, 1, 50, 95]),
    ([257, 513], [1100, 1600], 96, 48, 128, True, [0, 95]),
]


@pytest.mark.parametrize("counts,lens,Hq,Hkv,D,causal,heads", LARGE_CASES)
def test_cache_attention_large(rudder, counts, lens, Hq, Hkv, D, causal, heads):
    log(f"case large {counts} {lens} Hq={Hq} Hkv={Hkv} D={D} causal={causal}")
    g = torch.Generator().manual_seed(31)
    codes, scales, table = _cache(g, lens, Hkv, D)
    starts = _starts(counts)
    q = (torch.randn(int(starts[-1]), Hq, D, generator=g) * 2).to(torch.bfloat16)
    sm = 1 / math.sqrt(D)
    want, bound = ref.cache_attention(q, starts, lens, table, codes, scales, sm, causal, heads)
    got = _run_cache(rudder, q, starts, lens, table, codes, scales, sm, causal)
    ref.assert_within("O", got[:, heads], want[:, heads], bound[:, heads])


@pytest.mark.parametrize("counts,lens,Hq,Hkv,D,heads", [
    ([300, 41], [1100, 1030], 4, 2, 128, [0, 3]),
    ([1100, 700], [1025, 1500], 32, 32, 128, [0, 31]),
    ([700], [1400], 96, 96, 64, [0, 95]),
])
def test_cross_attention_large(rudder, counts, lens, Hq, Hkv, D, heads):
    log(f"case cross large {counts} {lens} Hq={Hq} Hkv={Hkv} D={D}")
    g = torch.Generator().manual_seed(32)
    starts, kv_start = _starts(counts), _starts(lens)[:-1]
    q = (torch.randn(int(starts[-1]), Hq, D, generator=g) * 2).to(torch.bfloat16)
    kv = torch.randn(sum(lens), 2 * Hkv, D, generator=g).to(torch.bfloat16)
    sm = 1 / math.sqrt(D)
    want, bound = ref.cross_attention(q, kv[:, :Hkv], kv[:, Hkv:], starts, kv_start, lens, sm,
                                      heads)
    dev = kv.cuda()
    got = rudder.cross_attention(q.cuda(), dev[:, :Hkv], dev[:, Hkv:], starts.cuda(),
                                 kv_start.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                                 max(counts), max(lens), sm)
    ref.assert_within("O", got[:, heads], want[:, heads], bound[:, heads])


@pytest.mark.parametrize("rows,ctx", [(3, 90), (3, 3000), (150, 300), (300, 1200)])
def test_rows_that_are_not_finite(rudder, rows, ctx):
    """A query row with a NaN, an infinity of either sign or both gives NaN in its row and head
    and leaves the others, in every kernel; a negative softmax scale."""
    log(f"case not finite rows={rows} ctx={ctx}")
    g = torch.Generator().manual_seed(33)
    Hq, Hkv, D = 2, 1, 128
    codes, scales, table = _cache(g, [ctx], Hkv, D)
    q = torch.randn(rows, Hq, D, generator=g).to(torch.bfloat16)
    clean = q.clone()
    bad = [(0, 0, float("nan")), (1, 1, float("inf")), (2, 0, -float("inf"))]
    for r, h, v in bad:
        q[r, h, 7 * r] = v
    starts = _starts([rows])
    for causal in (False, True):
        want, bound = ref.cache_attention(clean, starts, [ctx], table, codes, scales, -0.1, causal)
        got = _run_cache(rudder, q, starts, [ctx], table, codes, scales, -0.1, causal).cpu()
        for r, h, _ in bad:
            assert torch.isnan(got[r, h]).all(), (r, h)
            got[r, h], want[r, h], bound[r, h] = 0.0, 0.0, 0.0
        ref.assert_within("O", got, want, bound)


@pytest.mark.parametrize("rows,ctx", [(3, 2), (3, 0), (150, 100), (150, 0), (300, 2000)])
def test_masked_rows_that_are_not_finite(rudder, rows, ctx):
    """A row whose mask leaves nothing gives zeros whatever its query, in every kernel, also where
    the sequence stands beside one that is split over its tokens."""
    log(f"case masked, not finite rows={rows} ctx={ctx}")
    g = torch.Generator().manual_seed(36)
    D, lens = 128, [ctx, 4000]
    codes, scales, table = _cache(g, lens, 1, D)
    q = torch.full((2 * rows, 1, D), float("nan"), dtype=torch.bfloat16)
    q[rows:] = torch.randn(rows, 1, D, generator=g).to(torch.bfloat16)
    starts = _starts([rows, rows])
    for causal in (False, True):
        got = _run_cache(rudder, q, starts, lens, table, codes, scales, 0.1, causal).cpu()
        none = rows if ctx == 0 else max(rows - ctx, 0) if causal else 0
        assert not got[:none].any()
        assert torch.isnan(got[none:rows]).all()
        assert torch.isfinite(got[rows:]).all()


@pytest.mark.parametrize("sm", [0.0, -2.0])
@pytest.mark.parametrize("rows,causal", [(2, True), (40, True), (300, False)])
def test_scales_of_the_softmax(rudder, rows, causal, sm):
    """A softmax scale of zero weighs the visible tokens alike, a negative one turns them round."""
    log(f"case softmax scale {sm} rows={rows}")
    g = torch.Generator().manual_seed(37)
    D, lens = 128, [1100]
    codes, scales, table = _cache(g, lens, 1, D)
    q = torch.randn(rows, 1, D, generator=g).to(torch.bfloat16)
    starts = _starts([rows])
    want, bound = ref.cache_attention(q, starts, lens, table, codes, scales, sm, causal)
    got = _run_cache(rudder, q, starts, lens, table, codes, scales, sm, causal)
    ref.assert_within("O", got, want, bound)


@pytest.mark.parametrize("rows,causal", [(1, True), (30, True), (280, False)])
def test_pages_and_rows_far_apart(rudder, rows, causal):
    """Pages behind 4 GiB of codes, and query and output rows 2^25 elements apart (280 of them
    span 17 GiB): offsets pass 32 bits."""
    log(f"case far apart rows={rows}")
    g = torch.Generator().manual_seed(38)
    Hkv, D, ctx, far = 32, 128, 1100, 8400                     # pages of 512 KiB
    small_codes, small_scales, small_table = _cache(g, [ctx], Hkv, D)
    n = len(small_codes)
    codes = torch.zeros(far + n, Hkv, 2, PAGE * D, dtype=torch.int8, device="cuda")
    scales = torch.zeros(far + n, Hkv, 2, device="cuda")
    codes[far:], scales[far:] = small_codes.cuda(), small_scales.cuda()
    table = torch.where(small_table >= 0, small_table + far, small_table)
    small = torch.randn(rows, Hkv, D, generator=g).to(torch.bfloat16)
    apart = (1 << 25) if rows > 100 else (1 << 27)
    wide = torch.empty((rows - 1) * apart + 2 * Hkv * D, dtype=torch.bfloat16, device="cuda")
    q = wide.as_strided((rows, Hkv, D), (apart, D, 1))
    out = wide.as_strided((rows, Hkv, D), (apart, D, 1), Hkv * D)
    q.copy_(small.cuda())
    starts, heads = _starts([rows]), [0, 31]
    nb = rudder.attention_workspace_bytes(1, rows, rows, ctx, Hkv, Hkv, D)
    ws = torch.empty(max(nb, 16), dtype=torch.uint8, device="cuda")
    rudder.rudder_cache_attention(q, starts.cuda(), torch.tensor([ctx], dtype=torch.int32).cuda(),
                                  table.cuda(), codes, scales, 1, rows, rows, ctx, table.shape[1],
                                  far + n, Hkv, Hkv, D, 0.1, causal, ws, out)
    got = out.cpu()[:, heads]
    want, bound = ref.cache_attention(small[:, heads], starts, [ctx], small_table,
                                      small_codes[:, heads], small_scales[:, heads], 0.1, causal)
    ref.assert_within("O", got, want, bound)
    assert torch.equal(q.cpu(), small)
    # the same pages again, written by an append over them
    k = torch.randn(ctx, Hkv, D, generator=g).to(torch.bfloat16)
    rudder.cache_append(k.cuda(), k.cuda(), _starts([ctx]).cuda(),
                        torch.zeros(1, dtype=torch.int32).cuda(), table.cuda(), ctx, codes, scales)
    pages = table[0, :(ctx + PAGE - 1) // PAGE].cuda()
    K, V = rudder.cache_dequant(codes, scales, pages)
    back = K[:, 31].reshape(-1, D)[:ctx].cpu()
    # half a step of a block whose largest magnitude is below 6
    assert (back - k[:, 31].float()).abs().max() <= 6 / 127 / 2 * (1 + 2.0 ** -20)
    K, V = (x.transpose(1, 2).reshape(-1, Hkv, D)[:ctx] for x in (K, V))
    assert torch.equal(K, V)                       # the slots behind ctx keep their old codes
    assert not codes[:far].any()


@pytest.mark.parametrize("D,causal", [(64, True), (128, False), (128, True)])
def test_loose_bounds(rudder, D, causal):
    """max_rows and max_kv far above what the sequences hold, and sequences of very different
    lengths beside each other: other kernels and splits, the same results within the bounds."""
    log(f"case loose bounds D={D} causal={causal}")
    g = torch.Generator().manual_seed(40)
    counts, lens = [1, 5, 0, 40, 3], [1, 700, 64, 2100, 3]
    codes, scales, table = _cache(g, lens, 2, D)
    starts = _starts(counts)
    q = torch.randn(int(starts[-1]), 4, D, generator=g).to(torch.bfloat16)
    want, bound = ref.cache_attention(q, starts, lens, table, codes, scales, 0.1, causal)
    for max_rows, max_kv in ((40, 2100), (49, 100000), (1 << 20, 1 << 20), (129, 2304)):
        got = _run_cache(rudder, q, starts, lens, table, codes, scales, 0.1, causal, max_rows,
                         max_kv)
        ref.assert_within(f"O {max_rows} {max_kv}", got, want, bound)


@pytest.mark.parametrize("D", [64, 128])
def test_many_tokens(rudder, D):
    """Single tokens of many sequences with ragged contexts: whole stretches, two pieces and three
    a pair."""
    g = torch.Generator().manual_seed(41)
    for B, H, ctx in ((20, 8, 300), (24, 12, 2100), (90, 5, 1800)):
        log(f"case many tokens D={D} B={B} H={H} ctx={ctx}")
        lens = torch.randint(1, ctx + 1, (B,), generator=g).tolist()
        lens[3], lens[4] = ctx, 0
        codes, scales, table = _cache(g, lens, H, D)
        starts = _starts([1] * B)
        q = torch.randn(B, H, D, generator=g).to(torch.bfloat16)
        heads = [0, H - 1]
        want, bound = ref.cache_attention(q, starts, lens, table, codes, scales, 0.1, True, heads)
        got = _run_cache(rudder, q, starts, lens, table, codes, scales, 0.1, True)
        ref.assert_within("O", got[:, heads], want[:, heads], bound[:, heads])


def test_long_tables(rudder):
    """More than 64 pages a wave and more than 64 pieces' worth of tiles: page numbers are
    fetched anew."""
    log("case long tables")
    g = torch.Generator().manual_seed(34)
    D, ctx = 64, 64 * 700 + 5
    codes, scales, table = _cache(g, [ctx], 1, D)
    table[0, 600] = -1
    for rows, B in ((1, 1), (1, 300), (20, 1), (140, 60)):
        # many sequences leave one piece to each, so that a wave walks all of the table
        q = torch.randn(B * rows, 1, D, generator=g).to(torch.bfloat16)
        starts = (torch.arange(B + 1) * rows).to(torch.int32)
        two = starts[:2]
        want, bound = ref.cache_attention(q[:rows], two, [ctx], table, codes, scales, 0.1, False)
        got = _run_cache(rudder, q, starts, [ctx] * B, table.expand(B, -1).contiguous(), codes,
                         scales, 0.1, False)
        ref.assert_within(f"O rows={rows} B={B}", got[:rows], want, bound)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("counts,lens", [([1, 1], [500, 1000]), ([70], [400])])
def test_scales_of_all_sizes(rudder, D, counts, lens):
    """V scales from 2^-35 to 2^25 (and K scales to match) and blocks of zeros: the pages'
    shares of the sum stay right however far apart their scales are."""
    log(f"case scales D={D} {counts} {lens}")
    g = torch.Generator().manual_seed(22)
    codes, scales, table = _cache(g, lens, 1, D)
    P = len(codes)
    scales[:, :, 1] = 2.0 ** torch.randint(-35, 26, (P, 1), generator=g)
    for p in table[0, [1, 3]].tolist():                       # zero blocks
        codes[p, :, 1] = 0
        scales[p, :, 1] = 0
    starts = _starts(counts)
    q = torch.randn(int(starts[-1]), 2, D, generator=g).to(torch.bfloat16)
    want, bound = ref.cache_attention(q, starts, lens, table, codes, scales, 0.05, False)
    got = _run_cache(rudder, q, starts, lens, table, codes, scales, 0.05, False)
    ref.assert_within("O", got, want, bound)


def test_zero_and_far_blocks_keep_their_weight(rudder):
    """A block of zeros beside one of large values: the zeros' tokens still count in the
    denominator."""
    log("case zero blocks")
    D = 64
    codes = torch.zeros(2, 1, 2, PAGE * D, dtype=torch.int8)
    scales = torch.zeros(2, 1, 2)
    codes[1, 0, 1], scales[1, 0, 1] = 100, 2.0 ** 30
    table = torch.tensor([[0, 1]], dtype=torch.int32)
    for order in ([0, 1], [1, 0]):
        t = table[:, order]
        q = torch.ones(1, 1, D, dtype=torch.bfloat16)
        got = _run_cache(rudder, q, _starts([1]), [128], t, codes, scales, 1.0, False)
        # every weight is 1 / 128, half of the tokens have the value 100 * 2^30
        assert (got == 50 * 2.0 ** 30).all()


@pytest.mark.parametrize("D,rows", [(64, 1), (128, 1), (128, 40)])
def test_sharp_and_large_queries(rudder, D, rows):
    """Queries of very different magnitudes: near one-hot rows, rows of zeros and rows near the
    type's ends."""
    log(f"case sharp D={D} rows={rows}")
    g = torch.Generator().manual_seed(23)
    lens = [600]
    codes, scales, table = _cache(g, lens, 2, D)
    for scale, sm in ((30.0, 0.3), (1e30, 1e-31), (1e-30, 1e29), (0.0, 0.1)):
        q = (torch.randn(rows, 4, D, generator=g) * scale).to(torch.bfloat16)
        starts = _starts([rows])
        want, bound = ref.cache_attention(q, starts, lens, table, codes, scales, sm, True)
        got = _run_cache(rudder, q, starts, lens, table, codes, scales, sm, True)
        ref.assert_within(f"O at {scale}", got, want, bound)


@pytest.mark.parametrize("rows", [1, 50])
def test_absent_pages_and_bounds(rudder, rows):
    """Pages outside the pool hold no tokens; lengths behind the table or max_kv are cut; rows
    behind max_rows and behind the last sequence stay as they were."""
    log(f"case absent pages rows={rows}")
    g = torch.Generator().manual_seed(24)
    Hq, Hkv, D = 2, 2, 64
    lens = [400, 130]
    codes, scales, table = _cache(g, lens, Hkv, D)
    P = len(codes)
    table[0, 0], table[0, 3], table[1, 1] = -1, P, 2 ** 31 - 1
    starts = _starts([rows, rows])
    T = 2 * rows + 3
    q = torch.randn(T, Hq, D, generator=g).to(torch.bfloat16)
    sm = 1 / math.sqrt(D)
    want, bound = ref.cache_attention(q, starts, lens, table, codes, scales, sm, True)
    O = torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    n = rudder.attention_workspace_bytes(2, T, rows, 400, Hq, Hkv, D)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")

    def run(lens, max_rows, max_kv):
        O.fill_(7.0)
        rudder.rudder_cache_attention(
            q.cuda(), starts.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), table.cuda(),
            codes.cuda(), scales.cuda(), 2, T, max_rows, max_kv, table.shape[1], P, Hq, Hkv, D,
            sm, True, ws, O)
        return O.cpu()

    got = run(lens, rows, 400)
    ref.assert_within("O", got[:2 * rows], want[:2 * rows], bound[:2 * rows])
    assert (got[2 * rows:] == 7.0).all()
    # a length beyond max_kv
    cut, cut_bound = ref.cache_attention(q, starts, [300, 130], table, codes, scales, sm, True)
    got = run([2 ** 31 - 1, 130], rows, 300)
    ref.assert_within("O cut", got[:2 * rows], cut[:2 * rows], cut_bound[:2 * rows])
    # a negative length: no tokens
    got = run([-5, 130], rows, 400)
    assert not got[:rows].any()
    if rows > 1:
        got = run(lens, rows - 10, 400)
        assert (got[rows - 10:rows] == 7.0).all()
        ref.assert_within("O first rows", got[:rows - 10], want[:rows - 10], bound[:rows - 10])


def test_rows_are_independent(rudder):
    """A NaN query stays in its row and head; strided Q and O; other elements stay."""
    log("case strided, NaN query")
    g = torch.Generator().manual_seed(25)
    Hq, Hkv, D, rows = 4, 2, 64, 37
    lens = [150]
    codes, scales, table = _cache(g, lens, Hkv, D)
    buf = torch.randn(rows, 3 * Hq, D, generator=g).to(torch.bfloat16)
    buf[5, Hq + 1, 3] = float("nan")
    q = buf[:, Hq:2 * Hq]
    starts = _starts([rows])
    want, bound = ref.cache_attention(torch.nan_to_num(q), starts, lens, table, codes, scales,
                                      0.1, True)
    out = torch.full((rows, Hq + 2, D), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(max(16, rudder.attention_workspace_bytes(1, rows, rows, 150, Hq, Hkv, D)),
                     dtype=torch.uint8, device="cuda")
    rudder.rudder_cache_attention(
        buf.cuda()[:, Hq:2 * Hq], starts.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
        table.cuda(), codes.cuda(), scales.cuda(), 1, rows, rows, 150, table.shape[1], len(codes),
        Hq, Hkv, D, 0.1, True, ws, out[:, 1:1 + Hq])
    out = out.cpu()
    assert (out[:, 0] == 7.0).all() and (out[:, -1] == 7.0).all()
    got = out[:, 1:1 + Hq].clone()
    assert torch.isnan(got[5, 1]).all()
    got[5, 1] = 0.0
    want[5, 1], bound[5, 1] = 0.0, 0.0
    ref.assert_within("O", got, want, bound)


CROSS_CASES = [
    # counts, lens, Hq, Hkv, D
    ([1], [1], 1, 1, 64),
    ([1, 1, 1], [77, 0, 300], 4, 4, 128),
    ([5, 40], [64, 65], 6, 2, 64),
    ([200, 1], [512, 3], 2, 2, 128),
    ([96], [77], 4, 1, 128),
    ([3], [2000], 2, 2, 64),
    ([129, 130], [1, 63], 1, 1, 128),
]


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("counts,lens,Hq,Hkv,D", CROSS_CASES)
def test_cross_attention(rudder, counts, lens, Hq, Hkv, D, packed):
    """Padded and packed states; what lies in the padding (NaN, infinities) does not matter."""
    log(f"case cross {counts} {lens} Hq={Hq} Hkv={Hkv} D={D} packed={packed}")
    g = torch.Generator().manual_seed(26)
    starts = _starts(counts)
    T, B, L = int(starts[-1]), len(lens), max(lens) + 3
    q = (torch.randn(T, Hq, D, generator=g) * 2).to(torch.bfloat16)
    if packed:
        kv_start = _starts(lens)[:-1]
        rows = max(sum(lens), 1)
    else:
        kv_start = (torch.arange(B) * L).to(torch.int32)
        rows = B * L
    kv = torch.full((rows, 2 * Hkv, D), float("nan"), dtype=torch.bfloat16)
    kv[::2] = float("inf")
    for b, n in enumerate(lens):
        at = int(kv_start[b])
        kv[at:at + n] = torch.randn(n, 2 * Hkv, D, generator=g).to(torch.bfloat16)
    sm = 1 / math.sqrt(D)
    want, bound = ref.cross_attention(q, kv[:, :Hkv], kv[:, Hkv:], starts, kv_start, lens, sm)
    dev = kv.cuda()
    got = rudder.cross_attention(q.cuda(), dev[:, :Hkv], dev[:, Hkv:], starts.cuda(),
                                 kv_start.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                                 max(counts), max(lens), sm)
    ref.assert_within("O", got, want, bound)


def test_cross_rows_far_apart(rudder):
    """States whose rows are 2^24 elements apart, 200 of them over 6 GiB."""
    log("case cross far apart")
    g = torch.Generator().manual_seed(39)
    H, D, L, apart = 2, 128, 200, 1 << 24
    wide = torch.empty((L - 1) * apart + 2 * H * D, dtype=torch.bfloat16, device="cuda")
    K = wide.as_strided((L, H, D), (apart, D, 1))
    V = wide.as_strided((L, H, D), (apart, D, 1), H * D)
    k = torch.randn(L, 2 * H, D, generator=g).to(torch.bfloat16)
    K.copy_(k[:, :H].cuda())
    V.copy_(k[:, H:].cuda())
    q = torch.randn(140, H, D, generator=g).to(torch.bfloat16)
    starts = _starts([140])
    got = rudder.cross_attention(q.cuda(), K, V, starts.cuda(),
                                 torch.zeros(1, dtype=torch.int32).cuda(),
                                 torch.tensor([L], dtype=torch.int32).cuda(), 140, L, 0.1)
    want, bound = ref.cross_attention(q, k[:, :H], k[:, H:], starts, torch.tensor([0]), [L], 0.1)
    ref.assert_within("O", got, want, bound)


def test_cross_bounds(rudder):
    """Key rows that the arrays place outside the buffer do not exist."""
    log("case cross bounds")
    g = torch.Generator().manual_seed(27)
    D, H, Tkv = 64, 2, 100
    q = torch.randn(4, H, D, generator=g).to(torch.bfloat16)
    kv = torch.randn(Tkv, 2 * H, D, generator=g).to(torch.bfloat16)
    starts = _starts([2, 2])
    dev = kv.cuda()
    got = rudder.cross_attention(q.cuda(), dev[:, :H], dev[:, H:], starts.cuda(),
                                 torch.tensor([90, 2 ** 31 - 1], dtype=torch.int32).cuda(),
                                 torch.tensor([50, 50], dtype=torch.int32).cuda(), 2, 50, 0.1)
    want, bound = ref.cross_attention(q, kv[:, :H], kv[:, H:], starts, torch.tensor([90, 0]),
                                      [10, 0], 0.1)
    ref.assert_within("O", got, want, bound)


@pytest.mark.parametrize("rows,causal", [(2, True), (40, True), (300, False)])
@pytest.mark.parametrize("power,sm_power", [(-108, 107), (-120, 118), (-131, 126)])
def test_smallest_queries(rudder, rows, causal, power, sm_power):
    """Rows down to the type's subnormal numbers under softmax scales to match: they keep the bits
    that their type has, in every kernel."""
    log(f"case smallest queries 2^{power} rows={rows}")
    g = torch.Generator().manual_seed(43)
    D, lens = 128, [1100]
    codes, scales, table = _cache(g, lens, 1, D)
    q = (torch.randn(rows, 2, D, generator=g).double() * 2.0 ** power).to(torch.bfloat16)
    assert q.abs().max() > 0
    starts, sm = _starts([rows]), 2.0 ** sm_power
    want, bound = ref.cache_attention(q, starts, lens, table, codes, scales, sm, causal)
    got = _run_cache(rudder, q, starts, lens, table, codes, scales, sm, causal)
    ref.assert_within("O", got, want, bound)
