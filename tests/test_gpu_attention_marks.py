"""Which tokens a row sees, token by token, in every kernel and split: states whose tokens can be
told apart (attention_marks)."""
import pytest
import torch

import attention_marks as marks
from attention_reference import BF16, FP16, visible
from gpu_harness import log

pytestmark = pytest.mark.gpu
PAGE, SM, SCALE = 64, 0.125, 1.0 / marks.MARK


@pytest.fixture(scope="module")
def rudder():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    from w4a4_quantized_gemm_rudder_amd import rudder as r
    r.load_library()
    return r


def _i32(x):
    return torch.tensor(x, dtype=torch.int32)


def _pages(tokens, H, D):
    """Codes [n, H, 2, 64 D] of one sequence's pages; behind its last token codes of 127."""
    n = (tokens + PAGE - 1) // PAGE
    k, v = marks.token_marks(torch.arange(n * PAGE), D)
    k, v = k * marks.MARK, v * marks.MARK
    k[tokens:], v[tokens:] = 127, 127
    k = k.view(n, PAGE * D)
    v = v.view(n, PAGE, D).transpose(1, 2).reshape(n, PAGE * D)
    return torch.stack([k, v], 1)[:, None].expand(-1, H, -1, -1)


def _classes(rows, kv, heads, D):
    """Classes [rows, heads]: the row's last causal token's, the next one's and the one's before,
    further heads spread over the others."""
    last = kv - rows + torch.arange(rows)[:, None]
    step = torch.arange(heads)[None, :]
    offset = torch.where(step == 2, -1, torch.where(step < 2, step, step * D // heads + 1))
    return (last + offset) % D


def _check(got, rows, kv, classes, heads, D, causal, there=None, half_step=FP16):
    see = visible(rows, kv, causal)
    if there is not None:
        see = see & there[None, :]
    for h in heads:
        want = marks.expected(classes[:, h], see, D, 1.0)
        over = (got[:, h].double() - want).abs() - marks.bound(want, 1.0, half_step)
        assert over.numel() == 0 or float(over.max()) <= 0, (
            h, float(over.max()), [int(x) for x in (over > 0).nonzero()[0]],
            int((over > 0).sum()))


# (sequences' rows, keys, bound on the keys or None, Hq, Hkv, D, causal, heads compared)
CASES = [
    # at most 16 rows: whole stretches by one workgroup, pieces
    ([1, 2], [500, 64], None, 8, 1, 128, True, range(8)),
    ([1] * 64, [1300 - 20 * i for i in range(64)], None, 16, 2, 128, True, range(16)),
    ([1, 1], [9000, 8999], None, 16, 1, 128, True, range(16)),
    ([2, 1], [4000, 130], 4096, 8, 1, 64, True, range(8)),
    ([3], [2500], None, 4, 1, 128, False, range(4)),
    # 128 rows a workgroup: whole, in pieces, the last ones in pieces
    ([33, 129], [200, 129], None, 4, 2, 128, True, range(4)),
    ([70], [180], None, 3, 1, 64, False, range(3)),
    ([20], [3000], None, 4, 4, 64, True, range(4)),
    ([300, 17], [2500, 1000], None, 4, 1, 128, True, range(4)),
    ([96, 96], [4100, 4000], None, 2, 2, 128, False, range(2)),
    ([130], [900], None, 260, 260, 128, False, [0, 1, 2, 200, 257, 258, 259]),
    ([500], [1500], None, 96, 48, 64, True, [0, 1, 2, 50, 95]),
    # 256 rows a workgroup
    ([300, 41], [1100, 1030], None, 4, 2, 128, False, range(4)),
    ([130, 140], [1100, 64], None, 128, 128, 128, False, [0, 1, 2, 64, 127]),
    ([600], [5000], None, 3, 1, 128, False, range(3)),
]


@pytest.mark.parametrize("counts,lens,max_kv,Hq,Hkv,D,causal,heads", CASES)
def test_cache_tokens(rudder, counts, lens, max_kv, Hq, Hkv, D, causal, heads):
    log(f"case marks {counts[:3]} {lens[:3]} Hq={Hq} Hkv={Hkv} D={D} causal={causal}")
    g = torch.Generator().manual_seed(91)
    need = [(n + PAGE - 1) // PAGE for n in lens]
    order = torch.randperm(sum(need) + 1, generator=g)
    codes = torch.full((sum(need) + 1, Hkv, 2, PAGE * D), 127, dtype=torch.int8)
    table = torch.full((len(lens), max(need) + 1), -1, dtype=torch.int32)
    at, absent = 0, []
    for b, n in enumerate(need):
        pages = order[at:at + n]
        codes[pages] = _pages(lens[b], Hkv, D)
        table[b, :n] = pages.to(torch.int32)
        at += n
        # one page of the longer ones is not there
        absent.append(n // 2 if n > 6 else -1)
        if n > 6:
            table[b, n // 2] = len(codes) + b
    scales = torch.full((len(codes), Hkv, 2), SCALE)
    classes = [_classes(r, n, Hq, D) for r, n in zip(counts, lens)]
    q = torch.cat([marks.queries(c, D, SM, 1.0) for c in classes])
    starts = _i32([0] + counts).cumsum(0).to(torch.int32)
    got = rudder.cache_attention(q.cuda(), starts.cuda(), _i32(lens).cuda(), table.cuda(),
                                 codes.cuda(), scales.cuda(), max(counts),
                                 max(lens) if max_kv is None else max_kv, SM, causal).cpu()
    for b, n in enumerate(lens):
        there = torch.arange(n) // PAGE != absent[b]
        _check(got[int(starts[b]):int(starts[b + 1])], counts[b], n, classes[b], heads, D, causal,
               there)


@pytest.mark.parametrize("counts,lens,max_kv,Hq,Hkv,D,causal,heads",
                         [c for c in CASES if not c[6]] + [
                             ([1, 3], [77, 2000], None, 4, 2, 64, False, range(4)),
                             ([1] * 40, list(range(1, 512, 13)), None, 8, 8, 128, False,
                              range(8))])
def test_cross_tokens(rudder, counts, lens, max_kv, Hq, Hkv, D, causal, heads):
    log(f"case cross marks {counts[:3]} {lens[:3]} Hq={Hq} Hkv={Hkv} D={D}")
    k, v = (torch.cat(x).to(torch.bfloat16)[:, None].expand(-1, Hkv, -1)
            for x in zip(*(marks.token_marks(torch.arange(n), D) for n in lens)))
    classes = [_classes(r, n, Hq, D) for r, n in zip(counts, lens)]
    q = torch.cat([marks.queries(c, D, SM, 1.0) for c in classes])
    starts = _i32([0] + counts).cumsum(0).to(torch.int32)
    kv_start = _i32([0] + lens).cumsum(0).to(torch.int32)[:-1]
    got = rudder.cross_attention(q.cuda(), k.contiguous().cuda(), v.contiguous().cuda(),
                                 starts.cuda(), kv_start.cuda(), _i32(lens).cuda(), max(counts),
                                 max(lens) if max_kv is None else max_kv, SM).cpu()
    for b, n in enumerate(lens):
        _check(got[int(starts[b]):int(starts[b + 1])], counts[b], n, classes[b], heads, D, False,
               half_step=BF16)


# More than 64 tiles of one stretch, the page numbers fetched anew.  Rows, sequences (that share
# the pages), D, pages, and what the sizes make of them:
#   345 pairs of 16 rows: three pieces of 367 tiles, 92 for each of four waves
#   units that are whole rounds: 700 tiles each; less than half a round: two pieces of 350
LONG = [(1, 345, 64, 1100), (20, 768, 64, 200), (20, 512, 128, 300), (20, 200, 128, 700),
        (130, 256, 128, 300), (130, 100, 128, 700)]


@pytest.mark.parametrize("rows,B,D,pages", LONG)
def test_long_stretches(rudder, rows, B, D, pages):
    log(f"case long stretches rows={rows} B={B} D={D} pages={pages}")
    g = torch.Generator().manual_seed(92)
    kv, Hq = pages * PAGE - 59, 16 if rows == 1 else 1
    order = torch.randperm(pages, generator=g)
    codes = torch.empty(pages, 1, 2, PAGE * D, dtype=torch.int8)
    codes[order] = _pages(kv, 1, D)
    table = order.to(torch.int32)[None].repeat(B, 1)
    table[:, pages // 3] = -1
    classes = _classes(rows, kv, Hq, D)
    q = marks.queries(classes, D, SM, 1.0).repeat(B, 1, 1)
    starts = (torch.arange(B + 1) * rows).to(torch.int32)
    got = rudder.cache_attention(q.cuda(), starts.cuda(), _i32([kv] * B).cuda(), table.cuda(),
                                 codes.cuda(), torch.full((pages, 1, 2), SCALE).cuda(), rows, kv,
                                 SM, False).cpu().view(B, rows, Hq, D)
    assert torch.equal(got, got[:1].expand_as(got))
    _check(got[0], rows, kv, classes, range(Hq), D, False,
           torch.arange(kv) // PAGE != pages // 3)
