"""Causal attention of packed prompts against its 64-bit form, and what a row may and may not
see."""
import math

import pytest
import torch

import attention_reference as aref
import block_reference as ref
from gpu_harness import log

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rudder():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    from w4a4_quantized_gemm_rudder_amd import rudder as r
    r.load_library()
    return r


def _starts(counts):
    return torch.tensor([0] + counts, dtype=torch.int32).cumsum(0).to(torch.int32)


def _inputs(counts, Hq, Hkv, D, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    T = sum(counts)
    q = (torch.randn(T, Hq, D, generator=g) * scale).to(torch.bfloat16)
    k = torch.randn(T, Hkv, D, generator=g).to(torch.bfloat16)
    v = torch.randn(T, Hkv, D, generator=g).to(torch.bfloat16)
    return q, k, v


def _run(rudder, q, k, v, counts, sm, max_rows=None):
    got = rudder.prompt_attention(q.cuda(), k.cuda(), v.cuda(), _starts(counts).cuda(),
                                  max(counts) if max_rows is None else max_rows, sm)
    return got.cpu()


COUNTS = [[1], [2], [31, 32, 33], [63, 64, 65, 1], [0, 130, 0, 0, 7], [127, 128, 129], [200, 3, 257],
          [511], [1, 700, 1], [1030]]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 2), (6, 2), (8, 1), (5, 1)])
@pytest.mark.parametrize("counts", COUNTS)
def test_prompts(rudder, counts, Hq, Hkv, D):
    """Lengths around every tile's end, empty prompts, grouped heads of every kind."""
    log(f"case prompt {counts} Hq={Hq} Hkv={Hkv} D={D}")
    q, k, v = _inputs(counts, Hq, Hkv, D, sum(counts) + D, 1.5)
    sm = 1 / math.sqrt(D)
    got = _run(rudder, q, k, v, counts, sm)
    heads = sorted({0, Hq // 2, Hq - 1})
    want, bound = ref.prompt(q, k, v, _starts(counts).tolist(), sm, heads)
    aref.assert_within("O", got[:, heads], want[:, heads], bound[:, heads])


# prompts of enough tokens and heads for every kernel
LONG = [([4192, 4192], 16, 16, 128), ([1500, 700, 1111], 24, 8, 64), ([5000, 20, 3000], 8, 2, 128),
        ([9001], 4, 1, 64), ([6000], 32, 8, 128), ([300] * 24, 16, 4, 128), ([8300], 16, 16, 128),
        ([40] * 100, 4, 2, 64)]


@pytest.mark.parametrize("counts,Hq,Hkv,D", LONG)
def test_long_prompts(rudder, counts, Hq, Hkv, D):
    log(f"case long prompt {counts} Hq={Hq} Hkv={Hkv} D={D}")
    q, k, v = _inputs(counts, Hq, Hkv, D, 17, 1.5)
    sm = 1 / math.sqrt(D)
    got = _run(rudder, q, k, v, counts, sm)
    starts = _starts(counts).tolist()
    longest = max(counts)
    g = torch.Generator().manual_seed(1)
    rows = torch.cat([torch.arange(3), torch.randint(0, longest, (60,), generator=g),
                      torch.tensor([63, 64, 127, 128, 255, 256, longest - 2, longest - 1])])
    rows = rows.unique()
    heads = sorted({0, Hq // 2 + 1, Hq - 1})
    want, bound = ref.prompt(q, k, v, starts, sm, heads, rows)
    at = torch.cat([r0 + rows[rows < r1 - r0] for r0, r1 in zip(starts, starts[1:])])
    pick = lambda x: x[at][:, heads]  # noqa: E731
    aref.assert_within("O", pick(got), pick(want), pick(bound))
    # every row and head: close to bf16's rounding as a whole
    dev = [x.cuda() for x in (q, k, v)]
    for r0, r1 in zip(starts, starts[1:]):
        for h in heads:
            qq, kk, vv = dev[0][r0:r1, h].double(), dev[1][r0:r1, h * Hkv // Hq].double(), \
                dev[2][r0:r1, h * Hkv // Hq].double()
            i = torch.arange(r1 - r0, device="cuda")
            s = (qq @ kk.t().contiguous()) * sm
            s.masked_fill_(i[None, :] > i[:, None], -math.inf)
            full = torch.softmax(s, -1) @ vv
            err = (got[r0:r1, h].cuda().double() - full).norm() / full.norm()
            # a rounding to bf16 is off by 2^-9 / sqrt(3) to 2^-8 / sqrt(3) of a value; half a
            # step at most, the weights' 2^-11 beside it
            assert err <= aref.BF16, float(err)


@pytest.mark.parametrize("rows,D", [(70, 64), (70, 128), (700, 64), (1500, 128)])
@pytest.mark.parametrize("scale,sm", [(1.0, 0.0), (1.0, -2.0), (30.0, 0.3), (1e30, 1e-31),
                                      (1e30, 0.0), (1e-30, 1e29), (0.0, 0.1)])
def test_scales_of_softmax_and_queries(rudder, rows, D, scale, sm):
    """Softmax scales of zero and below, near one-hot rows, rows of zeros and near the type's ends."""
    log(f"case prompt scale={scale} sm={sm} rows={rows} D={D}")
    counts = [rows, 1, 40]
    q, k, v = _inputs(counts, 2, 1, D, 31, scale)
    got = _run(rudder, q, k, v, counts, sm)
    some = torch.randperm(rows, generator=torch.Generator().manual_seed(2))[:70]
    starts = _starts(counts).tolist()
    want, bound = ref.prompt(q, k, v, starts, sm, rows=some)
    at = torch.cat([r0 + some[some < r1 - r0] for r0, r1 in zip(starts, starts[1:])])
    aref.assert_within("O", got[at], want[at], bound[at])


@pytest.mark.parametrize("rows,D", [(48, 64), (400, 64), (1300, 128)])
def test_weights_keep_their_bits(rudder, rows, D):
    """Values of +1 and -1 in turn under nearly equal weights: the outputs are differences of
    weights, in which a weight's rounding shows.  Bound: fp16's half step a weight."""
    log(f"case prompt weights rows={rows} D={D}")
    q, k, _ = _inputs([rows], 2, 2, D, 33)
    k = (k.float() * 0.1).to(torch.bfloat16)
    sign = torch.ones(rows, 1, D)
    sign[::2] = -1.0
    v = (sign * torch.where(torch.arange(D) % 2 > 0, 1.0, -1.0)).expand(-1, 2, -1)
    v = v.contiguous().to(torch.bfloat16)
    sm = 1 / math.sqrt(D)
    got = _run(rudder, q, k, v, [rows], sm)
    some = torch.arange(1, rows, max(1, rows // 60))
    want, bound = ref.prompt(q, k, v, [0, rows], sm, rows=some)
    aref.assert_within("O", got[some], want[some], bound[some])


@pytest.mark.parametrize("rows,D", [(200, 64), (200, 128), (900, 128), (1100, 64)])
def test_sizes_of_values(rudder, rows, D):
    """Values whose tiles of 64 tokens are of very different sizes, in both orders, tiles of zeros
    among them, up to the type's ends: a tile's values keep their bits beside any other tile's."""
    log(f"case prompt value sizes rows={rows} D={D}")
    q, k, v = _inputs([rows], 3, 1, D, 35)
    tile = torch.arange(rows) // 64
    for powers in ([0, 20, -20, 3, 60, -60], [100, 0, -100], [-126, -100, -60, 0],
                   [8, 7, 6, 7, 8, -1, -2], [115]):
        e = torch.tensor(powers)[tile % len(powers)].double()
        vv = (v.double() * (2.0 ** e)[:, None, None]).to(torch.bfloat16)
        vv[tile == 1] = 0
        got = _run(rudder, q, k, vv, [rows], 0.1)
        some = torch.cat([torch.arange(70), torch.arange(70, rows, 13)])
        # weights of a tile beside one of values 2^d as large lose 2^-33 of the largest weight at
        # that one's size, and values 2^-32 of their tile's largest: counted in `bound` by the
        # largest value a row sees
        for t in some.tolist():
            want, bound = ref.prompt(q[:t + 1], k[:t + 1], vv[:t + 1], [0, t + 1], 0.1,
                                     rows=torch.tensor([t]))
            aref.assert_within(f"{powers} row {t}", got[t:t + 1], want[t:], bound[t:])


@pytest.mark.parametrize("rows,D", [(130, 64), (130, 128), (800, 128), (1200, 64)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 3.3e38])
def test_rows_see_nothing_behind_them(rudder, rows, D, bad):
    """Keys and values of the rows behind a row, of other prompts and of rows of no prompt may hold
    anything: its output has the same bits; the rows that see a value that is not finite are NaN
    in the heads that read it."""
    log(f"case prompt behind rows={rows} D={D} bad={bad}")
    counts, Hq, Hkv = [rows, 50], 4, 2
    q, k, v = _inputs(counts + [30], Hq, Hkv, D, 37)
    sm = 0.1
    clean = _run(rudder, q, k, v, counts, sm)
    for at in (0, 1, 63, 64, 100, rows - 1):
        kk, vv = k.clone(), v.clone()
        vv[at, 1, 5] = bad
        vv[sum(counts):] = bad
        kk[sum(counts):] = bad
        got = _run(rudder, q, kk, vv, counts, sm)
        assert torch.equal(got[:, :2], clean[:, :2]), at           # heads of the other key head
        if math.isfinite(bad):
            # a tile's largest value sets the size of its values' last bits: whole tiles in front
            # keep their bits, rows of the same tile 2^-32 of that value
            whole = at // 64 * 64
            assert torch.equal(got[:whole, 2:], clean[:whole, 2:]), at
        else:
            assert torch.equal(got[:at, 2:], clean[:at, 2:]), at
            assert torch.isnan(got[at:rows, 2:]).all(), at
        assert torch.equal(got[rows:], clean[rows:]), at
        kk, vv = k.clone(), v.clone()
        kk[at, 1] = bad
        got = _run(rudder, q, kk, vv, counts, sm)
        assert torch.equal(got[:at], clean[:at]) and torch.equal(got[rows:], clean[rows:]), at
        assert torch.equal(got[:, :2], clean[:, :2]), at
        if math.isnan(bad):
            assert torch.isnan(got[at:rows, 2:]).all(), at


def test_rows_of_a_long_prompt_see_nothing_behind_them(rudder):
    """The same on the kernel of eight waves, and tiles of larger and smaller values among them."""
    log("case long prompt behind")
    n, H = 8300, 16
    q, k, v = (x.cuda() for x in _inputs([n], H, H, 128, 38))
    starts = _starts([n]).cuda()
    run = lambda kk, vv: rudder.prompt_attention(q, kk, vv, starts, n, 0.1)  # noqa: E731
    clean = run(k, v)
    for at, bad in ((5000, float("nan")), (8299, float("inf")), (64, -float("inf"))):
        vv = v.clone()
        vv[at, 3, 9] = bad
        got = run(k, vv)
        assert torch.equal(got[:at], clean[:at]) and torch.isnan(got[at:, 3]).all()
        got[at:, 3] = clean[at:, 3]
        assert torch.equal(got, clean)
        kk = k.clone()
        kk[at, 3] = bad
        assert torch.equal(run(kk, v)[:at], clean[:at])
    for power in (30, -30):                        # 2^30 times as large, or all but these
        e = torch.where((torch.arange(n, device="cuda") // 64) % 5 == 2, 2.0 ** power, 1.0)
        vv = (v.float() * e[:, None, None]).to(torch.bfloat16)
        got = run(k, vv)
        for h in (0, 7):
            s = q[:, h].double() @ k[:, h].double().t().contiguous() * 0.1
            i = torch.arange(n, device="cuda")
            s.masked_fill_(i[None, :] > i[:, None], -math.inf)
            p = torch.softmax(s, -1)
            want, size = p @ vv[:, h].double(), p @ vv[:, h].double().abs()
            # weights' half step, four times over for the exponents' roundings, and bf16's
            bound = 4 * aref.FP16 * size + aref.BF16 * want.abs()
            assert ((got[:, h].double() - want).abs() <= bound + 2.0 ** -134).all(), (power, h)


def test_queries_that_are_not_finite(rudder):
    """NaN in their row and head alone."""
    log("case prompt queries not finite")
    for rows, D in ((70, 64), (300, 128), (1300, 128)):
        q, k, v = _inputs([rows, 9], 4, 2, D, 39)
        clean = _run(rudder, q, k, v, [rows, 9], 0.1)
        bad = q.clone()
        spots = [(0, 1, float("nan")), (33, 0, float("inf")), (64, 3, -float("inf")),
                 (rows - 1, 2, float("inf")), (rows + 3, 1, float("nan"))]
        for t, h, x in spots:
            bad[t, h, 7] = x
        got = _run(rudder, bad, k, v, [rows, 9], 0.1)
        for t, h, _ in spots:
            assert torch.isnan(got[t, h]).all(), (t, h)
            got[t, h] = clean[t, h]
        assert torch.equal(got, clean)


def test_strides_and_rows_left_alone(rudder):
    """Q, K and V as parts of one buffer, outputs any distance apart; rows behind the last prompt,
    behind max_rows and between the outputs stay; arrays that point outside are clamped."""
    log("case prompt strides")
    for counts, D in (([90, 40], 64), ([600, 300], 128)):
        Hq, Hkv, T = 4, 2, sum(counts) + 20
        q, k, v = _inputs([T], Hq, Hkv, D, 41)
        buf = torch.cat([q, k, v], 1).cuda()
        out = torch.full((T, Hq * D + 64), 7.0, dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(rudder.prompt_attention_workspace_bytes(2, T, max(counts), Hq, Hkv, D),
                         dtype=torch.uint8, device="cuda")
        starts = _starts(counts).cuda()
        parts = buf[:, :Hq], buf[:, Hq:Hq + Hkv], buf[:, Hq + Hkv:]
        rudder.rudder_prompt_attention(*parts, starts, 2, T, max(counts), Hq, Hkv, D, 0.1, ws,
                                       out[:, :Hq * D])
        want = _run(rudder, q, k, v, counts, 0.1)
        used = sum(counts)
        assert torch.equal(out[:used, :Hq * D].cpu().view(used, Hq, D), want[:used])
        assert (out[used:] == 7.0).all() and (out[:, Hq * D:] == 7.0).all()
        # a bound below the longest prompt leaves its last rows; a loose one may choose another
        # kernel, whose sums are rounded in another order: held to the formula as well
        short = max(counts) - 25
        cut = rudder.prompt_attention(*parts, starts, short, 0.1).cpu()
        assert torch.equal(cut[:short], want[:short]) and not cut[short:counts[0]].any()
        assert torch.equal(cut[counts[0]:], want[counts[0]:])
        loose = rudder.prompt_attention(*parts, starts, 10 * T, 0.1).cpu()
        rows = torch.cat([torch.arange(40), torch.arange(40, max(counts), 17)])
        formula, bound = ref.prompt(q, k, v, _starts(counts).tolist(), 0.1, rows=rows)
        at = torch.cat([r0 + rows[rows < n] for r0, n in zip([0, counts[0]], counts)])
        aref.assert_within("loose", loose[at], formula[at], bound[at])
        assert not loose[used:].any()
        # the first and the last sequence are clamped to the buffer, the second is empty
        odd = torch.tensor([-9, counts[0], counts[0] - 50, 10**9], dtype=torch.int32).cuda()
        got = rudder.prompt_attention(*parts, odd, T, 0.1).cpu()
        at = rows[rows < counts[0] - 50]
        aref.assert_within("clamped", got[at], formula[at], bound[at])
        tail = _run(rudder, q[counts[0] - 50:], k[counts[0] - 50:], v[counts[0] - 50:],
                    [T - counts[0] + 50], 0.1)
        assert torch.allclose(got[counts[0]:].float(), tail[50:].float(), rtol=4 * aref.BF16,
                              atol=4 * aref.BF16)


def test_same_bits_again(rudder):
    """Ten runs of a ragged batch, among others on the stream, have the same bits."""
    log("case prompt repeats")
    counts = [1500, 64, 900, 3, 2200]
    q, k, v = _inputs(counts, 8, 2, 128, 43)
    first = _run(rudder, q, k, v, counts, 0.09)
    for _ in range(9):
        assert torch.equal(_run(rudder, q, k, v, counts, 0.09), first)
    # a prompt's rows do not depend on the others of the batch
    alone = _run(rudder, q[:1500], k[:1500], v[:1500], [1500], 0.09)
    err = (alone.double() - first[:1500].double()).norm() / alone.double().norm()
    assert err <= aref.BF16 / 2, float(err)


def test_offsets_past_32_bits(rudder):
    """Rows so far apart that the last ones start past 2^31 elements."""
    log("case prompt offsets")
    T, D, ld = 70000, 64, 32768
    counts = [69000, 700, 300]
    q, k, v = _inputs([T], 1, 1, D, 45)
    far = torch.empty(T * ld, dtype=torch.bfloat16, device="cuda")
    part = [far.as_strided((T, 1, D), (ld, D, 1), i * D) for i in range(4)]
    for p, x in zip(part, (q, k, v)):
        p.copy_(x)
    part[3].zero_()
    n = rudder.prompt_attention_workspace_bytes(3, T, max(counts), 1, 1, D)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    rudder.rudder_prompt_attention(part[0], part[1], part[2], _starts(counts).cuda(), 3, T,
                                   max(counts), 1, 1, D, 0.125, ws, part[3])
    got = part[3].contiguous().cpu()
    rows = torch.tensor([0, 77, 299, 699, 30000, 68999])
    want, bound = ref.prompt(q, k, v, _starts(counts).tolist(), 0.125, rows=rows)
    at = torch.cat([r0 + rows[rows < n] for r0, n in zip(_starts(counts).tolist(), counts)])
    aref.assert_within("O", got[at], want[at], bound[at])


# Prompts of no rows behind the others: enough work units for the kernel for many rows at any size.
EMPTY = [0] * 600


def _run_many(rudder, q, k, v, counts, sm):
    n = rudder.prompt_attention_workspace_bytes(len(counts + EMPTY), q.shape[0], max(counts),
                                                q.shape[1], k.shape[1], q.shape[2])
    assert n > 0
    return _run(rudder, q, k, v, counts + EMPTY, sm)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (6, 2), (8, 1), (5, 1)])
@pytest.mark.parametrize("counts", COUNTS)
def test_prompts_among_many(rudder, counts, Hq, Hkv, D):
    log(f"case prompt among many {counts} Hq={Hq} Hkv={Hkv} D={D}")
    q, k, v = _inputs(counts, Hq, Hkv, D, sum(counts) + D + 1, 1.5)
    sm = 1 / math.sqrt(D)
    got = _run_many(rudder, q, k, v, counts, sm)
    heads = sorted({0, Hq // 2, Hq - 1})
    want, bound = ref.prompt(q, k, v, _starts(counts).tolist(), sm, heads)
    aref.assert_within("O", got[:, heads], want[:, heads], bound[:, heads])


@pytest.mark.parametrize("rows,D", [(70, 64), (330, 128)])
@pytest.mark.parametrize("scale,sm", [(1.0, 0.0), (1.0, -2.0), (30.0, 0.3), (1e30, 1e-31),
                                      (1e30, 0.0), (1e-30, 1e29), (0.0, 0.1)])
def test_scales_among_many(rudder, rows, D, scale, sm):
    log(f"case prompt among many scale={scale} sm={sm} rows={rows} D={D}")
    counts = [rows, 1, 40]
    q, k, v = _inputs(counts, 2, 1, D, 51, scale)
    got = _run_many(rudder, q, k, v, counts, sm)
    want, bound = ref.prompt(q, k, v, _starts(counts).tolist(), sm)
    aref.assert_within("O", got, want, bound)


@pytest.mark.parametrize("rows,D", [(200, 64), (400, 128)])
def test_sizes_of_values_among_many(rudder, rows, D):
    log(f"case prompt among many value sizes rows={rows} D={D}")
    q, k, v = _inputs([rows], 3, 1, D, 53)
    tile = torch.arange(rows) // 64
    for powers in ([0, 20, -20, 3, 60, -60], [100, 0, -100], [-126, -100, -60, 0],
                   [8, 7, 6, 7, 8, -1, -2], [115]):
        e = torch.tensor(powers)[tile % len(powers)].double()
        vv = (v.double() * (2.0 ** e)[:, None, None]).to(torch.bfloat16)
        vv[tile == 1] = 0
        got = _run_many(rudder, q, k, vv, [rows], 0.1)
        for t in list(range(70)) + list(range(70, rows, 13)):
            want, bound = ref.prompt(q[:t + 1], k[:t + 1], vv[:t + 1], [0, t + 1], 0.1,
                                     rows=torch.tensor([t]))
            aref.assert_within(f"{powers} row {t}", got[t:t + 1], want[t:], bound[t:])


@pytest.mark.parametrize("rows,D", [(130, 64), (400, 128)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 3.3e38])
def test_rows_among_many_see_nothing_behind_them(rudder, rows, D, bad):
    log(f"case prompt among many behind rows={rows} D={D} bad={bad}")
    counts, Hq, Hkv = [rows, 50], 4, 2
    q, k, v = _inputs(counts + [30], Hq, Hkv, D, 57)
    clean = _run_many(rudder, q, k, v, counts, 0.1)
    for at in (0, 1, 63, 64, 100, rows - 1):
        kk, vv = k.clone(), v.clone()
        vv[at, 1, 5] = bad
        vv[sum(counts):] = bad
        kk[sum(counts):] = bad
        got = _run_many(rudder, q, kk, vv, counts, 0.1)
        assert torch.equal(got[:, :2], clean[:, :2]), at           # heads of the other key head
        if math.isfinite(bad):
            # whole tiles in front keep their bits, as in test_rows_see_nothing_behind_them
            whole = at // 64 * 64
            assert torch.equal(got[:whole, 2:], clean[:whole, 2:]), at
        else:
            assert torch.equal(got[:at, 2:], clean[:at, 2:]), at
            assert torch.isnan(got[at:rows, 2:]).all(), at
        assert torch.equal(got[rows:], clean[rows:]), at
        kk = k.clone()
        kk[at, 1] = bad
        got = _run_many(rudder, q, kk, v, counts, 0.1)
        assert torch.equal(got[:at], clean[:at]) and torch.equal(got[rows:], clean[rows:]), at
        assert torch.equal(got[:, :2], clean[:, :2]), at
        if math.isnan(bad):
            assert torch.isnan(got[at:rows, 2:]).all(), at


@pytest.mark.parametrize("D", [64, 128])
def test_queries_among_many_that_are_not_finite(rudder, D):
    log(f"case prompt among many queries not finite D={D}")
    rows = 150
    q, k, v = _inputs([rows, 9], 4, 2, D, 59)
    clean = _run_many(rudder, q, k, v, [rows, 9], 0.1)
    bad = q.clone()
    spots = [(0, 1, float("nan")), (33, 0, float("inf")), (64, 3, -float("inf")),
             (rows - 1, 2, float("inf")), (rows + 3, 1, float("nan"))]
    for t, h, x in spots:
        bad[t, h, 7] = x
    got = _run_many(rudder, bad, k, v, [rows, 9], 0.1)
    for t, h, _ in spots:
        assert torch.isnan(got[t, h]).all(), (t, h)
        got[t, h] = clean[t, h]
    assert torch.equal(got, clean)


@pytest.mark.parametrize("D,Hq,Hkv,rows", [(64, 24, 8, 300), (64, 24, 8, 682), (64, 24, 8, 683),
                                           (128, 16, 16, 512), (128, 16, 16, 513),
                                           (128, 16, 16, 1024), (128, 16, 16, 1025)])
def test_sizes_beside_the_limits_of_a_kernel(rudder, D, Hq, Hkv, rows):
    """The last and the first sizes of each kernel, with the workspace that the library asks for and
    not a byte more."""
    log(f"case prompt limits D={D} Hq={Hq} Hkv={Hkv} rows={rows}")
    q, k, v = _inputs([rows], Hq, Hkv, D, 61)
    sm = 1 / math.sqrt(D)
    n = rudder.prompt_attention_workspace_bytes(1, rows, rows, Hq, Hkv, D)
    buf = torch.full((n + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    O = torch.zeros(rows, Hq, D, dtype=torch.bfloat16, device="cuda")
    rudder.rudder_prompt_attention(q.cuda(), k.cuda(), v.cuda(), _starts([rows]).cuda(), 1, rows,
                                   rows, Hq, Hkv, D, sm, buf[:n] if n else None, O)
    some = torch.cat([torch.arange(40), torch.arange(40, rows, 17), torch.tensor([rows - 1])]).unique()
    heads = [0, Hq - 1]
    want, bound = ref.prompt(q, k, v, [0, rows], sm, heads, some)
    got = O.cpu()
    aref.assert_within("O", got[some][:, heads], want[some][:, heads], bound[some][:, heads])
    assert (buf[n:] == 0xA5).all()
