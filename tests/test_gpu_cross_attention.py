"""Cross attention where its roundings and its checks of a row show: weights that cancel, softmax
scales of zero, below zero and of any size, queries that are not finite, single rows with strides
of their own; on the kernels of 128 and of 256 rows a workgroup, whole and split over the keys."""
import math

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


def _i32(x):
    return torch.tensor(x, dtype=torch.int32)


def _cross(rudder, q, k, v, counts, lens, sm, max_kv=None):
    starts = _i32([0] + counts).cumsum(0).to(torch.int32)
    kv_start = _i32([0] + lens).cumsum(0).to(torch.int32)[:-1]
    got = rudder.cross_attention(q.cuda(), k.cuda(), v.cuda(), starts.cuda(), kv_start.cuda(),
                                 _i32(lens).cuda(), max(counts),
                                 max(lens) if max_kv is None else max_kv, sm)
    return got.cpu(), starts, kv_start


# rows a sequence, bound on the keys, D: one tile of 128 rows, tiles split over the keys, 256 rows
# a workgroup (128 channels, over 128 rows, 16 tiles of keys and more)
KERNELS = [(1, 64, 64), (40, 64, 128), (3, 2000, 64), (140, 300, 128), (300, 1200, 128)]


@pytest.mark.parametrize("rows,max_kv,D", KERNELS)
def test_weights_keep_their_bits(rudder, rows, max_kv, D):
    """Values of +1 and -1 in equal shares under weights that differ by a few percent: the outputs
    are differences of weights, so that a weight's rounding shows in them, not beside the
    outputs' own.  Weights count with half a step of 2^-16: the rounding of a rounding's rest."""
    log(f"case weights rows={rows} max_kv={max_kv} D={D}")
    g = torch.Generator().manual_seed(81)
    counts, lens, H = [rows, max(rows - 1, 1)], [2, 48], 2
    q = torch.randn(sum(counts), H, D, generator=g).to(torch.bfloat16)
    k = (torch.randn(sum(lens), H, D, generator=g) * 0.1).to(torch.bfloat16)
    sign = torch.ones(sum(lens), 1, D)
    sign[::2] = -1.0
    v = (sign * torch.where(torch.arange(D) % 2 > 0, 1.0, -1.0)).expand(-1, H, -1)
    v = v.contiguous().to(torch.bfloat16)
    sm = 1 / math.sqrt(D)
    got, starts, kv_start = _cross(rudder, q, k, v, counts, lens, sm, max_kv)
    for b, n in enumerate(lens):
        r0, r1, k0 = int(starts[b]), int(starts[b + 1]), int(kv_start[b])
        for h in range(H):
            want, bound = ref.rows_attention(
                q[r0:r1, h].double(), k[k0:k0 + n, h].double(), v[k0:k0 + n, h].double(),
                torch.ones(r1 - r0, n, dtype=torch.bool), sm, ref.BF16 ** 2, 0.0)
            ref.assert_within(f"O {b} {h}", got[r0:r1, h], want, bound)


@pytest.mark.parametrize("scale,sm", [(1.0, 0.0), (1.0, -2.0), (30.0, 0.3), (1e30, 1e-31),
                                      (1e30, 0.0), (1e-30, 1e29), (0.0, 0.1)])
@pytest.mark.parametrize("rows,max_kv,D", KERNELS)
def test_scales_of_softmax_and_queries(rudder, rows, max_kv, D, scale, sm):
    """Softmax scales of zero and below, near one-hot rows, rows of zeros and rows near the type's
    ends, beside a sequence without states: a scale of zero weighs the states alike however large
    the queries are."""
    log(f"case cross scale={scale} sm={sm} rows={rows} max_kv={max_kv} D={D}")
    g = torch.Generator().manual_seed(82)
    counts, lens, H = [rows, 1, rows], [min(max_kv, 70), 0, max_kv], 2
    q = (torch.randn(sum(counts), 2 * H, D, generator=g) * scale).to(torch.bfloat16)
    k = torch.randn(sum(lens), H, D, generator=g).to(torch.bfloat16)
    v = torch.randn(sum(lens), H, D, generator=g).to(torch.bfloat16)
    got, starts, kv_start = _cross(rudder, q, k, v, counts, lens, sm)
    want, bound = ref.cross_attention(q, k, v, starts, kv_start, lens, sm)
    ref.assert_within("O", got, want, bound)
    if sm == 0.0:                                  # plain means
        for b, n in enumerate(lens):
            if n:
                at = int(kv_start[b])
                mean = v[at:at + n].double().mean(0).repeat_interleave(2, 0)
                rows_b = got[int(starts[b]):int(starts[b + 1])].double()
                assert (rows_b - mean).abs().max() <= 2 * ref.BF16 * float(mean.abs().max())


@pytest.mark.parametrize("sm", [0.1, -0.1, 0.0])
@pytest.mark.parametrize("rows,max_kv,D", [(3, 64, 64), (40, 64, 128), (3, 2000, 64),
                                           (140, 300, 128), (300, 1200, 128)])
def test_queries_that_are_not_finite(rudder, rows, max_kv, D, sm):
    """A query row with a NaN, an infinity of either sign or both gives NaN in its row and head
    and leaves the others; one of a sequence without states gives zeros."""
    log(f"case cross not finite rows={rows} max_kv={max_kv} D={D} sm={sm}")
    g = torch.Generator().manual_seed(83)
    counts, lens, H = [rows, 2], [max_kv, 0], 2
    q = torch.randn(sum(counts), H, D, generator=g).to(torch.bfloat16)
    k = torch.randn(sum(lens), H, D, generator=g).to(torch.bfloat16)
    v = torch.randn(sum(lens), H, D, generator=g).to(torch.bfloat16)
    clean, bad = q.clone(), [(0, 0, math.nan), (1, 1, math.inf), (2, 0, -math.inf)]
    for r, h, x in bad:
        q[r, h, 7 * r] = x
    q[rows], q[rows + 1, 0, 3] = math.nan, -math.inf
    got, starts, kv_start = _cross(rudder, q, k, v, counts, lens, sm)
    assert not got[rows:].any()
    want, bound = ref.cross_attention(clean, k, v, starts, kv_start, lens, sm)
    for r, h, _ in bad:
        assert torch.isnan(got[r, h]).all(), (r, h)
        got[r, h], want[r, h], bound[r, h] = 0.0, 0.0, 0.0
    ref.assert_within("O", got, want, bound)


def test_single_rows_with_any_stride(rudder):
    """One row has no distance to a next one: what its tensor's stride says does not matter."""
    log("case single row strides")
    g = torch.Generator().manual_seed(84)
    H, D, n = 2, 64, 70
    buf = torch.randn(1, 5 * H * D + 3, generator=g).to(torch.bfloat16).cuda()
    q = buf.as_strided((1, H, D), (5 * H * D + 3, D, 1))
    assert q.stride(0) % 8
    k = torch.randn(n, H, D, generator=g).to(torch.bfloat16)
    starts, zero = _i32([0, 1]).cuda(), _i32([0]).cuda()
    args = (k.cuda(), k.cuda(), starts, zero, _i32([n]).cuda(), 1, n, 0.1)
    want = rudder.cross_attention(q.contiguous().clone(), *args)
    assert torch.equal(rudder.cross_attention(q, *args), want)
    codes, scales = rudder.new_cache(2, H, D)
    one, other = (codes.clone(), scales.clone()), (codes, scales)
    table = _i32([[1, 0]]).cuda()
    rudder.cache_append(q, q, starts, zero, table, 1, *one)
    rudder.cache_append(q.contiguous().clone(), q.contiguous().clone(), starts, zero, table, 1,
                        *other)
    assert torch.equal(one[0], other[0]) and torch.equal(one[1], other[1])
