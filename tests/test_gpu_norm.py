"""RMS norm with the residual's addition, its rows and its codes, against the definition bit for
bit; codes back as values."""
import numpy as np
import pytest
import torch

import block_reference as ref
from gpu_harness import log, tile_for
from tiled_layout import tile_codes_e2m3_a8

pytestmark = pytest.mark.gpu
EPS = 1e-6
INT, E2M3 = 0, 1


@pytest.fixture(scope="module")
def rudder():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    from w4a4_quantized_gemm_rudder_amd import rudder as r
    r.load_library()
    return r


def _inputs(M, K, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g)
    x[:, torch.randperm(K, generator=g)[: max(1, K // 50)]] *= 30.0
    x, r = x.to(torch.bfloat16), (torch.randn(M, K, generator=g) * 2).to(torch.bfloat16)
    gamma, smooth = torch.rand(K, generator=g) + 0.5, torch.rand(K, generator=g) * 3 + 0.2
    sid = torch.randint(0, 3, (M,), generator=g).to(torch.uint8)
    return x, r, gamma, smooth, sid, torch.rand(3, generator=g) * 0.02 + 0.01


def _equal(name, got, want):
    got, want = got.cpu().contiguous(), want.contiguous()
    assert got.shape == want.shape and got.dtype == want.dtype, name
    bad = got.view(torch.uint8) != want.view(torch.uint8)
    assert not bad.any(), f"{name}: {int(bad.sum())} bytes differ"


# few rows, whole rows a wave of every width, rows of many waves; odd counts and ragged pieces
SHAPES = [(1, 8), (3, 40), (1, 4096), (33, 2040), (513, 128), (600, 2048), (520, 2056), (515, 4096),
          (530, 8192), (7, 8200), (2, 65536), (700, 72)]


@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("M,K", SHAPES)
def test_rows(rudder, M, K, add):
    log(f"case norm rows M={M} K={K} add={add}")
    x, r, gamma, *_ = _inputs(M, K, M + K)
    want, h = ref.norm(x, gamma, EPS, r if add else None)
    got = rudder.norm(x.cuda(), gamma.cuda(), EPS, r.cuda() if add else None)
    _equal("y", got[0] if add else got, want)
    if add:
        _equal("h", got[1], h)


# K a multiple of 32 that is none of 64 in the int containers, few and many rows, padding rows
CODE_SHAPES = [(1, 64), (31, 96), (33, 2048), (200, 4096), (513, 224), (600, 2048), (545, 4096),
               (514, 8192), (9, 8256), (2, 65536)]


@pytest.mark.parametrize("mode", ["table", "row"])
@pytest.mark.parametrize("bits,codes", [(8, INT), (4, INT), (4, E2M3)])
@pytest.mark.parametrize("M,K", CODE_SHAPES)
def test_codes(rudder, M, K, bits, codes, mode):
    """Codes and row scales bit for bit, padding rows zero; and with the table exactly those of
    the norm's rows through the quantizer."""
    if codes == E2M3:
        K = (K + 63) // 64 * 64
    log(f"case norm codes M={M} K={K} bits={bits} codes={codes} {mode}")
    x, r, gamma, smooth, sid, table = _inputs(M, K, 3 * M + K)
    if bits == 4:
        table = table * 16
    add = M % 2 == 1
    y, h = ref.norm(x, gamma, EPS, r if add else None)
    q, s = ref.codes(y, smooth, bits, sid, table if mode == "table" else None)
    kw = dict(stream_id=sid.cuda(), act_scale=table.cuda()) if mode == "table" else {}
    if add:
        kw["residual"] = r.cuda()
    got = rudder.norm_quant(x.cuda(), gamma.cuda(), smooth.cuda(), EPS, bits, codes, **kw)
    _equal("row_scale", got[1], s)
    _equal("Xq", got[0], torch.from_numpy(tile_for(codes, q.numpy(), bits)))
    if add:
        _equal("h", got[2], h)
    _equal("values", rudder.dequant_act(got[0], got[1], M, K, bits, codes),
           q.float() * s[:, None])
    if mode == "table":
        yy = rudder.norm(x.cuda(), gamma.cuda(), EPS, r.cuda() if add else None)
        chain = rudder.quant_act(yy[0] if add else yy, sid.cuda(), smooth.cuda(), table.cuda(), 3,
                                 bits, codes)
        _equal("chain", got[0], chain[0].cpu())
        _equal("chain's scales", got[1], chain[1].cpu())


@pytest.mark.parametrize("M,K", [(1, 64), (40, 192), (33, 4096)])
@pytest.mark.parametrize("bits,codes", [(8, INT), (4, INT), (4, E2M3), (8, E2M3)])
def test_values_of_every_code(rudder, M, K, bits, codes):
    """Every code at every place of a slot, in each container."""
    log(f"case dequant M={M} K={K} bits={bits} codes={codes}")
    top = 127 if bits == 8 else 7
    q = (np.arange(M * K).reshape(M, K) * 7 % (2 * top + 1) - top).astype(np.int8)
    packed = tile_codes_e2m3_a8(q) if (bits, codes) == (8, E2M3) else tile_for(codes, q, bits)
    s = torch.rand(M, generator=torch.Generator().manual_seed(1)) + 0.1
    got = rudder.dequant_act(torch.from_numpy(packed).cuda(), s.cuda(), M, K, bits, codes)
    _equal("values", got, torch.from_numpy(q).float() * s[:, None])


@pytest.mark.parametrize("M", [5, 700])
def test_strides_and_aliases(rudder, M):
    """Rows any distance apart; the sum in the residual's place or in X's; rows in X's place;
    what lies between the rows stays."""
    log(f"case norm strides M={M}")
    K = 264
    x, r, gamma, *_ = _inputs(M, K, 9)
    want, h = ref.norm(x, gamma, EPS, r)
    wide = {n: torch.full((M, K + 8 * i), 7.0, dtype=torch.bfloat16, device="cuda")
            for i, n in enumerate("xrhy", 1)}
    for n, src in (("x", x), ("r", r)):
        wide[n][:, :K] = src.cuda()
    v = {n: t[:, :K] for n, t in wide.items()}
    g = gamma.cuda()
    rudder.rudder_norm(v["x"], v["r"], g, EPS, M, K, v["h"], v["y"])
    for n, src in (("x", x), ("r", r), ("h", h), ("y", want)):
        _equal(n, v[n], src)
        assert (wide[n][:, K:] == 7.0).all(), n
    rudder.rudder_norm(v["x"], v["r"], g, EPS, M, K, v["r"], v["x"])       # both in place
    _equal("h in R", v["r"], h)
    _equal("y in X", v["x"], want)
    v["x"].copy_(x)
    v["r"].copy_(r)
    rudder.rudder_norm(v["x"], v["r"], g, EPS, M, K, v["x"], v["r"])       # the other way round
    _equal("h in X", v["x"], h)
    _equal("y in R", v["r"], want)
    for n in "xrhy":
        assert (wide[n][:, K:] == 7.0).all(), n


def test_values_of_any_size(rudder):
    """Rows near the type's ends, of zeros, of one element, without eps: the formula's numbers."""
    log("case norm sizes")
    K = 256
    g = torch.Generator().manual_seed(4)
    x = torch.randn(600, K, generator=g)
    x *= torch.tensor([2.0 ** e for e in range(-140, 128, 2)] + [0.0]).repeat(5)[:600, None]
    x[7] = 0
    x[9, 1:] = 0
    x = x.clamp(-3.3e38, 3.3e38).to(torch.bfloat16)
    gamma = torch.rand(K, generator=g) + 0.5
    for eps in (EPS, 1.0, 1e-38):
        for rows in (600, 9):
            want, _ = ref.norm(x[:rows], gamma, eps)
            _equal(f"eps={eps} {rows}", rudder.norm(x[:rows].cuda(), gamma.cuda(), eps), want)
    # without eps rows of zeros are NaN, and rows whose 1 / sqrt passes 32 bits infinite
    got = rudder.norm(x.cuda(), gamma.cuda(), 0.0).cpu()
    want, _ = ref.norm(x, gamma, 0.0)
    assert torch.isnan(got[(x == 0).all(1)]).all()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got[~torch.isnan(want)], want[~torch.isnan(want)])


@pytest.mark.parametrize("M", [6, 600])
def test_rows_that_are_not_finite(rudder, M):
    """They give the formula's numbers, and leave the other rows; codes of a row's own step size
    come with one that is not finite."""
    log(f"case norm not finite M={M}")
    K = 512
    x, r, gamma, smooth, *_ = _inputs(M, K, 12)
    clean, _ = ref.norm(x, gamma, EPS, r)
    q, s = ref.codes(clean, smooth, 8)
    x[1, 3], x[2, 5], x[4, 100] = float("nan"), float("inf"), -float("inf")
    want, h = ref.norm(x, gamma, EPS, r)
    y, gh = rudder.norm(x.cuda(), gamma.cuda(), EPS, r.cuda())
    bad = torch.zeros(M, dtype=torch.bool)
    bad[[1, 2, 4]] = True
    _equal("y", y.cpu()[~bad], clean[~bad])
    assert torch.equal(torch.isnan(y.cpu()), torch.isnan(want))
    assert torch.equal(y.cpu().nan_to_num(), want.nan_to_num())
    got = rudder.norm_quant(x.cuda(), gamma.cuda(), smooth.cuda(), EPS, 8, residual=r.cuda())
    assert torch.equal(got[1].cpu()[~bad], s[~bad])
    assert not torch.isfinite(got[1].cpu()[bad]).any()
    rows = rudder.dequant_act(got[0], got[1], M, K, 8)
    _equal("values", rows.cpu()[~bad], (q.float() * s[:, None])[~bad])


def test_zero_rows_and_steps(rudder):
    """No rows; rows of zeros have a step size of 0 and codes of 0; a table's step size of 0."""
    log("case norm zeros")
    K = 128
    x, r, gamma, smooth, sid, table = _inputs(40, K, 5)
    assert rudder.norm(x[:0].cuda(), gamma.cuda(), EPS).shape == (0, K)
    assert rudder.dequant_act(torch.zeros(1, dtype=torch.uint8, device="cuda"),
                              torch.zeros(1, device="cuda"), 0, K, 8).shape == (0, K)
    x[3] = 0
    table[1] = 0
    for kw in ({}, dict(stream_id=sid.cuda(), act_scale=table.cuda())):
        y, _ = ref.norm(x, gamma, EPS)
        q, s = ref.codes(y, smooth, 8, sid, table if kw else None)
        got = rudder.norm_quant(x.cuda(), gamma.cuda(), smooth.cuda(), EPS, 8, **kw)
        _equal("row_scale", got[1], s)
        _equal("Xq", got[0], torch.from_numpy(tile_for(INT, q.numpy(), 8)))
        assert not q[3].any() and (kw or s[3] == 0)


def test_offsets_past_32_bits(rudder):
    """Rows so far apart that the last ones start past 2^31 elements."""
    log("case norm offsets")
    M, K, ld = 70000, 64, 32768
    x, _, gamma, smooth, *_ = _inputs(M, K, 6)
    wide = torch.empty(M * ld, dtype=torch.bfloat16, device="cuda").as_strided((M, K), (ld, 1))
    wide.copy_(x)
    want, _ = ref.norm(x, gamma, EPS)
    got = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    rudder.rudder_norm(wide, None, gamma.cuda(), EPS, M, K, None, got)
    _equal("y", got, want)
    rudder.rudder_norm(got, None, gamma.cuda(), EPS, M, K, None, wide)
    _equal("far y", wide, ref.norm(want, gamma, EPS)[0])
