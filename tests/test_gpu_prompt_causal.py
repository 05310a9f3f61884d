"""Causal attention of prompts whose tokens' values are of very different sizes: a row's output goes by what
the row sees, also inside the tile of 64 tokens that it stands in."""
import math

import pytest
import torch

import attention_reference as aref
from gpu_harness import log

pytestmark = pytest.mark.gpu
TILE = 64


@pytest.fixture(scope="module")
def rudder():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    from w4a4_quantized_gemm_rudder_amd import rudder as r
    r.load_library()
    return r


def _run(rudder, q, k, v, sm, among):
    """One prompt; `among` prompts of no rows behind it, for the kernel of many rows."""
    n = len(q)
    starts = torch.tensor([0] + [n] * (among + 1), dtype=torch.int32)
    need = rudder.prompt_attention_workspace_bytes(among + 1, n, n, q.shape[1], k.shape[1],
                                                   q.shape[2])
    assert (need > 0) == (among > 0)
    return rudder.prompt_attention(q.cuda(), k.cuda(), v.cuda(), starts.cuda(), n, sm).cpu()


def _bounds(q, k, v, sm, rows):
    """O and bound [rows, Hq, D] in 64 bits, on the tensors' device.

    A weight is off by fp16's half step, or by 2^-33 of the row's largest, and never by more than itself
    (0 is a number of fp16); a value by 2^-32 of the largest of its tile where the row sees the whole
    tile, and by 2^-24 of the largest of its own token where it does not.  The exponent's error and the
    sums' as in attention_reference.rows_attention; bf16 numbers below 2^-126 are 2^-133 apart, whose
    half is added."""
    G, n, D = q.shape[1] // k.shape[1], len(q), q.shape[2]
    o = torch.zeros(len(rows), *q.shape[1:], dtype=torch.float64, device=q.device)
    e = torch.zeros_like(o)
    j = torch.arange(n, device=q.device)[None, :]
    t = rows.to(q.device)[:, None]
    ends = torch.clamp((j // TILE + 1) * TILE, max=n) - 1        # the last token of a token's tile
    for h in range(q.shape[1]):
        kk, vv, qq = k[:, h // G].double(), v[:, h // G].double(), q[rows.to(q.device), h].double()
        tokens = vv.abs().amax(1)
        tiles = torch.stack([x.amax() for x in tokens.split(TILE)]).repeat_interleave(TILE)[:n]
        p = torch.softmax((qq @ kk.t().contiguous() * sm).masked_fill(j > t, -math.inf), -1)
        zmax = (qq.abs() @ kk.abs().t().contiguous()).masked_fill(j > t, 0).amax(1, keepdim=True)
        dz = zmax * abs(sm) / math.log(2) * (D + 14) * aref.FP32 + 244 * aref.FP32
        o[:, h] = p @ vv
        b = (p @ vv.abs()) * (aref.FP16 + 2 * math.log(2) * dz + 2 * (t + 71) * aref.FP32)
        b += torch.minimum(p, 2.0 ** -33 * p.amax(1, keepdim=True)) @ vv.abs()
        off = torch.where(ends <= t, 2.0 ** -32 * tiles[None, :], 2.0 ** -24 * tokens[None, :])
        b += (p * off).sum(1, keepdim=True)
        e[:, h] = b + aref.BF16 * (o[:, h].abs() + b) + 2.0 ** -134
    return o, e


# rows, prompts of no rows behind them
KERNELS = [(100, 0), (520, 0), (100, 600), (520, 600)]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows,among", KERNELS)
@pytest.mark.parametrize("large", [2.0 ** 9, 2.0 ** 24, 2.0 ** 32, -2.0 ** 60, 3.38e38])
def test_large_values_behind_a_row(rudder, D, rows, among, large):
    """One token's values are far larger than the others': the rows in front of it, in its tile and
    before, have the outputs that they have without it, within their own bound."""
    log(f"case prompt causal D={D} rows={rows}/{among} large={large}")
    g = torch.Generator().manual_seed(rows)
    q, k, v = (torch.randn(rows, h, D, generator=g).to(torch.bfloat16) for h in (3, 1, 1))
    for at in (1, 31, 40, 63, 64, 65, 95, rows - 1):
        vv = v.clone()
        vv[at, 0, at % D] = large
        got = _run(rudder, q, k, vv, 0.1, among)
        some = torch.cat([torch.arange(max(0, at - 40), min(rows, at + 12)),
                          torch.arange(0, rows, 29)]).unique()
        want, bound = _bounds(q, k, vv, 0.1, some)
        aref.assert_within(f"at {at}", got[some], want, bound)
        clean = _run(rudder, q, k, v, 0.1, among)
        assert torch.equal(got[:at // TILE * TILE], clean[:at // TILE * TILE]), at


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows,among", KERNELS)
def test_tokens_of_every_size(rudder, D, rows, among):
    """Every token's values times a power of two of its own, up, down and mixed, zeros among them, with
    near and far weights."""
    log(f"case prompt causal sizes D={D} rows={rows}/{among}")
    g = torch.Generator().manual_seed(rows + 1)
    q, k, v = (torch.randn(rows, h, D, generator=g) for h in (4, 2, 2))
    i = torch.arange(rows)
    mixed = lambda lo, hi: torch.randint(lo, hi, (rows,), generator=g)  # noqa: E731
    for name, e, sm in (("up", i // 2 - 100, 0.1), ("down", 100 - i // 2, 0.1),
                        ("mixed", mixed(-60, 61), 0.1), ("mixed far", mixed(-60, 61), 3.0),
                        ("some", mixed(0, 20) // 19 * 100, 0.5), ("ends", mixed(0, 2) * 240 - 118, 1.0),
                        ("small", mixed(-126, -100), 0.1)):
        vv = (v.double() * (2.0 ** e.double().clamp(-130, 122))[:, None, None]).to(torch.bfloat16)
        vv[mixed(0, 10) == 0] = 0
        qq, kk = q.to(torch.bfloat16), k.to(torch.bfloat16)
        got = _run(rudder, qq, kk, vv, sm, among)
        some = torch.cat([torch.arange(min(rows, 70)), torch.arange(70, rows, 17)])
        want, bound = _bounds(qq, kk, vv, sm, some)
        aref.assert_within(name, got[some], want, bound)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows,among", [(100, 0), (300, 600)])
def test_values_that_are_not_finite_among_uneven_ones(rudder, D, rows, among):
    """Infinities and NaN in a tile of uneven values: NaN from their row on, the rows in front as
    without them, rows behind the prompt and the other head's as they were."""
    log(f"case prompt causal not finite D={D} rows={rows}/{among}")
    g = torch.Generator().manual_seed(rows + 2)
    q, k, v = (torch.randn(rows, h, D, generator=g).to(torch.bfloat16) for h in (4, 2, 2))
    v[50, 1] *= 2.0 ** 70
    clean = _run(rudder, q, k, v, 0.1, among)
    for at in (20, 50, 60, 70):
        for bad in (math.nan, math.inf, -math.inf):
            vv = v.clone()
            vv[at, 1, 3] = bad
            got = _run(rudder, q, k, vv, 0.1, among)
            assert torch.equal(got[:, :2], clean[:, :2])
            assert torch.isnan(got[at:, 2:]).all()
            some = torch.arange(at)
            want, bound = _bounds(q[:at], k[:at], v[:at], 0.1, some)
            # the rows in front see none of it; their tile's even so counts as not seen whole
            aref.assert_within(f"{at} {bad}", got[:at], want, bound + 2.0 ** -24 * bound)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows,among", KERNELS)
def test_large_values_of_no_weight_beside_small_ones(rudder, D, rows, among):
    """A row's own tile holds a token of large values and no weight, and small values of a small weight
    beside a zero that takes the rest: the small ones are the output."""
    log(f"case prompt causal no weight D={D} rows={rows}/{among}")
    g = torch.Generator().manual_seed(rows + 4)
    for large, small in ((72, -66), (100, -30), (30, -100)):
        for at in (0, 30, 63):
            power, weight = torch.full((rows,), float(small) - 4), torch.full((rows,), -60.0)
            i = torch.arange(rows) % TILE
            power[i == at], weight[i == at] = large, -(large - small + 60.0)
            power[i == 4], weight[i == 4] = small, -20.0
            weight[i == 7] = 0.0
            q, k, v = (torch.randn(rows, h, D, generator=g) * 0.1 for h in (2, 1, 1))
            q[:, :, 0], k[:, :, 0] = 8.0, (weight * math.log(2) / 8.0)[:, None]
            v = (v + 1.0).double() * (2.0 ** power.double())[:, None, None]
            v[i == 7] = 0
            q, k, v = (x.to(torch.bfloat16) for x in (q, k, v))
            got = _run(rudder, q, k, v, 1.0, among)
            some = torch.cat([torch.arange(min(rows, 70)), torch.arange(70, rows, 9)])
            want, bound = _bounds(q, k, v, 1.0, some)
            aref.assert_within(f"{large} {small} {at}", got[some], want, bound)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows,among", KERNELS)
def test_zeros_in_front_of_large_values(rudder, D, rows, among):
    """Tiles of small values, then tiles of large ones whose first tokens are zeros: rows that see of these
    only the zeros have what the small ones give."""
    log(f"case prompt causal zeros D={D} rows={rows}/{among}")
    g = torch.Generator().manual_seed(rows + 5)
    q, k = (torch.randn(rows, h, D, generator=g).to(torch.bfloat16) for h in (2, 1))
    i = torch.arange(rows)
    for small, large in ((-90, 100), (-100, 20), (0, 120)):
        v = torch.randn(rows, 1, D, generator=g) + 2.0
        v = v.double() * (2.0 ** torch.where(i // TILE % 2 > 0, large, small).double())[:, None, None]
        v[i % (2 * TILE) // 10 == 6] = 0               # 60 .. 69 of every 128
        v = v.to(torch.bfloat16)
        got = _run(rudder, q, k, v, 0.1, among)
        some = torch.cat([torch.arange(50, min(rows, 90)), torch.arange(min(180, rows), rows, 5)])
        want, bound = _bounds(q, k, v, 0.1, some)
        aref.assert_within(f"{small} {large}", got[some], want, bound)


def test_tokens_of_every_size_in_a_long_prompt(rudder):
    """The same on the kernel of eight waves, all rows of two heads."""
    log("case long prompt causal sizes")
    n, H, D = 8300, 16, 128
    g = torch.Generator(device="cuda").manual_seed(3)
    q, k, v = (torch.randn(n, H, D, generator=g, device="cuda") for _ in range(3))
    e = torch.randint(-60, 61, (n,), generator=g, device="cuda").double()
    e = torch.where(torch.arange(n, device="cuda") // 200 % 2 > 0, e, 0.0)
    v = v.double() * (2.0 ** e)[:, None, None]
    q, k, v = (x.to(torch.bfloat16) for x in (q, k, v))
    starts = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    got = rudder.prompt_attention(q, k, v, starts, n, 0.3)
    for h in (0, 9):
        pick = lambda x: x[:, h:h + 1].contiguous()  # noqa: E731
        want, bound = _bounds(pick(q), pick(k), pick(v), 0.3, torch.arange(n))
        aref.assert_within(f"head {h}", got[:, h:h + 1], want.cpu(), bound.cpu())
