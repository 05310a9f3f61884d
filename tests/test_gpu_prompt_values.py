"""Causal attention of prompts whose values differ in size from tile to tile and from key to key: every
key's value keeps its bits, whatever weight the larger ones have."""
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


def _run(rudder, q, k, v, sm, among=0):
    """One prompt; `among` prompts of no rows behind it, for the kernel of many rows."""
    n = len(q)
    starts = torch.tensor([0] + [n] * (among + 1), dtype=torch.int32)
    if among:
        assert rudder.prompt_attention_workspace_bytes(among + 1, n, n, q.shape[1], k.shape[1],
                                                       q.shape[2]) > 0
    return rudder.prompt_attention(q.cuda(), k.cuda(), v.cuda(), starts.cuda(), n, sm).cpu()


def _by_tiles(q, k, v, sm, rows):
    """O and bound [rows, Hq, D] in 64 bits, value by value.

    A weight is off by fp16's half step, or by 2^-33 of the row's largest, and never by more than itself
    (0 is a number of fp16); a value by 2^-32 of the largest of its tile of 64 tokens.  The exponent's
    error and the sums' as in attention_reference.rows_attention.  bf16 numbers below 2^-126 are 2^-133
    apart, whose half is added."""
    G = q.shape[1] // k.shape[1]
    o = torch.zeros(len(rows), *q.shape[1:], dtype=torch.float64)
    e = torch.zeros_like(o)
    for h in range(q.shape[1]):
        kk, vv, qq = k[:, h // G].double(), v[:, h // G].double(), q[:, h].double()
        tops = torch.stack([x.abs().amax() for x in vv.split(TILE)]).repeat_interleave(TILE)
        for i, t in enumerate(rows.tolist()):
            ks, vs = kk[:t + 1], vv[:t + 1]
            s = ks @ qq[t] * sm
            p = torch.softmax(s, 0)
            zmax = float((ks.abs() @ qq[t].abs()).max()) * abs(sm) / math.log(2)
            dz = zmax * (ks.shape[1] + 8 + 6) * aref.FP32 + (3 * 80 + 4) * aref.FP32
            A = p @ vs.abs()
            o[i, h] = p @ vs
            bound = A * (aref.FP16 + 2 * math.log(2) * dz + 2 * (t + 71) * aref.FP32)
            bound += torch.minimum(p, 2.0 ** -33 * p.max()) @ vs.abs()
            bound += 2.0 ** -32 * (p * tops[:t + 1]).sum()
            e[i, h] = bound + aref.BF16 * (o[i, h].abs() + bound) + 2.0 ** -134
    return o, e


# rows, prompts of no rows behind them
KERNELS = [(520, 0), (520, 600), (1100, 0), (1500, 600)]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows,among", KERNELS)
@pytest.mark.parametrize("power", [16, 24, 32, 60, 100])
@pytest.mark.parametrize("where", ["first", "middle", "last", "all but one"])
def test_large_values_of_no_weight(rudder, D, rows, among, power, where):
    """Tiles of values 2^power as large whose softmax weights are 2^-(power + 40): the outputs are
    those of the other tiles, whatever the order."""
    log(f"case prompt values of no weight D={D} rows={rows}/{among} 2^{power} {where}")
    g = torch.Generator().manual_seed(power + rows)
    tiles = (rows + TILE - 1) // TILE
    large = {"first": [0], "middle": [3], "last": [tiles - 1],
             "all but one": [t for t in range(tiles) if t != 2]}[where]
    is_large = torch.tensor([t in large for t in range(tiles)]).repeat_interleave(TILE)[:rows]
    q = torch.randn(rows, 2, D, generator=g) * 0.1
    k = torch.randn(rows, 1, D, generator=g) * 0.1
    v = torch.randn(rows, 1, D, generator=g) + 1.0
    # the first channel carries the weight: log2 of it is -(power + 40) for the large ones
    q[:, :, 0] = 8.0
    k[:, :, 0] = torch.where(is_large, -(power + 40) * math.log(2) / 8.0, 0.0)[:, None]
    v *= torch.where(is_large, 2.0 ** power, 1.0)[:, None, None]
    q, k, v = (x.to(torch.bfloat16) for x in (q, k, v))
    got = _run(rudder, q, k, v, 1.0, among)
    some = torch.cat([torch.arange(0, rows, 37), torch.tensor([63, 64, 127, 128, 191, 192, 200,
                                                                255, 256, rows - 1])]).unique()
    want, bound = _by_tiles(q, k, v, 1.0, some)
    aref.assert_within("O", got[some], want, bound)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows,among", KERNELS)
def test_a_row_each_way(rudder, D, rows, among):
    """Rows side by side of which every second one sees only the large tiles and the others only the
    small ones."""
    log(f"case prompt values a row each way D={D} rows={rows}/{among}")
    g = torch.Generator().manual_seed(rows)
    tile = torch.arange(rows) // TILE
    q = torch.randn(rows, 3, D, generator=g) * 0.1
    k = torch.randn(rows, 1, D, generator=g) * 0.1
    q[:, :, 0] = torch.where(torch.arange(rows) % 2 > 0, 12.0, -12.0)[:, None]
    for powers in ([40, 0], [0, 40], [100, 0, -20, 50], [0, 8, -8, 16], [-100, 20], [120, -120]):
        e = torch.tensor(powers)[tile % len(powers)].double()
        vv = (torch.randn(rows, 1, D, generator=g).double() * (2.0 ** e)[:, None, None])
        kk = k.clone()
        kk[:, :, 0] = torch.where(e > sorted(powers)[0], 10.0, -10.0)[:, None].float()
        qq, kk, vv = (x.to(torch.bfloat16) for x in (q, kk, vv.float()))
        got = _run(rudder, qq, kk, vv, 1.0, among)
        some = torch.cat([torch.arange(60, 70), torch.arange(1, rows, 41),
                          torch.tensor([rows - 2, rows - 1])]).unique()
        want, bound = _by_tiles(qq, kk, vv, 1.0, some)
        aref.assert_within(f"{powers}", got[some], want, bound)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows,among", KERNELS)
def test_small_weights_keep_their_bits(rudder, D, rows, among):
    """A first token of value zero takes nearly all of the weight, the others have 2^-20 of its each:
    the outputs are theirs, in tiles of different sizes."""
    log(f"case prompt small weights D={D} rows={rows}/{among}")
    g = torch.Generator().manual_seed(rows + 1)
    q = torch.randn(rows, 2, D, generator=g) * 0.1
    k = torch.randn(rows, 1, D, generator=g) * 0.1
    q[:, :, 0], k[:, :, 0] = 4.0, 0.0
    k[0, :, 0] = 20 * math.log(2) / 4.0
    for powers in ([0], [0, 8], [8, 0, 16], [0, -8, -24, 7]):
        e = torch.tensor(powers)[torch.arange(rows) // TILE % len(powers)].double()
        v = torch.rand(rows, 1, D, generator=g).double() + 0.5
        v = v * (2.0 ** e)[:, None, None]
        v[0] = 0
        qq, kk, vv = (x.to(torch.bfloat16) for x in (q, k, v.float()))
        got = _run(rudder, qq, kk, vv, 1.0, among)
        some = torch.cat([torch.arange(1, 70, 6), torch.arange(70, rows, 41)])
        want, bound = _by_tiles(qq, kk, vv, 1.0, some)
        aref.assert_within(f"{powers}", got[some], want, bound)


@pytest.mark.parametrize("power", [32, 100])
def test_large_values_of_no_weight_in_a_long_prompt(rudder, power):
    """The same on the kernel of eight waves; the bound as in _by_tiles, all rows of two heads."""
    log(f"case long prompt values of no weight 2^{power}")
    n, H, D = 8300, 16, 128
    g = torch.Generator(device="cuda").manual_seed(power)
    r = lambda h: torch.randn(n, h, D, generator=g, device="cuda")  # noqa: E731
    q, k, v = r(H) * 0.1, r(H) * 0.1, r(H) + 1.0
    large = (torch.arange(n, device="cuda") // TILE) % 5 == 2
    q[:, :, 0] = 8.0
    k[:, :, 0] = torch.where(large, -(power + 40) * math.log(2) / 8.0, 0.0)[:, None]
    v *= torch.where(large, 2.0 ** power, 1.0)[:, None, None]
    q, k, v = (x.to(torch.bfloat16) for x in (q, k, v))
    starts = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    got = rudder.prompt_attention(q, k, v, starts, n, 1.0)
    i = torch.arange(n, device="cuda")
    for h in (0, 9):
        qq, kt, vv = q[:, h].double(), k[:, h].double().t().contiguous(), v[:, h].double()
        tops = torch.stack([x.abs().amax() for x in vv.split(TILE)]).repeat_interleave(TILE)[:n]
        p = torch.softmax((qq @ kt).masked_fill_(i[None, :] > i[:, None], -math.inf), -1)
        want = p @ vv
        zmax = float((qq.abs() @ kt.abs()).max()) / math.log(2)
        dz = zmax * (D + 14) * aref.FP32 + 244 * aref.FP32
        bound = (p @ vv.abs()) * (aref.FP16 + 2 * math.log(2) * dz + 2 * (n + 70) * aref.FP32)
        bound += torch.minimum(p, 2.0 ** -33 * p.amax(-1, keepdim=True)) @ vv.abs()
        bound += 2.0 ** -32 * (p @ tops)[:, None]
        bound = bound + aref.BF16 * (want.abs() + bound) + 2.0 ** -134
        aref.assert_within(f"head {h}", got[:, h], want.cpu(), bound.cpu())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows,among", KERNELS)
@pytest.mark.parametrize("step", [12, 16, 24, 25, 26, 31])
def test_a_maximum_that_jumps(rudder, D, rows, among, step):
    """Every 32, 64 or 96 keys the scores go up by 2^step, and the values down by as much: the weights in
    front of a jump count as those behind it."""
    log(f"case prompt maximum that jumps D={D} rows={rows}/{among} 2^{step}")
    g = torch.Generator().manual_seed(step)
    for keys in (32, 64, 96):
        level = torch.clamp(torch.arange(rows) // keys, max=3).float()
        q = torch.randn(rows, 2, D, generator=g) * 0.1
        k = torch.randn(rows, 1, D, generator=g) * 0.1
        v = torch.rand(rows, 1, D, generator=g) + 0.5
        q[:, :, 0] = 16.0
        k[:, :, 0] = (level * step * math.log(2) / 16.0)[:, None]
        v *= (2.0 ** (-level * step))[:, None, None]
        q, k, v = (x.to(torch.bfloat16) for x in (q, k, v))
        got = _run(rudder, q, k, v, 1.0, among)
        some = torch.cat([torch.arange(24, rows if rows < 300 else 300, 8), torch.tensor([rows - 1])])
        want, bound = _by_tiles(q, k, v, 1.0, some)
        aref.assert_within(f"{keys}", got[some], want, bound)


@pytest.mark.parametrize("rows", [640, 641])
def test_sizes_beside_a_limit(rudder, rows):
    """16 heads of 128 channels: 320 work units of the few rows' kernel, and one more."""
    log(f"case prompt values beside a limit rows={rows}")
    g = torch.Generator().manual_seed(rows)
    q, k, v = (torch.randn(rows, 16, 128, generator=g).to(torch.bfloat16) for _ in range(3))
    got = _run(rudder, q, k, v, 0.09)
    some = torch.cat([torch.arange(0, rows, 61), torch.arange(rows - 3, rows)])
    pick = lambda x: x[:, [0, 7, 15]].contiguous()  # noqa: E731
    want, bound = _by_tiles(pick(q), pick(k), pick(v), 0.09, some)
    aref.assert_within("O", pick(got)[some], want, bound)
