"""Causal attention of prompts whose scores are far from zero: weights go by the scores' differences."""
import math

import pytest
import torch

import attention_reference as aref
from gpu_harness import log

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rudder():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    from w4a4_quantized_gemm_rudder_amd import rudder as r
    r.load_library()
    return r


def _run(rudder, q, k, v, counts, sm, many):
    """`many`: prompts of no rows behind the others, for the kernel of many rows."""
    starts = torch.tensor([0] + counts + [0] * (600 if many else 0), dtype=torch.int32)
    starts = starts.cumsum(0).to(torch.int32)
    need = rudder.prompt_attention_workspace_bytes(len(starts) - 1, len(q), max(counts),
                                                   q.shape[1], k.shape[1], q.shape[2])
    assert (need > 0) == many
    return rudder.prompt_attention(q.cuda(), k.cuda(), v.cuda(), starts.cuda(), max(counts),
                                   sm).cpu()


def _heads(first, second, T, D, seed):
    """q, k of one head whose products are those of the first two channels."""
    q, k = torch.zeros(T, 1, D), torch.zeros(T, 1, D)
    q[:, 0, :2], k[:, 0, :2] = first, second
    v = torch.randn(T, 1, D, generator=torch.Generator().manual_seed(seed))
    out = [x.to(torch.bfloat16) for x in (q, k, v)]
    assert torch.equal(out[0].float(), q) and torch.equal(out[1].float(), k)
    return out


def _softmax(q, k, v, sm):
    """O and bound of one prompt in 64 bits, all rows.  Products of two channels of few bits are exact in
    32, so a weight is off by its exponent's roundings alone: c to two half steps and the sum to one, of
    the difference from the largest score (45 in base 2 at most: beyond, what is off is less than
    2^-45), and the exponential's four; fp16's half step; and in all by 2^-33 of the largest."""
    z = q[:, 0].double() @ k[:, 0].double().t() * sm
    n = len(z)
    z = z.masked_fill(torch.arange(n)[None, :] > torch.arange(n)[:, None], -math.inf)
    p, vv = torch.softmax(z, -1), v[:, 0].double()
    o = p @ vv
    dz = (3 * 45 + 4) * aref.FP32
    e = (p @ vv.abs()) * (aref.FP16 + 2 * math.log(2) * dz + 2 * (n + 70) * aref.FP32)
    e = e + 2.0 ** -33 * vv.abs().sum(0)
    return o, e + aref.BF16 * (o.abs() + e)


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_rows_of_one_key(rudder, D, sign, many):
    """A row that sees one key has its value, bit for bit, whatever the score."""
    log(f"case prompt scores of one key D={D} sign={sign} many={many}")
    g = torch.Generator().manual_seed(5)
    e = torch.tensor([0, 10, 18, 20, 21, 22, 23, 24, 26, 27, 28, 29, 30, 31, 40, 64, 100, 122] * 12)
    T = len(e)
    a = torch.zeros(T, 2)
    b = torch.zeros(T, 2)
    a[:, 0] = torch.randint(128, 256, (T,), generator=g) * 2.0 ** -7
    b[:, 0] = sign * torch.randint(128, 256, (T,), generator=g) * 2.0 ** -7
    for sm in (1.0, 0.0883883, 1.1e-6, -3.7):
        first = a * (2.0 ** (e // 2))[:, None]
        second = b * (2.0 ** (e - e // 2))[:, None]
        q, k, v = _heads(first, second, T, D, 6)
        got = _run(rudder, q, k, v, [1] * T, sm, many)
        assert torch.equal(got, v), (sm, int((got != v).any(-1).sum()))


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("power", [20, 22, 23, 26, 28, 30, 100])
def test_keys_alike(rudder, D, power, many):
    """Keys of one score: the outputs are means."""
    log(f"case prompt scores alike D={D} 2^{power} many={many}")
    T = 400
    for x in (1.0, -1.0, 1.625, -1.4140625, 1.9921875):
        first, second = torch.zeros(T, 2), torch.zeros(T, 2)
        first[:, 0], second[:, 0] = abs(x) * 2.0 ** (power // 2), math.copysign(2.0 ** (
            power - power // 2), x)
        q, k, v = _heads(first, second, T, D, 7)
        got = _run(rudder, q, k, v, [T], 1.0, many)
        want, bound = _softmax(q, k, v, 1.0)
        aref.assert_within(f"{x}", got[:, 0], want, bound)


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("order", ["up", "down", "mixed"])
@pytest.mark.parametrize("power", [24, 27, 30, 64, 115])
def test_the_largest_score_takes_all(rudder, D, power, order, many):
    """Scores up to 2^power of eight bits each: steps so wide that only the largest have weights."""
    log(f"case prompt scores one takes all D={D} 2^{power} {order} many={many}")
    T = 500
    g = torch.Generator().manual_seed(power)
    for sign in (1.0, -1.0, 0.0):
        s = torch.randint(128, 256, (T,), generator=g).float()
        if sign == 0.0:                            # on both sides of zero
            s *= torch.randint(0, 2, (T,), generator=g) * 2.0 - 1.0
        else:
            s *= sign
        if order != "mixed":
            s = s.sort(descending=order == "down").values
        first, second = torch.zeros(T, 2), torch.zeros(T, 2)
        first[:, 0], second[:, 0] = 2.0 ** (power // 2 - 7), s * 2.0 ** (power - power // 2)
        q, k, v = _heads(first, second, T, D, 8)
        got = _run(rudder, q, k, v, [T], 1.0, many)
        want, bound = _softmax(q, k, v, 1.0)
        aref.assert_within(f"{sign}", got[:, 0], want, bound)


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("offset", [0, 2 ** 19, -2 ** 20, 2 ** 21, -2 ** 22, 2 ** 22, 2 ** 23, -2 ** 23])
def test_differences_far_from_zero(rudder, D, offset, many):
    """Whole numbers up to 100 apart beside an offset that both share: products and their sums are
    exact in 32 bits, and the weights go by the differences."""
    log(f"case prompt scores offset {offset} D={D} many={many}")
    T = 450
    g = torch.Generator().manual_seed(9)
    for order in ("mixed", "up", "down"):
        s = torch.randint(0, 101, (T,), generator=g).float()
        if order != "mixed":
            s = s.sort(descending=order == "down").values
        root = 2.0 ** (int(math.log2(abs(offset))) // 2) if offset else 0.0
        first, second = torch.ones(T, 2), torch.zeros(T, 2)
        first[:, 0], second[:, 0], second[:, 1] = root, offset / root if offset else 0.0, s
        q, k, v = _heads(first, second, T, D, 10)
        for sm in (0.5, 0.0625):
            got = _run(rudder, q, k, v, [T], sm, many)
            want, bound = _softmax(q, k, v, sm)
            aref.assert_within(f"{order} {sm}", got[:, 0], want, bound)


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_scores_of_every_size(rudder, D, many):
    """Near and far scores of both signs in any order, rows of every kind side by side."""
    log(f"case prompt scores of every size D={D} many={many}")
    T = 600
    g = torch.Generator().manual_seed(11)
    for seed in range(4):
        size = torch.randint(0, 5, (T // 20,), generator=g).repeat_interleave(20)
        s = torch.randint(-100, 101, (T,), generator=g).float() / 16
        s *= torch.tensor([1.0, 1.0, 2.0 ** 12, 2.0 ** 24, 2.0 ** 60])[size]
        if seed == 1:
            s = -s.abs()
        if seed == 2:
            s = s.sort().values
        first, second = torch.zeros(T, 2), torch.zeros(T, 2)
        first[:, 0] = torch.where(torch.arange(T) % 3 > 0, 1.0, -1.0) * torch.where(
            torch.arange(T) % 5 > 0, 1.0, 2.0 ** -24)
        second[:, 0] = s
        q, k, v = _heads(first, second, T, D, 12)
        got = _run(rudder, q, k, v, [T], 1.0, many)
        want, bound = _softmax(q, k, v, 1.0)
        aref.assert_within(f"{seed}", got[:, 0], want, bound)
