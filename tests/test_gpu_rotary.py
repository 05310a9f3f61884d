"""Rotary positions against the formula in 64 bits."""
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


def _i32(x):
    return torch.tensor(x, dtype=torch.int32)


def _positions(counts, pos, T):
    out = torch.full((T,), -1, dtype=torch.int64)
    at = 0
    for n, p in zip(counts, pos):
        if p >= 0:
            out[at:at + n] = p + torch.arange(n)
        at += n
    return out


def _check(name, got, x, positions, freq, magnitude, pairs):
    want, bound = ref.rotary(x, positions, freq, magnitude, pairs)
    aref.assert_within(name, got, want, bound)


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("D,part", [(64, 64), (64, 16), (64, 48), (128, 128), (128, 64),
                                    (128, 112)])
@pytest.mark.parametrize("counts,Hq,Hkv", [([1], 1, 1), ([1, 1, 0, 1], 12, 3), ([3, 2], 40, 8),
                                           ([5, 0, 130, 1], 7, 7), ([64], 24, 2)])
def test_layouts(rudder, counts, Hq, Hkv, D, part, pairs):
    """Both layouts, whole and part of the head, one row to many, heads that do and do not fill a
    wave, as two parts of one buffer; channels behind the part are copied bit for bit."""
    log(f"case rotary {counts} Hq={Hq} Hkv={Hkv} D={D} part={part} pairs={pairs}")
    g = torch.Generator().manual_seed(sum(counts) + D + part)
    T = sum(counts)
    pos = [int(p) for p in torch.randint(0, 5000, (len(counts),), generator=g)]
    buf = torch.randn(T, Hq + 2 * Hkv, D, generator=g).to(torch.bfloat16)
    dev = buf.cuda()
    freq = ref.frequencies(part // 2)
    starts = _i32([0] + counts).cumsum(0).to(torch.int32).cuda()
    q, k = rudder.rotary(dev[:, :Hq], dev[:, Hq:Hq + Hkv], starts, freq.cuda(), max(counts),
                         _i32(pos).cuda(), layout=int(pairs))
    at = _positions(counts, pos, T)
    _check("q", q, buf[:, :Hq], at, freq, 1.0, pairs)
    _check("k", k, buf[:, Hq:Hq + Hkv], at, freq, 1.0, pairs)
    assert torch.equal(dev.cpu(), buf)
    assert torch.equal(q.cpu()[..., part:], buf[:, :Hq, part:])
    # in place the same bits, and nothing beside them
    rudder.rotary(dev[:, :Hq], dev[:, Hq:Hq + Hkv], starts, freq.cuda(), max(counts),
                  _i32(pos).cuda(), layout=int(pairs), in_place=True)
    assert torch.equal(dev[:, :Hq], q) and torch.equal(dev[:, Hq:Hq + Hkv], k)
    assert torch.equal(dev[:, Hq + Hkv:].cpu(), buf[:, Hq + Hkv:])


@pytest.mark.parametrize("pos", [0, 1, 16383, 1 << 20, 100_000_007, 2**31 - 3])
@pytest.mark.parametrize("magnitude", [1.0, -1.25, 0.0])
def test_far_positions(rudder, pos, magnitude):
    """Angles are right up to the last position there is, where 32 bits would leave nothing of
    them; row i of the last sequence passes 2^31."""
    log(f"case rotary pos={pos} magnitude={magnitude}")
    g = torch.Generator().manual_seed(3)
    counts, D = [7, 1], 128
    q = torch.randn(8, 3, D, generator=g).to(torch.bfloat16)
    for freq in (ref.frequencies(64), ref.frequencies(64, scaling="parts", factor=8.0,
                                                      trained=8192.0),
                 torch.linspace(3.0, 100.0, 64, dtype=torch.float64)):
        got, none = rudder.rotary(q.cuda(), None, _i32([0, 7, 8]).cuda(), freq.cuda(), 7,
                                  _i32([pos, pos // 2]).cuda(), magnitude)
        assert none is None
        # an angle of 2^38 radians and its product with 1 / (2 pi) in plain 64 bits are off by
        # 2^-16 turns, so the expectation is formed with whole turns taken off exactly
        positions = _positions(counts, [pos, pos // 2], 8)
        a = torch.tensor([[_turned(int(p), float(f)) for f in freq] for p in positions])
        one = torch.ones(8, dtype=torch.int64)
        for t in range(8):
            want, bound = ref.rotary(q[t:t + 1], one[:1], a[t], magnitude, False)
            aref.assert_within(f"row {t}", got[t:t + 1], want, bound)


def _turned(position, freq):
    """position * freq without its whole turns, by exact arithmetic (2 pi to 60 digits)."""
    from fractions import Fraction
    two_pi = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494459")
    a = position * Fraction(freq)
    return float(a - round(a / two_pi) * two_pi)


def test_rows_left_alone(rudder):
    """Rows behind the last sequence, of skipped sequences and behind max_rows stay as they were;
    arrays that point outside the buffers are clamped to them."""
    log("case rotary rows left alone")
    g = torch.Generator().manual_seed(8)
    T, D = 40, 64
    q = torch.randn(T, 2, D, generator=g).to(torch.bfloat16)
    freq = ref.frequencies(D // 2)
    counts, pos = [9, 5, 8], [3, -1, 0]
    dev = q.cuda()
    rudder.rotary(dev, None, _i32([0, 9, 14, 22]).cuda(), freq.cuda(), 7, _i32(pos).cuda(),
                  in_place=True)
    at = _positions(counts, pos, T)
    at[7:9] = at[21] = -1
    _check("q", dev, q, at, freq, 1.0, False)
    assert torch.equal(dev.cpu()[at < 0], q[at < 0])
    dev = q.cuda()
    rudder.rotary(dev, None, _i32([-5, 3, 2, 10**9, T]).cuda(), freq.cuda(), 1000, None,
                  in_place=True)
    at = torch.full((T,), -1, dtype=torch.int64)
    at[:3], at[2:] = torch.arange(3), torch.arange(T - 2)
    # row 2 belongs to two sequences: whichever came first, it has been turned by some angle
    keep = torch.arange(T) != 2
    want, bound = ref.rotary(q, at, freq, 1.0, False)
    aref.assert_within("clamped", dev[keep.cuda()], want[keep], bound[keep])


def test_offsets_past_32_bits(rudder):
    log("case rotary offsets")
    T, D, ld = 70000, 64, 32768
    g = torch.Generator().manual_seed(2)
    q = torch.randn(T, 1, D, generator=g).to(torch.bfloat16)
    far = torch.empty(T * ld, dtype=torch.bfloat16, device="cuda").as_strided((T, 1, D), (ld, D, 1))
    far.copy_(q)
    freq = ref.frequencies(D // 2)
    rudder.rotary(far, far, _i32([0, T]).cuda(), freq.cuda(), T, None, in_place=False)
    rudder.rotary(far, None, _i32([0, T]).cuda(), freq.cuda(), T, None, in_place=True)
    _check("q", far, q, torch.arange(T), freq, 1.0, False)


def test_relative_positions(rudder):
    """What rotary positions are for: products of turned rows depend on the positions' distance."""
    log("case rotary distance")
    g = torch.Generator().manual_seed(5)
    q, k = (torch.randn(1, 1, 128, generator=g).to(torch.bfloat16) for _ in range(2))
    freq = rudder.rotary_frequencies(128, scaling="base", factor=4.0)

    def product(i, j):
        turn = lambda x, p: rudder.rotary(x.cuda(), None, _i32([0, 1]).cuda(), freq, 1,  # noqa: E731
                                          _i32([p]).cuda())[0].double()
        return float((turn(q, i) * turn(k, j)).sum())

    size = float((q.double().norm() * k.double().norm()))
    base = product(37, 0)
    for shift in (1, 1000, 123456):
        # two bf16 roundings of each row, each at most half a step of an element
        assert abs(product(37 + shift, shift) - base) <= 4 * aref.BF16 * size
    assert abs(product(38, 0) - base) > 1e-3 * size
