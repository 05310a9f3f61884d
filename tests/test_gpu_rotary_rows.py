"""Rotary positions where a launch's workgroups take several turns: far more rows, or a bound on them far
above the sequences' lengths."""
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


@pytest.mark.parametrize("pairs", [False, True])
def test_a_loose_bound_on_many_sequences(rudder, pairs):
    """65535 sequences, all but a few of one row or none, with a bound of all rows there are: the rows
    are those of each sequence turned on its own."""
    log(f"case rotary loose bound pairs={pairs}")
    g = torch.Generator().manual_seed(1)
    B, D = 65535, 64
    counts = torch.randint(0, 2, (B,), generator=g)
    counts[[7, 40000, B - 1]] = torch.tensor([5000, 77, 300])
    T = int(counts.sum()) + 9
    starts = torch.zeros(B + 1, dtype=torch.int32)
    starts[1:] = counts.cumsum(0)
    pos = torch.randint(-3, 1000, (B,), generator=g).clamp(min=-1).to(torch.int32)
    pos[[7, 40000, B - 1]] = torch.tensor([11, 0, 500], dtype=torch.int32)
    q = torch.randn(T, 2, D, generator=g).to(torch.bfloat16)
    freq = ref.frequencies(D // 2)
    dev = q.cuda()
    rudder.rotary(dev, None, starts.cuda(), freq.cuda(), 1 << 25, pos.cuda(), layout=int(pairs),
                  in_place=True)
    at = torch.full((T,), -1, dtype=torch.int64)
    of = torch.repeat_interleave(torch.arange(B), counts)
    rows = torch.arange(len(of))
    at[:len(of)] = torch.where(pos[of] >= 0, pos[of].long() + rows - starts[of].long(), -1)
    want, bound = ref.rotary(q, at, freq, 1.0, pairs)
    aref.assert_within("q", dev, want, bound)
    assert torch.equal(dev.cpu()[at < 0], q[at < 0])


def test_more_rows_than_a_launch_takes_at_once(rudder):
    """One sequence of 2^22 rows and some: as its two parts, each at its own position."""
    log("case rotary long sequence")
    T, D, cut = (1 << 22) + 1003, 64, 1 << 21
    g = torch.Generator(device="cuda").manual_seed(2)
    q = torch.randn(T, 1, D, generator=g, device="cuda", dtype=torch.bfloat16)
    freq = ref.frequencies(D // 2).cuda()
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    whole, _ = rudder.rotary(q, None, i32(0, T), freq, T, i32(5))
    parts, _ = rudder.rotary(q, None, i32(0, cut, T), freq, T - cut, i32(5, 5 + cut))
    assert torch.equal(whole, parts)
    some = torch.tensor([0, 1, cut, (1 << 22) - 1, 1 << 22, (1 << 22) + 5, T - 1])
    want, bound = ref.rotary(q[some.cuda()].cpu(), some + 5, freq.cpu(), 1.0, False)
    aref.assert_within("q", whole[some.cuda()], want, bound)
