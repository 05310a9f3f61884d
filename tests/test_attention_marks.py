"""The marked states tell mistakes apart (no GPU needed): tokens that a row should not have seen, or
should have and did not, leave the bound the kernels are held to."""
import pytest
import torch

import attention_marks as marks
from attention_reference import visible

PAGE = 64


def _outside(classes, seen, should, D):
    """Rows whose output over the tokens `seen` is outside the bound around `should`."""
    want = marks.expected(classes, should, D, 1.0)
    got = marks.expected(classes, seen, D, 1.0)
    return int(((got - want).abs() > marks.bound(want, 1.0, 2.0 ** -8)).any(1).sum())


@pytest.mark.parametrize("D,rows,kv", [(64, 20, 3000), (128, 1, 9000), (128, 300, 2500),
                                       (64, 1, 70405), (128, 20, 44805)])
def test_mistakes_are_outside(D, rows, kv):
    g = torch.Generator().manual_seed(1)
    pages = (kv + PAGE - 1) // PAGE
    page = torch.arange(kv) // PAGE
    # one row of every class, everything visible: a page that is dropped shows
    classes = torch.arange(D)
    full = torch.ones(D, kv, dtype=torch.bool)
    for p in [0, 1, pages - 1] + torch.randint(0, pages, (5,), generator=g).tolist():
        assert _outside(classes, full & (page != p), full, D) > 0, p
    # pages that stand in each other's places: all behind the 64th one further on, the last ones
    # replaced by the first
    v = marks.token_marks(torch.arange(kv), D)[1].double()
    want = marks.expected(classes, full, D, 1.0)
    for places in (torch.where(page < 64, page, torch.clamp(page + 1, max=pages - 1)),
                   torch.where(page >= pages - 5, page - (pages - 5), page)):
        token = torch.clamp(places * PAGE + torch.arange(kv) % PAGE, max=kv - 1)
        if torch.equal(token, torch.arange(kv)):
            continue
        mine = ((token % D)[None, :] == classes[:, None]).double()
        got = mine @ v[token] / mine.sum(1, keepdim=True).clamp(min=1)
        assert ((got - want).abs() > marks.bound(want, 1.0, 2.0 ** -8)).any()
    # a causal limit one too low shows in the row whose class is its last token's, one too
    # high in the row whose class is the next one's (but in the last row, which has no next)
    see = visible(rows, kv, True)
    last = kv - rows + torch.arange(rows)
    assert _outside(last % D, see & (torch.arange(kv) < last[:, None]), see, D) == rows
    more = torch.arange(kv)[None, :] <= last[:, None] + 1
    assert _outside((last + 1) % D, more, see, D) == rows - 1
