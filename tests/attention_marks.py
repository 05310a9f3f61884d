"""States in which every token can be told from every other: which of them a row saw, and no
other, stands in its output.

Token j of a sequence has one mark in its key, at channel j % D, and one in its value, at channel
(j // D) % D.  A query that is one-hot at channel c weighs the visible tokens with j % D = c alike
and all others with exp(-30): its output is 1 / (their number) at the channels of their values and 0
elsewhere.  One token too many or too few changes one channel of one row from or to 0."""
import torch

MARK = 100                 # code of a mark
SHARPNESS = 30.0           # a marked token's exponent above the others'
LEAK = 1e-12               # exp(-30) and what 10000 tokens make of it, relative to a mark's share


def token_marks(tokens, D):
    """Keys and values [n, D] (0 or 1) of the tokens with these numbers."""
    eye = torch.eye(D, dtype=torch.int8)
    return eye[tokens % D], eye[(tokens // D) % D]


def queries(classes, D, sm, key_value):
    """One-hot queries [..., D], so large that sm * q . k is SHARPNESS at a mark (to bf16's
    rounding, the same for all)."""
    q = torch.zeros(*classes.shape, D)
    q.scatter_(-1, classes[..., None], SHARPNESS / (sm * key_value))
    return q.to(torch.bfloat16)


def expected(classes, visible, D, value):
    """classes [n], visible [n, kv] -> O [n, D] in 64 bits: the mean of the values of the visible
    tokens of a row's class, or of all visible tokens where there is none of the class; zeros
    where nothing is visible."""
    tokens = torch.arange(visible.shape[1])
    mine = visible & ((tokens % D)[None, :] == classes[:, None])
    mine = torch.where(mine.any(1, keepdim=True), mine, visible).double()
    v = token_marks(tokens, D)[1].double() * value
    return mine @ v / mine.sum(1, keepdim=True).clamp(min=1)


def bound(want, value, half_step):
    """The weights of a row's tokens are one number, rounded to the product's type (half_step) in
    the numerator and not in the sum; sums of equal terms and the division in 32 bits, below 2^-16
    for 2^8 additions of 2^-24 each on either side of the quotient; the other tokens' leak;
    the rounding to bf16."""
    e = want * (half_step + 2.0 ** -15) + LEAK * 1e4 * value
    return e + 2.0 ** -8 * (want + e)
