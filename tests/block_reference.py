"""Plain forms of the norms, rotary positions and prompt attention from the
definitions in the header, on the CPU, and the bounds their kernels are held to."""
import math

import torch

import attention_reference as ref

FP32 = ref.FP32
QMAX = {8: 127.0, 4: 7.0}


# --- norms -------------------------------------------------------------------
# Bit for bit: squares of bf16 values and, but for 2^-53, their sums are exact in 64 bits, so that
# only what the definition rounds is rounded.

def norm(x, gamma, eps, residual=None):
    """(y, h) in bf16."""
    h = x if residual is None else (residual.float() + x.float()).to(torch.bfloat16)
    f = h.float()
    mean = (f.double() ** 2).sum(1, keepdim=True) / x.shape[1]
    r = (1 / torch.sqrt(mean + float(torch.tensor(eps, dtype=torch.float32)))).float()
    return ((f * r) * gamma).to(torch.bfloat16), h


def codes(y, inv_smooth, bits, sid=None, table=None):
    """(integer codes int8 [M, K], row scales): the quantizer's rule, a step size a row without a
    table."""
    q = QMAX[bits]
    u = y.float() * inv_smooth
    s = (u.abs().amax(1).double() / q).float() if table is None else table[sid.long()]
    c = torch.round(torch.clamp(u * ref.recip(s)[:, None], -q, q))
    return c.to(torch.int8), s


# --- rotary positions ----------------------------------------------------------

def frequencies(n, base=10000.0, scaling="plain", factor=1.0, trained=0.0, low=1.0, high=32.0):
    """Pair by pair, in Python's own floats."""
    out = []
    for i in range(n):
        b = base * factor ** (n / (n - 1)) if scaling == "base" and n > 1 else base
        f = b ** (-i / n)
        if scaling == "linear":
            f /= factor
        if scaling == "parts":
            turns = trained * f / (2 * math.pi)
            keep = min(max((turns - low) / (high - low), 0.0), 1.0)
            f = f / factor * (1 - keep) + f * keep
        out.append(f)
    return torch.tensor(out, dtype=torch.float64)


def rotary(x, positions, freq, magnitude, pairs):
    """x [T, H, D] at positions [T] (negative: untouched) -> (values in 64 bits, bound).

    The angle is off by 2^-26 turns from its rounding to 32 bits and the library's sine and cosine
    by 4 half steps of one, their magnitude's product and the two products and the sum by half a
    step each; the rounding to bf16."""
    n = freq.numel()
    x = x.double()
    out, e = x.clone(), torch.zeros_like(x)
    a = positions.double()[:, None] * freq
    c, s = (magnitude * f(a)[:, None] for f in (torch.cos, torch.sin))
    lo, hi = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if pairs else (slice(0, n), slice(n, 2 * n))
    u, v = x[..., lo], x[..., hi]
    there = (positions >= 0)[:, None, None]
    size = (u.abs() + v.abs()) * abs(magnitude)
    err = size * (2 * math.pi * 2.0 ** -26 + 8 * FP32)
    for at, val in ((lo, u * c - v * s), (hi, v * c + u * s)):
        out[..., at] = torch.where(there, val, out[..., at])
        e[..., at] = torch.where(there, err + ref.BF16 * (val.abs() + err), 0.0)
    return out, e


# --- prompt attention ------------------------------------------------------------

def prompt(q, k, v, starts, sm, heads=None, rows=None):
    """O and bound [T, Hq, D] in 64 bits; `heads`, `rows` (of every prompt): those computed.

    As attention over other keys, with weights rounded to fp16; a value is off by at most 2^-32 of
    its tile's largest; and bf16 numbers below 2^-126 are 2^-133 apart, whose half is added."""
    T, Hq, D = q.shape
    G = Hq // k.shape[1]
    o = torch.zeros(T, Hq, D, dtype=torch.float64)
    e = torch.zeros_like(o)
    for r0, r1 in zip(starts, starts[1:]):
        at = torch.arange(r1 - r0) if rows is None else rows[rows < r1 - r0]
        if not len(at):
            continue
        vis = torch.arange(int(at.max()) + 1)[None, :] <= at[:, None]
        end = r0 + vis.shape[1]
        for h in range(Hq) if heads is None else heads:
            vv = v[r0:end, h // G].double()
            oo, ee = ref.rows_attention(q[r0 + at, h].double(), k[r0:end, h // G].double(), vv, vis,
                                        sm, ref.FP16, 0.0)
            o[r0 + at, h], e[r0 + at, h] = oo, (
                ee + 2.0 ** -32 * float(vv.abs().max()) + 2.0 ** -134)
    return o, e
