"""Plain 64-bit forms of the group-scaled few-row product, the 8-bit cache and
the two attention calls, and the bounds their kernels are held to.  On the
CPU, sequence by sequence, from the definitions in the headers."""
import math

import torch

PAGE = 64
BF16, FP16, FP32 = 2.0 ** -8, 2.0 ** -11, 2.0 ** -24      # half a step, relative


def f32(x):
    return x.to(torch.float32)


def recip(s):
    """fl32(1 / s), 0 for 0."""
    d = s.double()
    return f32(torch.where(d > 0, 1 / torch.where(d > 0, d, 1.0), 0.0))


# --- group-scaled weights -------------------------------------------------

def group_codes(W, group):
    """Codes int8 [K, N] and bf16 scales [K / group, N]."""
    K, N = W.shape
    w = f32(W).view(K // group, group, N)
    s = f32(w.abs().amax(1).double() / 7).to(torch.bfloat16)
    q = torch.round(torch.clamp(w * recip(s)[:, None], -7, 7))
    return q.to(torch.int8).view(K, N), s


def pack_grouped(q, s):
    """Codes and scales in the library's layout (uint8 tensor, bf16 in tile order)."""
    K, N = q.shape
    Kp, Np = (K + 127) // 128 * 128, (N + 15) // 16 * 16
    full = torch.zeros(Kp, Np, dtype=torch.int64)
    full[:K, :N] = q
    out = torch.zeros(Kp * Np // 2, dtype=torch.uint8).numpy()
    nib = (full + 8).numpy()
    for k in range(Kp):
        word = (k % 128) // 32
        shift = (k % 8) // 2 + 4 * (k % 2)
        for n in range(Np):
            tile = (n // 16) * (Kp // 128) + k // 128
            lane = n % 16 + 16 * ((k % 32) // 8)
            at = tile * 1024 + 16 * lane + 4 * word + shift // 2
            out[at] |= int(nib[k, n]) << (4 * (shift % 2))
    group = K // s.shape[0]
    sp = torch.zeros(Kp // group, Np, dtype=torch.bfloat16)
    sp[:s.shape[0], :N] = s
    # [k tile, group of the tile, n tile, n / 4, n % 4] -> [n tile, k tile, n / 4, group, n % 4]
    sp = sp.view(Kp // 128, 128 // group, Np // 16, 4, 4).permute(2, 0, 3, 1, 4)
    return torch.from_numpy(out), sp.reshape(-1)


def matvec(x, q, s, group, sid=None, a=None, b=None):
    """Y in 64 bits, and the bound on a kernel's distance from it.

    Sums of one group: (24 + q) * x and x, each at most 31 * sum |x| large, counted here as 143 (a
    wider offset's), and of `group` fp32 additions, their difference one more rounding; then K / group fused additions; the
    compensation's fma; the rounding to bf16."""
    x, q, s = x.double(), q.double(), s.double()
    K, N = q.shape
    w = q * s.repeat_interleave(group, 0)
    t = x @ w
    ax = x.abs().view(len(x), K // group, group).sum(2)
    e = 2 * (group + 4) * 143 * FP32 * (ax @ s) + (K // group + 4) * FP32 * (x.abs() @ w.abs())
    y = t
    if a is not None:
        a, b = a.double()[sid.long()], b.double()[sid.long()]
        y = a * t + b
        e = a.abs() * e + 2 * FP32 * (a * t).abs() + 2 * FP32 * b.abs()
    return y, e + BF16 * (y.abs() + e)


# --- the cache -------------------------------------------------------------

def append(K, V, row_start, pos, table, codes, scales):
    """The append rule, token by token from its definition; codes [P, H, 2, 64 D] int8 and
    scales [P, H, 2] are changed in place."""
    P, H = codes.shape[:2]
    D = codes.shape[3] // PAGE
    for b in range(len(pos)):
        r0, r1, p0 = int(row_start[b]), int(row_start[b + 1]), int(pos[b])
        i = 0
        while i < r1 - r0:
            no, slot = (p0 + i) // PAGE, (p0 + i) % PAGE
            n = min(PAGE - slot, r1 - r0 - i)
            page = int(table[b, no]) if no < table.shape[1] else -1
            if 0 <= page < P:
                for h in range(H):
                    for half, X in ((0, K), (1, V)):
                        x = f32(X[r0 + i:r0 + i + n, h])
                        had = scales[page, h, half].clone() if slot else torch.tensor(0.0)
                        s = torch.maximum(had, f32(x.abs().max().double() / 127))
                        c = codes[page, h, half]
                        c = c.view(PAGE, D) if half == 0 else c.view(D, PAGE).t()
                        if slot and s > had:
                            ratio = f32(had.double() / s.double())
                            c[:slot] = torch.round(f32(c[:slot]) * ratio).to(torch.int8)
                        q = torch.round(torch.clamp(x * recip(s), -127, 127))
                        c[slot:slot + n] = q.to(torch.int8)
                        scales[page, h, half] = s
            i += n


def values(codes, scales, pages):
    """K and V of whole pages, 64 bits [n, H, 64, D]."""
    P, H = codes.shape[:2]
    D = codes.shape[3] // PAGE
    c, s = codes[pages.long()].double(), scales[pages.long()].double()
    k = c[:, :, 0].reshape(-1, H, PAGE, D) * s[:, :, 0, None, None]
    v = c[:, :, 1].reshape(-1, H, D, PAGE).transpose(2, 3) * s[:, :, 1, None, None]
    return k, v


# --- attention -------------------------------------------------------------

def rows_attention(q, k, v, visible, sm, p_half_step, q_step):
    """q [n, D], k, v [kv, D] in 64 bits, visible [n, kv]: (o, bound).

    With A = sum p |v|: the weights' rounding (p_half_step), the two rounded sums over the keys
    ((kv + 70) additions or rescalings of 32 bits each) and the weights' relative error from an
    error dz of the exponent, in numerator and denominator: 2 ln 2 dz.  dz: the fp32 product
    of D terms and its scaling, (D + 8) half steps of c sum |q k|; q's own rounding (q_step of the
    row's largest element, for the cache half a unit 2^-14 of the largest power of
    two in the row, or one unit for the largest itself: 2^-15); three roundings at the exponent's
    own magnitude and that of log2 of a scale (80 at most).  Then the absolute floor of weights
    held in fp16 (2^-33 of the largest a key), and the rounding to bf16."""
    if not len(k):
        z = torch.zeros(len(q), v.shape[1], dtype=torch.float64)
        return z, z
    c = sm / math.log(2)
    s = q @ k.t() * sm
    s = s.masked_fill(~visible, -math.inf)
    m = s.amax(1, keepdim=True)
    p = torch.exp(s - torch.where(m > -math.inf, m, 0.0))
    total = p.sum(1, keepdim=True)
    p = torch.where(total > 0, p / torch.where(total > 0, total, 1.0), 0.0)
    o = p @ v
    kv, D = k.shape
    ak = k.abs().amax(0).sum()                           # at least sum |k| of any one key
    zmax = (q.abs() @ k.abs().t()).amax(1, keepdim=True) * abs(c)
    dz = zmax * (D + 8) * FP32 + abs(c) * q.abs().amax(1, keepdim=True) * ak * q_step
    dz = dz + 3 * FP32 * (2 * zmax + 80) + 4 * FP32
    A = p @ v.abs()
    e = A * (p_half_step + 2 * math.log(2) * dz + 2 * (kv + 70) * FP32)
    e = e + kv * 2.0 ** -33 * v.abs().max()
    return o, e + BF16 * (o.abs() + e)


def visible(n, kv, causal):
    j = torch.arange(kv)[None, :]
    i = torch.arange(n)[:, None]
    return (j <= kv - n + i) if causal else torch.ones(n, kv, dtype=torch.bool)


def cache_attention(q, row_start, kv_len, table, codes, scales, sm, causal, heads=None):
    """O and bound [T, Hq, D] in 64 bits (zeros in rows of no sequence); pages outside the pool
    are not visible.  `heads`: those that are computed, all by default."""
    T, Hq, D = q.shape
    P, H = codes.shape[:2]
    o = torch.zeros(T, Hq, D, dtype=torch.float64)
    e = torch.zeros_like(o)
    for b in range(len(kv_len)):
        r0, r1 = int(row_start[b]), int(row_start[b + 1])
        kv = min(int(kv_len[b]), table.shape[1] * PAGE)
        pages = table[b, :(kv + PAGE - 1) // PAGE]
        good = (pages >= 0) & (pages < P)
        k, v = values(codes, scales, torch.where(good, pages, 0))
        there = good.repeat_interleave(PAGE)[:kv]
        vis = visible(r1 - r0, kv, causal) & there[None, :]
        for h in range(Hq) if heads is None else heads:
            g = h // (Hq // H)
            kk = torch.where(there[:, None], k[:, g].reshape(-1, D)[:kv], 0.0)
            vv = torch.where(there[:, None], v[:, g].reshape(-1, D)[:kv], 0.0)
            o[r0:r1, h], e[r0:r1, h] = rows_attention(q[r0:r1, h].double(), kk, vv, vis, sm, FP16,
                                                          2.0 ** -15)
    return o, e


def cross_attention(q, k, v, row_start, kv_start, kv_len, sm, heads=None):
    T, Hq, D = q.shape
    H = k.shape[1]
    o = torch.zeros(T, Hq, D, dtype=torch.float64)
    e = torch.zeros_like(o)
    for b in range(len(kv_len)):
        r0, r1 = int(row_start[b]), int(row_start[b + 1])
        k0, n = int(kv_start[b]), int(kv_len[b])
        vis = torch.ones(r1 - r0, n, dtype=torch.bool)
        for h in range(Hq) if heads is None else heads:
            g = h // (Hq // H)
            o[r0:r1, h], e[r0:r1, h] = rows_attention(
                q[r0:r1, h].double(), k[k0:k0 + n, g].double(), v[k0:k0 + n, g].double(), vis, sm,
                BF16, 0.0)
    return o, e


def assert_within(name, got, want, bound):
    got = got.double().cpu()
    assert torch.isfinite(got).all(), f"{name}: {int((~torch.isfinite(got)).sum())} not finite"
    over = (got - want).abs() - bound
    worst = float(over.max()) if over.numel() else 0.0
    at = int(over.reshape(-1).argmax()) if over.numel() else 0
    assert worst <= 0, (f"{name}: {int((over > 0).sum())} of {over.numel()} outside the bound, "
                        f"worst at {at}: got {float(got.reshape(-1)[at])}, want "
                        f"{float(want.reshape(-1)[at])}, bound {float(bound.reshape(-1)[at])}")
