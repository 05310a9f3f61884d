"""Cases of the operators around a block's linears, their plain forms and their
definitions in 64 bits.

Operators ("op" of a case):
  norm    root-mean-square norm of the residual stream, with the residual's
          addition in front of it; its output bf16 rows, or the next linear's
          packed codes (8 bits, or 4 bits in the E2M3 container) with step sizes
          from a table or one a row, read back as the values they stand for
  rotary  rotary positions on a QKV output's query and key heads: both layouts,
          a part of the head, frequencies scaled for long contexts
  prompt  causal attention of whole prompts packed one behind the other,
          grouped heads, bf16 keys and values

`own` False: elementary torch operations in 32 bits (64 for the norm's mean
square and the angles).  `own` True: the calls a user's program makes.
"""
import math

import torch

own = False

EPS = 1e-6


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one token between two linears of a hidden-4096 block, bf16 rows for the few-row products
        dict(name="norm_token_1x4096", op="norm", M=1, K=4096, out="bf16", add=True),
        # the proprio and action tokens of a hidden-4096 step and some more, a step size a row
        dict(name="norm_actions_201x4096_row8", op="norm", M=201, K=4096, out="row8", add=True),
        # the first norm of a hidden-2048 block on two rollouts: W4A8 codes, table step sizes
        dict(name="norm_frame_8384x2048_int8", op="norm", M=8384, K=2048, out="int8", add=False),
        # the norm in front of a hidden-4096 backbone's W4A4 up projection
        dict(name="norm_backbone_16576x4096_e2m3", op="norm", M=16576, K=4096, out="e2m3",
             add=True),
        # one new token of each of 48 rollouts, far into a context stretched eightfold
        dict(name="rotary_48_tokens_far", op="rotary", B=48, rows=1, pos=120000, Hq=32, Hkv=8,
             D=128, part=128, layout="half", scaling="parts"),
        # a frame (video, proprio and action tokens) of two rollouts
        dict(name="rotary_frame_2x4192", op="rotary", B=2, rows=4192, pos=1000, Hq=16, Hkv=16,
             D=128, part=128, layout="half", scaling="plain"),
        # ragged prompts, small heads of which half is rotated, pairs side by side
        dict(name="rotary_prompts_3x9001_part", op="rotary", B=3, rows=9001, pos=0, Hq=24, Hkv=8,
             D=64, part=32, layout="pairs", scaling="base"),
        # an instruction on its own: latency
        dict(name="prompt_instruction_1x77", op="prompt", B=1, rows=77, Hq=16, Hkv=16, D=128),
        # ragged prompts, small heads, grouped
        dict(name="prompt_ragged_3x1500_d64", op="prompt", B=3, rows=1500, Hq=24, Hkv=8, D=64),
        # a batch of prompts, from short ones to 4801 tokens, four query heads to a key head
        dict(name="prompt_ragged_12x4801", op="prompt", B=12, rows=4801, Hq=32, Hkv=8, D=128),
        # the tokens of two rollouts' frames, each token seeing those in front of it
        dict(name="prompt_frame_2x4192", op="prompt", B=2, rows=4192, Hq=16, Hkv=16, D=128),
        # one long prompt: the backbone's 16576 tokens
        dict(name="prompt_long_1x16576", op="prompt", B=1, rows=16576, Hq=32, Hkv=8, D=128),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "rotary", "rotary", "prompt", "prompt"])
    if op == "norm":
        out = rng.choice(["bf16", "row8", "int8", "e2m3", "int4"])
        K = 64 * _log_int(rng, 2, 128)                 # 128 .. 8192 channels
        return dict(op=op, M=_log_int(rng, 1, 60_000_000 // K if K > 3500 else 16576), K=K,
                    out=out, add=rng.random() < 0.6)
    D, Hkv = rng.choice([64, 128]), rng.choice([1, 2, 8, 16])
    Hq = Hkv * rng.choice([1, 1, 3, 4])
    if op == "rotary":
        rows = 1 if rng.random() < 0.3 else _log_int(rng, 2, 9001)
        return dict(op=op, B=_log_int(rng, 1, max(1, min(64, 16000 // rows))), rows=rows,
                    pos=_log_int(rng, 1, 1_000_000), Hq=Hq, Hkv=Hkv, D=D,
                    part=rng.choice([16, D // 2, D - 16, D, D]),
                    layout=rng.choice(["half", "pairs"]),
                    scaling=rng.choice(["plain", "linear", "base", "parts"]))
    rows = _log_int(rng, 1, 6000)
    return dict(op=op, B=_log_int(rng, 1, max(1, min(32, 12000 // rows))), rows=rows, Hq=Hq,
                Hkv=Hkv, D=D)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _counts(case):
    """Row counts of a case's sequences, the longest `rows`: its own, whatever the seed, so that
    outputs keep their shapes.  Frames of rollouts and single tokens have the same count each."""
    B, rows = case["B"], case["rows"]
    if rows in (1, 4192):
        return torch.full((B,), rows, dtype=torch.int64)
    g = torch.Generator().manual_seed(rows * 1009 + B)
    n = torch.clamp((rows * torch.rand(B, generator=g)).long(), min=1)
    n[B // 2] = rows
    return n


def _frequencies(case):
    """Radians a position of each pair of channels (fp64) and the factor on cosines and sines."""
    n = case["part"]
    i = torch.arange(n // 2, dtype=torch.float64)
    base, factor, trained = 10000.0, 8.0, 16384.0
    kind = case["scaling"]
    if kind == "base" and n > 2:
        base *= factor ** (n / (n - 2))
    f = base ** (-2 * i / n)
    if kind == "linear":
        f = f / factor
    if kind != "parts":
        return f, 1.0
    # turns over the trained length: below 1 a pair is stretched, above 32 it is left
    keep = ((trained * f / (2 * math.pi) - 1.0) / (32.0 - 1.0)).clamp(0, 1)
    return f / factor * (1 - keep) + f * keep, 0.1 * math.log(factor) + 1.0


_CODES = {"row8": (8, 0), "int8": (8, 0), "int4": (4, 0), "e2m3": (4, 1)}   # bits, container


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    gh = torch.Generator().manual_seed(seed)
    st = dict(case)
    if own:
        from w4a4_quantized_gemm_rudder_amd import rudder
        st["rudder"] = rudder
    if case["op"] == "norm":
        M, K, S = case["M"], case["K"], 3
        bf16 = torch.bfloat16
        x = torch.randn(M, K, generator=g, device="cuda", dtype=bf16)
        hot = torch.randperm(K, generator=gh)[: max(1, K // 100)].cuda()
        x[:, hot] *= 30.0                              # outlier channels
        st["x"] = x
        st["r"] = None
        if case["add"]:
            st["r"] = torch.randn(M, K, generator=g, device="cuda", dtype=bf16) * 2
        st["gamma"] = 0.8 + 0.4 * torch.rand(K, generator=g, device="cuda")
        st["sid"] = torch.randint(0, S, (M,), generator=g, device="cuda").to(torch.uint8)
        smooth = 0.7 + 0.6 * torch.rand(K, generator=g, device="cuda")
        smooth[hot] *= 5.0
        st["inv_smooth"] = (1 / smooth.double()).float()
        if case["out"] != "bf16":
            st["bits"], st["codes"] = _CODES[case["out"]]
            top = 3.0 if st["bits"] == 8 else 2.0
            st["table"] = None if case["out"] == "row8" else (
                top * (0.8 + 0.4 * torch.rand(S, generator=g, device="cuda"))
                / (127 if st["bits"] == 8 else 7))
        if own:
            st["h"] = torch.empty_like(x) if case["add"] else None
            if case["out"] == "bf16":
                st["y"] = torch.empty_like(x)
            else:
                n = st["rudder"].packed_act_bytes(M, K, st["bits"], st["codes"])
                st["q"] = torch.empty(n, dtype=torch.uint8, device="cuda")
                st["scale"] = torch.empty(M, device="cuda")
                st["values"] = torch.empty(M, K, device="cuda")
        return st
    B, Hq, Hkv, D = (case[k] for k in ("B", "Hq", "Hkv", "D"))
    n_rows = _counts(case)
    start = torch.zeros(B + 1, dtype=torch.int64)
    start[1:] = torch.cumsum(n_rows, 0)
    T = st["T"] = int(start[-1])
    st["row_start"] = start.to(torch.int32).cuda()
    # a QKV projection's output; its three parts are used as they lie
    qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=g, device="cuda", dtype=torch.bfloat16)
    st["q"], st["k"], st["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    if case["op"] == "rotary":
        f, st["magnitude"] = _frequencies(case)
        st["freq"] = f.cuda()
        far = torch.randint(0, max(1, case["pos"]) // 2 + 1, (B,), generator=gh)
        st["pos"] = (case["pos"] - far).to(torch.int32).cuda()
        if own:
            st["kind"] = {"half": st["rudder"].ROTARY_HALF,
                          "pairs": st["rudder"].ROTARY_PAIRS}[case["layout"]]
            st["qo"] = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
            st["ko"] = torch.empty(T, Hkv, D, dtype=torch.bfloat16, device="cuda")
        return st
    st["q"].mul_(1.5)
    st["sm"] = 1.0 / math.sqrt(D)
    if own:
        r, rows = st["rudder"], case["rows"]
        st["o"] = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
        st["ws"] = torch.empty(r.prompt_attention_workspace_bytes(B, T, rows, Hq, Hkv, D),
                               dtype=torch.uint8, device="cuda")
    return st


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(st):
    op = st["op"]
    if own:
        return _OWN[op](st)
    return _PLAIN[op](st)


def _own_norm(st):
    r, M, K = st["rudder"], st["M"], st["K"]
    if st["out"] == "bf16":
        r.rudder_norm(st["x"], st["r"], st["gamma"], EPS, M, K, st["h"], st["y"])
        out = {"y": st["y"]}
    else:
        r.rudder_norm_quant(st["x"], st["r"], st["sid"], st["gamma"], st["inv_smooth"],
                            st["table"], EPS, M, K, 3, st["bits"], st["codes"], st["h"], st["q"],
                            st["scale"])
        r.rudder_dequant_act(st["q"], st["scale"], M, K, st["bits"], st["codes"], st["values"])
        out = {"values": st["values"], "scale": st["scale"]}
    return {**out, "h": st["h"]} if st["add"] else out


def _own_rotary(st):
    st["rudder"].rudder_rotary(
        st["q"], st["k"], st["row_start"], st["pos"], st["freq"], st["magnitude"], st["B"],
        st["T"], st["rows"], st["Hq"], st["Hkv"], st["D"], st["part"], st["kind"], st["qo"],
        st["ko"])
    return {"q": st["qo"], "k": st["ko"]}


def _own_prompt(st):
    st["rudder"].rudder_prompt_attention(
        st["q"], st["k"], st["v"], st["row_start"], st["B"], st["T"], st["rows"], st["Hq"],
        st["Hkv"], st["D"], st["sm"], st["ws"], st["o"])
    return st["o"]


def _plain_norm(st):
    h = st["x"]
    if st["add"]:
        h = (st["r"].float() + h.float()).to(torch.bfloat16)
    x = h.float()
    mean = x.double().square().sum(-1, keepdim=True) / st["K"]
    y = (x * (1 / torch.sqrt(mean + EPS)).float()) * st["gamma"]
    y = y.to(torch.bfloat16)
    if st["out"] == "bf16":
        out = {"y": y}
    else:
        most = 127 if st["bits"] == 8 else 7
        u = y.float() * st["inv_smooth"]
        if st["table"] is None:
            scale = (u.abs().amax(1).double() / most).float()
        else:
            scale = st["table"][st["sid"].long()]
        inv = torch.where(scale > 0, 1 / scale.double(), 0.0).float()
        q = torch.round(torch.clamp(u * inv[:, None], -most, most))
        out = {"values": q * scale[:, None], "scale": scale}
    return {**out, "h": h} if st["add"] else out


def _positions(st):
    """Position of every row, int64 [T]."""
    i = torch.arange(st["T"], device="cuda")
    start = st["row_start"].long()
    b = torch.searchsorted(start, i, right=True) - 1
    return st["pos"].long()[b] + i - start[b]


def _pairs(x, n, layout):
    """The two halves of the rotated part of x [..., D]."""
    if layout == "half":
        return x[..., :n // 2], x[..., n // 2:n]
    return x[..., 0:n:2], x[..., 1:n:2]


def _rotate(x, cos, sin, n, layout):
    a, b = _pairs(x, n, layout)
    c, d = a * cos - b * sin, b * cos + a * sin
    turned = torch.cat([c, d], -1) if layout == "half" else torch.stack([c, d], -1).flatten(-2)
    return torch.cat([turned, x[..., n:]], -1)


def _plain_rotary(st):
    angle = _positions(st).double()[:, None, None] * st["freq"]
    cos = (torch.cos(angle) * st["magnitude"]).float()
    sin = (torch.sin(angle) * st["magnitude"]).float()
    n, layout = st["part"], st["layout"]
    return {"q": _rotate(st["q"].float(), cos, sin, n, layout).to(torch.bfloat16),
            "k": _rotate(st["k"].float(), cos, sin, n, layout).to(torch.bfloat16)}


def _plain_prompt(st):
    """Sequences padded to the longest; keys behind a row are masked, so no other mask is needed."""
    B, rows, Hq, Hkv, D = (st[n] for n in ("B", "rows", "Hq", "Hkv", "D"))
    start = st["row_start"].long()
    i = torch.arange(rows, device="cuda")
    have = i[None, :] < (start[1:] - start[:-1])[:, None]
    row = torch.where(have, start[:-1, None] + i[None, :], 0)
    q = st["q"][row].float().view(B, rows, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4)
    q = q.reshape(B, Hkv, -1, D)
    k = st["k"][row].float().permute(0, 2, 3, 1).contiguous()
    v = st["v"][row].float().transpose(1, 2).contiguous()
    s = (q @ k).view(B, Hq, rows, rows)
    s *= st["sm"]
    s.masked_fill_(i[None, :] > i[:, None], -math.inf)
    s.sub_(s.amax(-1, keepdim=True)).exp_()
    total = s.sum(-1, keepdim=True)
    o = (s.view(B, Hkv, -1, rows) @ v).view(B, Hq, rows, D)
    return (o / total).permute(0, 2, 1, 3)[have].to(torch.bfloat16)


_OWN = {"norm": _own_norm, "rotary": _own_rotary, "prompt": _own_prompt}
_PLAIN = {"norm": _plain_norm, "rotary": _plain_rotary, "prompt": _plain_prompt}


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    if case["op"] == "norm":
        M, K, out = case["M"], case["K"], case["out"]
        size = 6 if case["add"] else 2                 # x, and r and h
        # bf16 rows; or codes, and the values read back
        size += {"bf16": 2, "row8": 5, "int8": 5, "int4": 4.5, "e2m3": 4.75}[out]
        rest = 4 * K if out == "bf16" else 8 * K + 5 * M
        return {"bytes": size * M * K + rest, "flops": (6 if out == "bf16" else 10) * M * K}
    n = _counts(case)
    T, Hq, Hkv, D = int(n.sum()), case["Hq"], case["Hkv"], case["D"]
    if case["op"] == "rotary":
        return {"bytes": 4 * T * (Hq + Hkv) * D, "flops": 3 * T * (Hq + Hkv) * case["part"]}
    return {"bytes": 4 * T * (Hq + Hkv) * D, "flops": 4 * D * Hq * int((n * (n + 1) // 2).sum())}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    return {"norm": _exact_norm, "rotary": _exact_rotary, "prompt": _exact_prompt}[case["op"]](st)


def _exact_norm(st):
    """bf16 rows in 64 bits.  Codes are decided in 32 bits by definition (1 / sqrt is formed in 64
    bits and rounded, each product rounded, the rows rounded to bf16 before the quantizer)."""
    h = st["x"].double()
    if st["add"]:
        h = (st["r"].double() + h).to(torch.bfloat16).double()
    k = (h * h).mean(1, keepdim=True).add(float(EPS)).rsqrt()
    out = {"h": h} if st["add"] else {}
    if st["out"] == "bf16":
        return {**out, "y": h * k * st["gamma"].double()}
    most = 2.0 ** (st["bits"] - 1) - 1
    y = ((h * k.float().double()).float().double() * st["gamma"].double()).float()
    u = (y.to(torch.bfloat16).double() * st["inv_smooth"].double()).float().double()
    if st["table"] is None:
        scale = (u.abs().amax(1) / most).float().double()
    else:
        scale = st["table"].double().index_select(0, st["sid"].int())
    inv = torch.where(scale > 0, scale.reciprocal(), torch.zeros_like(scale)).float().double()
    q = (u * inv[:, None]).float().double().clamp(-most, most).round()
    return {**out, "values": q * scale[:, None], "scale": scale}


def _exact_rotary(st):
    """As a product of complex numbers, sequence by sequence."""
    start, n = st["row_start"].tolist(), st["part"]
    out = {"q": st["q"].double().clone(), "k": st["k"].double().clone()}
    for b, p in enumerate(st["pos"].tolist()):
        at = torch.arange(p, p + start[b + 1] - start[b], dtype=torch.float64, device="cuda")
        angle = torch.outer(at, st["freq"])[:, None]
        turn = torch.polar(torch.full_like(angle, st["magnitude"]), angle)
        for name in ("q", "k"):
            x = out[name][start[b]:start[b + 1], :, :n]
            re = slice(0, n // 2) if st["layout"] == "half" else slice(0, n, 2)
            im = slice(n // 2, n) if st["layout"] == "half" else slice(1, n, 2)
            z = torch.complex(x[..., re].contiguous(), x[..., im].contiguous()) * turn
            x[..., re], x[..., im] = z.real, z.imag
    return out


def _exact_prompt(st):
    """Sequence by sequence, some heads' rows at a time."""
    H, G, D = st["Hkv"], st["Hq"] // st["Hkv"], st["D"]
    start = st["row_start"].tolist()
    o = torch.zeros(st["T"], st["Hq"], D, dtype=torch.float64, device="cuda")
    for r0, r1 in zip(start, start[1:]):
        for h in range(H):
            k, v = (st[x][r0:r1, h].double().contiguous() for x in ("k", "v"))
            kt = k.t().contiguous()
            for a in range(r0, r1, 4096):
                e = min(a + 4096, r1)
                i = torch.arange(a - r0, e - r0, device="cuda")[:, None]
                hidden = torch.arange(e - r0, device="cuda")[None, :] > i
                for g in range(G):
                    s = st["q"][a:e, h * G + g].double() @ kt[:, :e - r0] * st["sm"]
                    s = s.masked_fill(hidden, -math.inf)
                    o[a:e, h * G + g] = torch.softmax(s, -1) @ v[:e - r0]
    return o
