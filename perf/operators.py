"""Cases of the attention and few-row operators, their plain forms and their
definitions in 64 bits.

Operators ("op" of a case):
  matvec  few rows times 4-bit weights with one scale per group of input
          channels and output channel, with the per-stream compensation
  append  new keys and values quantized into the paged 8-bit cache (64 tokens
          a page, one scale per page, head and K|V), and the touched pages
          read back as values
  cache   attention over that cache, bidirectional or causal, grouped heads
  cross   attention of a block's tokens to an encoder's states (bf16)

`own` False: elementary torch operations in 32 bits.  `own` True: the calls a
user's program makes.
"""
import math

import torch

own = False

PAGE = 64


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one token through the attention output projection of a hidden-2048 block
        dict(name="matvec_o_1x2048x2048", op="matvec", M=1, K=2048, N=2048, group=128, comp=True),
        # one token through the QKV projection of a hidden-4096 block
        dict(name="matvec_qkv_1x4096x12288", op="matvec", M=1, K=4096, N=12288, group=64,
             comp=True),
        # the MLP down projection for 13 action tokens decoded together, fine groups
        dict(name="matvec_down_13x16384x4096", op="matvec", M=13, K=16384, N=4096, group=32,
             comp=False),
        # one new token of each of 48 rollouts written to the cache
        dict(name="append_48_tokens", op="append", B=48, rows=1, ctx=4096, Hq=32, Hkv=8, D=128),
        # a whole frame (video, proprio and action tokens) of two rollouts, from the QKV output
        dict(name="append_frame_2x4192", op="append", B=2, rows=4192, ctx=1000, Hq=16, Hkv=16,
             D=128),
        # one rollout, one token, a short context: latency
        dict(name="cache_token_ctx777", op="cache", B=1, rows=1, ctx=777, Hq=16, Hkv=16, D=128,
             causal=True),
        # 48 rollouts, one token each, ragged contexts, four query heads to a cached head
        dict(name="cache_48_tokens_ctx8192", op="cache", B=48, rows=1, ctx=8192, Hq=32, Hkv=8,
             D=128, causal=True),
        # the 96 proprio and action tokens of a denoising step against eight cached frames
        dict(name="cache_actions_2x96_ctx33536", op="cache", B=2, rows=96, ctx=33536, Hq=16,
             Hkv=16, D=128, causal=False),
        # ragged prompts prefilled causally, small heads, grouped
        dict(name="cache_prefill_3x1500_d64", op="cache", B=3, rows=1500, ctx=1700, Hq=24, Hkv=8,
             D=64, causal=True),
        # a whole frame of two rollouts against three cached frames, all of it visible
        dict(name="cache_frame_2x4192_ctx12576", op="cache", B=2, rows=4192, ctx=12576, Hq=16,
             Hkv=16, D=128, causal=False),
        # the action tokens' cross attention to a short instruction
        dict(name="cross_96_len77", op="cross", B=1, rows=96, ctx=77, Hq=16, Hkv=16, D=128),
        # a block's cross attention: two rollouts of 4192 tokens, encoder states up to 512 long
        dict(name="cross_2x4192_len512", op="cross", B=2, rows=4192, ctx=512, Hq=16, Hkv=16,
             D=128),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["matvec", "append", "cache", "cache", "cross"])
    if op == "matvec":
        group = rng.choice([32, 64, 128])
        K = group * max(1, _log_int(rng, 256, 16384) // group)
        return dict(op=op, M=_log_int(rng, 1, 16), K=K, N=_log_int(rng, 64, 12288), group=group,
                    comp=rng.random() < 0.5)
    D, Hkv = rng.choice([64, 128]), rng.choice([1, 4, 8, 16])
    Hq = Hkv * rng.choice([1, 1, 3, 4])
    if op == "append":
        rows = 1 if rng.random() < 0.4 else _log_int(rng, 2, 3000)
        B = _log_int(rng, 1, max(1, min(48, 6000 // rows)))
        return dict(op=op, B=B, rows=rows, ctx=_log_int(rng, 1, 4096), Hq=Hq, Hkv=Hkv, D=D)
    if op == "cross":
        rows = 1 if rng.random() < 0.3 else _log_int(rng, 2, 4192)
        return dict(op=op, B=_log_int(rng, 1, 2 if rows > 500 else 16), rows=rows,
                    ctx=_log_int(rng, 1, 1024), Hq=Hq, Hkv=Hkv, D=D)
    kind = rng.choice(["token", "token", "few", "chunk"])
    if kind == "token":
        return dict(op=op, B=_log_int(rng, 1, 48), rows=1, ctx=_log_int(rng, 16, 8192), Hq=Hq,
                    Hkv=Hkv, D=D, causal=True)
    rows = _log_int(rng, 2, 200) if kind == "few" else _log_int(rng, 200, 2000)
    return dict(op=op, B=rng.choice([1, 2, 3]), rows=rows, ctx=rows + _log_int(rng, 16, 8192),
                Hq=Hq, Hkv=Hkv, D=D, causal=rng.random() < 0.5)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _spread(g, n, most, fixed):
    """n lengths up to `most`: all of them `fixed`, or ragged with the longest at `most`."""
    if fixed:
        return torch.full((n,), most, dtype=torch.int64)
    r = torch.rand(n, generator=g)
    v = torch.clamp((most * (0.3 + 0.7 * r)).long(), min=1)
    v[0] = most
    return v


def _rows(case):
    """Row counts of the sequences, the contexts' lengths before an append and the generator of
    further lengths: a case's own, whatever the seed, so that its outputs keep their shapes."""
    B, rows, ctx = case["B"], case["rows"], case["ctx"]
    g = torch.Generator().manual_seed(rows * 1009 + ctx)
    n_rows = _spread(g, B, rows, rows == 1 or not case.get("causal", False))
    return n_rows, ctx + torch.randint(0, PAGE, (B,), generator=g), g


def _lengths(case, n_rows, g):
    """Key lengths of an attention case."""
    cache = case["op"] == "cache"
    lens = _spread(g, case["B"], case["ctx"], cache and case["rows"] > 1 and not case["causal"])
    return torch.maximum(lens, n_rows) if cache else lens


def _layout(rows):
    """Row counts -> (row_start int32 [B+1] on the GPU, total rows)."""
    start = torch.zeros(len(rows) + 1, dtype=torch.int64)
    start[1:] = torch.cumsum(rows, 0)
    return start.to(torch.int32).cuda(), int(start[-1])


def _pool(g, gh, lens, Hkv, D):
    """A cache pool holding `lens` tokens per sequence in shuffled pages, and some pages more.
    K codes are [page, head, token, channel], V codes [page, head, channel, token]."""
    B = len(lens)
    need = (lens + PAGE - 1) // PAGE
    width = max(1, int(need.max()))
    total = int(need.sum())
    num_pages = total + 3
    order = torch.randperm(num_pages, generator=gh)[:total].to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32)
    table[torch.arange(width)[None, :] < need[:, None]] = order
    codes = torch.empty(num_pages, Hkv, 2, PAGE * D, dtype=torch.int8, device="cuda")
    x = torch.randn(num_pages, Hkv, 2, PAGE * D, generator=g, device="cuda",
                    dtype=torch.bfloat16)
    x *= 0.5 + torch.rand(num_pages, Hkv, 2, 1, generator=g, device="cuda").to(torch.bfloat16)
    scales = (x.abs().amax(-1).float().double() / 127).float()
    codes.copy_(torch.round(x.float() * (1 / scales.double()).float()[..., None])
                .clamp_(-127, 127))
    return codes, scales, table.cuda(), num_pages, width


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    gh = torch.Generator().manual_seed(seed)
    st = dict(case)
    op = case["op"]
    if op == "matvec":
        M, K, N, S = case["M"], case["K"], case["N"], 3
        x = torch.randn(M, K, generator=g, device="cuda")
        hot = torch.randperm(K, generator=gh)[: max(1, K // 100)]
        x[:, hot.cuda()] *= 30.0                       # outlier channels
        W = (torch.randn(K, N, generator=g, device="cuda") * 0.02).to(torch.bfloat16)
        st["x"] = x.to(torch.bfloat16)
        st["sid"] = torch.randint(0, S, (M,), generator=g, device="cuda").to(torch.uint8)
        st["a"] = torch.rand(S, N, generator=g, device="cuda") * 0.2 + 0.9
        st["b"] = torch.randn(S, N, generator=g, device="cuda") * 0.01
        if own:
            from w4a4_quantized_gemm_rudder_amd import rudder
            st["rudder"] = rudder
            st["Wq"], st["ws"] = rudder.quantize_weights_grouped(W, case["group"])
            st["y"] = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
        else:
            st["q"], st["s"] = _group_codes(W, case["group"])
        return st
    B, rows, ctx, Hkv, D = (case[k] for k in ("B", "rows", "ctx", "Hkv", "D"))
    n_rows, pos, gl = _rows(case)
    if op == "append":
        # contexts of `ctx` tokens and some, the last page of most of them begun
        lens = pos + n_rows
        first, last = pos // PAGE, (lens - 1) // PAGE
        st["codes"], st["scales"], st["table"], st["num_pages"], st["width"] = _pool(
            g, gh, lens, Hkv, D)
        st["pos"] = pos.to(torch.int32).cuda()
        n = (last - first + 1)
        at = torch.arange(int(n.max()))
        inside = at[None, :] < n[:, None]
        st["page_seq"] = torch.arange(B)[:, None].expand_as(inside)[inside].cuda()
        st["page_no"] = (first[:, None] + at[None, :])[inside].cuda()
        st["pages"] = st["table"][st["page_seq"], st["page_no"]].contiguous()
        st["row_start"], T = _layout(n_rows)
        Hq = case["Hq"]
        qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=g, device="cuda").to(torch.bfloat16)
        st["k"], st["v"] = qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    else:
        Hq = case["Hq"]
        st["row_start"], T = _layout(n_rows)
        lens = _lengths(case, n_rows, gl)
        if op == "cache":
            st["codes"], st["scales"], st["table"], st["num_pages"], st["width"] = _pool(
                g, gh, lens, Hkv, D)
        else:
            kv = torch.randn(B * ctx, 2 * Hkv * D, generator=g, device="cuda").to(torch.bfloat16)
            st["k"] = kv[:, :Hkv * D].view(B * ctx, Hkv, D)
            st["v"] = kv[:, Hkv * D:].view(B * ctx, Hkv, D)
            st["kv_start"] = (torch.arange(B) * ctx).to(torch.int32).cuda()
        st["kv_len"] = lens.to(torch.int32).cuda()
        st["q"] = (torch.randn(T, Hq, D, generator=g, device="cuda") * 1.5).to(torch.bfloat16)
        st["sm"] = 1.0 / math.sqrt(D)
    st["T"] = T
    if own:
        from w4a4_quantized_gemm_rudder_amd import rudder
        st["rudder"] = rudder
        if op == "append":
            n = st["pages"].numel()
            st["K_out"] = torch.empty(n, Hkv, PAGE, D, device="cuda")
            st["V_out"] = torch.empty(n, Hkv, PAGE, D, device="cuda")
        else:
            st["o"] = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
            st["ws"] = torch.empty(
                rudder.attention_workspace_bytes(B, T, rows, ctx, Hq, Hkv, D),
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


def _own_matvec(st):
    comp = st["comp"]
    st["rudder"].rudder_matvec_w4(
        st["x"], st["sid"] if comp else None, st["Wq"], st["ws"], st["a"] if comp else None,
        st["b"] if comp else None, st["M"], st["N"], st["K"], st["group"], 3, st["y"])
    return st["y"]


def _own_append(st):
    r = st["rudder"]
    r.rudder_cache_append(st["k"], st["v"], st["row_start"], st["pos"], st["table"], st["B"],
                          st["T"], st["rows"], st["width"], st["num_pages"], st["Hkv"], st["D"],
                          st["codes"], st["scales"])
    r.rudder_cache_dequant(st["codes"], st["scales"], st["pages"], st["pages"].numel(),
                           st["num_pages"], st["Hkv"], st["D"], st["K_out"], st["V_out"])
    return {"k": st["K_out"], "v": st["V_out"], "scales": st["scales"]}


def _own_cache(st):
    st["rudder"].rudder_cache_attention(
        st["q"], st["row_start"], st["kv_len"], st["table"], st["codes"], st["scales"], st["B"],
        st["T"], st["rows"], st["ctx"], st["width"], st["num_pages"], st["Hq"], st["Hkv"],
        st["D"], st["sm"], st["causal"], st["ws"], st["o"])
    return st["o"]


def _own_cross(st):
    st["rudder"].rudder_cross_attention(
        st["q"], st["k"], st["v"], st["row_start"], st["kv_start"], st["kv_len"], st["B"],
        st["T"], st["k"].shape[0], st["rows"], st["ctx"], st["Hq"], st["Hkv"], st["D"],
        st["sm"], st["ws"], st["o"])
    return st["o"]


def _group_codes(W, group):
    """Symmetric 4-bit codes int8 [K, N] and bf16 scales [K/group, N] of the weights."""
    K, N = W.shape
    w = W.float().view(K // group, group, N)
    s = (w.abs().amax(1).double() / 7).float().to(torch.bfloat16)
    inv = torch.where(s > 0, 1 / s.double(), 0.0).float()
    q = torch.round(torch.clamp(w * inv[:, None, :], -7, 7))
    return q.to(torch.int8).view(K, N), s


def _plain_matvec(st):
    K, N, group = st["K"], st["N"], st["group"]
    w = (st["q"].float().view(K // group, group, N) * st["s"].float()[:, None, :]).view(K, N)
    y = st["x"].float() @ w
    if st["comp"]:
        sid = st["sid"].long()
        y = st["a"][sid] * y + st["b"][sid]
    return y.to(torch.bfloat16)


def _new_codes(x, old, s_old, fresh, new):
    """The append rule on one K or V half: x [n, H, 64, D] the new tokens' values (0 elsewhere),
    old codes [n, H, 64, D], s_old [n, H], slot masks [n, 64] -> (codes, scales)."""
    s_old = torch.where(fresh[:, None], 0.0, s_old)
    s = torch.maximum(s_old, (x.abs().amax((2, 3)).double() / 127).float())
    inv = torch.where(s > 0, 1 / s.double(), 0.0).float()[:, :, None, None]
    ratio = torch.where(s > 0, s_old.double() / s.double(), 1.0).float()[:, :, None, None]
    c = torch.round(torch.clamp(x * inv, -127, 127))
    kept = (~new & (torch.cumsum(new, 1) == 0))[:, None, :, None]
    o = torch.where(kept, torch.round(old * ratio), old)
    return torch.where(new[:, None, :, None], c, o), s


def _plain_append(st):
    Hkv, D = st["Hkv"], st["D"]
    pages, seq = st["pages"].long(), st["page_seq"]
    n = pages.numel()
    at = st["page_no"][:, None] * PAGE + torch.arange(PAGE, device="cuda")[None, :]
    i = at - st["pos"].long()[seq][:, None]                  # index among the sequence's new rows
    count = (st["row_start"][1:] - st["row_start"][:-1]).long()[seq][:, None]
    new = (i >= 0) & (i < count)
    row = torch.where(new, i + st["row_start"].long()[seq][:, None], 0)
    fresh = new[:, 0]
    old = st["codes"][pages]                                  # [n, H, 2, 64 D]
    mask = new[:, None, :, None]
    k_old = old[:, :, 0].view(n, Hkv, PAGE, D).float()
    v_old = old[:, :, 1].view(n, Hkv, D, PAGE).transpose(2, 3).float()
    x = torch.where(mask, st["k"][row].float().transpose(1, 2), 0.0)
    kc, ks = _new_codes(x, k_old, st["scales"][pages][:, :, 0], fresh, new)
    x = torch.where(mask, st["v"][row].float().transpose(1, 2), 0.0)
    vc, vs = _new_codes(x, v_old, st["scales"][pages][:, :, 1], fresh, new)
    halves = [kc.reshape(n, Hkv, PAGE * D), vc.transpose(2, 3).reshape(n, Hkv, PAGE * D)]
    st["codes"][pages] = torch.stack(halves, 2).to(torch.int8)
    st["scales"][pages] = torch.stack([ks, vs], 2)
    out = {"k": kc * ks[:, :, None, None], "v": vc * vs[:, :, None, None]}
    return {**out, "scales": st["scales"]}


def _rows_of(st):
    """Padded row numbers [B, rows] and which of them a sequence has."""
    start = st["row_start"].long()
    i = torch.arange(st["rows"], device="cuda")[None, :]
    have = i < (start[1:] - start[:-1])[:, None]
    return torch.where(have, start[:-1, None] + i, 0), have


def _plain_attention(st, k, v):
    """q against k, v [B, Hkv, L, D] in 32 bits (zeros behind a sequence's length)."""
    B, rows, Hq, Hkv, D = (st[n] for n in ("B", "rows", "Hq", "Hkv", "D"))
    L = k.shape[2]
    row, have = _rows_of(st)
    q = st["q"][row].float().view(B, rows, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4)
    q = q.reshape(B, Hkv, -1, D)
    s = (q @ k.transpose(2, 3).contiguous()).view(B, Hq, rows, L)
    s *= st["sm"]
    j = torch.arange(L, device="cuda")[None, None, :]
    limit = st["kv_len"].long()[:, None].expand(B, rows)
    if st.get("causal"):
        count = have.sum(1, keepdim=True)
        limit = limit - count + 1 + torch.arange(rows, device="cuda")[None, :]
        limit = torch.minimum(limit, st["kv_len"].long()[:, None])
    s.masked_fill_((j >= limit[:, :, None])[:, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    s.sub_(torch.where(m > -math.inf, m, 0.0)).exp_()
    total = s.sum(-1, keepdim=True)
    o = (s.view(B, Hkv, -1, L) @ v).view(B, Hq, rows, D)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 2, 1, 3)
    return o[have].to(torch.bfloat16)


def _plain_cache(st):
    B, W, Hkv, D = st["B"], st["width"], st["Hkv"], st["D"]
    pages = st["table"].long().clamp_(min=0)
    at = torch.arange(W * PAGE, device="cuda")[None, :] < st["kv_len"][:, None]
    at = at[:, None, :, None]
    c, s = st["codes"][pages], st["scales"][pages]            # [B, W, H, 2, 64 D], [B, W, H, 2]
    k = c[:, :, :, 0].view(B, W, Hkv, PAGE, D).float() * s[:, :, :, 0, None, None]
    k = k.permute(0, 2, 1, 3, 4).reshape(B, Hkv, W * PAGE, D)
    v = c[:, :, :, 1].view(B, W, Hkv, D, PAGE).float() * s[:, :, :, 1, None, None]
    v = v.permute(0, 2, 1, 4, 3).reshape(B, Hkv, W * PAGE, D)
    return _plain_attention(st, torch.where(at, k, 0.0), torch.where(at, v, 0.0))


def _plain_cross(st):
    L = st["ctx"]
    j = torch.arange(L, device="cuda")[None, :]
    have = j < st["kv_len"].long()[:, None]
    at = torch.where(have, st["kv_start"].long()[:, None] + j, 0)
    have = have[:, None, :, None]
    k = torch.where(have, st["k"][at].float().transpose(1, 2), 0.0)
    v = torch.where(have, st["v"][at].float().transpose(1, 2), 0.0)
    return _plain_attention(st, k, v)


_OWN = {"matvec": _own_matvec, "append": _own_append, "cache": _own_cache, "cross": _own_cross}
_PLAIN = {"matvec": _plain_matvec, "append": _plain_append, "cache": _plain_cache,
          "cross": _plain_cross}


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "matvec":
        M, K, N = case["M"], case["K"], case["N"]
        extra = 2 * 4 * N * min(M, 3) + M if case["comp"] else 0
        return {"bytes": K * N / 2 + 2 * (K // case["group"]) * N + 2 * M * K + 2 * M * N + extra,
                "flops": 2 * M * K * N}
    B, rows, ctx, Hkv, D = (case[k] for k in ("B", "rows", "ctx", "Hkv", "D"))
    n_rows, pos, gl = _rows(case)
    T = int(n_rows.sum())
    if op == "append":
        pages = int(((pos + n_rows - 1) // PAGE - pos // PAGE + 1).sum())     # touched
        new = 2 * T * Hkv * D                                 # values of K and V
        return {"bytes": 2 * new + new + pages * 2 * Hkv * PAGE * D * 5, "flops": 4 * new}
    Hq = case["Hq"]
    lens = _lengths(case, n_rows, gl)
    if op == "cache":
        kv = 2 * Hkv * D * int(lens.sum()) + 8 * Hkv * int(((lens + PAGE - 1) // PAGE).sum())
    else:
        kv = 4 * Hkv * D * int(lens.sum())
    pairs = (n_rows * lens).sum()
    if case.get("causal"):
        pairs = pairs - (n_rows * (n_rows - 1) // 2).sum()
    return {"bytes": kv + 4 * T * Hq * D, "flops": 4 * D * Hq * int(pairs)}


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
    return {"matvec": _exact_matvec, "append": _exact_append, "cache": _exact_attention,
            "cross": _exact_attention}[case["op"]](st)


def _exact_matvec(st):
    s = st["s"].double().repeat_interleave(st["group"], 0)
    y = torch.matmul(st["x"].double(), st["q"].double() * s)
    if st["comp"]:
        a, b = st["a"].double(), st["b"].double()
        y = torch.stack([a[i] * y[m] + b[i] for m, i in enumerate(st["sid"].tolist())])
    return y


def _exact_append(st):
    """Page by page.  The codes are decided in 32 bits by definition (absmax / 127, its
    reciprocal and the product are each rounded to 32 bits); the values are code * scale."""
    H, D = st["Hkv"], st["D"]
    scales = st["scales"].double()
    outs = {"k": [], "v": []}
    start, pos = st["row_start"].tolist(), st["pos"].tolist()
    for p, b, no in zip(st["pages"].tolist(), st["page_seq"].tolist(), st["page_no"].tolist()):
        lo = max(pos[b], no * PAGE)
        hi = min(pos[b] + start[b + 1] - start[b], (no + 1) * PAGE)
        r = start[b] + lo - pos[b]
        slot = lo - no * PAGE
        for name, half in (("k", 0), ("v", 1)):
            c = st["codes"][p, :, half].double()
            c = c.view(H, PAGE, D) if half == 0 else c.view(H, D, PAGE).transpose(1, 2)
            c = c.clone()
            x = st[name][r:r + hi - lo].double().transpose(0, 1)          # [H, n, D]
            fine = (x.abs().amax((1, 2)) / 127).float().double()
            had = scales[p, :, half] if slot else torch.zeros_like(fine)
            s = torch.maximum(had, fine)
            s1 = torch.where(s > 0, s, 1.0)
            c[:, :slot] = torch.round((c[:, :slot] * (had / s1).float().double()[:, None, None])
                                      .float()).double()
            q = (x * (1 / s1).float().double()[:, None, None]).float()
            c[:, slot:slot + hi - lo] = torch.round(q.clamp(-127, 127)).double()
            scales[p, :, half] = s
            outs[name].append(c * s[:, None, None])
    return {"k": torch.stack(outs["k"]), "v": torch.stack(outs["v"]), "scales": scales}


def _exact_attention(st):
    """Sequence by sequence, some heads' rows at a time."""
    H, G, D = st["Hkv"], st["Hq"] // st["Hkv"], st["D"]
    start, lens = st["row_start"].tolist(), st["kv_len"].tolist()
    o = torch.zeros(st["T"], st["Hq"], D, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        rows = range(start[b], start[b + 1])
        if st["op"] == "cross":
            at = int(st["kv_start"][b])
            k = st["k"][at:at + n].double().transpose(0, 1)
            v = st["v"][at:at + n].double().transpose(0, 1)
        else:
            used = st["table"][b, :(n + PAGE - 1) // PAGE].long()
            c, s = st["codes"][used].double(), st["scales"][used].double()
            k = (c[:, :, 0].view(-1, H, PAGE, D) * s[:, :, 0, None, None])
            v = (c[:, :, 1].view(-1, H, D, PAGE) * s[:, :, 1, None, None]).transpose(2, 3)
            k, v = (t.transpose(0, 1).reshape(H, -1, D)[:, :n] for t in (k, v))
        k, v = k.contiguous(), v.contiguous()
        for h in range(H):
            kt = k[h].t().contiguous()
            for r in range(rows.start, rows.stop, 4096):
                e = min(r + 4096, rows.stop)
                for g in range(G):
                    s = st["q"][r:e, h * G + g].double() @ kt * st["sm"]
                    if st.get("causal"):
                        i = torch.arange(r, e, device="cuda")[:, None] - start[b]
                        j = torch.arange(n, device="cuda")[None, :]
                        s = s.masked_fill(j > i + n - len(rows), -math.inf)
                    o[r:e, h * G + g] = torch.softmax(s, -1) @ v[h]
    return o
