"""The operators around the linears as a block uses them: norm and codes, QKV linear, rotary
positions, append and prompt attention, O linear, norm with the residual, up and down linears; single
tokens through the few-row products; captured in a graph and on two streams."""
import math

import pytest
import torch

import attention_reference as aref
import block_reference as ref
from gpu_harness import log

pytestmark = pytest.mark.gpu
PAGE, EPS = 64, 1e-5


@pytest.fixture(scope="module")
def rudder():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    from w4a4_quantized_gemm_rudder_amd import rudder as r
    r.load_library()
    return r


def _i32(x):
    return torch.tensor(x, dtype=torch.int32)


class Block:
    """Weights of a small block (W4A8 attention projections, W4A4 up projection in E2M3)."""

    def __init__(self, rudder, Hq, Hkv, D, K, F, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.r, self.Hq, self.Hkv, self.D, self.K, self.F = rudder, Hq, Hkv, D, K, F
        self.N = (Hq + 2 * Hkv) * D

        def layer(k, n, codes):
            w = (torch.randn(k, n, generator=g, device="cuda") * 0.08).to(torch.bfloat16)
            one = torch.ones(1, n, device="cuda")
            return (*rudder.quantize_weights(w, torch.ones(k, device="cuda"), codes), one, 0 * one)

        self.qkv, self.out = layer(K, self.N, 0), layer(Hq * D, K, 0)
        self.up = layer(K, F, 1)
        self.g1, self.g2 = (torch.rand(K, generator=g, device="cuda") + 0.5 for _ in range(2))
        self.freq = rudder.rotary_frequencies(D, scaling="parts", factor=4.0, trained=2048)
        self.table = torch.full((1,), 0.5, device="cuda")

    def linear(self, w, xq, rs, sid, M, k, n, bits, codes=0):
        return self.r.linear(xq, rs, sid, w[0], w[1], w[3], w[4], M, n, k, 1, bits, codes)


def test_prompt_through_a_block(rudder):
    """Two prompts: each stage against its plain form on the previous stage's GPU output."""
    log("case block prompt")
    Hq, Hkv, D, K, F, counts = 4, 2, 64, 256, 384, [150, 37]
    b = Block(rudder, Hq, Hkv, D, K, F, 71)
    M, sm = sum(counts), 1 / math.sqrt(D)
    g = torch.Generator().manual_seed(72)
    x = torch.randn(M, K, generator=g).to(torch.bfloat16)
    sid = torch.zeros(M, dtype=torch.uint8, device="cuda")
    starts = _i32([0] + counts).cumsum(0).to(torch.int32)
    ds = starts.cuda()
    xq, rs = rudder.norm_quant(x.cuda(), b.g1, b.qkv[2], EPS, 8)
    Y = b.linear(b.qkv, xq, rs, sid, M, K, b.N, 8).view(M, -1, D)
    plain = Y.cpu().clone()
    q, k, v = Y[:, :Hq], Y[:, Hq:Hq + Hkv], Y[:, Hq + Hkv:]
    rudder.rotary(q, k, ds, b.freq, max(counts), in_place=True)
    codes, scales = rudder.new_cache(8, Hkv, D)
    table = _i32([[3, 0, 6], [1, -1, -1]])
    rudder.cache_append(k, v, ds, _i32([0, 0]).cuda(), table.cuda(), max(counts), codes, scales)
    O = rudder.prompt_attention(q, k, v, ds, max(counts), sm)
    oq, ors = rudder.quant_act(O.view(M, -1), sid, b.out[2], None, 1, 8)
    Z = b.linear(b.out, oq, ors, sid, M, Hq * D, K, 8)
    uq, urs, h = rudder.norm_quant(Z, b.g2, b.up[2], EPS, 4, 1, sid, b.table, residual=x.cuda())
    U = b.linear(b.up, uq, urs, sid, M, K, F, 4, 1)

    y, _ = ref.norm(x, b.g1.cpu(), EPS)
    c, s = ref.codes(y, torch.ones(K), 8)
    assert torch.equal(rudder.dequant_act(xq, rs, M, K, 8).cpu(), c.float() * s[:, None])
    at = torch.cat([torch.arange(n) for n in counts])
    for name, got, p in (("q", q, plain[:, :Hq]), ("k", k, plain[:, Hq:Hq + Hkv])):
        want, bound = ref.rotary(p, at, b.freq.cpu(), 1.0, False)
        aref.assert_within(name, got, want, bound)
    host = Y.cpu()
    want, bound = ref.prompt(*(t.cpu() for t in (q, k, v)), starts.tolist(), sm)
    aref.assert_within("O", O, want, bound)
    hc, hs = torch.zeros_like(codes).cpu(), torch.zeros_like(scales).cpu()
    aref.append(host[:, Hq:Hq + Hkv], host[:, Hq + Hkv:], starts, _i32([0, 0]), table, hc, hs)
    assert torch.equal(codes.cpu(), hc) and torch.equal(scales.cpu(), hs)
    # the cache's answer to the same rows: K and V in 8 bits, half a step of the page's largest
    C = rudder.cache_attention(q, ds, _i32(counts).cuda(), table.cuda(), codes, scales,
                               max(counts), max(counts), sm)
    err = (C.double() - O.double()).norm() / O.double().norm()
    assert err < 0.03, float(err)
    y, hh = ref.norm(Z.cpu(), b.g2.cpu(), EPS, x)
    assert torch.equal(h.cpu(), hh)
    c, s = ref.codes(y, torch.ones(K), 4, sid.cpu(), b.table.cpu())
    assert torch.equal(rudder.dequant_act(uq, urs, M, K, 4, 1).cpu(), c.float() * s[:, None])
    wq = torch.empty(K, F, device="cuda")
    rudder.rudder_dequant_weights(b.up[0], b.up[1], K, F, 1, wq)
    act = rudder.dequant_act(uq, urs, M, K, 4, 1).double()
    full = act @ wq.double()
    # the linear: exact integer sums, three roundings to fp32 and one to bf16; the values multiplied
    # here were each rounded to fp32, which counts with the terms' size, not the sum's
    bound = (aref.BF16 + 4 * aref.FP32) * full.abs() + 3 * aref.FP32 * (act.abs() @ wq.double().abs())
    assert ((U.double() - full).abs() <= bound).all()


def test_tokens_behind_a_prompt(rudder):
    """A prompt of 100 tokens, then 30 single tokens through norm, few-row product, rotary
    positions, append and attention to the cache: the last outputs against their plain forms."""
    log("case block tokens")
    Hq, Hkv, D, K, group = 4, 2, 64, 256, 64
    g = torch.Generator().manual_seed(73)
    N = (Hq + 2 * Hkv) * D
    W = (torch.randn(K, N, generator=g) * 0.1).to(torch.bfloat16)
    wq = rudder.quantize_weights_grouped(W.cuda(), group)
    gamma = torch.rand(K, generator=g) + 0.5
    freq = rudder.rotary_frequencies(D)
    codes, scales = rudder.new_cache(4, Hkv, D)
    table = _i32([[2, 0, 3]]).cuda()
    x = torch.randn(130, K, generator=g).to(torch.bfloat16)
    res = torch.zeros(1, K, dtype=torch.bfloat16, device="cuda")
    ks = []
    for t, n in [(0, 100)] + [(t, 1) for t in range(100, 130)]:
        xt = x[t:t + n].cuda()
        if n == 1:
            y, res = rudder.norm(xt, gamma.cuda(), EPS, res)
        else:
            y = rudder.norm(xt, gamma.cuda(), EPS)
        Y = rudder.matvec_w4(y, *wq, N, group).view(n, -1, D)
        before = Y.clone()
        q, k, v = Y[:, :Hq], Y[:, Hq:Hq + Hkv], Y[:, Hq + Hkv:]
        starts, pos = _i32([0, n]).cuda(), _i32([t]).cuda()
        rudder.rotary(q, k, starts, freq, n, pos, in_place=True)
        rudder.cache_append(k, v, starts, pos, table, n, codes, scales)
        O = rudder.cache_attention(q, starts, _i32([t + n]).cuda(), table, codes, scales, n, 192,
                                   0.125)
        ks.append(k.cpu().clone())
    acc = torch.zeros(1, K, dtype=torch.bfloat16)
    for t in range(100, 130):
        want, acc = ref.norm(x[t:t + 1], gamma, EPS, acc)
    assert torch.equal(res.cpu(), acc) and torch.equal(y.cpu(), want)
    for name, got, p in (("q", q, before[:, :Hq]), ("k", k, before[:, Hq:Hq + Hkv])):
        want, bound = ref.rotary(p.cpu(), _i32([129]).long(), freq.cpu(), 1.0, False)
        aref.assert_within(name, got, want, bound)
    want, bound = aref.cache_attention(q.cpu(), [0, 1], [130], table.cpu(), codes.cpu(),
                                       scales.cpu(), 0.125, True)
    aref.assert_within("O", O, want, bound)
    # the cached keys are the turned ones, but for their step size
    got, _ = rudder.cache_dequant(codes, scales, _i32([2, 0, 3]).cuda())
    got = got.permute(0, 2, 1, 3).reshape(-1, Hkv, D)[:130].cpu()
    err = (got - torch.cat(ks).float()).norm() / got.norm()
    assert err < 0.02, float(err)


def _case(rudder, counts, Hq, Hkv, D, seed):
    """The calls with preallocated buffers: (run, outputs)."""
    r = rudder
    g = torch.Generator(device="cuda").manual_seed(seed)
    M, B, rows, K = sum(counts), len(counts), max(counts), Hq * D
    bf = dict(dtype=torch.bfloat16, device="cuda")
    buf = torch.randn(M, Hq + 2 * Hkv, D, generator=g, device="cuda").to(torch.bfloat16)
    x = torch.randn(M, K, generator=g, device="cuda").to(torch.bfloat16)
    gamma = torch.rand(K, generator=g, device="cuda") + 0.5
    smooth = torch.rand(K, generator=g, device="cuda") + 0.5
    starts = _i32([0] + counts).cumsum(0).to(torch.int32).cuda()
    freq = r.rotary_frequencies(D)
    qo, ko = torch.zeros(M, Hq, D, **bf), torch.zeros(M, Hkv, D, **bf)
    O, h, y = torch.zeros(M, Hq, D, **bf), torch.zeros(M, K, **bf), torch.zeros(M, K, **bf)
    xq = torch.zeros(r.packed_act_bytes(M, K, 8), dtype=torch.uint8, device="cuda")
    rs, values = torch.zeros(M, device="cuda"), torch.zeros(M, K, device="cuda")
    ws = torch.empty(max(16, r.prompt_attention_workspace_bytes(B, M, rows, Hq, Hkv, D)),
                     dtype=torch.uint8, device="cuda")

    def run():
        r.rudder_rotary(buf[:, :Hq], buf[:, Hq:Hq + Hkv], starts, None, freq, 1.0, B, M, rows, Hq,
                        Hkv, D, D, r.ROTARY_PAIRS, qo, ko)
        r.rudder_prompt_attention(qo, ko, buf[:, Hq + Hkv:], starts, B, M, rows, Hq, Hkv, D, 0.1,
                                  ws, O)
        r.rudder_norm(O.view(M, K), x, gamma, EPS, M, K, h, y)
        r.rudder_norm_quant(y, x, None, gamma, smooth, None, EPS, M, K, 1, 8, 0, h, xq, rs)
        r.rudder_dequant_act(xq, rs, M, K, 8, 0, values)

    return run, [qo, ko, O, h, y, xq, rs, values], (x, buf)


CASES = [([1], 2, 1, 64), ([70, 9], 4, 2, 64), ([1500, 300, 1], 8, 2, 128), ([2500, 2100], 16, 4, 64)]


@pytest.mark.parametrize("counts,Hq,Hkv,D", CASES)
def test_graph_replays(rudder, counts, Hq, Hkv, D):
    """The captured calls replayed on changed inputs, with eager work between, equal the eager run
    bit for bit."""
    log(f"case block graph {counts}")
    run, outputs, inputs = _case(rudder, counts, Hq, Hkv, D, 81)
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    scratch = torch.randn(512, 512, device="cuda")
    for rep in range(3):
        for t in inputs:
            t.mul_(1.25)
        run()
        torch.cuda.synchronize()
        want = [o.clone() for o in outputs]
        for o in outputs:
            o.fill_(9)
        (scratch @ scratch).sum().item()
        graph.replay()
        torch.cuda.synchronize()
        for i, (o, w) in enumerate(zip(outputs, want)):
            assert torch.equal(o.view(torch.uint8), w.view(torch.uint8)), (rep, i)


def test_two_streams(rudder):
    """Two sets of calls with buffers of their own on two streams at a time equal the same alone."""
    log("case block two streams")
    cases = [_case(rudder, [1500, 700], 8, 2, 128, 82), _case(rudder, [900, 1100, 30], 8, 8, 64, 83)]
    wants = []
    for run, outputs, _ in cases:
        run()
        torch.cuda.synchronize()
        wants.append([o.clone() for o in outputs])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for (run, _o, _i), st in zip(cases, streams):
            with torch.cuda.stream(st):
                run()
    torch.cuda.synchronize()
    for (_, outputs, _i), want in zip(cases, wants):
        for o, w in zip(outputs, want):
            assert torch.equal(o.view(torch.uint8), w.view(torch.uint8))


def test_conveniences_on_a_given_stream(rudder):
    """The allocating forms on a stream that is not the current one."""
    log("case block given stream")
    g = torch.Generator(device="cuda").manual_seed(84)
    T, H, D = 700, 4, 64
    q, k, v = (torch.randn(T, H, D, generator=g, device="cuda").to(torch.bfloat16)
               for _ in range(3))
    starts, freq = _i32([0, 300, 700]).cuda(), rudder.rotary_frequencies(D)
    gamma, smooth = torch.rand(H * D, device="cuda") + 0.5, torch.rand(H * D, device="cuda") + 0.5
    calls = [
        lambda **s: rudder.norm(q.view(T, -1), gamma, EPS, k.view(T, -1), **s),
        lambda **s: rudder.norm_quant(q.view(T, -1), gamma, smooth, EPS, 4, 1, **s),
        lambda **s: (rudder.dequant_act(torch.full((704 * 256,), 3, dtype=torch.uint8,
                                                   device="cuda"), gamma.repeat(3), T, 256, 8,
                                        **s),),
        lambda **s: rudder.rotary(q, k, starts, freq, 400, **s),
        lambda **s: (rudder.prompt_attention(q, k, v, starts, 400, 0.125, **s),),
    ]
    wants = [c() for c in calls]
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    for stream in (st, st.cuda_stream):
        for c, want in zip(calls, wants):
            got = c(stream=stream)
            st.synchronize()
            for a, b in zip(got, want):
                assert torch.equal(a, b)
