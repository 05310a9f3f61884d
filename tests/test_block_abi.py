"""Host-side checks of the norms, rotary positions and prompt attention (no GPU needed): sizes,
frequencies, and every refusal before anything is launched."""
import math

import pytest
import torch

import block_reference as ref

P = 0x1000              # never dereferenced


@pytest.fixture(scope="module")
def r():
    from w4a4_quantized_gemm_rudder_amd import rudder
    rudder.load_library()
    return rudder


def _status(r, name, args, kw):
    args = dict(args)
    for k in kw:
        assert k in args, k
    args.update(kw)
    status = getattr(r.load_library(), name)(*args.values(), None)
    assert (r.load_library().rudder_last_error() == b"") == (status == 0)
    return status


NORM = dict(X=P, R=P, gamma=P, eps=1e-6, M=4, K=256, ldx=256, ldr=512, ldh=264, ldy=256, H=P,
            Y=2 * P)
QUANT = dict(X=P, R=P, sid=P, gamma=P, inv_smooth=P, table=P, eps=1e-6, M=4, K=256, S=3, abits=8,
             codes=0, ldx=256, ldr=512, ldh=264, H=P, Xq=P, row_scale=P)
BOTH = [
    (dict(X=None), 1), (dict(gamma=None), 1), (dict(R=None), 1), (dict(H=None), 1),
    (dict(M=-1), 1), (dict(K=0), 1), (dict(K=-8), 1), (dict(K=252), 1), (dict(ldx=248), 1),
    (dict(ldx=260), 1), (dict(ldr=255), 1), (dict(ldh=252), 1), (dict(eps=-1e-9), 1),
    (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(X=P + 8), 1),
    (dict(R=P + 2), 1), (dict(H=P + 8), 1), (dict(gamma=P + 4), 1),
    (dict(K=65536 + 64, ldx=70400, ldr=70400, ldh=70400), 2), (dict(M=(1 << 25) + 1), 2),
    (dict(M=1 << 25, K=2048, ldx=2048, ldr=2048, ldh=2048), 2),
    (dict(M=0), 0), (dict(M=0, R=None, H=None, ldr=0, ldh=0), 0), (dict(M=0, eps=0.0), 0),
]


@pytest.mark.parametrize("kw,status", BOTH + [
    (dict(Y=None), 1), (dict(ldy=248), 1), (dict(Y=P + 8), 1), (dict(Y=P), 1),
    (dict(M=0, K=264, ldx=264, ldr=264, ldh=264, ldy=264), 0),
])
def test_norm_refusals(r, kw, status):
    kw = dict(kw)
    if kw.get("K", 0) > 256:
        kw["ldy"] = kw["ldx"]
    assert _status(r, "rudder_norm", NORM, kw) == status


@pytest.mark.parametrize("kw,status", BOTH + [
    (dict(inv_smooth=None), 1), (dict(Xq=None), 1), (dict(row_scale=None), 1),
    (dict(sid=None), 1), (dict(K=240), 1), (dict(K=224, codes=1), 1),
    (dict(S=0), 1), (dict(S=9), 1), (dict(abits=6), 1), (dict(codes=2), 1), (dict(Xq=P + 8), 1),
    (dict(inv_smooth=P + 4), 1), (dict(codes=1), 2), (dict(M=0, sid=None, table=None, S=0), 0),
    (dict(M=0, table=None, S=0), 0), (dict(M=0, abits=4, codes=1), 0),
])
def test_norm_quant_refusals(r, kw, status):
    assert _status(r, "rudder_norm_quant", QUANT, kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(Xq=None), 1), (dict(row_scale=None), 1), (dict(out=None), 1), (dict(M=-1), 1),
    (dict(K=0), 1), (dict(K=48), 1), (dict(K=96, codes=1), 1), (dict(abits=5), 1),
    (dict(codes=-1), 1), (dict(Xq=P + 4), 1), (dict(out=P + 4), 1), (dict(K=1 << 17), 2),
    (dict(M=(1 << 25) + 1), 2), (dict(M=1 << 25, K=2048), 2), (dict(M=0), 0),
    (dict(M=0, codes=1), 0),
])
def test_dequant_act_refusals(r, kw, status):
    args = dict(Xq=P, row_scale=P, M=4, K=64, abits=8, codes=0, out=P)
    assert _status(r, "rudder_dequant_act", args, kw) == status


ROTARY = dict(Q=P, K=P, row_start=P, pos=P, freq=P, magnitude=1.0, B=2, T=4, max_rows=2, Hq=4,
              Hkv=2, D=64, part=32, layout=0, ldq=512, ldk=512, ldqo=256, ldko=128, Qo=P, Ko=P)


@pytest.mark.parametrize("kw,status", [
    (dict(Q=None), 1), (dict(K=None), 1), (dict(row_start=None), 1), (dict(freq=None), 1),
    (dict(Qo=None), 1), (dict(Ko=None), 1), (dict(B=-1), 1), (dict(T=-1), 1),
    (dict(max_rows=-1), 1), (dict(Hq=0), 1), (dict(Hkv=-1), 1), (dict(layout=2), 1),
    (dict(part=0), 1), (dict(part=24), 1), (dict(part=80), 1), (dict(ldq=248), 1),
    (dict(ldk=132), 1), (dict(ldqo=255), 1), (dict(ldko=120), 1),
    (dict(magnitude=float("inf")), 1), (dict(magnitude=float("nan")), 1), (dict(Q=P + 8), 1),
    (dict(Ko=P + 2), 1), (dict(D=96, part=96), 2), (dict(B=65536), 2),
    (dict(Hq=5000, ldq=320000, ldqo=320000), 2), (dict(T=1 << 26, max_rows=1 << 26), 2),
    (dict(B=0), 0), (dict(T=0), 0), (dict(max_rows=0), 0), (dict(T=0, pos=None), 0),
    (dict(T=0, Hkv=0, K=None, Ko=None, ldk=0, ldko=0), 0),
])
def test_rotary_refusals(r, kw, status):
    assert _status(r, "rudder_rotary", ROTARY, kw) == status


PROMPT = dict(Q=P, K=P, V=P, row_start=P, B=2, T=4, max_rows=2, Hq=4, Hkv=2, D=64, ldq=512,
              ldk=512, ldv=512, ldo=256, sm=0.1, ws=P, wbytes=1 << 40, O=P)


@pytest.mark.parametrize("kw,status", [
    (dict(Q=None), 1), (dict(K=None), 1), (dict(V=None), 1), (dict(row_start=None), 1),
    (dict(O=None), 1), (dict(B=-1), 1), (dict(T=-2), 1), (dict(max_rows=-1), 1), (dict(Hq=3), 1),
    (dict(Hq=0), 1), (dict(Hkv=0), 1), (dict(ldq=255), 1), (dict(ldk=120), 1), (dict(ldv=132), 1),
    (dict(ldo=248), 1), (dict(sm=float("nan")), 1), (dict(sm=float("inf")), 1),
    (dict(sm=-3e38), 1), (dict(Q=P + 8), 1), (dict(V=P + 2), 1), (dict(O=P + 8), 1),
    (dict(ws=P + 4), 1), (dict(D=80), 2), (dict(B=40000), 2),
    (dict(Hkv=5000, Hq=5000, ldq=320000, ldk=320000, ldv=320000, ldo=320000), 2),
    (dict(T=1 << 25, max_rows=1 << 25), 2), (dict(B=3000, T=1 << 20, max_rows=1 << 20), 2),
    (dict(B=0), 0), (dict(T=0), 0), (dict(max_rows=0, ws=None, wbytes=0), 0),
])
def test_prompt_refusals(r, kw, status):
    assert _status(r, "rudder_prompt_attention", PROMPT, kw) == status


def test_prompt_workspace(r):
    """Too small a workspace is refused, with the size in the message; sizes that the call refuses
    have none; smaller calls never need more."""
    need = r.prompt_attention_workspace_bytes
    for bad in ((1, 9, 9, 15, 2, 64), (1, 9, 9, 4, 2, 96), (-1, 9, 9, 4, 2, 64),
                (0, 9, 9, 4, 2, 64), (1, 0, 9, 4, 2, 64)):
        assert need(*bad) == 0
    big = need(2, 8384, 4192, 16, 16, 128)
    if big:
        args = dict(PROMPT, B=2, T=8384, max_rows=4192, Hq=16, Hkv=16, D=128, ldq=2048, ldk=2048,
                    ldv=2048, ldo=2048)
        assert _status(r, "rudder_prompt_attention", args, dict(wbytes=big - 1)) == 1
        assert str(big) in r.load_library().rudder_last_error().decode()
        assert _status(r, "rudder_prompt_attention", args, dict(ws=None)) == 1
    for D in (64, 128):
        for B, T, rows in ((4, 9000, 3000), (1, 700, 700), (40, 4000, 100), (3, 2000, 2000)):
            most = need(B, T, rows, 8, 2, D)
            for b in (1, 2, B):
                for t in (1, 63, T // 3, T):
                    for n in (1, 64, rows // 2, rows):
                        assert need(min(b, B), t, n, 8, 2, D) <= most


# n, base, scaling, factor, trained, low, high
@pytest.mark.parametrize("case", [
    (32, 10000.0, "plain", 1.0, 0.0, 1.0, 32.0), (8, 500000.0, "plain", 9.0, 0.0, 1.0, 32.0),
    (16, 10000.0, "linear", 4.0, 0.0, 1.0, 32.0), (64, 10000.0, "base", 8.0, 0.0, 1.0, 32.0),
    (1, 10000.0, "base", 8.0, 0.0, 1.0, 32.0), (64, 10000.0, "parts", 16.0, 4096.0, 1.0, 32.0),
    (48, 500000.0, "parts", 8.0, 8192.0, 1.0, 4.0),
])
def test_frequencies(r, case):
    n, base, scaling, factor, trained, low, high = case
    got = r.rotary_frequencies(2 * n, base, scaling, factor, trained, low, high, device="cpu")
    want = ref.frequencies(n, base, scaling, factor, trained, low, high)
    assert got.dtype == torch.float64 and got.shape == (n,)
    assert ((got - want).abs() <= 1e-13 * want).all()


def test_frequencies_by_scaling(r):
    """What the scalings are for: the slowest pair's turns over a stretched context are those of
    the trained one, the fastest pair stays where the scaling keeps it."""
    n, factor = 64, 8.0
    plain = r.rotary_frequencies(2 * n, device="cpu")
    assert plain[0] == 1 and plain[-1] == pytest.approx(10000.0 ** (-(n - 1) / n), rel=1e-14)
    base = r.rotary_frequencies(2 * n, scaling="base", factor=factor, device="cpu")
    assert base[0] == 1 and base[-1] * factor == pytest.approx(float(plain[-1]), rel=1e-12)
    parts = r.rotary_frequencies(2 * n, scaling="parts", factor=factor, trained=4096, device="cpu")
    turns = 4096 * plain / (2 * math.pi)
    assert torch.equal(parts[turns >= 32], plain[turns >= 32])
    assert torch.equal(parts[turns <= 1], plain[turns <= 1] / factor)
    assert (parts < plain)[turns < 32].all() and (parts * factor > plain)[turns > 1].all()


@pytest.mark.parametrize("kw,status", [
    (dict(freq=None), 1), (dict(n=0), 1), (dict(n=-2), 1), (dict(n=7), 1), (dict(base=0.0), 1),
    (dict(base=float("nan")), 1), (dict(base=float("inf")), 1), (dict(scaling=4), 1),
    (dict(scaling=-1), 1), (dict(factor=0.5), 1), (dict(factor=float("nan")), 1),
    (dict(trained=0.0), 1), (dict(low=-1.0), 1), (dict(high=1.0), 1), (dict(high=math.inf), 1),
    (dict(n=(1 << 16) + 2), 2),
])
def test_frequencies_refusals(r, kw, status):
    buf = torch.zeros(64, dtype=torch.float64)
    args = dict(n=64, base=1e4, scaling=3, factor=8.0, trained=4096.0, low=1.0, high=32.0,
                freq=buf.data_ptr())
    args.update(kw)
    assert r.load_library().rudder_rotary_frequencies(*args.values()) == status
    assert not buf.any()


def test_frequencies_binding(r):
    for bad in (torch.zeros(8), torch.zeros(3, dtype=torch.float64)):
        with pytest.raises(ValueError, match="fp64"):
            r.rudder_rotary_frequencies(16, 1e4, 0, 1.0, 0.0, 1.0, 32.0, bad)
    with pytest.raises(r.RudderError, match="even"):
        r.rotary_frequencies(15, device="cpu")
    with pytest.raises(KeyError):
        r.rotary_frequencies(16, scaling="other", device="cpu")


def test_frequencies_of_one_element_many_times(r):
    """An expanded or strided tensor has the elements but not the memory behind each other."""
    one, far = torch.zeros(1, dtype=torch.float64), torch.zeros(16, dtype=torch.float64)
    for bad in (one.expand(8), far[::2]):
        with pytest.raises(ValueError, match="contiguous fp64"):
            r.rudder_rotary_frequencies(16, 1e4, 0, 1.0, 0.0, 1.0, 32.0, bad)
    assert not one.any() and not far.any()


def test_conveniences_check_shapes(r):
    """Vectors of other widths and codes of other sizes, also where there is nothing to do."""
    x, g, wide = torch.zeros(3, 64, dtype=torch.bfloat16), torch.zeros(64), torch.zeros(128)
    for n in (3, 0):
        with pytest.raises(ValueError, match="gamma of 128 elements.*K=64"):
            r.norm(x[:n], wide, 1e-6)
        with pytest.raises(ValueError, match="gamma of 128 elements.*K=64"):
            r.norm_quant(x[:n], wide, g, 1e-6, 8)
        with pytest.raises(ValueError, match="inv_smooth of 128 elements.*K=64"):
            r.norm_quant(x[:n], g, wide, 1e-6, 8)
    for M, K, abits, codes in ((32, 64, 8, 0), (32, 64, 4, 1), (64, 64, 4, 0), (32, 128, 4, 0)):
        Xq = torch.zeros(r.packed_act_bytes(M, K, abits, codes), dtype=torch.uint8)
        with pytest.raises(ValueError, match="codes of M=32, K=64, abits=4, codes=0"):
            r.dequant_act(Xq, torch.zeros(32), 32, 64, 4)


def test_binding_refuses_host_tensors(r):
    """Tensors of the wrong place, type, size or layout never reach the library."""
    bf, i32 = torch.bfloat16, torch.int32
    x, g = torch.zeros(4, 64, dtype=bf), torch.zeros(64)
    with pytest.raises(ValueError, match="X"):
        r.rudder_norm(x, None, g, 1e-6, 4, 64, None, x, stream=0)
    with pytest.raises(ValueError, match="X"):
        r.rudder_norm(x, None, P, 1e-6, 5, 64, None, P, stream=0)
    with pytest.raises(ValueError, match="gamma"):
        r.rudder_norm(P, None, g[:60], 1e-6, 4, 64, None, P, stream=0)
    with pytest.raises(ValueError, match="Xq"):
        r.rudder_norm_quant(P, None, None, P, P, None, 1e-6, 4, 64, 1, 8, 0, None,
                            torch.zeros(32 * 64 - 1, dtype=torch.uint8), P, stream=0)
    with pytest.raises(ValueError, match="out"):
        r.rudder_dequant_act(P, P, 4, 64, 8, 0, torch.zeros(4, 63), stream=0)
    q = torch.zeros(4, 2, 64, dtype=bf)
    with pytest.raises(ValueError, match="freq"):
        r.rudder_rotary(P, None, P, None, torch.zeros(32), 1.0, 1, 4, 4, 2, 0, 64, 64, 0, P, None,
                        stream=0)
    with pytest.raises(ValueError, match="Q"):
        r.rudder_rotary(q.transpose(1, 2), None, P, None, P, 1.0, 1, 4, 4, 2, 0, 64, 64, 0, P,
                        None, stream=0)
    with pytest.raises(ValueError, match="row_start"):
        r.rudder_prompt_attention(P, P, P, torch.zeros(2, dtype=i32), 2, 4, 4, 2, 2, 64, 0.1, None,
                                  P, stream=0)
    with pytest.raises(ValueError, match="V"):
        r.rudder_prompt_attention(P, P, q.float(), P, 2, 4, 4, 2, 2, 64, 0.1, None, P, stream=0)
    assert q.sum() == 0 and x.sum() == 0
    # sizes of no work pass through without a device
    r.rudder_norm(P, None, P, 1e-6, 0, 64, None, 2 * P, stream=0)
