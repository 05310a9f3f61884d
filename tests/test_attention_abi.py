"""Host-side checks of the cache, attention and few-row calls (no GPU
needed): sizes, and every refusal before anything is launched."""
import pytest
import torch

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
    return getattr(r.load_library(), name)(*args.values(), None)


MATVEC = dict(X=P, sid=P, Wq=P, gs=P, a=P, b=P, M=4, N=48, K=256, group=64, S=3, Y=P)


@pytest.mark.parametrize("kw,status", [
    (dict(X=None), 1), (dict(Wq=None), 1), (dict(gs=None), 1), (dict(Y=None), 1),
    (dict(a=None), 1), (dict(b=None), 1), (dict(sid=None), 1), (dict(M=-1), 1), (dict(N=0), 1),
    (dict(K=0), 1), (dict(K=96), 1), (dict(group=16), 1), (dict(group=0), 1), (dict(S=0), 1),
    (dict(S=9), 1), (dict(X=P + 2), 1), (dict(Wq=P + 8), 1), (dict(gs=P + 2), 1),
    (dict(K=65536 + 64), 2), (dict(N=(1 << 24) + 1), 2), (dict(M=(1 << 19) + 1), 2),
    (dict(M=0), 0), (dict(M=0, sid=None, a=None, b=None, S=0), 0),
])
def test_matvec_refusals(r, kw, status):
    assert _status(r, "rudder_matvec_w4", MATVEC, kw) == status
    assert (r.load_library().rudder_last_error() == b"") == (status == 0)


@pytest.mark.parametrize("kw,status", [
    (dict(W=None), 1), (dict(Wq=None), 1), (dict(gs=None), 1), (dict(K=100), 1), (dict(N=-1), 1),
    (dict(group=48), 1), (dict(Wq=P + 4), 1), (dict(K=65536 * 2), 2),
])
def test_quantize_weights_grouped_refusals(r, kw, status):
    args = dict(W=P, K=256, N=48, group=64, Wq=P, gs=P)
    assert _status(r, "rudder_quantize_weights_grouped", args, kw) == status


def test_sizes(r):
    assert r.grouped_weight_bytes(256, 48) == 256 * 48 // 2
    assert r.grouped_weight_bytes(96, 17) == 128 * 32 // 2        # padded to 128 and 16
    assert r.grouped_weight_bytes(0, 17) == 0
    assert r.grouped_scale_count(96, 17, 32) == 4 * 32            # padded likewise
    assert r.grouped_scale_count(96, 17, 64) == 0
    assert r.cache_page_bytes(8, 128) == 8 * 2 * 64 * 128
    assert r.cache_page_bytes(8, 96) == 0 and r.cache_page_bytes(0, 64) == 0
    # whole rounds of row tiles need no pieces; one row of a long cache does
    assert r.attention_workspace_bytes(2, 8192, 4096, 4192, 16, 16, 128) == 0
    one = r.attention_workspace_bytes(1, 1, 1, 40000, 16, 16, 128)
    assert one > 0 and one % (16 * 130 * 4) == 0
    # bounded by T, not by a loose max_rows
    assert r.attention_workspace_bytes(1, 1, 1000, 40000, 16, 16, 128) == one
    for bad in ((1, 1, 1, 100, 15, 2, 64), (1, 1, 1, 100, 4, 2, 96), (-1, 1, 1, 100, 4, 2, 64),
                (1, 1, 1, -1, 4, 2, 64)):
        assert r.attention_workspace_bytes(*bad) == 0


APPEND = dict(K=P, V=P, row_start=P, pos=P, table=P, B=2, T=4, max_rows=2, max_pages=3,
              num_pages=9, Hkv=2, D=64, ldk=128, ldv=384, codes=P, scales=P)


@pytest.mark.parametrize("kw,status", [
    (dict(K=None), 1), (dict(V=None), 1), (dict(row_start=None), 1), (dict(pos=None), 1),
    (dict(table=None), 1), (dict(codes=None), 1), (dict(scales=None), 1), (dict(B=-1), 1),
    (dict(T=-1), 1), (dict(max_rows=-1), 1), (dict(max_pages=0), 1), (dict(num_pages=0), 1),
    (dict(Hkv=0), 1), (dict(ldk=127), 1), (dict(ldk=120), 1), (dict(ldv=132), 1),
    (dict(K=P + 8), 1), (dict(codes=P + 1), 1), (dict(D=96), 2), (dict(B=65536), 2),
    (dict(Hkv=5000, ldk=5000 * 64, ldv=5000 * 64), 2),
    (dict(T=1 << 30, max_rows=1 << 30), 2), (dict(B=0), 0), (dict(T=0), 0),
    (dict(max_rows=0), 0),
])
def test_append_refusals(r, kw, status):
    assert _status(r, "rudder_cache_append", APPEND, kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(codes=None), 1), (dict(scales=None), 1), (dict(pages=None), 1), (dict(k=None), 1),
    (dict(v=None), 1), (dict(n=-1), 1), (dict(num_pages=0), 1), (dict(Hkv=-2), 1),
    (dict(k=P + 4), 1), (dict(D=32), 2), (dict(n=(1 << 23) + 1), 2), (dict(n=0), 0),
])
def test_dequant_refusals(r, kw, status):
    args = dict(codes=P, scales=P, pages=P, n=3, num_pages=9, Hkv=2, D=64, k=P, v=P)
    assert _status(r, "rudder_cache_dequant", args, kw) == status


CACHE = dict(Q=P, row_start=P, kv_len=P, table=P, codes=P, scales=P, B=2, T=4, max_rows=2,
             max_kv=100, max_pages=3, num_pages=9, Hq=4, Hkv=2, D=64, ldq=256, ldo=256, sm=0.1,
             causal=1, ws=P, wbytes=1 << 40, O=P)
CROSS = dict(Q=P, K=P, V=P, row_start=P, kv_start=P, kv_len=P, B=2, T=4, Tkv=100, max_rows=2,
             max_kv=50, Hq=4, Hkv=2, D=64, ldq=256, ldk=128, ldv=128, ldo=256, sm=0.1, ws=P,
             wbytes=1 << 40, O=P)
BOTH = [
    (dict(Q=None), 1), (dict(row_start=None), 1), (dict(kv_len=None), 1), (dict(O=None), 1),
    (dict(B=-1), 1), (dict(T=-2), 1), (dict(max_rows=-1), 1), (dict(max_kv=-1), 1),
    (dict(Hq=3), 1), (dict(Hq=0), 1), (dict(Hkv=0), 1), (dict(ldq=255), 1), (dict(ldq=248), 1),
    (dict(ldo=260), 1), (dict(sm=float("nan")), 1), (dict(sm=float("inf")), 1),
    (dict(Q=P + 8), 1), (dict(O=P + 2), 1), (dict(ws=P + 4), 1), (dict(D=80), 2),
    (dict(B=70000), 2), (dict(B=40000), 2), (dict(T=1 << 25, max_rows=1 << 25), 2),
    (dict(max_kv=(1 << 30) + 1), 2),
    (dict(B=3000, T=1 << 20, max_rows=1 << 20), 2),
    (dict(B=0), 0), (dict(T=0), 0), (dict(max_rows=0), 0),
    (dict(max_kv=1 << 20, ws=None), 1), (dict(max_kv=1 << 20, wbytes=1000), 1),   # a workspace
]


@pytest.mark.parametrize("kw,status", BOTH + [
    (dict(table=None), 1), (dict(codes=None), 1), (dict(scales=None), 1), (dict(max_pages=0), 1),
    (dict(num_pages=-1), 1), (dict(codes=P + 4), 1),
])
def test_cache_attention_refusals(r, kw, status):
    assert _status(r, "rudder_cache_attention", CACHE, kw) == status


@pytest.mark.parametrize("kw,status", BOTH + [
    (dict(K=None), 1), (dict(V=None), 1), (dict(kv_start=None), 1), (dict(Tkv=-1), 1),
    (dict(ldk=100), 1), (dict(ldv=129), 1), (dict(K=P + 2), 1), (dict(V=P + 4), 1),
])
def test_cross_attention_refusals(r, kw, status):
    assert _status(r, "rudder_cross_attention", CROSS, kw) == status


def test_binding_checks_tensors(r):
    """Types, sizes and layouts of tensors are checked against the sizes passed."""
    T, H, D = 4, 2, 64
    i32 = torch.zeros(8, dtype=torch.int32)
    q = torch.zeros(T, H, D, dtype=torch.bfloat16)
    codes = torch.zeros(3, H, 2, 64 * D, dtype=torch.int8)
    scales = torch.zeros(3, H, 2)
    ok = dict(Q=q, row_start=i32, kv_len=i32, page_table=i32, codes=codes, scales=scales, B=2,
              T=T, max_rows=2, max_kv=100, max_pages=2, num_pages=3, Hq=H, Hkv=H, D=D, sm=0.1,
              causal=True, workspace=None, O=q.clone(), stream=0)
    # addresses pass as they are: what is under test is the one tensor
    addresses = {k: P for k in ("Q", "row_start", "kv_len", "page_table", "codes", "scales", "O")}
    for kw in (dict(Q=q.float()), dict(Q=q[:3]), dict(Q=q.transpose(0, 1)), dict(Q=q[..., ::2]),
               dict(row_start=i32.long()), dict(row_start=i32[:2]), dict(kv_len=i32[:1]),
               dict(page_table=i32[:3]), dict(page_table=i32[::2]), dict(codes=codes[:2]),
               dict(scales=scales[:2]), dict(scales=scales.double()), dict(O=q[:2]),
               dict(Q=q, ldq=2 * H * D)):
        with pytest.raises(ValueError, match="expected at least"):
            r.rudder_cache_attention(**{**ok, **addresses, **kw})
    with pytest.raises(ValueError, match="Wq.*expected at least"):
        r.rudder_matvec_w4(P, None, torch.zeros(100, dtype=torch.uint8), P, None, None, T, 32, 128,
                           64, 1, P, stream=0)
    # host memory is not taken for device memory
    for name in ("Q", "row_start", "codes", "O"):
        with pytest.raises(ValueError, match=f"{name}: not on a GPU"):
            r.rudder_cache_attention(**{**ok, **addresses, name: ok[name]})
    with pytest.raises(r.RudderError) as e:
        r.rudder_cache_attention(**{**ok, **addresses, "sm": float("nan")})
    assert e.value.status == r.RUDDER_ERR_INVALID_ARG


def test_binding_checks_arguments(r):
    """What is neither a tensor nor an address, sizes that are no 32-bit integers, tensors without
    memory and wrong argument counts are Python errors, and nothing is called."""
    ok = dict(X=P, stream_id=None, Wq=P, g_scale=P, comp_a=None, comp_b=None, M=0, N=64, K=128,
              group=64, S=1, Y=P, stream=0)
    r.rudder_matvec_w4(**ok)
    for kw, error in ((dict(X="rows"), TypeError), (dict(X=3.5), TypeError),
                      (dict(M=1 << 32), OverflowError), (dict(N=-(1 << 40)), OverflowError),
                      (dict(K=128.0), TypeError), (dict(X=-1 << 70), OverflowError),
                      (dict(X=torch.empty(0, 128, dtype=torch.bfloat16, device="meta")),
                       ValueError)):
        with pytest.raises(error):
            r.rudder_matvec_w4(**{**ok, **kw})
    with pytest.raises(TypeError):
        r._load_bind().matvec_w4(P, None)
    with pytest.raises(ImportError):
        r._load_bind().use("/nowhere/librudder.so")
    r.rudder_matvec_w4(**ok)


@pytest.mark.parametrize("sm,status", [(3e38, 1), (-3e38, 1), (2.0 ** 127, 0), (-2.0 ** 127, 0)])
def test_largest_softmax_scales(r, sm, status):
    """The kernels' scale is sm * log2(e): what would make it infinite is refused."""
    for name, args in (("rudder_cache_attention", CACHE), ("rudder_cross_attention", CROSS)):
        assert _status(r, name, args, dict(sm=sm, B=0)) == status


def _calls(r):
    """Every call of the operators between the linears with addresses in all places, and the names
    of its device arrays."""
    T, H, D, P_ = 4, 2, 64, P
    row = dict(row_start=P_, B=2, T=T, max_rows=2)
    cache = dict(page_table=P_, codes=P_, scales=P_, max_pages=2, num_pages=3)
    return [
        (r.rudder_quantize_weights_grouped, dict(W=P_, K=128, N=0, group=64, Wq=P_, g_scale=P_),
         ("W", "Wq", "g_scale")),
        (r.rudder_matvec_w4,
         dict(X=P_, stream_id=P_, Wq=P_, g_scale=P_, comp_a=P_, comp_b=P_, M=0, N=64, K=128,
              group=64, S=1, Y=P_), ("X", "stream_id", "Wq", "g_scale", "comp_a", "comp_b", "Y")),
        (r.rudder_cache_append, dict(K=P_, V=P_, pos=P_, Hkv=H, D=D, **{**row, "B": 0}, **cache),
         ("K", "V", "row_start", "pos", "page_table", "codes", "scales")),
        (r.rudder_cache_dequant, dict(codes=P_, scales=P_, pages=P_, n=0, num_pages=3, Hkv=H, D=D,
                                      K_out=P_, V_out=P_),
         ("codes", "scales", "pages", "K_out", "V_out")),
        (r.rudder_cache_attention,
         dict(Q=P_, kv_len=P_, max_kv=100, Hq=H, Hkv=H, D=D, sm=0.1, causal=True, workspace=P_,
              O=P_, **{**row, "B": 0}, **cache),
         ("Q", "row_start", "kv_len", "page_table", "codes", "scales", "workspace", "O")),
        (r.rudder_cross_attention,
         dict(Q=P_, K=P_, V=P_, kv_start=P_, kv_len=P_, Tkv=T, max_kv=100, Hq=H, Hkv=H, D=D,
              sm=0.1, workspace=P_, O=P_, **{**row, "B": 0}),
         ("Q", "K", "V", "row_start", "kv_start", "kv_len", "workspace", "O")),
    ]


def _like(name, device):
    """A tensor for that argument, large enough, of a device that need not be there."""
    from torch._subclasses.fake_tensor import FakeTensorMode
    kind = {"Wq": torch.uint8, "stream_id": torch.uint8, "workspace": torch.uint8,
            "comp_a": torch.float32, "comp_b": torch.float32, "scales": torch.float32,
            "K_out": torch.float32, "V_out": torch.float32, "codes": torch.int8,
            "row_start": torch.int32, "pos": torch.int32, "page_table": torch.int32,
            "kv_len": torch.int32, "kv_start": torch.int32, "pages": torch.int32}
    shape = ((4, 2, 64) if name in ("Q", "K", "V", "O") else (1 << 20,))
    with FakeTensorMode(allow_non_fake_inputs=True):
        return torch.empty(shape, dtype=kind.get(name, torch.bfloat16), device=device)


def test_binding_refuses_tensors_of_another_device(r, monkeypatch):
    """Every device array has to lie on the current device, whether a stream is given or not."""
    monkeypatch.setattr(r, "_get_device", lambda: 0)
    monkeypatch.setattr(r, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    for call, args, names in _calls(r):
        for name in names:
            for stream in ({}, {"stream": 0}):
                with pytest.raises(ValueError, match=f"{name}: on cuda:1.*cuda:0"):
                    call(**{**args, **stream, name: _like(name, "cuda:1")})
            # one of the current device passes the binding; without memory it is a null pointer
            try:
                call(**{**args, name: _like(name, "cuda:0")})
            except r.RudderError as e:
                assert "null pointer" in str(e) or "compensation" in str(e)

    class Stream:
        cuda_stream, device_index = 0, 1

    for call, args, _ in _calls(r):
        with pytest.raises(ValueError, match="stream of cuda:1.*cuda:0"):
            call(**args, stream=Stream())


def test_conveniences_check_shapes(r):
    """What the allocating forms take their sizes from has to agree: the rows' heads and channels
    with the cache's, also where there is nothing to do, and the weights and scales with the
    product's sizes and group."""
    bf16, i32 = torch.bfloat16, torch.int32
    q, k = torch.zeros(5, 4, 64, dtype=bf16), torch.zeros(5, 2, 64, dtype=bf16)
    rows, two = torch.zeros(3, dtype=i32), torch.zeros(2, dtype=i32)
    table = torch.zeros(2, 3, dtype=i32)
    for heads, D in ((4, 64), (2, 128), (4, 128), (1, 64)):
        cache = r.new_cache(3, heads, D, device="cpu")
        for n in (5, 0):
            with pytest.raises(ValueError, match="codes.*2 heads of 64 channels"):
                r.cache_append(k[:n], k[:n], rows, two, table, 5, *cache)
    for n in (5, 0):
        cache = r.new_cache(3, 2, 128, device="cpu")
        with pytest.raises(ValueError, match="codes.*2 heads of 64 channels"):
            r.cache_attention(q[:n], rows, two, table, *cache, 5, 100, 0.1)
        flat = (cache[0].view(3, 2, -1), cache[1])
        with pytest.raises(ValueError, match="codes.*2 heads of 64 channels"):
            r.cache_attention(q[:n], rows, two, table, *flat, 5, 100, 0.1)
    r._check_cache(r.new_cache(3, 2, 64, device="cpu")[0].view(3, -1), 2, 64)    # pages in a row
    x = torch.zeros(3, 256, dtype=bf16)
    for K, N, group in ((256, 48, 32), (256, 48, 128), (256, 64, 64), (128, 48, 64),
                        (512, 48, 64)):
        Wq = torch.zeros(r.grouped_weight_bytes(K, N), dtype=torch.uint8)
        gs = torch.zeros(r.grouped_scale_count(K, N, group), dtype=bf16)
        with pytest.raises(ValueError, match="K=256, N=48, group=64"):
            r.matvec_w4(x, Wq, gs, 48, 64)
        with pytest.raises(ValueError, match="K=256, N=48, group=64"):
            r.matvec_w4(x[:0], Wq, gs, 48, 64)


def test_workspace_bound_holds_for_smaller_sizes(r):
    """A buffer for the largest sizes serves every smaller call, though single calls' needs do not
    grow with their sizes."""
    import random
    assert (r.attention_workspace_bytes(2, 8192, 4096, 16384, 16, 16, 128) <
            r.attention_workspace_bytes(2, 2, 1, 16384, 16, 16, 128))
    rng = random.Random(7)
    grow = lambda lo, hi: int(round(lo * (hi / lo) ** rng.random()))
    for _ in range(400):
        D, Hkv = rng.choice([64, 128]), rng.choice([1, 2, 5, 8, 16, 48, 128])
        Hq = Hkv * rng.choice([1, 2, 3, 8, 16, 17])
        B, rows, kv = grow(1, 300), grow(1, 5000), grow(1, 200000)
        T = grow(1, B * rows)
        if min(rows, T) * Hq > 1 << 26:
            continue
        bound = r.attention_workspace_bound(B, T, rows, kv, Hq, Hkv, D)
        # a round of partial rows, or three pieces of 16 rows a sequence and head
        assert bound <= max(98304, 16 * max(1364, 3 * B * Hkv)) * (D + 2) * 4
        for _ in range(60):
            b, m, n = rng.randint(1, B), min(rows, grow(1, rows)), min(kv, grow(1, kv))
            t = rng.choice([T, rng.randint(1, T)])
            need = r.attention_workspace_bytes(b, t, m, n, Hq, Hkv, D)
            assert need <= bound, (b, t, m, n, Hq, Hkv, D)
            assert r.attention_workspace_bound(b, t, m, n, Hq, Hkv, D) <= bound
    for bad in ((1, 1, 1, 100, 15, 2, 64), (1, 1, 1, 100, 4, 2, 96), (-1, 1, 1, 100, 4, 2, 64),
                (1, 1, 1, -1, 4, 2, 64)):
        assert r.attention_workspace_bound(*bad) == 0
