"""GPU parity of matmul_i8 against exact integer products (bounds derived in oracle/norm.py), and of the
8-bit path run as it is used: chunk vectors -> norm -> 8 bits -> projection -> upsampling."""
import numpy as np
import pytest

from oracle import norm as o

pytestmark = pytest.mark.gpu


def _operand(rng, R, K, pad=None):
    """int8 rows inside a buffer padded with 77 behind each row (bytes that must not count)."""
    import torch
    ld = max(16, (K + 15) // 16 * 16 if pad is None else pad)
    v = rng.integers(-128, 128, (R, K)).astype(np.int8)
    buf = torch.full((R, ld), 77, dtype=torch.int8, device="cuda")
    buf[:, :K] = torch.from_numpy(v).cuda()
    return v, buf[:, :K]


def _scale(rng, n):
    return (rng.uniform(0.01, 0.03, n) * rng.choice([-1, 1], n)).astype(np.float32)


def _case(rng, M, N, K, T, bias, pad=None, out=None, st=None):
    import dynamic_byte_chunking_b200 as dbc
    import torch
    a, at = _operand(rng, M, K, pad)
    b, bt = _operand(rng, N, K, pad)
    sa, sb = _scale(rng, M), _scale(rng, N)
    bv = None if bias is None else o.store(rng.standard_normal(N).astype(np.float32), bias)
    dt = torch.bfloat16 if T == "bf16" else torch.float32
    bd = None if bv is None else torch.from_numpy(bv).cuda().to(torch.bfloat16 if bias == "bf16" else torch.float32)
    got = dbc.matmul_i8(at, torch.from_numpy(sa).cuda(), bt, torch.from_numpy(sb).cuda(), bias=bd, out_dtype=dt,
                        out=out, dev_status=st)
    ref = o.matmul_i8(a, sa.astype(np.float64), b, sb.astype(np.float64), bv)
    g = got.double().cpu().numpy()
    assert g.shape == ref.shape
    bound = o.matmul_i8_bound(ref, bv, T)
    bad = ~(np.abs(g - ref) <= bound)
    assert not bad.any(), f"{M}x{N}x{K} {T}: {bad.sum()} off, worst {np.max(np.abs(g - ref) / bound):.2f}, first {np.argwhere(bad)[:4].tolist()}"


SIZES = [1, 2, 3, 4, 5, 7, 8, 9, 15, 16, 17, 31, 32, 33, 48, 63, 64, 65, 100, 127, 128, 129, 200, 255, 256, 257, 300]


@pytest.mark.parametrize("M", SIZES)
def test_rows(M):
    """Every row count around the tile edges, with odd and even channel counts and depths."""
    import torch
    rng = np.random.default_rng(M)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for k, (N, K) in enumerate([(1, 1), (8, 16), (77, 100), (128, 128), (130, 257), (256, 512), (513, 96), (1000, 1536)]):
        _case(rng, M, N, K, "bf16" if k % 2 else "f32", [None, "bf16", "f32"][k % 3], st=st)
    assert st.item() == 0


@pytest.mark.parametrize("N", SIZES)
def test_channels(N):
    import torch
    rng = np.random.default_rng(1000 + N)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for k, (M, K) in enumerate([(1, 300), (6, 64), (40, 1000), (150, 128), (520, 272)]):
        _case(rng, M, N, K, "f32" if k % 2 else "bf16", [None, "bf16", "f32"][k % 3], st=st)
    assert st.item() == 0


@pytest.mark.parametrize("K", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 96, 127, 128, 129, 255, 256, 257, 640, 1023, 1024,
                               1025, 4096, 10000])
def test_depths(K):
    import torch
    rng = np.random.default_rng(2000 + K)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for M, N in [(1, 40), (4, 130), (20, 33), (130, 70), (300, 264)]:
        _case(rng, M, N, K, "f32", "f32", st=st)
    assert st.item() == 0


@pytest.mark.parametrize("M,N,K", [(1, 8192, 2048), (3, 20000, 513), (16, 4096, 8192), (61, 1543, 1531), (64, 256, 16384),
                                   (2500, 1536, 512), (1111, 2222, 777), (4096, 4096, 1024), (20000, 64, 64),
                                   (33, 40000, 128)])
def test_larger(M, N, K):
    import torch
    rng = np.random.default_rng(M + N + K)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    _case(rng, M, N, K, "bf16", "bf16", st=st)
    assert st.item() == 0


@pytest.mark.parametrize("M", [1, 5, 40, 200])
def test_largest_sums_are_exact(M):
    """All operands -128 at the largest depth: the sums reach 131071 * 16384 = 2^31 - 16384."""
    import dynamic_byte_chunking_b200 as dbc
    import torch
    K, N = 131071, 136
    a = torch.full((M, K + 1), -128, dtype=torch.int8, device="cuda")[:, :K]
    b = torch.full((N, K + 1), -128, dtype=torch.int8, device="cuda")[:, :K]
    b[1] = 127
    one = torch.ones(max(M, N), device="cuda")
    out = dbc.matmul_i8(a, one[:M], b, one[:N], out_dtype=torch.float32).double().cpu().numpy()
    assert np.array_equal(out[:, 0], np.full(M, float(np.float32(131071 * 16384))))
    assert np.array_equal(out[:, 1], np.full(M, float(np.float32(-131071 * 16256))))


@pytest.mark.parametrize("M", [1, 9, 70, 300])
@pytest.mark.parametrize("T", ["bf16", "f32"])
def test_outputs_inside_wider_buffers(M, T):
    """Strided outputs, even and odd, on and off the 16-byte grid: nothing outside them is written."""
    import torch
    rng = np.random.default_rng(M)
    dt = torch.bfloat16 if T == "bf16" else torch.float32
    for N, ld, c0, pad in [(64, 80, 8, 160), (129, 200, 3, 144), (256, 257, 1, 272), (300, 304, 0, 144)]:
        buf = torch.full((M + 2, ld), 5.0, dtype=dt, device="cuda")
        _case(rng, M, N, 130, T, "bf16", pad=pad, out=buf[1:M + 1, c0:c0 + N])
        buf[1:M + 1, c0:c0 + N] = 5.0
        assert bool((buf == 5.0).all())


def test_unaligned_and_transposed_operands_are_copied():
    import dynamic_byte_chunking_b200 as dbc
    import torch
    rng = np.random.default_rng(5)
    for M in (1, 6, 90):
        a = torch.from_numpy(rng.integers(-128, 128, (M, 75)).astype(np.int8)).cuda()     # rows of 75 bytes
        b = torch.from_numpy(rng.integers(-128, 128, (75, 50)).astype(np.int8)).cuda().t()
        out = dbc.matmul_i8(a, torch.ones(M, device="cuda"), b, torch.ones(50, device="cuda"), out_dtype=torch.float32)
        assert torch.equal(out.double(), a.double() @ b.double().t())


def test_empty_and_refused():
    import dynamic_byte_chunking_b200 as dbc
    import torch
    i8 = lambda *s: torch.ones(*s, dtype=torch.int8, device="cuda")  # noqa: E731
    f = lambda n: torch.ones(n, device="cuda")  # noqa: E731
    assert dbc.matmul_i8(i8(0, 32), f(0), i8(4, 32), f(4)).shape == (0, 4)
    assert dbc.matmul_i8(i8(4, 32), f(4), i8(0, 32), f(0)).shape == (4, 0)
    bias = torch.arange(300, device="cuda", dtype=torch.float32)
    for M in (1, 7, 200):
        out = dbc.matmul_i8(i8(M, 0), f(M), i8(300, 0), f(300), bias=bias, out_dtype=torch.float32)
        assert torch.equal(out, bias.expand(M, 300))
        assert not dbc.matmul_i8(i8(M, 0), f(M), i8(300, 0), f(300)).any()
    rows = 65535 * 128 + 5                               # more token tiles than a grid's second dimension
    out = dbc.matmul_i8(i8(rows, 0), f(rows), i8(2, 0), f(2), bias=bias[1:3], out_dtype=torch.float32)
    assert torch.equal(out, bias[1:3].expand(rows, 2))
    with pytest.raises(ValueError):
        dbc.matmul_i8(i8(4, 32), f(4), i8(4, 48), f(4))
    with pytest.raises(ValueError):
        dbc.matmul_i8(i8(4, 32), f(3), i8(4, 32), f(4))
    with pytest.raises(ValueError):
        dbc.matmul_i8(i8(4, 32), f(4), i8(4, 32), f(4), bias=f(5))
    with pytest.raises(ValueError):
        dbc.matmul_i8(i8(4, 32), f(4), i8(4, 32), f(4), out=torch.zeros(4, 5, device="cuda"))
    with pytest.raises(TypeError):
        dbc.matmul_i8(f(32).view(1, 32), f(1), i8(4, 32), f(4))
    with pytest.raises(TypeError):
        dbc.matmul_i8(i8(4, 32), f(4), i8(4, 32), f(4), out_dtype=torch.float16)
    with pytest.raises(dbc.DbcError):
        dbc.matmul_i8(i8(1, 131072), f(1), i8(1, 131072), f(1))


def test_non_finite_scales_reach_their_rows_only():
    import dynamic_byte_chunking_b200 as dbc
    import torch
    for M in (3, 80, 300):
        a, b = torch.ones(M, 64, dtype=torch.int8, device="cuda"), torch.ones(140, 64, dtype=torch.int8, device="cuda")
        sa, sb = torch.ones(M, device="cuda"), torch.ones(140, device="cuda")
        sa[1] = float("nan")
        out = dbc.matmul_i8(a, sa, b, sb, out_dtype=torch.float32)
        assert bool(out[1].isnan().all()) and bool((out[[0] + list(range(2, M))] == 64).all())


@pytest.mark.parametrize("M", [2, 50, 400])
def test_streams_and_graphs(M):
    import dynamic_byte_chunking_b200 as dbc
    import torch
    torch.manual_seed(M)
    b = torch.randint(-127, 128, (520, 256), device="cuda", dtype=torch.int8)
    sb = torch.rand(520, device="cuda")
    sides = [torch.cuda.Stream() for _ in range(2)]
    graphs = []
    for side in sides:
        a = torch.zeros(M, 256, dtype=torch.int8, device="cuda")
        sa = torch.ones(M, device="cuda")
        side.wait_stream(torch.cuda.current_stream())
        dbc.matmul_i8(a, sa, b, sb, stream=side)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            out = dbc.matmul_i8(a, sa, b, sb, out_dtype=torch.float32)
        graphs.append((g, a, sa, out, side))
    for _ in range(3):
        data = [torch.randint(-127, 128, (M, 256), device="cuda", dtype=torch.int8) for _ in graphs]
        torch.cuda.synchronize()
        for (g, a, sa, out, side), v in zip(graphs, data):
            with torch.cuda.stream(side):
                a.copy_(v)
                g.replay()
        torch.cuda.synchronize()
        for (g, a, sa, out, side), v in zip(graphs, data):
            ref = (v.double() @ b.double().t()) * sb.double()
            assert torch.all((out.double() - ref).abs() <= ref.abs() * 4 * o.U32)


@pytest.mark.parametrize("rows,T,d,d_g", [(2, 1024, 256, 256), (3, 777, 512, 1536)])
def test_chunk_path_in_8_bits(rows, T, d, d_g):
    """Coding rate -> Top-K -> chunk vectors -> norm, 8 bits, projection -> upsampling -> next norm."""
    import dynamic_byte_chunking_b200 as dbc
    import torch
    torch.manual_seed(rows)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    H = (torch.randn(rows, T, d, device="cuda") / d ** 0.5).bfloat16()
    dR = dbc.chunk_coding_rate(H, 0.5, dev_status=st)
    K = T // 4
    idx, io = dbc.chunk_topk_select(dR, K, rows=rows, T=T, dev_status=st)
    w = (1 + 0.1 * torch.randn(d, device="cuda")).bfloat16()
    W = (torch.randn(d, d_g, device="cuda") / d ** 0.5).bfloat16()
    Wq, Ws = dbc.quantize_rows_i8(W.t(), dev_status=st)
    Z, G = dbc.chunk_project_i8(H, idx, io, w, Wq, Ws, rows=rows, T=T, dev_status=st)
    z = H.view(rows, T, d).gather(1, idx.view(rows, K, 1).expand(-1, -1, d)).reshape(-1, d)
    assert torch.equal(Z, z)
    zn, wn = z.double().cpu().numpy(), w.double().cpu().numpy()
    q, sc = o.rms_norm_i8(zn, wn, 1e-6)
    wq, wsc = o.quantize_rows_i8(W.t().double().cpu().numpy())
    assert np.array_equal(Wq.cpu().numpy(), wq)
    ref = o.matmul_i8(q, sc, wq, wsc, None)
    g = G.double().cpu().numpy()
    # the two scales are off by their own roundings, then the product's bound
    slack = np.abs(ref) * (o.CHAIN / 2 + o.OPS + 2) * o.U32
    assert np.all(np.abs(g - ref) <= o.matmul_i8_bound(ref, None, "bf16") + slack)
    # and it stands for the unquantised projection: half a code of each operand per product, at random signs
    full = o.rms_norm(zn, wn, 1e-6) @ W.double().cpu().numpy()
    y = o.rms_norm(zn, wn, 1e-6)
    step = 0.5 * (sc[:, None] * np.abs(W.double().cpu().numpy()).sum(0) + np.abs(y).sum(1)[:, None] * wsc +
                  0.5 * d * sc[:, None] * wsc)
    assert np.all(np.abs(g - full) <= step + np.abs(full) * 2.0 ** -8 + slack)
    Wb = (torch.randn(16, d_g, d, device="cuda") / d_g ** 0.5).bfloat16()
    S = dbc.chunk_upsample(G, H, idx, io, Wb, rows=rows, T=T, dev_status=st)
    y2, s2 = dbc.rms_norm(S, w, eps=1e-6, residual=H.view(-1, d).float(), out_dtype=torch.bfloat16, dev_status=st)
    ref2 = o.rms_norm(s2.double().cpu().numpy(), wn, 1e-6)
    assert np.all(np.abs(y2.double().cpu().numpy() - ref2) <= o.rms_norm_bound(ref2, "bf16"))
    assert st.item() == 0


@pytest.mark.parametrize("M,N,K", [(3, 40, 512), (70, 300, 64), (16, 300, 2048), (200, 256, 4096), (1500, 1536, 256)])
def test_scales_far_from_one(M, N, K):
    """Results inside fp32's range from scales whose product with the sum alone is not: the largest with sums of 2^22
    and more, the smallest (subnormal) with the largest."""
    import dynamic_byte_chunking_b200 as dbc
    import torch
    rng = np.random.default_rng(M)
    a, at = _operand(rng, M, K)
    b, bt = _operand(rng, N, K)
    a[::2], b[::2] = 127, 127
    at.copy_(torch.from_numpy(a)), bt.copy_(torch.from_numpy(b))
    ea = np.where(np.arange(M) % 3 == 0, 120, np.where(np.arange(M) % 3 == 1, -135, 3))
    for eb in (-110, 0, 100):
        sa = (rng.uniform(1, 2, M) * 2.0 ** ea).astype(np.float32)
        sb = (rng.uniform(1, 2, N) * 2.0 ** eb).astype(np.float32)
        for bias in (None, "f32"):
            bv = None if bias is None else o.store(rng.standard_normal(N).astype(np.float32), "f32")
            out = dbc.matmul_i8(at, torch.from_numpy(sa).cuda(), bt, torch.from_numpy(sb).cuda(), out_dtype=torch.float32,
                                bias=None if bv is None else torch.from_numpy(bv).float().cuda())
            ref = o.matmul_i8(a, sa.astype(np.float64), b, sb.astype(np.float64), bv)
            g = out.double().cpu().numpy()
            keep = np.abs(ref) < 2.0 ** 127
            bound = o.matmul_i8_bound(ref, bv, "f32") + o.TINY["f32"]
            assert np.all(np.abs(g - ref)[keep] <= bound[keep]), (eb, bias)
            assert np.all(np.isinf(g[np.abs(ref) > 2.0 ** 128 * (1 + 2.0 ** -20)]))


# From M > 128 and 24 tiles of 256 x 256 on the wide kernel runs, below it the split one.
@pytest.mark.parametrize("bias", [None, "bf16", "f32"])
@pytest.mark.parametrize("T", ["bf16", "f32"])
def test_wide_kernel(T, bias):
    """6 x 6 tiles with ragged edges; outputs packed, and inside wider buffers on (tile stores) and off the 16-byte
    grid (element stores; a width that ends inside 16 bytes among them), whose guards stay; depths shorter than a
    step and ending inside one."""
    import torch
    rng = np.random.default_rng(7)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    dt = torch.bfloat16 if T == "bf16" else torch.float32
    M = 1300
    for N, ld, c0 in [(1283, None, 0), (1288, None, 0), (1283, 1304, 8), (1288, 1304, 8), (1300, 1312, 8),
                      (1288, 1297, 3)]:
        for K in (1, 17, 33, 129, 777):
            if ld is None:
                _case(rng, M, N, K, T, bias, st=st)
                continue
            buf = torch.full((M + 2, ld), 5.0, dtype=dt, device="cuda")
            _case(rng, M, N, K, T, bias, out=buf[1:M + 1, c0:c0 + N], st=st)
            buf[1:M + 1, c0:c0 + N] = 5.0
            assert bool((buf == 5.0).all())
    assert st.item() == 0


# tiles of 128 tokens, depth not split and split in two (20 and 18 wide tiles); tiles of 64 and 32 tokens with the
# depth in 4 and 2; both sides of the switch to the wide kernel (23 and 24 tiles) with a deep product
@pytest.mark.parametrize("M,N,K", [(1280, 1000, 100), (600, 1536, 777), (300, 1000, 2000), (260, 1000, 1100), (5888, 256, 2048),
                                   (5889, 256, 2048), (130, 5888, 1500), (257, 3100, 1500)])
@pytest.mark.parametrize("T,bias", [("f32", "bf16"), ("bf16", "f32"), ("f32", None)])
def test_split_kernel_and_the_switch(M, N, K, T, bias):
    import torch
    rng = np.random.default_rng(M + K)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    _case(rng, M, N, K, T, bias, st=st)
    assert st.item() == 0


def test_wide_kernel_largest_sums():
    """Sums of 2^31 - 16384, and a NaN scale that reaches its row (or channel) only."""
    import dynamic_byte_chunking_b200 as dbc
    import torch
    K, M, N = 131071, 1300, 1283
    a = torch.full((M, K + 1), -128, dtype=torch.int8, device="cuda")[:, :K]
    b = torch.full((N, K + 1), -128, dtype=torch.int8, device="cuda")[:, :K]
    b[1] = 127
    sa, sb = torch.ones(M, device="cuda"), torch.ones(N, device="cuda")
    out = dbc.matmul_i8(a, sa, b, sb, out_dtype=torch.float32)
    assert bool((out[:, 1] == float(np.float32(-131071 * 16256))).all())
    out[:, 1] = out[0, 0]
    assert bool((out == float(np.float32(131071 * 16384))).all())
    sa[700], sb[600] = float("nan"), float("nan")
    out = dbc.matmul_i8(a, sa, b, sb, out_dtype=torch.float32)
    assert bool(out[700].isnan().all()) and bool(out[:, 600].isnan().all())
    out[700], out[:, 600] = 0, 0
    assert not bool(out.isnan().any())


def test_wide_kernel_on_two_streams_and_in_graphs():
    import dynamic_byte_chunking_b200 as dbc
    import torch
    torch.manual_seed(3)
    M, N, K = 1500, 1536, 256
    b = torch.randint(-127, 128, (N, K), device="cuda", dtype=torch.int8)
    sb = torch.rand(N, device="cuda")
    graphs = []
    for _ in range(2):
        side = torch.cuda.Stream()
        a, sa = torch.zeros(M, K, dtype=torch.int8, device="cuda"), torch.rand(M, device="cuda")
        side.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            out = dbc.matmul_i8(a, sa, b, sb, out_dtype=torch.float32)
        graphs.append((g, a, sa, out, side))
    for _ in range(3):
        data = [torch.randint(-127, 128, (M, K), device="cuda", dtype=torch.int8) for _ in graphs]
        torch.cuda.synchronize()
        for (g, a, sa, out, side), v in zip(graphs, data):
            with torch.cuda.stream(side):
                a.copy_(v)
                g.replay()
                eager = dbc.matmul_i8(a, sa, b, sb, out_dtype=torch.float32)
            side.synchronize()
            assert torch.equal(out, eager)
        for (g, a, sa, out, side), v in zip(graphs, data):
            ref = (v.double() @ b.double().t()) * sa.double()[:, None] * sb.double()
            assert torch.all((out.double() - ref).abs() <= ref.abs() * 4 * o.U32)


@pytest.mark.parametrize("N", [16400, 16401])
def test_outputs_past_32_bits(N):
    """More than 2^31 outputs (tile and element stores): the last rows as a call of their own gives them."""
    import dynamic_byte_chunking_b200 as dbc
    import torch
    torch.manual_seed(N)
    M, K = 140_000, 32
    a = torch.randint(-127, 128, (M, K), device="cuda", dtype=torch.int8)
    b = torch.randint(-127, 128, (N, K), device="cuda", dtype=torch.int8)
    sa, sb = torch.rand(M, device="cuda"), torch.rand(N, device="cuda")
    out = dbc.matmul_i8(a, sa, b, sb)
    for r in (slice(0, 40), slice(131_000, 131_040), slice(M - 40, M)):
        assert torch.equal(out[r], dbc.matmul_i8(a[r], sa[r], b, sb))
