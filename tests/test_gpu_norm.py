"""GPU parity of rms_norm, rms_norm_i8, quantize_rows_i8 and rms_norm_backward against the float64 oracle, with
the elementwise bounds that oracle/norm.py derives; 8-bit codes have to be equal."""
import numpy as np
import pytest

from oracle import norm as o

pytestmark = pytest.mark.gpu

EPS = 1e-6
# one thread, tiles and their edges, odd widths, every width class up to the limit
WIDTHS = [1, 2, 7, 8, 31, 64, 72, 100, 128, 136, 255, 256, 257, 264, 512, 520, 1000, 1024, 1032, 1536, 2048, 2056,
          2600, 4096, 4104, 5001, 8192, 8200, 16376, 16383, 16384]


def _rows(d):
    """Row counts: a few for wide rows, enough for several blocks for narrow ones."""
    return [1, 3, 37] if d > 2048 else [1, 2, 5, 333]


def _t(v, T, dev="cuda"):
    import torch
    return torch.from_numpy(np.ascontiguousarray(v)).to(dev).to(torch.bfloat16 if T == "bf16" else torch.float32)


def _np(t):
    return t.detach().double().cpu().numpy()


def _vals(rng, shape, T):
    return o.store(rng.standard_normal(shape).astype(np.float32), T)


def _weight(rng, d, T):
    return o.store((1 + 0.2 * rng.standard_normal(d)).astype(np.float32), T)


def _close(got, ref, bound, what):
    got = _np(got)
    assert got.shape == ref.shape, what
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.max(np.abs(got - ref) / bound):.2f} bounds"


def _status():
    import torch
    return torch.zeros(1, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("d", WIDTHS)
def test_rms_norm(d):
    import dynamic_byte_chunking_b200 as dbc
    import torch
    rng = np.random.default_rng(d)
    st = _status()
    for k, N in enumerate(_rows(d)):
        for T, TY, res in (("bf16", "bf16", True), ("f32", "bf16", k % 2 == 0), ("bf16", "f32", False), ("f32", "f32", True)):
            x = _vals(rng, (N, d), T)
            r = _vals(rng, (N, d), T) if res else None
            w = _weight(rng, d, "bf16" if k % 2 else "f32") if d % 3 else None
            s = o.residual_sum(x, r, T)
            y, sg = dbc.rms_norm(_t(x, T), None if w is None else _t(w, "bf16" if k % 2 else "f32"), eps=EPS,
                                 residual=None if r is None else _t(r, T),
                                 out_dtype=torch.bfloat16 if TY == "bf16" else torch.float32, dev_status=st)
            assert (sg is None) == (r is None)
            if r is not None:
                assert np.array_equal(_np(sg), s), (N, T)
            ref = o.rms_norm(s, w, EPS)
            _close(y, ref, o.rms_norm_bound(ref, TY), f"N={N} {T}->{TY}")
    assert st.item() == 0


@pytest.mark.parametrize("d", WIDTHS)
def test_rms_norm_i8_and_quantize(d):
    import dynamic_byte_chunking_b200 as dbc
    rng = np.random.default_rng(1000 + d)
    st = _status()
    for k, N in enumerate(_rows(d)):
        for T in ("bf16", "f32"):
            x = _vals(rng, (N, d), T)
            r = _vals(rng, (N, d), T) if k % 2 == 0 else None
            w = _weight(rng, d, "bf16") if d % 3 else None
            s = o.residual_sum(x, r, T)
            q, sc, sg = dbc.rms_norm_i8(_t(x, T), None if w is None else _t(w, "bf16"), eps=EPS,
                                        residual=None if r is None else _t(r, T), dev_status=st)
            qr, sr = o.rms_norm_i8(s, w, EPS)
            assert np.array_equal(q.cpu().numpy(), qr), (N, T)
            assert q.stride(0) % 16 == 0 or N == 1
            _close(sc, sr, np.abs(sr) * (o.CHAIN / 2 + o.OPS) * o.U32, f"scale N={N} {T}")
            if r is not None:
                assert np.array_equal(_np(sg), s)
            q, sc = dbc.quantize_rows_i8(_t(x, T), dev_status=st)
            qr, sr = o.quantize_rows_i8(x)
            assert np.array_equal(q.cpu().numpy(), qr), (N, T)
            _close(sc, sr, np.abs(sr) * 2 * o.U32, f"quantize scale N={N} {T}")
    assert st.item() == 0


@pytest.mark.parametrize("d", WIDTHS)
def test_rms_norm_backward(d):
    import dynamic_byte_chunking_b200 as dbc
    rng = np.random.default_rng(2000 + d)
    st = _status()
    for k, N in enumerate(_rows(d)):
        for TY, T, has in (("bf16", "bf16", True), ("f32", "bf16", False), ("bf16", "f32", False), ("f32", "f32", True)):
            s, dy = _vals(rng, (N, d), T), _vals(rng, (N, d), TY)
            ds = _vals(rng, (N, d), T) if has else None
            w = _weight(rng, d, "bf16") if (d + k) % 3 else None
            dx, dw = dbc.rms_norm_backward(_t(dy, TY), _t(s, T), None if w is None else _t(w, "bf16"), eps=EPS,
                                           dsum=None if ds is None else _t(ds, T), dev_status=st)
            rx, rw = o.rms_norm_backward(dy, s, w, EPS, ds)
            bx, bw = o.backward_bounds(dy, s, w, EPS, ds, T)
            _close(dx, rx, bx, f"dx N={N} {TY} {T}")
            _close(dw, rw, bw, f"dw N={N} {TY} {T}")
            none, nodw = dbc.rms_norm_backward(_t(dy, TY), _t(s, T), None if w is None else _t(w, "bf16"), eps=EPS,
                                               dsum=None if ds is None else _t(ds, T), want_dw=False)
            assert nodw is None and np.array_equal(_np(none), _np(dx))
    assert st.item() == 0


@pytest.mark.parametrize("N,d", [(20011, 64), (70001, 256), (9001, 1000), (3001, 4096)])
def test_many_rows(N, d):
    """More rows than the grid holds at once; dw from long sums, twice the same bits."""
    import dynamic_byte_chunking_b200 as dbc
    import torch
    rng = np.random.default_rng(N)
    x, r, dy = (_vals(rng, (N, d), "bf16") for _ in range(3))
    w = _weight(rng, d, "bf16")
    s = o.residual_sum(x, r, "bf16")
    xt, rt, dyt, wt = _t(x, "bf16"), _t(r, "bf16"), _t(dy, "bf16"), _t(w, "bf16")
    y, sg = dbc.rms_norm(xt, wt, eps=EPS, residual=rt)
    ref = o.rms_norm(s, w, EPS)
    _close(y, ref, o.rms_norm_bound(ref, "bf16"), "y")
    assert np.array_equal(_np(sg), s)
    q, sc, _ = dbc.rms_norm_i8(xt, wt, eps=EPS, residual=rt)
    qr, sr = o.rms_norm_i8(s, w, EPS)
    assert np.array_equal(q.cpu().numpy(), qr)
    dx, dw = dbc.rms_norm_backward(dyt, sg, wt, eps=EPS)
    rx, rw = o.rms_norm_backward(dy, s, w, EPS, None)
    bx, bw = o.backward_bounds(dy, s, w, EPS, None, "bf16")
    _close(dx, rx, bx, "dx")
    _close(dw, rw, bw, "dw")
    again = dbc.rms_norm_backward(dyt, sg, wt, eps=EPS)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


@pytest.mark.parametrize("T", ["bf16", "f32"])
@pytest.mark.parametrize("d", [40, 256, 1000, 2048])
def test_extreme_rows(T, d):
    """Zero rows, rows whose squares overflow or vanish in fp32, tiny maxima, exact halves under the code."""
    import dynamic_byte_chunking_b200 as dbc
    rng = np.random.default_rng(d)
    base = _vals(rng, (8, d), T)
    x = base.copy()
    x[0] = 0
    x[1] = o.store(base[1] * 2.0 ** 100, T)       # squares overflow
    x[2] = o.store(base[2] * 2.0 ** -90, T)       # squares vanish
    x[3] = o.store(base[3] * 2.0 ** -128, T)      # subnormal values
    x[4] = 0
    x[4, -1] = o.store(np.array(-3e38), T)
    x[5] = np.arange(d) % 128 - 0.5               # halves: p = j + 1/2 under a maximum of 127
    x[5, 0] = 127
    x[6] = -x[5]
    st = _status()
    w = o.store(2.0 ** rng.integers(-1, 1, d), T)
    for eps in (EPS, 1e-30):
        y, _ = dbc.rms_norm(_t(x, T), _t(w, T), eps=eps, dev_status=st)
        ref = o.rms_norm(x, w, eps)
        _close(y, ref, o.rms_norm_bound(ref, T), f"eps={eps}")
        q, sc, _ = dbc.rms_norm_i8(_t(x, T), _t(w, T), eps=eps, dev_status=st)
        qr, sr = o.rms_norm_i8(x, w, eps)
        assert np.array_equal(q.cpu().numpy(), qr)
        _close(sc, sr, np.abs(sr) * (o.CHAIN / 2 + o.OPS) * o.U32 + o.TINY["f32"], "scale")
        dy = _vals(rng, (8, d), T)
        dx, _ = dbc.rms_norm_backward(_t(dy, T), _t(x, T), _t(w, T), eps=eps, want_dw=False, dev_status=st)
        rx, _ = o.rms_norm_backward(dy, x, w, eps, None)
        bx, _ = o.backward_bounds(dy, x, w, eps, None, T)
        with np.errstate(over="ignore"):
            rx32 = rx.astype(np.float32)
        keep = np.isfinite(rx32)                   # a gradient above the type's range becomes an infinity
        got = _np(dx)
        assert np.all(np.abs(got - rx)[keep] <= bx[keep])
    q, sc = dbc.quantize_rows_i8(_t(x, T), dev_status=st)
    qr, sr = o.quantize_rows_i8(x)
    assert np.array_equal(q.cpu().numpy(), qr)
    _close(sc, sr, np.abs(sr) * 2 * o.U32 + o.TINY["f32"], "quantize scale")
    assert st.item() == 0


@pytest.mark.parametrize("d", [33, 256, 1536, 6000])
@pytest.mark.parametrize("T", ["bf16", "f32"])
def test_non_finite_rows_stay_alone(T, d):
    import dynamic_byte_chunking_b200 as dbc
    rng = np.random.default_rng(d)
    x = _vals(rng, (7, d), T)
    clean = x.copy()
    x[2, d // 2] = np.nan
    x[4, 0] = np.inf
    x[5, -1] = -np.inf
    x[5, 0] = np.nan
    good = [0, 1, 3, 6]
    st = _status()
    y, _ = dbc.rms_norm(_t(x, T), None, eps=EPS, dev_status=st)
    assert st.item() == 1 << dbc.ERR_NONFINITE
    yc, _ = dbc.rms_norm(_t(clean, T), None, eps=EPS)
    y, yc = _np(y), _np(yc)
    assert np.array_equal(y[good], yc[good])
    assert np.isnan(y[2]).all() and np.isnan(y[5]).all() and np.isnan(y[4, 0]) and not y[4, 1:].any()
    for call in (lambda s_: dbc.rms_norm_i8(_t(x, T), None, eps=EPS, dev_status=s_)[:2],
                 lambda s_: dbc.quantize_rows_i8(_t(x, T), dev_status=s_)):
        st = _status()
        q, sc = call(st)
        assert st.item() == 1 << dbc.ERR_NONFINITE
        q, sc = q.cpu().numpy(), _np(sc)
        assert not q[[2, 4, 5]].any() and np.isnan(sc[[2, 4, 5]]).all()
        assert np.isfinite(sc[good]).all() and np.array_equal(q[good], o.quantize_rows_i8(clean)[0][good])
    st = _status()
    dx, _ = dbc.rms_norm_backward(_t(clean, T), _t(x, T), None, eps=EPS, want_dw=False, dev_status=st)
    assert st.item() == 1 << dbc.ERR_NONFINITE
    dc, _ = dbc.rms_norm_backward(_t(clean, T), _t(clean, T), None, eps=EPS, want_dw=False)
    assert np.array_equal(_np(dx)[good], _np(dc)[good])


@pytest.mark.parametrize("T", ["bf16", "f32"])
@pytest.mark.parametrize("d,pad,shift", [(256, 64, 0), (256, 8, 8), (256, 3, 1), (1024, 1, 0), (100, 28, 5), (31, 1, 1),
                                         (4096, 24, 8), (2051, 2, 1)])
def test_strided_and_unaligned_rows(T, d, pad, shift):
    """Rows inside wider buffers, some off the 16-byte grid: same results, neighbours untouched."""
    import dynamic_byte_chunking_b200 as dbc
    import torch
    rng = np.random.default_rng(d + pad)
    N, ld = 9, d + pad + shift
    dt = torch.bfloat16 if T == "bf16" else torch.float32

    def inside(v):
        buf = torch.full((N, ld), 7.0, dtype=dt, device="cuda")
        view = buf[:, shift:shift + d]
        if v is not None:
            view.copy_(_t(v, T))
        return buf, view

    def kept(buf):
        b = buf.clone()
        b[:, shift:shift + d] = 7.0
        return bool((b == 7.0).all())

    x, r, dy, ds = (_vals(rng, (N, d), T) for _ in range(4))
    w = _weight(rng, d, T)
    xv, rv, dyv, dsv = (inside(v)[1] for v in (x, r, dy, ds))
    (sb, s), (yb, y), (xb, dx) = inside(None), inside(None), inside(None)
    dbc.rms_norm(xv, _t(w, T), eps=EPS, residual=rv, y=y, s=s)
    yr, sr = dbc.rms_norm(_t(x, T), _t(w, T), eps=EPS, residual=_t(r, T))
    assert torch.equal(s, sr) and kept(sb) and kept(yb)
    ref = o.rms_norm(o.residual_sum(x, r, T), w, EPS)
    _close(y, ref, o.rms_norm_bound(ref, T), "y")
    dbc.rms_norm_backward(dyv, s, _t(w, T), eps=EPS, dsum=dsv, dx=dx)
    rx, _ = o.rms_norm_backward(dy, _np(sr), w, EPS, ds)
    bx, _ = o.backward_bounds(dy, _np(sr), w, EPS, ds, T)
    _close(dx, rx, bx, "dx")
    assert kept(xb)
    qb = torch.full((N, ld), 99, dtype=torch.int8, device="cuda")
    q, sc, _ = dbc.rms_norm_i8(xv, _t(w, T), eps=EPS, residual=rv, q=qb[:, shift:shift + d])
    qr, _, _ = dbc.rms_norm_i8(_t(x, T), _t(w, T), eps=EPS, residual=_t(r, T))
    assert torch.equal(q, qr)
    qb[:, shift:shift + d] = 99
    assert bool((qb == 99).all())
    # a transposed and a broadcast input are copied first
    xt = _t(x, T).t().contiguous().t()
    one = _t(r[:1], T).expand(N, d)
    y2, s2 = dbc.rms_norm(xt, _t(w, T), eps=EPS, residual=one)
    y3, s3 = dbc.rms_norm(_t(x, T), _t(w, T), eps=EPS, residual=one.contiguous())
    assert torch.equal(y2, y3) and torch.equal(s2, s3)


@pytest.mark.parametrize("d", [96, 256, 257, 1536, 8192])
def test_in_place_forms(d):
    """s over residual or x, y over x, dx over s, dsum or dy."""
    import dynamic_byte_chunking_b200 as dbc
    import torch
    rng = np.random.default_rng(d)
    N = 301
    x, r, w = _t(_vals(rng, (N, d), "bf16"), "bf16"), _t(_vals(rng, (N, d), "bf16"), "bf16"), _t(_weight(rng, d, "bf16"), "bf16")
    y, s = dbc.rms_norm(x, w, eps=EPS, residual=r)
    r2, x2 = r.clone(), x.clone()
    y2, _ = dbc.rms_norm(x2, w, eps=EPS, residual=r2, s=r2, y=x2)
    assert torch.equal(y2, y) and torch.equal(r2, s) and y2 is x2
    x3 = x.clone()
    y3, _ = dbc.rms_norm(x3, w, eps=EPS, residual=r, s=x3)
    assert torch.equal(y3, y) and torch.equal(x3, s)
    q, sc, _ = dbc.rms_norm_i8(x, w, eps=EPS, residual=r)
    r4 = r.clone()
    q4, sc4, _ = dbc.rms_norm_i8(x, w, eps=EPS, residual=r4, s=r4)
    assert torch.equal(q4, q) and torch.equal(sc4, sc) and torch.equal(r4, s)
    dy, ds = _t(_vals(rng, (N, d), "bf16"), "bf16"), _t(_vals(rng, (N, d), "bf16"), "bf16")
    dx, dw = dbc.rms_norm_backward(dy, s, w, eps=EPS, dsum=ds)
    for k in range(3):
        c = [dy.clone(), s.clone(), ds.clone()]
        dx2, dw2 = dbc.rms_norm_backward(c[0], c[1], w, eps=EPS, dsum=c[2], dx=c[k])
        assert torch.equal(dx2, dx) and torch.equal(dw2, dw)


def test_shapes_and_empty_batches():
    import dynamic_byte_chunking_b200 as dbc
    import torch
    x = torch.randn(3, 5, 48, device="cuda")
    y, _ = dbc.rms_norm(x, eps=EPS)
    q, sc, s = dbc.rms_norm_i8(x, eps=EPS, residual=x)
    assert y.shape == x.shape and q.shape == x.shape and sc.shape == (3, 5) and s.shape == x.shape
    one, _ = dbc.rms_norm(x[0, 0], eps=EPS)
    assert torch.equal(one, y[0, 0])
    e = torch.empty(0, 64, device="cuda", dtype=torch.bfloat16)
    assert dbc.rms_norm(e)[0].shape == (0, 64) and dbc.quantize_rows_i8(e)[0].shape == (0, 64)
    dx, dw = dbc.rms_norm_backward(e, e)
    assert dx.shape == (0, 64) and not dw.any() and dw.shape == (64,)


def test_binding_refusals():
    import dynamic_byte_chunking_b200 as dbc
    import torch
    x = torch.zeros(4, 64, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        dbc.rms_norm(x, torch.ones(63, device="cuda"))
    with pytest.raises(TypeError):
        dbc.rms_norm(x, torch.ones(64, device="cuda", dtype=torch.float16))
    with pytest.raises(TypeError):
        dbc.rms_norm(x.half())
    with pytest.raises(ValueError):
        dbc.rms_norm(x, residual=x.float())
    with pytest.raises(ValueError):
        dbc.rms_norm(x, residual=x[:2])
    with pytest.raises(ValueError):
        dbc.rms_norm(x, s=x)
    with pytest.raises(ValueError):
        dbc.rms_norm(x, y=torch.zeros(64, 4, device="cuda", dtype=torch.bfloat16).t())
    with pytest.raises(ValueError):
        dbc.rms_norm(x, y=x.clone(), out_dtype=torch.float32)
    with pytest.raises(ValueError):
        dbc.rms_norm(x, torch.ones(64))
    with pytest.raises(ValueError):
        dbc.rms_norm_i8(x, scale=torch.zeros(3, device="cuda"))
    with pytest.raises(ValueError):
        dbc.rms_norm_backward(x[:2], x)
    with pytest.raises(ValueError):
        dbc.rms_norm_backward(x, x, want_dw=False, dw=torch.zeros(64, device="cuda"))
    with pytest.raises(TypeError):
        dbc.rms_norm(x, dev_status=torch.zeros(1, device="cuda"))
    with pytest.raises(dbc.DbcError):
        dbc.rms_norm(x, eps=0.0)
    with pytest.raises(dbc.DbcError):
        dbc.quantize_rows_i8(torch.zeros(1, 16385, device="cuda"))


def test_other_stream_and_captured_graphs():
    """A stream argument orders the copies too; graphs replay on new data, two of them at once."""
    import dynamic_byte_chunking_b200 as dbc
    import torch
    torch.manual_seed(0)
    x, r = torch.randn(2, 700, 512, device="cuda").bfloat16()
    w = torch.randn(512, device="cuda").bfloat16()
    y, s = dbc.rms_norm(x, w, residual=r)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2, s2 = dbc.rms_norm(x.t().contiguous().t(), w, residual=r, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, y2) and torch.equal(s, s2)

    graphs = []
    for k in range(2):
        ins = [torch.zeros_like(x), torch.zeros_like(r)]
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            def body():
                y_, s_ = dbc.rms_norm(ins[0], w, residual=ins[1])
                q_, c_, _ = dbc.rms_norm_i8(ins[0], w, residual=ins[1])
                dx_, dw_ = dbc.rms_norm_backward(y_, s_, w, dsum=ins[0])
                return y_, s_, q_, c_, dx_, dw_
            body()
        torch.cuda.current_stream().wait_stream(st)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            outs = body()
        graphs.append((g, ins, outs, st, body))
    for trial in range(3):
        data = [torch.randn(2, 700, 512, device="cuda").bfloat16() for _ in graphs]
        torch.cuda.synchronize()
        for (g, ins, outs, st, body), v in zip(graphs, data):
            with torch.cuda.stream(st):
                ins[0].copy_(v[0])
                ins[1].copy_(v[1])
                g.replay()
        torch.cuda.synchronize()
        for (g, ins, outs, st, body), v in zip(graphs, data):
            for a, b in zip(outs, body()):
                assert torch.equal(a, b)


def test_row_offsets_past_32_bits():
    """A batch whose last rows lie past 2^31 elements and 2^32 bytes."""
    import dynamic_byte_chunking_b200 as dbc
    import torch
    N, d = 8_400_003, 264                          # 2.2e9 elements
    x = torch.zeros(N, d, dtype=torch.bfloat16, device="cuda")
    x[-5:] = torch.randn(5, d, device="cuda").bfloat16()
    tail = x[-5:].clone()
    y, _ = dbc.rms_norm(x, eps=EPS)
    assert torch.equal(y[-5:], dbc.rms_norm(tail, eps=EPS)[0]) and not y[:1000].any()
    dx, dw = dbc.rms_norm_backward(x, x, eps=EPS, dx=y)
    rx, rw = dbc.rms_norm_backward(tail, tail, eps=EPS)
    assert torch.equal(dx[-5:], rx)
    assert torch.allclose(dw, rw, rtol=1e-5, atol=1e-5)
    del y, dx
    q, sc = dbc.quantize_rows_i8(x)
    assert torch.equal(q[-5:], dbc.quantize_rows_i8(tail)[0]) and torch.equal(sc[-5:], dbc.quantize_rows_i8(tail)[1])


@pytest.mark.parametrize("T", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 200, 256, 700, 1536, 333, 1333])
def test_codes_under_an_fp32_weight_and_near_ties(T, d):
    """Products of more than 16 significant bits; rows whose quotients are, or are within a rounding of,
    halves: p = (k + 1/2) m / 127 for all k, one step of fp32 up and down."""
    import dynamic_byte_chunking_b200 as dbc
    rng = np.random.default_rng(d)
    N = 96
    x = _vals(rng, (N, d), T)
    w = _weight(rng, d, "f32")
    q, sc, _ = dbc.rms_norm_i8(_t(x, T), _t(w, "f32"), eps=EPS)
    qr, sr = o.rms_norm_i8(x, w, EPS)
    assert np.array_equal(q.cpu().numpy(), qr)
    _close(sc, sr, np.abs(sr) * (o.CHAIN / 2 + o.OPS) * o.U32, "scale")
    if T == "f32":
        m = rng.uniform(0.5, 2.0, (N, 1)).astype(np.float32) * np.float32(2.0) ** rng.integers(-60, 60, (N, 1)).astype(np.float32)
        k = rng.integers(-127, 127, (N, d))
        p = ((k + 0.5) / 127.0 * m.astype(np.float64)).astype(np.float32)
        step = rng.integers(-1, 2, (N, d))
        p = np.where(step > 0, np.nextafter(p, np.float32(np.inf)), np.where(step < 0, np.nextafter(p, np.float32(-np.inf)), p))
        p[:, :1] = m
        p = p.astype(np.float64)
        q, sc = dbc.quantize_rows_i8(_t(p, T))
        assert np.array_equal(q.cpu().numpy(), o.quantize_rows_i8(p)[0])


def test_stored_sums_of_all_exponent_gaps():
    """s = bf16(fp32(x + r)) bit for bit, over random bit patterns (subnormals, opposite signs, overflow)."""
    import dynamic_byte_chunking_b200 as dbc
    import torch
    g = torch.Generator(device="cuda").manual_seed(1)
    for d in (256, 1536, 777):
        bits = torch.randint(-32768, 32768, (2, 2000, d), generator=g, device="cuda", dtype=torch.int32).to(torch.int16)
        x, r = bits.view(torch.bfloat16)
        x, r = torch.where(x.isfinite(), x, 1.0), torch.where(r.isfinite(), r, -1.0)
        # half of the pairs close to each other in size
        r = torch.where(torch.rand(r.shape, generator=g, device="cuda") < 0.5, (x.float() * 1.37).clamp(-3e38, 3e38).bfloat16().neg(), r)
        _, s = dbc.rms_norm(x, residual=r)
        ref = (x.float() + r.float()).bfloat16()
        same = (s.view(torch.int16) == ref.view(torch.int16)) | (s.isnan() & ref.isnan())
        assert bool(same.all())


def test_first_call_of_a_process_may_be_captured():
    """No call needs one before it outside a capture (a child process: its first calls are captured)."""
    import subprocess
    import sys
    import os
    code = """
import sys
sys.path.insert(0, ROOT)
import torch, dynamic_byte_chunking_b200 as dbc
x = torch.randn(300, 512, device='cuda').bfloat16(); z = torch.randn(300, 99, device='cuda').bfloat16()
st = torch.zeros(1, dtype=torch.int32, device='cuda')
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    q, sc, s = dbc.rms_norm_i8(x, residual=x, dev_status=st)
    y, _ = dbc.rms_norm(z, dev_status=st)
    dx, dw = dbc.rms_norm_backward(x, s, dev_status=st)
    o1 = dbc.matmul_i8(q, sc, q[:40], sc[:40], out_dtype=torch.float32, dev_status=st)
    o2 = dbc.matmul_i8(q[:3], sc[:3], q, sc, dev_status=st)
g.replay()
torch.cuda.synchronize()
assert st.item() == 0
ref = (q.double() @ q[:40].double().t()) * sc.double()[:, None] * sc[:40].double()
assert torch.allclose(o1.double(), ref, rtol=1e-6)
assert torch.equal(y, dbc.rms_norm(z)[0]) and torch.equal(dx, dbc.rms_norm_backward(x, s)[0])
print('fine')
""".replace("ROOT", repr(os.path.dirname(os.path.dirname(os.path.abspath(__file__)))))
    p = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert p.returncode == 0 and p.stdout.strip().endswith("fine"), p.stderr[-2000:]


@pytest.mark.parametrize("d", [96, 256, 1000, 2048, 99, 501, 1531, 3001])
def test_sum_that_is_not_stored(d):
    """The library's calls with a residual and no s (the binding always stores it)."""
    import ctypes
    import dynamic_byte_chunking_b200 as dbc
    import torch
    rng = np.random.default_rng(d)
    N = 700
    x, r, w = (_t(_vals(rng, s, "bf16"), "bf16") for s in ((N, d), (N, d), (d,)))
    y, _ = dbc.rms_norm(x, w, residual=r)
    q, sc, _ = dbc.rms_norm_i8(x, w, residual=r)
    y2, q2, sc2 = torch.zeros_like(y), torch.zeros(N, d, dtype=torch.int8, device="cuda"), torch.zeros_like(sc)
    L, st = dbc.lib(), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert L.rms_norm(x.data_ptr(), d, 1, r.data_ptr(), d, w.data_ptr(), 1, N, d, 1e-6, None, 0, y2.data_ptr(), d, 1,
                      None, st) == 0
    assert L.rms_norm_i8(x.data_ptr(), d, 1, r.data_ptr(), d, w.data_ptr(), 1, N, d, 1e-6, None, 0, q2.data_ptr(), d,
                         sc2.data_ptr(), None, st) == 0
    # (q2's rows are d bytes apart, q's on 16-byte boundaries: two routes through memory, the same codes)
    assert torch.equal(y, y2) and torch.equal(q, q2) and torch.allclose(sc, sc2, rtol=1e-6)


@pytest.mark.parametrize("T", ["bf16", "f32"])
@pytest.mark.parametrize("d", [40, 200, 256, 512, 1000, 2048, 8192, 33, 257, 500, 777, 1531, 3001])
def test_gradients_whose_products_leave_fp32(T, d):
    """dy so small that dy w s vanishes in fp32 while dy and s do not: the projection term of dx stays.  Rows of
    zeros, rows with one such gradient and ordinary rows between them (bounds: backward_bounds)."""
    import dynamic_byte_chunking_b200 as dbc
    rng = np.random.default_rng(d)
    N = 11
    s, dy = _vals(rng, (N, d), T), _vals(rng, (N, d), T)
    for r, es, ey in ((0, -50, -106), (2, -45, -100), (3, -40, -118), (4, -50, -60), (7, -49, -110), (10, -48, -104)):
        s[r], dy[r] = o.store(s[r] * 2.0 ** es, T), o.store(dy[r] * 2.0 ** ey, T)
    dy[5] = 0
    dy[7, 1:] = 0
    w = _weight(rng, d, T)
    st = _status()
    for eps in (1e-30, EPS):
        dx, dw = dbc.rms_norm_backward(_t(dy, T), _t(s, T), _t(w, T), eps=eps, dev_status=st)
        rx, rw = o.rms_norm_backward(dy, s, w, eps, None)
        bx, bw = o.backward_bounds(dy, s, w, eps, None, T)
        # Below 2^-126 fp32 has a step of 2^-149: dy w, its difference from xhat c and c itself are each off by half
        # of it there, whatever their size (an element of row 3 that is 2^-8 of the others is there), and dx is
        # rstd times that.
        rs = o.rstd_of(s, eps)
        _close(dx, rx, bx + rs * 2.0 ** -150 * (2 + np.abs(s * rs)), f"dx eps={eps}")
        _close(dw, rw, bw, f"dw eps={eps}")
    assert st.item() == 0


@pytest.mark.parametrize("TY,T,d,N", [("bf16", "bf16", 64, 600_000), ("f32", "bf16", 256, 160_000), ("bf16", "bf16", 512, 100_000),
                                      ("bf16", "bf16", 1536, 40_000), ("f32", "f32", 1536, 40_000), ("bf16", "f32", 4096, 20_000),
                                      ("bf16", "bf16", 8192, 10_000), ("f32", "bf16", 16384, 5_000), ("f32", "f32", 12000, 5_000),
                                      ("bf16", "bf16", 33, 2_000_000), ("bf16", "f32", 77, 600_000),
                                      ("f32", "bf16", 257, 310_000), ("bf16", "bf16", 500, 160_000), ("f32", "f32", 1531, 40_000),
                                      ("bf16", "bf16", 5001, 10_000), ("bf16", "f32", 9001, 5_000)])
def test_dw_of_many_rows_keeps_small_terms(TY, T, d, N):
    """dw where every column's terms are 1 in the first 1/64 of the rows and less than half a step of fp32 at 1 in
    the others: one fp32 chain over a thread's rows loses all of those, 63 roundings of the result (half of it where
    only every other thread has such rows in front).

    Rows of +-1 have one rstd, off by half a rounding of 1/d, half of the mean and two steps (four roundings) of
    rsqrtf; the products with it round once, sixteen of them add up in fp32 (15 roundings, all terms are positive)
    before they join fp64 sums, and so does the result: 22 in all, and one for the fp64 additions."""
    import dynamic_byte_chunking_b200 as dbc
    import torch
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}
    g = torch.Generator(device="cuda").manual_seed(d)
    s = torch.randint(0, 2, (N, d), generator=g, device="cuda", dtype=torch.int8).mul_(2).sub_(1)
    first, small = N // 64, 255 * 2.0 ** -32
    dy = s.to(dt[TY])
    dy[first:] *= small
    _, dw = dbc.rms_norm_backward(dy, s.to(dt[T]), None, eps=1e-30)
    ref = np.full(d, first + (N - first) * small)
    _close(dw, ref, ref * 23 * o.U32, "dw")


@pytest.mark.parametrize("N,d", [(200003, 33), (100003, 131), (60001, 257), (20011, 777), (5003, 1531), (3001, 3333)])
def test_many_odd_rows(N, d):
    """Rows off the 16-byte grid, several tiles (or rows) to a CTA and several rows of a tile to a team: against the
    oracle, packed, inside wider buffers and in place."""
    import dynamic_byte_chunking_b200 as dbc
    import torch
    rng = np.random.default_rng(N)
    st = _status()
    x, r, dy, ds = (_vals(rng, (N, d), "bf16") for _ in range(4))
    w = _weight(rng, d, "bf16")
    xt, rt, dyt, dst, wt = (_t(v, "bf16") for v in (x, r, dy, ds, w))
    s = o.residual_sum(x, r, "bf16")
    ref = o.rms_norm(s, w, EPS)
    by = o.rms_norm_bound(ref, "bf16")

    def wider(t=None, dtype=torch.bfloat16):
        buf = torch.full((N, d + 4), 7, dtype=dtype, device="cuda")
        if t is not None:
            buf[:, 1:d + 1] = t
        return buf

    def kept(buf):
        return bool((buf[:, 0] == 7).all() and (buf[:, d + 1:] == 7).all())

    y, sg = dbc.rms_norm(xt, wt, eps=EPS, residual=rt, dev_status=st)
    _close(y, ref, by, "y")
    assert np.array_equal(_np(sg), s)
    yb, sb = wider(), wider()
    dbc.rms_norm(wider(xt)[:, 1:d + 1], wt, eps=EPS, residual=wider(rt)[:, 1:d + 1], y=yb[:, 1:d + 1], s=sb[:, 1:d + 1])
    _close(yb[:, 1:d + 1], ref, by, "strided y")
    assert torch.equal(sb[:, 1:d + 1], sg) and kept(yb) and kept(sb)
    x2, r2 = xt.clone(), rt.clone()
    dbc.rms_norm(x2, wt, eps=EPS, residual=r2, y=x2, s=r2)
    assert torch.equal(x2, y) and torch.equal(r2, sg)

    qr, sr = o.rms_norm_i8(s, w, EPS)
    q, sc, _ = dbc.rms_norm_i8(xt, wt, eps=EPS, residual=rt, dev_status=st)
    assert np.array_equal(q.cpu().numpy(), qr)
    _close(sc, sr, np.abs(sr) * (o.CHAIN / 2 + o.OPS) * o.U32, "scale")
    qb = wider(dtype=torch.int8)
    dbc.rms_norm_i8(wider(xt)[:, 1:d + 1], wt, eps=EPS, residual=rt, q=qb[:, 1:d + 1])
    assert torch.equal(qb[:, 1:d + 1], q) and kept(qb)
    r3 = rt.clone()
    q3, _, _ = dbc.rms_norm_i8(xt, wt, eps=EPS, residual=r3, s=r3, q=torch.empty(N, d, dtype=torch.int8, device="cuda"))
    assert torch.equal(q3, q) and torch.equal(r3, sg)
    qr, sr = o.quantize_rows_i8(x)
    q, sc = dbc.quantize_rows_i8(xt, dev_status=st)
    assert np.array_equal(q.cpu().numpy(), qr)
    _close(sc, sr, np.abs(sr) * 2 * o.U32, "quantize scale")
    del qr, sr, ref, by

    rx, rw = o.rms_norm_backward(dy, s, w, EPS, ds)
    bx, bw = o.backward_bounds(dy, s, w, EPS, ds, "bf16")
    dx, dw = dbc.rms_norm_backward(dyt, sg, wt, eps=EPS, dsum=dst, dev_status=st)
    _close(dx, rx, bx, "dx")
    _close(dw, rw, bw, "dw")
    xb = wider()
    _, dw2 = dbc.rms_norm_backward(wider(dyt)[:, 1:d + 1], sb[:, 1:d + 1], wt, eps=EPS, dsum=wider(dst)[:, 1:d + 1],
                                   dx=xb[:, 1:d + 1])
    _close(xb[:, 1:d + 1], rx, bx, "strided dx")
    _close(dw2, rw, bw, "strided dw")
    assert kept(xb)
    for k in range(3):
        c = [dyt.clone(), sg.clone(), dst.clone()]
        _, dw2 = dbc.rms_norm_backward(c[0], c[1], wt, eps=EPS, dsum=c[2], dx=c[k])
        assert torch.equal(c[k], dx) and torch.equal(dw2, dw)
    assert st.item() == 0
