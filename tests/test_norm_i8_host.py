"""Refusals of the norm / 8-bit entry points, decided on the host before any launch (no GPU needed)."""
import ctypes

import pytest

F = ctypes.c_float
P = ctypes.c_void_p(4096)           # never dereferenced: every case returns before a launch
ODD = ctypes.c_void_p(4097)
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    import dynamic_byte_chunking_b200 as dbc
    from dynamic_byte_chunking_b200 import build
    build.build()
    return dbc.lib()


def _norm(L, x=P, xs=64, dt=1, r=None, rs=0, w=None, wd=0, N=2, d=64, eps=1e-6, s=None, ss=0, y=P, ys=64, yd=1):
    return L.rms_norm(x, xs, dt, r, rs, w, wd, N, d, F(eps), s, ss, y, ys, yd, None, None)


def test_rms_norm_refusals(L):
    for eps in (0.0, -1.0, NAN, INF):
        assert _norm(L, eps=eps) == 1
    assert _norm(L, N=-1) == 1 and _norm(L, d=0) == 1
    assert _norm(L, x=None) == 1 and _norm(L, y=None) == 1
    assert _norm(L, xs=63) == 1 and _norm(L, ys=63) == 1
    assert _norm(L, r=P, rs=63) == 1 and _norm(L, r=P, rs=64, s=P, ss=63) == 1
    assert _norm(L, s=P, ss=64) == 1                                 # a sum without a residual
    assert _norm(L, x=ODD) == 1 and _norm(L, y=ODD) == 1 and _norm(L, r=ODD, rs=64) == 1 and _norm(L, w=ODD) == 1
    assert _norm(L, dt=2) == 2 and _norm(L, yd=7) == 2 and _norm(L, w=P, wd=5) == 2
    assert _norm(L, d=16385, xs=16385, ys=16385) == 2
    assert _norm(L, N=0, x=None, y=None) == 0                        # nothing to do


def test_rms_norm_i8_and_quantize_refusals(L):
    def i8(x=P, xs=64, N=2, d=64, eps=1e-6, q=P, qs=64, sc=P, dt=1):
        return L.rms_norm_i8(x, xs, dt, None, 0, None, 0, N, d, F(eps), None, 0, q, qs, sc, None, None)

    def qu(x=P, xs=64, N=2, d=64, q=P, qs=64, sc=P, dt=1):
        return L.quantize_rows_i8(x, xs, dt, N, d, q, qs, sc, None, None)

    assert i8(eps=0.0) == 1
    for f in (i8, qu):
        assert f(q=None) == 1 and f(sc=None) == 1 and f(x=None) == 1 and f(sc=ODD) == 1 and f(x=ODD) == 1
        assert f(qs=63) == 1 and f(xs=1) == 1 and f(N=-2) == 1 and f(d=-1) == 1
        assert f(dt=3) == 2 and f(d=1 << 15, xs=1 << 15, qs=1 << 15) == 2
        assert f(N=0, x=None, q=None, sc=None) == 0


def test_rms_norm_backward_refusals(L):
    import dynamic_byte_chunking_b200 as dbc
    need = dbc.rms_norm_backward_workspace(10, 64)
    assert 0 < need <= dbc.rms_norm_backward_workspace(10_000_000, 64) < 64 << 20
    assert dbc.rms_norm_backward_workspace(0, 64) == 0

    def f(dy=P, ys=64, yd=1, s=P, ss=64, dt=1, w=None, wd=0, ds=None, dss=0, N=10, d=64, eps=1e-6, dx=P, xs=64,
          dw=P, ws=P, wb=1 << 40):
        return L.rms_norm_backward(dy, ys, yd, s, ss, dt, w, wd, ds, dss, N, d, F(eps), dx, xs, dw, ws, wb, None,
                                   None)

    assert f(eps=0.0) == 1 and f(N=-1) == 1 and f(d=0) == 1
    assert f(dy=None) == 1 and f(s=None) == 1 and f(dx=None) == 1
    assert f(ys=1) == 1 and f(ss=1) == 1 and f(xs=1) == 1 and f(ds=P, dss=1) == 1
    assert f(dy=ODD) == 1 and f(s=ODD) == 1 and f(dx=ODD) == 1 and f(ds=ODD, dss=64) == 1 and f(dw=ODD) == 1
    assert f(dt=2) == 2 and f(yd=2) == 2 and f(w=P, wd=2) == 2 and f(d=20000, ys=20000, ss=20000, xs=20000) == 2
    assert f(ws=None) == 7 and f(wb=need - 1) == 7 and f(ws=ODD) == 7
    assert f(N=0, dw=None, dx=None, dy=None, s=None, ws=None) == 0


def test_matmul_i8_refusals(L):
    def f(a=P, lda=64, sa=P, b=P, ldb=64, sb=P, bias=None, bd=0, M=3, N=5, K=64, out=P, ldo=5, od=1):
        return L.matmul_i8(a, lda, sa, b, ldb, sb, bias, bd, M, N, K, out, ldo, od, None, None)

    assert f(M=-1) == 1 and f(N=-1) == 1 and f(K=-1) == 1
    assert f(lda=63) == 1 and f(lda=72) == 1 and f(ldb=48) == 1 and f(ldo=4) == 1
    for name in ("a", "sa", "b", "sb", "out"):
        assert f(**{name: None}) == 1, name
        assert f(**{name: ODD}) == 1, name
    assert f(a=ctypes.c_void_p(4104)) == 1 and f(b=ctypes.c_void_p(4104)) == 1      # 8-byte aligned only
    assert f(bias=ODD) == 1
    assert f(od=2) == 2 and f(bias=P, bd=9) == 2
    assert f(K=131072, lda=131072, ldb=131072) == 2                  # a sum could leave 32 bits
    assert f(M=(1 << 31) - 1) == 2 and f(N=1 << 31, ldo=1 << 31) == 2
    assert f(M=0, a=None, sa=None, out=None) == 0 and f(N=0, ldo=0, b=None, out=None) == 0


def test_binding_takes_cuda_tensors_only():
    torch = pytest.importorskip("torch")
    import dynamic_byte_chunking_b200 as dbc
    x, c = torch.zeros(2, 64), torch.zeros(2, 64, dtype=torch.int8)
    one = torch.ones(2)
    for call in (lambda: dbc.rms_norm(x), lambda: dbc.rms_norm_i8(x), lambda: dbc.quantize_rows_i8(x),
                 lambda: dbc.rms_norm_backward(x, x), lambda: dbc.matmul_i8(c, one, c, one)):
        with pytest.raises(ValueError, match="CUDA tensors only"):
            call()


def test_one_buffer_for_both_outputs_is_refused(L):
    """y over s would leave the sum nowhere; y over x with s over the residual is the in-place form."""
    Q = ctypes.c_void_p(8192)
    assert _norm(L, r=Q, rs=64, s=P, ss=64, y=P) == 1
    assert _norm(L, r=Q, rs=64, s=Q, ss=64, y=Q) == 1
    assert _norm(L, r=Q, rs=64, s=Q, ss=64, y=P, N=0) == 0
