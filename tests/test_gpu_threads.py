"""Host threads that call the same operators at different sizes, each on its own stream.  The threads call the
library itself, in a tight loop: the binding's Python part would run them mostly one after another."""
import ctypes
import threading

import pytest

pytestmark = pytest.mark.gpu

CALLS = 3000                                         # per thread


class Call:
    """One prepared call of the library: its arguments but the stream, the tensors they point into, its outputs."""

    def __init__(self, fn, args, keep, outs):
        self.fn, self.args, self.keep, self.outs = fn, args, keep, outs

    def __call__(self, stream):
        return self.fn(*self.args, stream)


def _p(t):
    return ctypes.c_void_p(t.data_ptr())


def _run_together(calls):
    """Every call CALLS times in a thread and on a stream of its own: none refused, and the last results those of
    a call made alone."""
    import torch
    want = []
    for c in calls:
        assert c(None) == 0
        torch.cuda.synchronize()
        want.append([t.clone() for t in c.outs])
        for t in c.outs:
            t.zero_()
    torch.cuda.synchronize()
    refused = [0] * len(calls)
    streams = [torch.cuda.Stream() for _ in calls]
    gate = threading.Barrier(len(calls))

    def work(i):
        call, stream = calls[i], ctypes.c_void_p(streams[i].cuda_stream)
        gate.wait()
        for _ in range(CALLS):
            if call(stream) != 0:
                refused[i] += 1

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not any(refused), f"calls refused per thread: {refused} of {CALLS}"
    for c, w in zip(calls, want):
        for a, b in zip(c.outs, w):
            assert torch.equal(a, b)


def _norm(op, d):
    import dynamic_byte_chunking_b200 as dbc
    import torch
    L, N = dbc.lib(), 3
    g = torch.Generator(device="cuda").manual_seed(d)
    x, r = (torch.randn(N, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    w = torch.randn(d, generator=g, device="cuda").bfloat16()
    s, y = torch.empty_like(x), torch.empty_like(x)
    q, sc, dw = torch.empty(N, d, dtype=torch.int8, device="cuda"), torch.empty(N, device="cuda"), torch.empty(d, device="cuda")
    ws = torch.empty(dbc.rms_norm_backward_workspace(N, d), dtype=torch.uint8, device="cuda")
    eps = ctypes.c_float(1e-6)
    keep = [x, r, w, ws]
    if op == "norm":
        return Call(L.rms_norm, (_p(x), d, 1, _p(r), d, _p(w), 1, N, d, eps, _p(s), d, _p(y), d, 1, None), keep, [s, y])
    if op == "norm_i8":
        return Call(L.rms_norm_i8, (_p(x), d, 1, _p(r), d, _p(w), 1, N, d, eps, _p(s), d, _p(q), d, _p(sc), None), keep,
                    [s, q, sc])
    if op == "quantize":
        return Call(L.quantize_rows_i8, (_p(x), d, 1, N, d, _p(q), d, _p(sc), None), keep, [q, sc])
    return Call(L.rms_norm_backward, (_p(x), d, 1, _p(r), d, 1, _p(w), 1, None, 0, N, d, eps, _p(y), d, _p(dw), _p(ws),
                                      ws.numel(), None), keep, [y, dw])


# pairs of widths that one kernel serves with different amounts of shared memory: wide rows, odd narrow rows
# (tiles), odd wide rows
@pytest.mark.parametrize("op", ["norm", "norm_i8", "quantize", "backward"])
@pytest.mark.parametrize("widths", [(4096, 1536), (499, 301), (2047, 1027)])
def test_norms_at_two_widths(op, widths):
    _run_together([_norm(op, d) for d in widths] + [_norm(op, d) for d in widths])


def _coding_rate(d):
    """The fp32 path (its factorisations' panels grow with d)."""
    import dynamic_byte_chunking_b200 as dbc
    import torch
    g = torch.Generator(device="cuda").manual_seed(d)
    H = torch.randn(70, d, generator=g, device="cuda").div(d ** 0.5)
    dR = torch.empty(70, device="cuda")
    ws = torch.empty(dbc.chunk_coding_rate_workspace(1, 70, 70, d), dtype=torch.uint8, device="cuda")
    return Call(dbc.lib().chunk_coding_rate, (_p(H), 0, None, 1, 70, 70, d, ctypes.c_float(0.5), _p(dR), _p(ws), ws.numel(),
                                              None), [H, ws], [dR])


def _step(d):
    import dynamic_byte_chunking_b200 as dbc
    import torch
    H = torch.zeros(1, 1, d, device="cuda")          # zeros leave the carried factor as it is
    B, dR = torch.eye(d, device="cuda"), torch.empty(1, device="cuda")
    return Call(dbc.lib().chunk_coding_rate_step, (_p(H), 0, 1, 1, d, ctypes.c_float(0.5), _p(B), _p(dR), None), [H, B], [dR])


@pytest.mark.parametrize("make,sizes", [(_coding_rate, (512, 64)), (_step, (256, 64))], ids=["coding_rate", "step"])
def test_chunker_at_two_sizes(make, sizes):
    _run_together([make(n) for n in sizes] + [make(n) for n in sizes])


def _product(M, N, K):
    import dynamic_byte_chunking_b200 as dbc
    import torch
    g = torch.Generator(device="cuda").manual_seed(M)
    a, b = (torch.randint(-127, 128, (R, K), generator=g, device="cuda", dtype=torch.int8) for R in (M, N))
    sa, sb = torch.rand(M, device="cuda"), torch.rand(N, device="cuda")
    out = torch.empty(M, N, device="cuda")
    return Call(dbc.lib().matmul_i8, (_p(a), K, _p(sa), _p(b), K, _p(sb), None, 0, M, N, K, _p(out), N, 0, None),
                [a, b, sa, sb], [out])


def _upsample():
    import dynamic_byte_chunking_b200 as dbc
    import torch
    g = torch.Generator(device="cuda").manual_seed(1)
    T, K, d = 128, 32, 256
    H, G = (torch.randn(n, d, generator=g, device="cuda").bfloat16() for n in (T, K))
    W = torch.randn(16, d, d, generator=g, device="cuda").bfloat16()
    idx, io = torch.arange(0, T, T // K, device="cuda"), torch.tensor([0, K], device="cuda")
    S = torch.empty(T, d, device="cuda")
    ws = torch.empty(dbc.chunk_upsample_workspace(1, T, 16), dtype=torch.uint8, device="cuda")
    return Call(dbc.lib().chunk_upsample, (_p(G), d, _p(H), 1, None, T, T, d, _p(idx), _p(io), 1, _p(W), 16, 0, _p(S), _p(ws),
                                           ws.numel(), None), [H, G, W, idx, io, ws], [S])


def _tensor_rate():
    import dynamic_byte_chunking_b200 as dbc
    import torch
    g = torch.Generator(device="cuda").manual_seed(2)
    T, d = 512, 256
    H = torch.randn(T, d, generator=g, device="cuda").div(16).bfloat16()
    dR = torch.empty(T, device="cuda")
    ws = torch.empty(dbc.chunk_coding_rate_workspace(1, T, T, d), dtype=torch.uint8, device="cuda")
    return Call(dbc.lib().chunk_coding_rate, (_p(H), 1, None, 1, T, T, d, ctypes.c_float(0.5), _p(dR), _p(ws), ws.numel(), None),
                [H, ws], [dR])


@pytest.mark.parametrize("make", [lambda: _product(5, 256, 512), lambda: _product(1500, 1536, 256), _upsample, _tensor_rate],
                         ids=["product_split", "product_wide", "upsample", "coding_rate"])
def test_first_cuda_call_of_a_thread(make):
    """A host thread that has made no CUDA call yet: the same kernels and results as in any other."""
    import dynamic_byte_chunking_b200 as dbc
    import torch
    call = make()
    before = dbc.launch_count()
    assert call(None) == 0
    launches = dbc.launch_count() - before
    torch.cuda.synchronize()
    want = [t.clone() for t in call.outs]
    for t in call.outs:
        t.zero_()
    torch.cuda.synchronize()
    rc = []
    before = dbc.launch_count()
    t = threading.Thread(target=lambda: rc.append(call(None)))
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert rc == [0] and dbc.launch_count() - before == launches
    for a, b in zip(call.outs, want):
        assert torch.equal(a, b)


def test_products_at_several_sizes():
    _run_together([_product(5, 256, 512), _product(14, 1536, 256), _product(130, 300, 256), _product(1500, 1536, 256)])
