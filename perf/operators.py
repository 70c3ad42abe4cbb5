"""Cases and reference forms of the residual / RMS norm / 8-bit product operators.

``rms_norm``           s = T(x + residual), y = s * rstd * w, rstd = 1 / sqrt(mean(s^2) + eps)
``rms_norm_i8``        the same row in 8 bits: p = fp32(s * w), m = max |p|, q = rint(127 p / m),
                       scale = m * rstd / 127
``rms_norm_backward``  dx (the gradient of x and of the residual) and dw
``quantize_rows_i8``   q = rint(127 x / m), scale = m / 127, m = max |x| of the row
``matmul_i8``          out = a_scale * b_scale * (a b^T in exact integers) (+ bias)

With ``own`` false :func:`run` evaluates them with elementary torch operations, with ``own`` true it calls
the library.  Sizes are the workload families' (8 x 8192 x 256 byteflow positions; 32 x 8192 x 512 wide
positions, 1024 chunk vectors a row, projected from 512 to 1536; a ragged batch of about 2.2 M positions x 256)
and generic ones.
"""
import math

import torch

own = False

EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
# per pass, of the largest listed cases
MOST_ELEMENTS = 2200003 * 256
MOST_PRODUCTS = 8192 * 4096 * 4096


def listed():
    return [
        # the decoder's first norm: the fp32 S of the upsampling, read once per byteflow batch
        dict(name="norm upsampled f32", op="norm", N=65536, d=256, dtype="f32", out="bf16", residual=False),
        # a norm inside a layer over the ragged batch: bf16 residual stream updated on the way (odd row count)
        dict(name="norm ragged bf16", op="norm", N=2200003, d=256, dtype="bf16", out="bf16", residual=True),
        # one byte of one stream while decoding: latency
        dict(name="norm i8 one row", op="norm_i8", N=1, d=256, dtype="bf16", residual=True),
        # chunk vectors of the wide batch at the global width, in 8 bits for the next product
        dict(name="norm i8 chunk vectors", op="norm_i8", N=32768, d=1536, dtype="bf16", residual=True),
        # training, byteflow batch, with the gradient that arrives at the residual stream
        dict(name="backward byteflow", op="norm_bwd", N=65536, d=256, dtype="bf16", dy="bf16", dsum=True),
        # training at the global width, odd row count, fp32 gradient of y
        dict(name="backward wide", op="norm_bwd", N=32749, d=1536, dtype="bf16", dy="f32", dsum=False),
        # the local-to-global projection's weight, once per load
        dict(name="quantize weight", op="quant", N=1536, d=512, dtype="bf16", stride=512),
        # activations without a norm in front: one part of a wider fused buffer, all positions of the wide batch
        dict(name="quantize positions", op="quant", N=262144, d=512, dtype="bf16", stride=1536),
        # one chunk vector while decoding: latency
        dict(name="product one token", op="matmul", M=1, N=1536, K=512, out="bf16", bias=False),
        # a decoding batch with odd sizes, bias and fp32 logits
        dict(name="product odd batch", op="matmul", M=61, N=1543, K=1531, out="f32", bias=True),
        # the projection of every chunk vector of the wide batch
        dict(name="product wide projection", op="matmul", M=32768, N=1536, K=512, out="bf16", bias=False),
        # a large square-ish layer of a global model
        dict(name="product large", op="matmul", M=8192, N=4096, K=4096, out="bf16", bias=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng):
    """A row width: mostly multiples of 64 up to 4096, sometimes any number."""
    if rng.random() < 0.7:
        return 64 * _log(rng, 1, 64)
    return _log(rng, 17, 4096)


def draw(rng):
    op = rng.choice(["norm", "norm_i8", "norm_bwd", "quant", "matmul", "matmul"])
    if op == "matmul":
        K = _width(rng)
        N = _width(rng)
        M = _log(rng, 1, min(65536, MOST_PRODUCTS // (N * K)))
        return dict(op=op, M=M, N=N, K=K, out=rng.choice(["bf16", "bf16", "f32"]), bias=rng.random() < 0.5)
    d = _width(rng)
    N = _log(rng, 1, MOST_ELEMENTS // 4 // d)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "norm":
        return dict(op=op, N=N, d=d, dtype=dtype, out=rng.choice(["bf16", "f32"]), residual=rng.random() < 0.7)
    if op == "norm_i8":
        return dict(op=op, N=N, d=d, dtype=dtype, residual=rng.random() < 0.7)
    if op == "norm_bwd":
        return dict(op=op, N=N, d=d, dtype=dtype, dy=rng.choice(["bf16", "f32"]), dsum=rng.random() < 0.5)
    return dict(op=op, N=N, d=d, dtype=dtype, stride=d * rng.choice([1, 1, 2]))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)

    st = dict(case)
    if case["op"] == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        ld = (K + 15) // 16 * 16   # the rows of 8-bit operands start on 16-byte boundaries

        def operand(rows):
            v = normal(rows, ld).mul_(36).round_().clamp_(-127, 127).to(torch.int8)   # |max| of a row of normals
            return v[:, :K]

        st["a"], st["b"] = operand(M), operand(N)
        st["a_scale"] = torch.rand(M, generator=g, device="cuda") * 0.02 + 0.01
        st["b_scale"] = (torch.rand(N, generator=g, device="cuda") * 0.02 + 0.01) / math.sqrt(K)
        st["bias"] = normal(N, dtype=torch.bfloat16) if case["bias"] else None
        return st
    N, d, dtype = case["N"], case["d"], DTYPES[case["dtype"]]
    if case["op"] == "quant":
        st["x"] = normal(N, case["stride"], dtype=dtype)[:, :d]
        return st
    st["x"] = normal(N, d, dtype=dtype)
    st["weight"] = (normal(d) * 0.1 + 1).to(torch.bfloat16)
    if case["op"] == "norm_bwd":
        st["dyv"] = normal(N, d, dtype=DTYPES[case["dy"]])
        st["dsumv"] = normal(N, d, dtype=dtype) if case["dsum"] else None
    else:
        st["res"] = normal(N, d, dtype=dtype) if case["residual"] else None
    return st


# ---------------------------------------------------------------- plain forms
def _sum(x, res):
    return x if res is None else (x.float() + res.float()).to(x.dtype)


def _rstd(sf):
    return 1.0 / torch.sqrt(sf.square().mean(-1, keepdim=True) + EPS)


def _codes(p):
    """(q, m): 64 bits, because a quotient next to a half decides the whole number."""
    m = p.abs().amax(-1, keepdim=True)
    q = torch.round(p.double() * 127.0 / m.double())
    return torch.where(m > 0, q, torch.zeros_like(q)).to(torch.int8), m


def _plain(st):
    op = st["op"]
    if op == "matmul":
        acc = st["a"].float() @ st["b"].float().t()
        acc = acc * st["a_scale"][:, None] * st["b_scale"]
        if st["bias"] is not None:
            acc = acc + st["bias"].float()
        return {"out": acc.to(DTYPES[st["out"]])}
    if op == "quant":
        q, m = _codes(st["x"].float())
        return {"q": q, "scale": m[:, 0] / 127.0}
    w = st["weight"].float()
    if op == "norm_bwd":
        sf, dy = st["x"].float(), st["dyv"].float()
        rs = _rstd(sf)
        gw = dy * w
        c = (gw * sf).mean(-1, keepdim=True) * rs * rs
        dx = rs * (gw - sf * c)
        if st["dsumv"] is not None:
            dx = dx + st["dsumv"].float()
        dw = (dy * sf * rs).sum(0, dtype=torch.float64)   # long sums in 64 bits
        return {"dx": dx.to(st["x"].dtype), "dw": dw.float()}
    s = _sum(st["x"], st["res"])
    sf = s.float()
    rs = _rstd(sf)
    out = {} if st["res"] is None else {"s": s}
    if op == "norm":
        return {**out, "y": (sf * rs * w).to(DTYPES[st["out"]])}
    q, m = _codes(sf * w)
    return {**out, "q": q, "scale": (m * rs)[:, 0] / 127.0}


# ---------------------------------------------------------------- the library's calls
def _own(st):
    import dynamic_byte_chunking_b200 as dbc
    op = st["op"]
    if op == "matmul":
        return {"out": dbc.matmul_i8(st["a"], st["a_scale"], st["b"], st["b_scale"], bias=st["bias"],
                                     out_dtype=DTYPES[st["out"]])}
    if op == "quant":
        q, scale = dbc.quantize_rows_i8(st["x"])
        return {"q": q, "scale": scale}
    if op == "norm_bwd":
        dx, dw = dbc.rms_norm_backward(st["dyv"], st["x"], st["weight"], eps=EPS, dsum=st["dsumv"])
        return {"dx": dx, "dw": dw}
    if op == "norm":
        y, s = dbc.rms_norm(st["x"], st["weight"], eps=EPS, residual=st["res"], out_dtype=DTYPES[st["out"]])
        return {"y": y} if st["res"] is None else {"s": s, "y": y}
    q, scale, s = dbc.rms_norm_i8(st["x"], st["weight"], eps=EPS, residual=st["res"])
    return {"q": q, "scale": scale} if st["res"] is None else {"s": s, "q": q, "scale": scale}


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    if case["op"] == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        size = 2 if case["out"] == "bf16" else 4
        return {"bytes": (M + N) * K + 4 * (M + N) + M * N * size + (2 * N if case["bias"] else 0),
                "flops": 2 * M * N * K}
    N, d = case["N"], case["d"]
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "quant":
        return {"bytes": N * d * (e + 1) + 4 * N, "flops": 3 * N * d}
    if case["op"] == "norm_bwd":
        dy = 2 if case["dy"] == "bf16" else 4
        return {"bytes": N * d * (dy + 2 * e + (e if case["dsum"] else 0)) + 6 * d, "flops": 12 * N * d}
    moved = e * (3 if case["residual"] else 1)
    if case["op"] == "norm":
        return {"bytes": N * d * (moved + (2 if case["out"] == "bf16" else 4)) + 2 * d, "flops": 5 * N * d}
    return {"bytes": N * d * (moved + 1) + 4 * N + 2 * d, "flops": 7 * N * d}


# ---------------------------------------------------------------- 64 bits, from the definitions
def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "matmul":
        out = torch.einsum("mk,nk->mn", st["a"].to(torch.float64), st["b"].to(torch.float64))
        out.mul_(st["a_scale"].to(torch.float64).unsqueeze(1)).mul_(st["b_scale"].to(torch.float64).unsqueeze(0))
        if case["bias"]:
            out.add_(st["bias"].to(torch.float64).unsqueeze(0))
        return {"out": out}
    if op == "quant":
        return {"q": None, "scale": st["x"].to(torch.float64).abs().max(dim=1).values.div(127)}
    x, w = st["x"].to(torch.float64), st["weight"].to(torch.float64)
    d = case["d"]
    if op == "norm_bwd":
        dy = st["dyv"].to(torch.float64)
        inv = (torch.einsum("nd,nd->n", x, x) / d + EPS).pow(-0.5).unsqueeze(1)
        xhat = x * inv
        dw = torch.einsum("nd,nd->d", dy, xhat)
        dy.mul_(w)
        dx = dy - xhat * (torch.einsum("nd,nd->n", dy, xhat) / d).unsqueeze(1)
        dx.mul_(inv)
        if case["dsum"]:
            dx.add_(st["dsumv"].to(torch.float64))
        return {"dx": dx, "dw": dw}
    out = {}
    if case["residual"]:
        out["s"] = x + st["res"].to(torch.float64)
        x = out["s"].to(DTYPES[case["dtype"]]).to(torch.float64)   # the stored sum is what is normalised
    inv = (torch.einsum("nd,nd->n", x, x) / d + EPS).pow(-0.5)
    x = x * w
    if op == "norm":
        out["y"] = x.mul_(inv.unsqueeze(1))
    else:
        out["q"], out["scale"] = None, x.abs().max(dim=1).values * inv / 127
    return out
