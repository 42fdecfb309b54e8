"""Workloads of the operators that lie between the lookup and the head of a student,
its residual blocks, at sizes from one decode step to a full training batch, with
their plain forms in float32 torch operations and their definitions in float64.

A block's output y is normed, weighted, gated and added to the residual stream h, and
the next block reads the normed sum; what the backward pass needs is stored in 8
bits, and a trained layer answers from 4 bits:

  norm       u = y r_y w_post (post) or y,  h' = alpha h + beta gate u,  x = h' r_h w_pre,
             r_v = (mean v^2 + eps)^(-1/2) per row; a gate row serves gate_rows rows
  norm_grad  from dx and dh' the gradients of h, y, w_post, w_pre and the gate, with r_y, r_h
             and y, h' as stored (stored8: as their 8-bit values)
  pack       microscaled storage and back: 32 values along a row share a power of two s,
             the smallest at which the largest of them does not round past the format's
             largest value; v = s q, q the nearest (ties to even) multiple of 1/64 up to
             127/64 ("int8") or of 0, 0.5, 1, 1.5, 2, 3, 4, 6 ("fp4") with its sign
  linear     Y = X W^T, W in fp4
  product    Y = X W^T, both in fp4
  wgrad      dW = dY^T X, X in int8

Layout of a packed matrix of c columns: codes [rows][ceil(c / 32) * 32 bytes] (int8) or
[rows][ceil(c / 32) * 16 bytes] (fp4: two to a byte, the even column in the low half;
bit 3 the sign, bits 0..2 the index of the magnitude), scales [rows][ceil(c / 32) bytes
rounded up to 16] holding log2 s + 127; what lies past c is zero.
"""
import math
import random

import torch

own = False

EPS = 1e-6
ALPHA, BETA = 0.9, 0.5


def _case(name, **kw):
    return dict(name=name, **kw)


def listed():
    return [
        # one decode step of 8 sequences: latency
        _case("norm_decode", op="norm", n=8, d=4096, dtype="bf16", post=True, gate_rows=8),
        # a training batch of 8 sequences, each with a gate of its own
        _case("norm_train", op="norm", n=16384, d=4096, dtype="bf16", post=True, gate_rows=2048),
        # a narrow student in f32, odd sizes, its block's output not normed, one gate for all tokens
        _case("norm_grad_student", op="norm_grad", n=2047, d=1000, dtype="f32", post=False, gate_rows=2047, stored8=False),
        # a training batch whose activations were stored in 8 bits
        _case("norm_grad_train", op="norm_grad", n=16384, d=4096, dtype="bf16", post=True, gate_rows=16384, stored8=True),
        # activations of a training batch, stored for the backward pass and read there
        _case("pack8_train", op="pack", n=16384, d=4096, dtype="bf16", fmt="int8"),
        # a student's f32 weights, odd sizes
        _case("pack4_student", op="pack", n=1000, d=333, dtype="f32", fmt="fp4"),
        # one decode step of 8 sequences through a feed-forward matrix: bound by reading W
        _case("linear_decode", op="linear", T=8, N=14336, K=4096, dtype="bf16"),
        # a ragged prompt through the other feed-forward matrix
        _case("linear_prompt", op="linear", T=2047, N=4096, K=14336, dtype="bf16"),
        # a small projected layer with both sides in 4 bits, odd sizes
        _case("product_odd", op="product", T=333, N=1000, K=1000, dtype="bf16"),
        # prompts of 8192 tokens through a feed-forward matrix
        _case("product_prompt", op="product", T=8192, N=14336, K=4096, dtype="bf16"),
        # a narrow student's layer in f32
        _case("wgrad_student", op="wgrad", T=2047, N=512, K=1000, dtype="f32"),
        # a training batch through an attention projection
        _case("wgrad_train", op="wgrad", T=16384, N=4096, K=4096, dtype="bf16"),
    ]


def _size(rng, lo, hi):
    """A size in [lo, hi], uniform in its logarithm: any odd number, or a power of two."""
    if rng.random() < 0.4:
        return 1 << rng.randint(math.ceil(math.log2(lo)), math.floor(math.log2(hi)))
    return min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))) | 1)


def draw(rng: random.Random):
    op = rng.choice(("norm", "norm_grad", "pack", "linear", "product", "wgrad"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    if op in ("norm", "norm_grad"):
        n, d = _size(rng, 1, 16384), _size(rng, 32, 8192)
        n = min(n, (16384 * 4096) // d)
        rows = rng.choice((0, 1, n, n, min(n, _size(rng, 2, 2048))))
        case = dict(op=op, n=n, d=d, dtype=dtype, post=rng.random() < 0.7, gate_rows=rows)
        if op == "norm_grad":
            case["stored8"] = rng.random() < 0.5
        return case
    if op == "pack":
        d = _size(rng, 32, 14336)
        n = min(_size(rng, 1, 16384), (16384 * 4096) // d)
        return dict(op=op, n=n, d=d, dtype=dtype, fmt=rng.choice(("int8", "fp4")))
    most = 2048 if dtype == "f32" and op != "product" else 8192  # the f32 products run at a sixteenth of the bf16 rate
    T = _size(rng, 1, most)
    if op == "linear" and rng.random() < 0.5:
        T = rng.randint(1, 64)  # decode steps
    return dict(op=op, T=T, N=_size(rng, 32, most), K=_size(rng, 32, most), dtype=dtype)


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


# ---------------------------------------------------------------- microscaled storage, plain

def _pow2(e):
    """2^(e - 127) for integer e in [0, 254], from its bits."""
    return torch.where(e > 0, e << 23, 0x400000).int().view(torch.float32)


def _pack(x, fmt):
    """(codes, scales) in the layout above."""
    n, c = x.shape
    nb = -(-c // 32)
    v = torch.zeros(n, nb * 32, device=x.device)
    v[:, :c] = x
    v = v.view(n, nb, 32)
    top = v.abs().amax(2).view(torch.int32)
    e, m = top >> 23, top & 0x7FFFFF
    byte = (e + (m >= 0x7F0000)).clamp(0, 254) if fmt == "int8" else (e - 2 + (m >= 0x600000)).clamp(0, 252)
    a = v * _pow2(254 - byte)[:, :, None]
    if fmt == "int8":
        q = torch.round(a * 64).clamp(-127, 127).to(torch.int8).view(n, nb * 32).view(torch.uint8)
    else:
        a, sign = a.abs(), a < 0
        i = torch.zeros_like(a, dtype=torch.int32)
        for k, edge in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)):  # ties to the even index
            i += (a > edge) if k % 2 == 0 else (a >= edge)
        i = (i + 8 * (sign & (i > 0))).view(n, nb * 16, 2)
        q = (i[:, :, 0] | i[:, :, 1] << 4).to(torch.uint8)
    s = torch.zeros(n, -(-nb // 16) * 16, dtype=torch.uint8, device=x.device)
    s[:, :nb] = byte.to(torch.uint8)
    return q, s


def _unpack(p):
    """The values of a packed matrix in float32."""
    q, s, c, fmt = p
    n, nb = q.shape[0], -(-c // 32)
    if fmt == "int8":
        v = q.view(torch.int8).float() * (1.0 / 64)
    else:
        i = torch.stack((q & 15, q >> 4), 2).int()
        mag, half = (i >> 1) & 3, (i & 1).float() * 0.5
        v = torch.where(mag > 0, (1.0 + half) * (1 << mag).float() * 0.5, half)
        v = torch.where(i >= 8, -v, v)
    return (v.view(n, nb, 32) * _pow2(s[:, :nb].int())[:, :, None]).view(n, nb * 32)[:, :c]


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = _dtype(case)
    op = case["op"]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    def features(n, d):
        """Activations: features of unequal variance, a few of them far above the rest."""
        scale = torch.exp(0.5 * randn(d))
        far = torch.rand(d, generator=g, device=dev) < 0.004
        return (randn(n, d) * torch.where(far, 20.0 * scale, scale)).to(dt)

    def packed(x, fmt):
        return _pack(x, fmt) + (x.shape[1], fmt)

    if op == "pack":
        x = features(case["n"], case["d"])
        if case["n"] > 4:
            x[torch.rand(case["n"], generator=g, device=dev) < 0.03] = 0  # padding
        return dict(op=op, x=x, fmt=case["fmt"])
    if op in ("linear", "product", "wgrad"):
        T, N, K = case["T"], case["N"], case["K"]
        x = features(T, K)
        if op == "wgrad":
            dy = (randn(T, N) * torch.exp(randn(T, 1)) * (1.0 / T)).to(dt)
            return dict(op=op, dy=dy, x=packed(x, "int8"))
        w = packed(randn(N, K) / math.sqrt(K), "fp4")
        return dict(op=op, x=packed(x, "fp4") if op == "product" else x, w=w, dtype=dt)
    n, d, rows = case["n"], case["d"], case["gate_rows"]
    h, y = features(n, d), features(n, d)
    w_pre = (1.0 + 0.2 * randn(d)).to(dt)
    w_post = (1.0 + 0.2 * randn(d)).to(dt) if case["post"] else None
    gate = (0.7 + 0.5 * randn(-(-n // rows), d)).to(dt) if rows else None
    s = dict(op=op, y=y, w_post=w_post, w_pre=w_pre, gate=gate, rows=max(rows, 1), post=case["post"])
    if op == "norm":
        return dict(s, h=h)
    out = _norm(dict(s, h=h))
    s.update(out=out["h"], r_post=out["r_post"], r_pre=out["r_pre"])
    if case["stored8"]:
        s.update(y=packed(y, "int8"), out=packed(s["out"], "int8"))
    return dict(s, dx=(randn(n, d) * (1.0 / n)).to(dt), dout=(randn(n, d) * (2.0 / n)).to(dt))


# ---------------------------------------------------------------- the framework's calls

def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    import weights_bf16_fp32_amd as spec
    op = s["op"]

    def mx(p):
        return spec.Mx(p[0], p[1], p[2], spec.MX_INT8 if p[3] == "int8" else spec.MX_FP4) if isinstance(p, tuple) else p

    if op == "pack":
        p = spec.mx_quantize(s["x"], spec.MX_INT8 if s["fmt"] == "int8" else spec.MX_FP4)
        return spec.mx_dequantize(p, s["x"].dtype)
    if op == "linear":
        return spec.mx_linear(s["x"], mx(s["w"]))
    if op == "product":
        return spec.mx_product(mx(s["x"]), mx(s["w"]), s["dtype"])
    if op == "wgrad":
        return spec.mx_weight_grad(s["dy"], mx(s["x"]))
    block = dict(post=s["post"], w_post=s["w_post"], w_pre=s["w_pre"], gate=s["gate"], gate_rows=s["rows"], alpha=ALPHA,
                 beta=BETA)
    if op == "norm":
        h, x, r_post, r_pre = spec.block_norm(s["h"], s["y"], eps=EPS, **block)
        return {"h": h, "x": x, "r_post": r_post, "r_pre": r_pre}
    dh, dy, dw_post, dw_pre, dgate = spec.block_norm_grad(s["dx"], s["dout"], mx(s["out"]), mx(s["y"]), s["r_pre"],
                                                          s["r_post"], **block)
    return {"dh": dh, "dy": dy, "dw_post": dw_post, "dw_pre": dw_pre, "dgate": dgate}


# ---------------------------------------------------------------- plain forms

def _rows_of(s, n):
    """The gate row of every row, or None."""
    return None if s["gate"] is None else torch.arange(n, device=s["gate"].device) // s["rows"]


def _norm(s):
    h, y, dt = s["h"].float(), s["y"].float(), s["h"].dtype
    r_post = None
    if s["post"]:
        r_post = 1.0 / torch.sqrt((y * y).mean(1) + EPS)
        y = y * r_post[:, None] * s["w_post"].float()
    if s["gate"] is not None:
        y = y * s["gate"].float()[_rows_of(s, y.shape[0])]
    h = ALPHA * h + BETA * y
    r_pre = 1.0 / torch.sqrt((h * h).mean(1) + EPS)
    return {"h": h.to(dt), "x": (h * r_pre[:, None] * s["w_pre"].float()).to(dt), "r_post": r_post, "r_pre": r_pre}


def _plain(s):
    op = s["op"]
    if op == "pack":
        return _unpack(_pack(s["x"], s["fmt"]) + (s["x"].shape[1], s["fmt"])).to(s["x"].dtype)
    if op == "linear":
        return torch.matmul(s["x"].float(), _unpack(s["w"]).t()).to(s["dtype"])
    if op == "product":
        return torch.matmul(_unpack(s["x"]), _unpack(s["w"]).t()).to(s["dtype"])
    if op == "wgrad":
        return torch.matmul(s["dy"].float().t(), _unpack(s["x"])).to(s["dy"].dtype)
    if op == "norm":
        return _norm(s)
    out, y = (_unpack(v) if isinstance(v, tuple) else v.float() for v in (s["out"], s["y"]))
    dx, dt = s["dx"].float(), s["dx"].dtype
    n = out * s["r_pre"][:, None]
    a = dx * s["w_pre"].float()
    dout = s["dout"].float() + s["r_pre"][:, None] * (a - n * (a * n).mean(1, keepdim=True))
    dw_pre = (dx * n).sum(0)
    n = y * s["r_post"][:, None] if s["post"] else y
    b = BETA * dout
    dgate = dw_post = None
    if s["gate"] is not None:
        rows = _rows_of(s, y.shape[0])
        dgate = torch.zeros(s["gate"].shape, device=y.device).index_add_(0, rows, b * n)
        if s["post"]:
            dgate = dgate * s["w_post"].float()
        b = b * s["gate"].float()[rows]
    if s["post"]:
        dw_post = (b * n).sum(0)
        b = b * s["w_post"].float()
        b = s["r_post"][:, None] * (b - n * (b * n).mean(1, keepdim=True))
    return {"dh": (ALPHA * dout).to(dt), "dy": b.to(dt), "dw_post": dw_post, "dw_pre": dw_pre, "dgate": dgate}


def _packed_bytes(rows, cols, fmt):
    """Codes and scales, without the padding."""
    return rows * (cols if fmt == "int8" else cols / 2) + rows * (-(-cols // 32))


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op in ("linear", "product", "wgrad"):
        T, N, K = case["T"], case["N"], case["K"]
        x = T * K * es if op == "linear" else _packed_bytes(T, K, "int8" if op == "wgrad" else "fp4")
        w = _packed_bytes(N, K, "fp4") if op != "wgrad" else N * K * es
        return {"bytes": x + w + T * N * es, "flops": 2 * T * N * K}
    n, d = case["n"], case["d"]
    if op == "pack":  # the packed matrix is written by one call and read by the other
        return {"bytes": 2 * n * d * es + 2 * _packed_bytes(n, d, case["fmt"]), "flops": 4 * n * d}
    rows = case["gate_rows"]
    gates = -(-n // rows) * d if rows else 0
    small = (1 + case["post"]) * n * 4
    if op == "norm":
        return {"bytes": 4 * n * d * es + gates * es + small, "flops": (12 if case["post"] else 8) * n * d}
    stored = 2 * _packed_bytes(n, d, "int8") if case["stored8"] else 2 * n * d * es
    return {"bytes": 4 * n * d * es + stored + gates * (es + 4) + small, "flops": (24 if case["post"] else 16) * n * d}


# ---------------------------------------------------------------- definitions in float64

_VALUES = {"int8": [(i if i < 128 else i - 256) / 64 for i in range(256)],
           "fp4": [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]}


def _exact_values(p):
    if not isinstance(p, tuple):
        return p.double()
    q, s, c, fmt = p
    table = torch.tensor(_VALUES[fmt], dtype=torch.float64, device=q.device)
    if fmt == "fp4":
        q = torch.stack((q % 16, q // 16), 2).flatten(1)
    scale = ((s.long() + (1023 - 127)) << 52).view(torch.float64).repeat_interleave(32, 1)
    return table[q[:, :c].long()] * scale[:, :c]


def _exact_pack(x, fmt):
    """The nearest values that the format holds, by search among them."""
    pos = sorted(v for v in set(_VALUES[fmt]) if v >= 0 and v < 2 or fmt == "fp4" and v >= 0)
    grid = torch.tensor(pos, dtype=torch.float64, device=x.device)
    n, c = x.shape
    v = torch.nn.functional.pad(x.double(), (0, -c % 32)).view(n, -1, 32)
    limit = 127.5 / 64 if fmt == "int8" else 7.0  # halfway from the largest value to the next
    e = torch.frexp(v.abs().amax(2, keepdim=True) / limit).exponent.clamp(-127, 127 if fmt == "int8" else 125)
    scale = ((e.long() + 1023) << 52).view(torch.float64)
    a = v.abs() / scale
    hi = torch.searchsorted(grid, a.flatten()).view(a.shape).clamp(1, len(pos) - 1)
    below, above = grid[hi - 1], grid[hi]
    up = (above - a < a - below) | ((above - a == a - below) & (hi % 2 == 0))
    return (torch.where(up, above, below) * scale * torch.sign(v)).view(n, -1)[:, :c]


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "pack":
        return _exact_pack(s["x"], s["fmt"])
    if op in ("linear", "product"):
        return torch.nn.functional.linear(_exact_values(s["x"]), _exact_values(s["w"]))
    if op == "wgrad":
        return torch.matmul(s["dy"].double().t().contiguous(), _exact_values(s["x"]))
    v = {k: s[k].double().requires_grad_() for k in ("w_post", "w_pre", "gate") if s[k] is not None}
    y = _exact_values(s["y"]).requires_grad_()
    n, d = y.shape

    def normed(x, weight, r=None):
        """x r(x), or for a given r at the present x its first-order form there."""
        if r is None:
            r = torch.rsqrt(torch.linalg.vector_norm(x, dim=1, keepdim=True) ** 2 / d + EPS)
            return x * r * weight, r[:, 0]
        r, at = r.double()[:, None], x.detach()
        r = r - r ** 3 * ((x - at) * at).mean(1, keepdim=True)
        return x * r * weight, r[:, 0]

    u, r_post = y, None
    if s["post"]:
        u, r_post = normed(y, v["w_post"], s.get("r_post"))
    if "gate" in v:
        u = u * torch.repeat_interleave(v["gate"], s["rows"], 0)[:n]
    if op == "norm":
        with torch.no_grad():
            h = s["h"].double() * ALPHA + u * BETA
            x, r_pre = normed(h, v["w_pre"])
            return {"h": h, "x": x, "r_post": r_post if r_post is None else r_post.detach(), "r_pre": r_pre}
    # a residual h whose sum with the rest is the stored h'
    at = _exact_values(s["out"])
    h = ((at - BETA * u) / ALPHA).detach().requires_grad_()
    out = ALPHA * h + BETA * u
    x = normed(out, v["w_pre"], s["r_pre"])[0]
    total = (x * s["dx"].double()).sum() + (out * s["dout"].double()).sum()
    names = ["dh", "dy", "dw_pre"] + (["dw_post"] if s["post"] else []) + (["dgate"] if "gate" in v else [])
    leaves = {"dh": h, "dy": y, "dw_pre": v.get("w_pre"), "dw_post": v.get("w_post"), "dgate": v.get("gate")}
    got = dict(zip(names, torch.autograd.grad(total, [leaves[k] for k in names])))
    return {k: got.get(k) for k in ("dh", "dy", "dw_post", "dw_pre", "dgate")}
