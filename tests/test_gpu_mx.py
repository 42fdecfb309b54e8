"""Microscaled storage and the products with it against their definitions in float64.

Storage is exact: the values, the scales and the padding are compared for equality.
Products: u = 2^-24, r the output type's unit roundoff (2^-8 bf16, 2^-24 f32).  The
operands are exact in the products' type, and a sum of m products accumulated in f32,
in any order, is off by at most (m + 2) u sum|terms|; the output is rounded once."""
import pytest

from gpu_util import print_case

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
FP4 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


@pytest.fixture(scope="module")
def spec():
    import torch
    import weights_bf16_fp32_amd as spec
    assert torch.cuda.is_available()
    spec.lib()
    return spec


def _dt(name):
    import torch
    return torch.bfloat16 if name == "bf16" else torch.float32


def _r(name):
    import torch
    return torch.finfo(_dt(name)).eps / 2


def _gen(seed):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _strided(x, pad, shift=0):
    """x with rows `pad` elements further apart, its first element `shift` elements into the buffer;
    NaN in between."""
    import torch
    n, d = x.shape
    buf = torch.full((n * (d + pad) + shift,), float("nan"), dtype=x.dtype, device=x.device)
    y = torch.as_strided(buf, (n, d), (d + pad, 1), shift)
    y.copy_(x)
    return y


def _fmt(spec, name):
    return spec.MX_INT8 if name == "int8" else spec.MX_FP4


def _pow2(e):
    """2^e in float64 for integers e, from its bits (torch's ldexp rounds)."""
    import torch
    return ((e.long() + 1023) << 52).view(torch.float64)


def _stored(x, fmt):
    """(values, scale bytes) of x [n, c] in float64: the nearest multiples, by search."""
    import torch
    n, c = x.shape
    grid = torch.tensor([i / 64 for i in range(128)] if fmt == "int8" else FP4, dtype=torch.float64, device=x.device)
    v = torch.nn.functional.pad(x.double(), (0, -c % 32)).view(n, (c + 31) // 32, 32)
    bad = ~v.isfinite().all(2, keepdim=True)
    top = torch.where(bad, 0.0, v.abs().amax(2, keepdim=True))
    # the smallest power of two at which top / scale lies below the middle to the next value that is not held
    _, e = torch.frexp(top / (127.5 / 64 if fmt == "int8" else 7.0))
    e = torch.where(top == 0, -127, e.clamp(-127, 127 if fmt == "int8" else 125))
    scale = _pow2(e)
    a = (v.abs() / scale).nan_to_num(0.0, 0.0).clamp(max=float(grid[-1]))
    hi = torch.searchsorted(grid, a.flatten()).view(a.shape).clamp(1, len(grid) - 1)
    lo = hi - 1
    d = (grid[hi] - a) - (a - grid[lo])
    i = torch.where((d < 0) | ((d == 0) & (hi % 2 == 0)), hi, lo)
    out = torch.where(bad, float("nan"), torch.copysign(grid[i] * scale, v))
    return out.flatten(1)[:, :c], torch.where(bad, 255, e + 127)[:, :, 0].to(torch.uint8)


def _values(spec, m):
    """The values of storage in float64, read from its bytes."""
    import torch
    q, s = m.q, m.s
    nb = (m.cols + 31) // 32
    if m.fmt == spec.MX_INT8:
        v = q[:, :nb * 32].view(torch.int8).double() / 64
    else:
        table = torch.tensor(FP4 + [-x for x in FP4], dtype=torch.float64, device=q.device)
        q = q[:, :nb * 16]
        v = table[torch.stack((q & 15, q >> 4), 2).flatten(1).long()]
    scale = _pow2(s[:, :nb].int() - 127)
    scale = torch.where(s[:, :nb] == 255, float("nan"), scale)
    return (v.view(len(q), nb, 32) * scale[:, :, None]).flatten(1)[:, :m.cols]


def _same(a, b):
    return bool(((a == b) | (a.isnan() & b.isnan())).all())


def _mixed(g, n, c):
    """Values over many magnitudes, with zero rows."""
    import torch
    x = torch.randn(n, c, generator=g, device="cuda") * torch.exp2(torch.randint(-6, 7, (n, c), generator=g, device="cuda").float())
    x = x * torch.exp2(torch.randint(-60, 60, (n, 1), generator=g, device="cuda").float())
    x[torch.rand(n, generator=g, device="cuda") < 0.1] = 0
    return x


# ---------------------------------------------------------------- storage

@pytest.mark.parametrize("fmt", ["int8", "fp4"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,c,pad,shift", [
    (1, 1, 0, 0), (3, 31, 0, 0), (2, 32, 0, 0), (5, 33, 7, 0), (9, 8, 0, 1), (7, 1000, 1, 3), (1, 14336, 0, 0),
    (130, 4104, 8, 0), (257, 520, 0, 0), (4, 8191, 0, 0), (1025, 65, 0, 0), (0, 64, 0, 0)])
def test_storage(spec, fmt, dtype, n, c, pad, shift):
    import torch
    print_case("mx_quantize", fmt=fmt, dtype=dtype, n=n, c=c, pad=pad, shift=shift)
    x = _strided(_mixed(_gen(n + c), n, c).to(_dt(dtype)), pad, shift) if n else torch.empty((0, c), dtype=_dt(dtype), device="cuda")
    lq, ls = spec._mx_rows(_fmt(spec, fmt), c)
    q = torch.full((n, lq + 16), 0xA5, dtype=torch.uint8, device="cuda")
    s = torch.full((n, ls + 16), 0xA5, dtype=torch.uint8, device="cuda")
    m = spec.mx_quantize(x, _fmt(spec, fmt), out=spec.Mx(q, s, c, _fmt(spec, fmt)))
    want, scales = _stored(x, fmt)
    assert _same(_values(spec, m), want)
    assert torch.equal(s[:, :scales.shape[1]], scales)
    # whole blocks and groups of scales are written, zero past the columns; nothing behind them
    assert not s[:, scales.shape[1]:ls].any() and bool((s[:, ls:] == 0xA5).all()) and bool((q[:, lq:] == 0xA5).all())
    used = c if fmt == "int8" else (c + 1) // 2
    assert not q[:, used:lq].any() and (fmt == "int8" or c % 2 == 0 or not (q[:, used - 1] >> 4).any())
    for out in ("bf16", "f32"):  # exact in both
        y = _strided(torch.zeros((n, c), dtype=_dt(out), device="cuda"), pad, shift) if n else None
        y = spec.mx_dequantize(m, _dt(out), out=y)
        assert y.dtype == _dt(out) and _same(y.double(), want)


@pytest.mark.parametrize("fmt", ["int8", "fp4"])
def test_storage_of_every_bf16(spec, fmt):
    """Every bf16 as the largest of a block and beside each of a few larger ones: NaN, infinities, zeros
    of both signs, subnormal and the largest values are among them."""
    import torch
    bits = torch.arange(65536, device="cuda").to(torch.int32).to(torch.int16).view(torch.bfloat16)
    one = torch.zeros((65536, 32), dtype=torch.bfloat16, device="cuda")
    one[:, 5] = bits
    beside = bits.view(2048, 32).clone()
    tops = torch.tensor([1.0, 1.75, 1.9921875, 6.0, 7.0, 127.0, 2.0 ** -126, 2.0 ** 127, 3.3895e38], device="cuda").bfloat16()
    finite = torch.where(bits.isfinite(), bits, torch.zeros_like(bits))
    for x in [one, beside] + [torch.cat((torch.where(finite.abs() <= t, finite, 0 * finite).view(-1, 16),
                                         t.expand(4096, 16)), 1) for t in tops]:
        m = spec.mx_quantize(x, _fmt(spec, fmt))
        want, scales = _stored(x, fmt)
        assert torch.equal(m.s[:, :scales.shape[1]], scales)
        assert _same(_values(spec, m), want)
        assert _same(spec.mx_dequantize(m, torch.float32).double(), want)
        y = spec.mx_dequantize(m).double()
        assert _same(y, want.bfloat16().double())  # (below 2^-133 nothing is held in bf16)


@pytest.mark.parametrize("fmt", ["int8", "fp4"])
def test_storage_ties_in_f32(spec, fmt):
    """Halfway between two held values, and next to it on both sides; every exponent of f32."""
    import torch
    if fmt == "int8":
        mid = torch.arange(127, device="cuda", dtype=torch.float64) / 64 + 1 / 128
    else:
        g = torch.tensor(FP4, dtype=torch.float64, device="cuda")
        mid = (g[1:] + g[:-1]) / 2
    rows = []
    for k in (-1, 0, 1):
        v = (mid.float().view(torch.int32) + k).view(torch.float32)
        v = torch.cat((v, -v))
        v = torch.nn.functional.pad(v, (0, -len(v) % 31)).view(-1, 31)
        rows.append(torch.cat((v, torch.full((len(v), 1), 1.5 if fmt == "int8" else 6.0, device="cuda")), 1))
    base = torch.cat(rows).double()
    x = (base[None] * _pow2(torch.arange(-127, 126, device="cuda"))[:, None, None]).float().view(-1, 32)
    m = spec.mx_quantize(x, _fmt(spec, fmt))
    want, scales = _stored(x, fmt)
    assert torch.equal(m.s[:, :1], scales) and _same(_values(spec, m), want)
    assert _same(spec.mx_dequantize(m, torch.float32).double(), want.float().double())


def test_storage_half_step(spec):
    """A value is off by half a step of its block at most, whatever the block."""
    import torch
    x = _mixed(_gen(3), 500, 640)
    top = x.view(500, 20, 32).abs().amax(2).double()
    for fmt, rel in (("int8", 1 / 127), ("fp4", 1 / 6)):  # half the largest step over the least top: 0.5 / 63.75, 1 / 3.5
        err = (_values(spec, spec.mx_quantize(x, _fmt(spec, fmt))) - x.double()).abs().view(500, 20, 32).amax(2)
        assert bool((err <= top * (rel if fmt == "int8" else 1 / 3.5)).all())


def test_storage_past_32_bits(spec):
    import torch
    n, c = 270000, 16384  # 4.4 GB of codes: the last rows lie past 2^32 bytes
    x = torch.empty((n, c), dtype=torch.bfloat16, device="cuda")
    x[:] = 1.0
    x[-2:] = torch.arange(c, device="cuda").remainder(61).bfloat16()
    m = spec.mx_quantize(x, spec.MX_INT8)
    y = spec.mx_dequantize(m)
    assert torch.equal(y[:3], x[:3]) and torch.equal(y[-3:], x[-3:])


# ---------------------------------------------------------------- products

def _operand(g, n, k, dtype):
    import torch
    return (torch.randn(n, k, generator=g, device="cuda") * torch.exp(torch.randn(k, generator=g, device="cuda"))).to(_dt(dtype))


def _close(got, a, b, dtype, base=None):
    """got = base + a b^T within the bound above."""
    import torch
    want, mag = a @ b.t().contiguous(), a.abs() @ b.abs().t().contiguous()
    if base is not None:
        want, mag = want + base, mag + base.abs()
    tol = (a.shape[1] + 3) * U * mag * 1.01 + _r(dtype) * want.abs() + 1e-37
    bad = (got.double() - want).abs() > tol
    assert not bad.any(), (int(bad.sum()), ((got.double() - want).abs() / tol).max().item())


SHAPES = [(1, 1, 1), (1, 32, 32), (1, 4096, 4096), (2, 100, 33), (7, 333, 1000), (8, 1024, 2048), (16, 50, 64), (17, 257, 96),
          (31, 130, 4096), (33, 1000, 520), (64, 512, 256), (65, 129, 1000), (130, 300, 31), (257, 1000, 777),
          (300, 512, 4096), (1000, 1023, 64), (600, 4096, 1024)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,N,K", SHAPES)
@pytest.mark.parametrize("pad,shift", [(0, 0), (5, 1)])
def test_linear(spec, dtype, T, N, K, pad, shift):
    import torch
    print_case("mx_linear", dtype=dtype, T=T, N=N, K=K, pad=pad, shift=shift)
    g = _gen(T + N + K)
    x = _strided(_operand(g, T, K, dtype), pad, shift)
    w = spec.mx_quantize(torch.randn(N, K, generator=g, device="cuda"), spec.MX_FP4)
    buf = torch.full((T, N + pad), 7.0, dtype=_dt(dtype), device="cuda")
    y = spec.mx_linear(x, w, out=buf[:, :N])
    _close(y, x.double(), _values(spec, w), dtype)
    assert bool((buf[:, N:] == 7.0).all())
    assert torch.equal(y, spec.mx_linear(x, w))  # the same in every run


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,N,K", SHAPES)
def test_product(spec, dtype, T, N, K):
    import torch
    print_case("mx_product", dtype=dtype, T=T, N=N, K=K)
    g = _gen(T * 3 + N + K)
    x = spec.mx_quantize(_operand(g, T, K, "f32"), spec.MX_FP4)
    w = spec.mx_quantize(torch.randn(N, K, generator=g, device="cuda"), spec.MX_FP4)
    buf = torch.full((T, N + 3), 7.0, dtype=_dt(dtype), device="cuda")
    y = spec.mx_product(x, w, _dt(dtype), out=buf[:, :N])
    _close(y, _values(spec, x), _values(spec, w), dtype)
    assert bool((buf[:, N:] == 7.0).all())
    assert torch.equal(y, spec.mx_product(x, w, _dt(dtype)))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,N,K", SHAPES + [(4096, 33, 70), (5000, 256, 256), (2049, 64, 1000)])
@pytest.mark.parametrize("pad,beta", [(0, 0.0), (3, 0.75)])
def test_weight_grad(spec, dtype, T, N, K, pad, beta):
    import torch
    print_case("mx_weight_grad", dtype=dtype, T=T, N=N, K=K, pad=pad, beta=beta)
    g = _gen(T * 5 + N + K)
    dy = _strided(_operand(g, T, N, dtype), pad)
    x = spec.mx_quantize(_operand(g, T, K, dtype), spec.MX_INT8)
    buf = torch.randn((N, K + pad), generator=g, device="cuda").to(_dt(dtype))
    if beta == 0.0:
        buf[:] = float("nan")  # what was there does not count
    before = buf.clone()
    got = spec.mx_weight_grad(dy, x, beta=beta, dW=buf[:, :K])
    _close(got, dy.double().t().contiguous(), _values(spec, x).t().contiguous(), dtype,
           None if beta == 0.0 else beta * before[:, :K].double())
    assert torch.equal(buf[:, K:].isnan(), before[:, K:].isnan()) and torch.equal(buf[:, K:].nan_to_num(), before[:, K:].nan_to_num())
    again = before.clone()
    assert torch.equal(got, spec.mx_weight_grad(dy, x, beta=beta, dW=again[:, :K]))


def test_products_without_rows(spec):
    import torch
    w = spec.mx_quantize(torch.randn(70, 64, device="cuda"), spec.MX_FP4)
    none = spec.mx_quantize(torch.empty(0, 64, device="cuda"), spec.MX_FP4)
    assert spec.mx_linear(torch.empty(0, 64, device="cuda"), w).shape == (0, 70)
    assert spec.mx_product(none, w).shape == (0, 70)
    none8 = spec.mx_quantize(torch.empty(0, 50, device="cuda"), spec.MX_INT8)
    dy = torch.empty(0, 40, device="cuda")
    assert not spec.mx_weight_grad(dy, none8).any()
    dw = torch.randn(40, 50, device="cuda")
    assert torch.equal(spec.mx_weight_grad(dy, none8, beta=0.5, dW=dw.clone()), 0.5 * dw)


def test_nan_blocks_reach_their_results_only(spec):
    """A NaN or an infinity in a row makes that row of the result NaN, and no other."""
    import torch
    g = _gen(5)
    for T in (5, 40, 200):
        x, w = torch.randn(T, 300, generator=g, device="cuda"), torch.randn(90, 300, generator=g, device="cuda")
        wq = spec.mx_quantize(w, spec.MX_FP4)
        clean = spec.mx_linear(x.bfloat16(), wq)
        x[2, 299], w[7, 0] = float("nan"), float("inf")
        wn, xq = spec.mx_quantize(w, spec.MX_FP4), spec.mx_quantize(x, spec.MX_FP4)
        y = spec.mx_linear(x.bfloat16(), wn)
        keep = torch.ones(T, 90, dtype=torch.bool, device="cuda")
        keep[2], keep[:, 7] = False, False
        assert torch.equal(y.isnan(), ~keep) and torch.equal(y[keep], clean[keep])
        p = spec.mx_product(xq, wn)
        assert torch.equal(p.isnan(), ~keep)
        dw = spec.mx_weight_grad(torch.ones(T, 33, device="cuda"), spec.mx_quantize(x, spec.MX_INT8))
        assert dw[:, 288:].isnan().all() and not dw[:, :288].isnan().any()


def test_products_from_rows_of_larger_storage(spec):
    """Views of rows, and row strides beyond a row's bytes."""
    import torch
    g = _gen(9)
    x, w = torch.randn(300, 200, generator=g, device="cuda"), torch.randn(150, 200, generator=g, device="cuda")
    big = [torch.full((400, 256), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(2)]
    wq = spec.mx_quantize(w, spec.MX_FP4, out=spec.Mx(big[0][20:170, 16:], big[1][20:170, 32:], 200, spec.MX_FP4))
    want = spec.mx_quantize(w, spec.MX_FP4)
    for T in (3, 300):
        assert torch.equal(spec.mx_linear(x[:T], wq), spec.mx_linear(x[:T], want))
        xq = spec.mx_quantize(x[:T], spec.MX_FP4)
        assert torch.equal(spec.mx_product(xq, wq), spec.mx_product(xq, want))


def test_products_captured_and_on_another_stream(spec):
    import torch
    g = _gen(11)
    T, N, K = 200, 300, 500
    x, dy = torch.randn(T, K, generator=g, device="cuda").bfloat16(), torch.randn(T, N, generator=g, device="cuda").bfloat16()
    w = torch.randn(N, K, generator=g, device="cuda").bfloat16()

    def step(x, dy, w):
        wq, xq, x8 = spec.mx_quantize(w, spec.MX_FP4), spec.mx_quantize(x, spec.MX_FP4), spec.mx_quantize(x, spec.MX_INT8)
        return (spec.mx_linear(x, wq), spec.mx_linear(x[:5], wq), spec.mx_product(xq, wq), spec.mx_weight_grad(dy, x8),
                spec.mx_dequantize(x8))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step(x, dy, w)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(other, step(x, dy, w)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(x, dy, w)
    for _ in range(4):
        for t in (x, dy, w):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, step(x, dy, w)))
