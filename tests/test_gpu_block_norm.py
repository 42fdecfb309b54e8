"""The norms around a residual block, and their gradients, against their definitions in float64.

Bounds.  u = 2^-24, r the output type's unit roundoff (2^-8 bf16, 2^-24 f32).  A sum of m
terms accumulated in f32, in any order, is off by at most (m + 2) u sum|terms|; a
product of k factors by k u; division and square root are correctly rounded or off by 2 u."""
import pytest

from gpu_util import print_case

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 1e-6


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


def _r(dt):
    import torch
    return torch.finfo(dt).eps / 2


def _strided(x, pad, shift=0):
    import torch
    n, d = x.shape
    buf = torch.full((n * (d + pad) + shift,), float("nan"), dtype=x.dtype, device=x.device)
    y = torch.as_strided(buf, (n, d), (d + pad, 1), shift)
    y.copy_(x)
    return y


class Case:
    """Inputs of one block; gate_rows 0: no gate."""

    def __init__(self, n, d, dtype, post=True, gate_rows=0, weights=True, pad=0, seed=0, alpha=0.9, beta=-0.6):
        import torch
        g = torch.Generator(device="cuda")
        g.manual_seed(seed + n + d)

        def rand(*s):
            return torch.randn(*s, generator=g, device="cuda")
        dt = _dt(dtype)
        self.n, self.d, self.dt, self.post, self.rows = n, d, dt, post, max(gate_rows, 1)
        self.alpha, self.beta = alpha, beta
        self.h, self.y, self.dx, self.dout = (
            _strided((rand(n, d) * torch.exp(0.5 * rand(d))).to(dt), pad, 1 if pad else 0) for _ in range(4))
        self.w_post = (1 + 0.3 * rand(d)).to(dt) if weights and post else None
        self.w_pre = (1 + 0.3 * rand(d)).to(dt) if weights else None
        self.gate = _strided(rand(-(-n // gate_rows), d).to(dt), pad) if gate_rows else None

    @property
    def args(self):
        return dict(post=self.post, w_post=self.w_post, w_pre=self.w_pre, gate=self.gate, gate_rows=self.rows,
                    alpha=self.alpha, beta=self.beta)

    def f64(self):
        """(w_post, w_pre, gate per row) in float64, ones where there are none."""
        import torch
        one = torch.ones(self.d, dtype=torch.float64, device="cuda")
        gate = one.expand(self.n, self.d)
        if self.gate is not None:
            gate = self.gate.double()[torch.arange(self.n, device="cuda") // self.rows]
        return (one if self.w_post is None else self.w_post.double()), (one if self.w_pre is None else self.w_pre.double()), gate


def _norm(v):
    return ((v * v).mean(1, keepdim=True) + EPS).rsqrt()


def _within(got, want, tol, what):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), ((got.double() - want).abs() / tol).max().item())


def check_forward(c, out):
    h2, x, r_post, r_pre = out
    w1, w2, g = c.f64()
    h, y = c.h.double(), c.y.double()
    r, rel = _r(c.dt), (c.d / 2 + 8) * U  # of a factor r_post or r_pre: half of the sum's, the mean's, eps', the root's
    u = y
    if c.post:
        ry = _norm(y)
        _within(r_post, ry[:, 0], rel * ry[:, 0], "r_post")
        u = y * ry * w1
    u = c.beta * g * u
    want = c.alpha * h + u
    dh = (rel + 5 * U) * u.abs() + 3 * U * (c.alpha * h).abs()
    _within(h2, want, dh + r * want.abs() + 1e-37, "Hout")
    rh = _norm(want)
    rrel = rel + (dh * dh).sum(1, keepdim=True).sqrt() / (want * want).sum(1, keepdim=True).sqrt().clamp(min=1e-30)
    _within(r_pre, rh[:, 0], (rrel * rh)[:, 0], "r_pre")
    wx = want * rh * w2
    _within(x, wx, (w2 * rh).abs() * dh + (rrel + 3 * U + r) * wx.abs() + 1e-37, "X")


def check_grad(c, y, h2, r_post, r_pre, got, dx=True, dout=True):
    """y, h2: the values (float64) that the gradients are formed from."""
    import torch
    dh, dy, dw_post, dw_pre, dgate = got
    w1, w2, g = c.f64()
    n, d, r = c.n, c.d, _r(c.dt)
    zero = torch.zeros(n, d, dtype=torch.float64, device="cuda")
    gx, go = c.dx.double() if dx else zero, c.dout.double() if dout else zero
    r2 = r_pre.double()[:, None]
    a, n2 = gx * w2, h2 * r2
    m = (a * n2).mean(1, keepdim=True)
    e_m = (d + 8) * U * (a * n2).abs().mean(1, keepdim=True)
    G = go + r2 * (a - n2 * m)
    mag = go.abs() + (r2 * a).abs()
    e_G = 5 * U * mag + (r2 * n2).abs() * (e_m + 5 * U * m.abs()) + 2 * U * G.abs()
    _within(dh, c.alpha * G, abs(c.alpha) * e_G + (r + 2 * U) * (c.alpha * G).abs() + 1e-37, "dH")
    if dx and c.w_pre is not None:
        _within(dw_pre, (gx * n2).sum(0), (n + 8) * U * (gx * n2).abs().sum(0) + 1e-37, "dw_pre")
    r1 = r_post.double()[:, None] if c.post else 1.0
    n1 = y * r1
    f = c.beta * g * w1
    b = f * G
    mb = (b * n1).mean(1, keepdim=True) if c.post else 0.0
    cf = (f * n1).abs()
    # mean(b n1) is formed as mean(f n1 base) - r2 m mean(f n1 n2)
    e_mb = ((d + 12) * U * ((cf * mag).mean(1, keepdim=True) + (r2 * m).abs() * (cf * n2.abs()).mean(1, keepdim=True)) +
            r2 * e_m * (cf * n2.abs()).mean(1, keepdim=True)) if c.post else 0.0
    want = r1 * (b - n1 * mb)
    e = r1 * (f.abs() * e_G + 5 * U * b.abs() + n1.abs() * (e_mb + 5 * U * (mb.abs() if c.post else 0.0)))
    _within(dy, want, e + (r + 2 * U) * want.abs() + 1e-37, "dY")
    s, e_s = c.beta * G * n1, abs(c.beta) * n1.abs() * (e_G + 5 * U * G.abs())
    if c.w_post is not None:
        _within(dw_post, (g * s).sum(0), (g.abs() * (e_s + (n + 10) * U * s.abs())).sum(0) + 1e-37, "dw_post")
    if c.gate is not None:
        k = torch.arange(n, device="cuda") // c.rows
        out = torch.zeros(dgate.shape, dtype=torch.float64, device="cuda")
        tol = torch.zeros_like(out)
        _within(dgate, out.index_add_(0, k, w1 * s), tol.index_add_(0, k, w1.abs() * (e_s + (c.rows + 10) * U * s.abs())) + 1e-37,
                "dgate")


SIZES = [(1, 1), (1, 4096), (3, 31), (8, 4096), (5, 513), (17, 1000), (130, 64), (700, 96), (33, 2047), (9, 2049),
         (6, 5000), (5, 8192), (3, 8193), (2, 16384), (2100, 1024), (600, 2056)]
GATES = ["none", "one", "each", "some"]


def _gate_rows(kind, n):
    return {"none": 0, "one": n, "each": 1, "some": max(1, n // 3)}[kind]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,d", SIZES)
@pytest.mark.parametrize("post,gate,weights,pad", [(True, "one", True, 0), (True, "some", True, 3), (False, "each", True, 0),
                                                   (False, "none", False, 8), (True, "none", False, 0)])
def test_block_norm(spec, dtype, n, d, post, gate, weights, pad):
    import torch
    print_case("block_norm", dtype=dtype, n=n, d=d, post=post, gate=gate, weights=weights, pad=pad)
    c = Case(n, d, dtype, post, _gate_rows(gate, n), weights, pad)
    out = spec.block_norm(c.h, c.y, eps=EPS, **c.args)
    check_forward(c, out)
    # in place, and with all three matrices stored as mx_quantize stores them
    h, y = c.h.clone(), c.y.clone()
    m = [spec.mx_empty(n, d, spec.MX_INT8) for _ in range(3)]
    for v in m:
        v.q.fill_(0xA5), v.s.fill_(0xA5)
    again = spec.block_norm(h, y, eps=EPS, Hout=h, X=y, y8=m[0], h8=m[1], x8=m[2], **c.args)
    for a, b in zip(out, again):
        assert (a is None and b is None) or torch.equal(a, b)
    for v, t in zip(m, (c.y, out[0], out[1])):
        q = spec.mx_quantize(t, spec.MX_INT8)
        assert torch.equal(v.q, q.q) and torch.equal(v.s, q.s)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,d", SIZES + [(1500, 128), (3000, 40)])
@pytest.mark.parametrize("post,gate,weights,pad,stored8", [
    (True, "one", True, 0, False), (True, "some", True, 3, True), (False, "each", True, 0, True),
    (False, "none", False, 8, False), (True, "each", True, 0, False), (True, "none", True, 0, True)])
def test_block_norm_grad(spec, dtype, n, d, post, gate, weights, pad, stored8):
    import torch
    print_case("block_norm_grad", dtype=dtype, n=n, d=d, post=post, gate=gate, weights=weights, pad=pad, stored8=stored8)
    c = Case(n, d, dtype, post, _gate_rows(gate, n), weights, pad)
    h2, x, r_post, r_pre = spec.block_norm(c.h, c.y, eps=EPS, **c.args)
    y = c.y
    if stored8:
        y, h2 = spec.mx_quantize(y, spec.MX_INT8), spec.mx_quantize(h2, spec.MX_INT8)
    yv, hv = (spec.mx_dequantize(t, torch.float32).double() if stored8 else t.double() for t in (y, h2))
    got = spec.block_norm_grad(c.dx, c.dout, h2, y, r_pre, r_post, **c.args)
    check_grad(c, yv, hv, r_post, r_pre, got)
    # the same in every run, and in place
    dx, dout = c.dx.clone(), c.dout.clone()
    again = spec.block_norm_grad(dx, dout, h2, y, r_pre, r_post, dH=dout, dY=dx, **c.args)
    for a, b in zip(got, again):
        assert (a is None and b is None) or torch.equal(a, b)


@pytest.mark.parametrize("n,d,rows", [(1030, 72, 2), (2600, 40, 5), (2600, 1056, 7), (1300, 1100, 3), (1024, 2064, 500),
                                      (3000, 64, 9), (5000, 33, 4999), (2048, 1032, 20)])
def test_gate_rows_of_all_kinds(spec, n, d, rows):
    """Whole gate rows to a worker, one gate row over many, and runs that end inside the last."""
    print_case("block_norm_grad gates", n=n, d=d, rows=rows)
    c = Case(n, d, "f32", True, rows)
    h2, x, r_post, r_pre = spec.block_norm(c.h, c.y, eps=EPS, **c.args)
    check_forward(c, (h2, x, r_post, r_pre))
    check_grad(c, c.y.double(), h2.double(), r_post, r_pre, spec.block_norm_grad(c.dx, c.dout, h2, c.y, r_pre, r_post, **c.args))


def test_parts_that_are_absent(spec):
    """The norm of the stream alone; only one of the two gradients; no rows."""
    import torch
    c = Case(37, 300, "bf16", True, 37)
    h, x, r_post, r_pre = spec.block_norm(c.h, eps=EPS, w_pre=c.w_pre)
    assert h is c.h and r_post is None
    hd = c.h.double()
    want = hd * _norm(hd) * c.w_pre.double()
    _within(x, want, (2.0 ** -8 + 200 * U) * want.abs(), "norm alone")
    dh, dy, dw_post, dw_pre, dgate = spec.block_norm_grad(c.dx, None, c.h, None, r_pre, w_pre=c.w_pre)
    assert dy is None and dw_post is None and dgate is None
    ref = hd.clone().requires_grad_()
    w = c.w_pre.double().requires_grad_()
    gh, gw = torch.autograd.grad((ref * _norm(ref) * w * c.dx.double()).sum(), (ref, w))
    # r_pre comes 158 u off, n2 twice in the mean's part and the mean of 300 terms 308 u: 3 of those of the largest term
    _within(dh, gh, 2.0 ** -8 * gh.abs() + 1000 * U * (r_pre[:, None] * c.dx.double() * c.w_pre.double()).abs().amax(), "dH of the norm alone")
    _within(dw_pre, gw, 210 * U * (hd * r_pre.double()[:, None] * c.dx.double()).abs().sum(0), "dw_pre of the norm alone")
    h2, x, r_post, r_pre = spec.block_norm(c.h, c.y, eps=EPS, **c.args)
    for dx, dout in ((True, False), (False, True)):
        got = spec.block_norm_grad(c.dx if dx else None, c.dout if dout else None, h2, c.y, r_pre, r_post, **c.args)
        check_grad(c, c.y.double(), h2.double(), r_post, r_pre, got, dx, dout)
        assert dx or got[3] is None
    c = Case(1, 65, "f32", True, 1)
    e = torch.empty(0, 65, device="cuda")
    args = dict(c.args, gate=c.gate[:0])
    out = spec.block_norm(e, e, eps=EPS, **args)
    assert [tuple(t.shape) for t in out] == [(0, 65), (0, 65), (0,), (0,)]
    got = spec.block_norm_grad(e, e, e, e, out[3], out[2], **args)
    assert not got[2].any() and not got[3].any() and got[4].shape == (0, 65)


def test_zero_rows_and_large_values(spec):
    """Rows of zeros, values whose squares leave f32, NaN in one row."""
    import torch
    for d in (100, 3000):
        c = Case(12, d, "f32", True, 12)
        c.h[3], c.y[3], c.y[4] = 0, 0, 0
        c.y[5] *= 1e25
        c.h[6] *= 1e30
        h2, x, r_post, r_pre = spec.block_norm(c.h, c.y, eps=EPS, **c.args)
        check_forward(c, (h2, x, r_post, r_pre))
        assert not x[3].any() and r_pre[3] == r_post[3] == r_post[4] == torch.tensor(EPS).rsqrt()
        c.y[7, d - 1] = float("nan")
        h3, x3, _, _ = spec.block_norm(c.h, c.y, eps=EPS, **c.args)
        rest = [i for i in range(12) if i != 7]
        assert x3[7].isnan().all() and torch.equal(x3[rest], x[rest]) and torch.equal(h3[rest], h2[rest])


def test_gradients_are_differences(spec):
    """<gradient, v> against the central difference of the float64 definition along v: for the residual
    stream, the block's output, both weights and the gate at once and one by one."""
    import torch
    c = Case(23, 140, "f32", True, 8)
    h2, x, r_post, r_pre = spec.block_norm(c.h, c.y, eps=EPS, **c.args)
    dh, dy, dw_post, dw_pre, dgate = spec.block_norm_grad(c.dx, c.dout, h2, c.y, r_pre, r_post, **c.args)
    at = [t.double() for t in (c.h, c.y, c.w_post, c.w_pre, c.gate)]
    grads = [t.double() for t in (dh, dy, dw_post, dw_pre, dgate)]

    def loss(h, y, w1, w2, gate):
        g = gate[torch.arange(c.n, device="cuda") // c.rows]
        o = c.alpha * h + c.beta * g * (y * _norm(y) * w1)
        return (o * _norm(o) * w2 * c.dx.double()).sum() + (o * c.dout.double()).sum()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    for only in (None, 0, 1, 2, 3, 4):
        v = [torch.randn(t.shape, generator=gen, device="cuda", dtype=torch.float64) * (only is None or only == i)
             for i, t in enumerate(at)]
        e = 1e-5
        diff = (loss(*[a + e * b for a, b in zip(at, v)]) - loss(*[a - e * b for a, b in zip(at, v)])) / (2 * e)
        dot = sum((a * b).sum() for a, b in zip(grads, v))
        mag = sum((a * b).abs().sum() for a, b in zip(grads, v))
        # the gradients' own errors (some tens of u each) and the difference's e^2 f''' / 6
        assert abs(dot - diff) <= 300 * U * mag + 1e-6, (only, dot.item(), diff.item())


def test_captured_and_on_another_stream(spec):
    """Two graphs that share a workspace, replayed in turn with eager calls between."""
    import torch
    cases = [Case(300, 1000, "bf16", True, 50), Case(40, 3000, "bf16", False, 40)]
    ws = torch.empty(max(spec.block_norm_grad_workspace(c.n, c.d, c.dt, c.gate.shape[0], c.rows) for c in cases),
                     dtype=torch.uint8, device="cuda")

    def step(c, ws=None):
        h2, x, r_post, r_pre = spec.block_norm(c.h, c.y, eps=EPS, **c.args)
        y8 = spec.mx_quantize(c.y, spec.MX_INT8)
        return [t for t in (h2, x) + spec.block_norm_grad(c.dx, c.dout, h2, y8, r_pre, r_post, ws=ws, **c.args) if t is not None]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step(cases[0])
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(other, step(cases[0])))
    graphs = []
    for c in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step(c, ws)
        graphs.append((c, g, out))
    for k in range(3):
        for c, g, out in graphs:
            for t in (c.h, c.y, c.dx, c.dout):
                t.copy_(torch.randn(t.shape, device="cuda"))
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, step(c)))
