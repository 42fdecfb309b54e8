"""Newton-Schulz orthogonalisation against its definition in float64.

Bounds (2-norm of the error over 2-norm of the result).  bf16 updates: emulated
in float64 with every f16 operand rounded as the kernels round it, gradients
with flat, decaying and rank-32 spectra are off by 0.5e-3 to 1.6e-3 before the
result is rounded to bf16 (1.7e-3 by itself); four times that, 7e-3, is
allowed.  f32 updates: the same emulation's unit is 2^-24 instead of 2^-12, and
products of up to 2000 terms in f32 add their own rounding, amplified alike; a
float32 evaluation of the formula on the CPU is off by 2e-6 to 2e-5 on these
spectra; 8e-5 is allowed."""
import pytest

from gpu_util import print_case

pytestmark = pytest.mark.gpu

LIMIT = {"bf16": 7e-3, "f32": 8e-5}
MUON = (3.4445, -4.7750, 2.0315)


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


def _update(kind, b, m, n, dtype, seed):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    if kind == "flat":
        G = randn(b, m, n)
    elif kind == "decay":  # 512 tokens, features of falling variance
        x = randn(b, 512, m) * torch.arange(1, m + 1, device="cuda").float().rsqrt()
        y = randn(b, 512, n) * torch.arange(1, n + 1, device="cuda").float().rsqrt()
        G = torch.matmul(x.transpose(1, 2).contiguous(), y)
    else:  # rank 32 and a little noise
        k = min(32, m, n)
        G = torch.matmul(randn(b, m, k), randn(b, k, n)) + 0.1 * randn(b, m, n)
    return G.to(_dt(dtype))


def _ref(G, coeffs, eps=1e-7, scale=1.0):
    import torch
    X = G.double()
    X = X / (torch.linalg.vector_norm(X, dim=(-2, -1), keepdim=True) + eps)
    tall = X.shape[-2] > X.shape[-1]
    if tall:
        X = X.transpose(-2, -1).contiguous()
    for a, b, c in coeffs:
        A = torch.matmul(X, X.transpose(-2, -1).contiguous())
        X = a * X + torch.matmul(b * A + c * torch.matmul(A, A), X)
    return scale * (X.transpose(-2, -1) if tall else X)


def _off(got, want):
    import torch
    return (torch.linalg.vector_norm(got.double() - want) / torch.linalg.vector_norm(want)).item()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["flat", "decay", "rank32"])
@pytest.mark.parametrize("m,n", [(64, 64), (128, 128), (129, 257), (100, 1000), (1000, 100), (333, 65), (65, 336),
                                 (512, 512), (1030, 520), (257, 2001)])
def test_orthogonalize(spec, dtype, kind, m, n):
    import torch
    print_case("orthogonalize", m=m, n=n, kind=kind, dtype=dtype)
    G = _update(kind, 1, m, n, dtype, m + n)[0]
    O = spec.orthogonalize(G)
    assert O.dtype == G.dtype and O.shape == G.shape
    assert _off(O, _ref(G, [MUON] * 5)) <= LIMIT[dtype]
    assert torch.equal(O, spec.orthogonalize(G))  # every run the same


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m,n", [(1, 1), (1, 7), (9, 1), (2, 3), (33, 2), (31, 31), (8, 40), (63, 1000)])
def test_small_shapes(spec, dtype, m, n):
    print_case("orthogonalize_small", m=m, n=n, dtype=dtype)
    G = _update("flat", 1, m, n, dtype, 3 * m + n)[0]
    assert _off(spec.orthogonalize(G), _ref(G, [MUON] * 5)) <= LIMIT[dtype]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("b,m,n,pad", [(3, 70, 130, 0), (5, 130, 70, 3), (2, 256, 256, 8), (33, 24, 16, 0)])
def test_batches_and_strides(spec, dtype, b, m, n, pad):
    import torch
    print_case("orthogonalize_batch", b=b, m=m, n=n, pad=pad, dtype=dtype)
    G0 = _update("decay", b, m, n, dtype, b + m)
    G0[1] *= 1e-4  # each matrix has its own norm
    buf = torch.full((b, m + 1, n + pad), float("nan"), dtype=G0.dtype, device="cuda")
    G = buf[:, :m, :n]
    G.copy_(G0)
    coeffs = [(3.0, -3.2, 1.2), (2.0, -1.5, 0.5), (1.875, -1.25, 0.375)]
    O = spec.orthogonalize(G, coeffs=coeffs, scale=0.2, out=torch.empty_like(buf)[:, :m, :n])
    want = _ref(G0, coeffs, scale=0.2)
    for k in range(b):
        assert _off(O[k], want[k]) <= LIMIT[dtype], k
    one = spec.orthogonalize(G[b - 1], coeffs=coeffs, scale=0.2)
    assert torch.equal(one, O[b - 1])
    spec.orthogonalize(G, coeffs=coeffs, scale=0.2, out=G)  # in place, the rest of the buffer untouched
    assert torch.equal(G, O) and bool(buf[:, m:].isnan().all()) and bool(buf[:, :, n:].isnan().all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_known_values(spec, dtype):
    """Matrices whose singular vectors are known: each value goes through the steps' polynomials.
    To first order, a step passes the error e of s on as |p'(s)| e, and adds what the rounding of
    the f16 operand (2^-12 of s, so 2^-11 of s^2) does to s (b s^2 + c s^4); the result is rounded once."""
    import torch
    a, b, c = MUON

    def p(s):
        for _ in range(5):
            s = s * (a + b * s ** 2 + c * s ** 4)
        return s

    def slack(s):
        e = 2.0 ** -20 * s
        for _ in range(5):
            e = (a + 3 * b * s ** 2 + 5 * c * s ** 4).abs() * e
            e += (2.0 ** -11 if dtype == "bf16" else 2.0 ** -21) * s ** 3 * (b + 2 * c * s ** 2).abs() + 2.0 ** -20 * s
            s = s * (a + b * s ** 2 + c * s ** 4)
        return 1.05 * e + torch.finfo(_dt(dtype)).eps / 2 * s.abs()
    n = 96
    s = torch.linspace(1.0, 0.01, n, dtype=torch.float64)
    G = torch.diag(s).to(_dt(dtype)).cuda()
    sv = G.double().diagonal()
    want = p(sv / sv.norm())
    O = spec.orthogonalize(G).double()
    assert bool(((O.diagonal() - want).abs() <= slack(sv / sv.norm())).all())
    assert not (O - torch.diag(O.diagonal())).any()
    one = torch.zeros(40, 300, dtype=_dt(dtype), device="cuda")
    one[17, 200] = -3.0  # rank one
    O = spec.orthogonalize(one).double()
    assert abs(O[17, 200].item() + p(3.0 / (3.0 + 1e-7))) <= slack(torch.ones(1, dtype=torch.float64)).item()
    O[17, 200] = 0.0
    assert not O.any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_extremes(spec, dtype):
    import torch
    assert not spec.orthogonalize(torch.zeros(70, 40, dtype=_dt(dtype), device="cuda")).any()
    G = _update("flat", 1, 65, 90, dtype, 1)[0]
    want = _ref(G, [MUON] * 5)
    for f in (2.0 ** 60, 2.0 ** -20):  # squares of the entries leave f32's range, the norm does not
        assert _off(spec.orthogonalize(G * f, eps=0.0), want) <= LIMIT[dtype]
    for bad in (float("nan"), float("inf")):
        H = G.clone()
        H[3, 4] = bad
        assert bool(spec.orthogonalize(H).isnan().any())
    B = torch.stack([H, G])  # and the next matrix of the batch is its own
    assert torch.equal(spec.orthogonalize(B)[1], spec.orthogonalize(G))


@pytest.mark.parametrize("steps", [1, 2, 3, 10])
def test_steps(spec, steps):
    G = _update("decay", 1, 200, 300, "bf16", steps)[0]
    cubic = [(1.5, -0.5, 0.0)] * steps  # s (3 - s^2) / 2
    assert _off(spec.orthogonalize(G, coeffs=cubic), _ref(G, cubic)) <= LIMIT["bf16"]


@pytest.mark.parametrize("m,n", [(2048, 2048), (1000, 4100), (4100, 1000)])
def test_large(spec, m, n):
    print_case("orthogonalize_large", m=m, n=n)
    G = _update("decay", 1, m, n, "bf16", m)[0]
    assert _off(spec.orthogonalize(G), _ref(G, [MUON] * 5)) <= LIMIT["bf16"]


def test_stream_and_graph(spec):
    import torch
    G = _update("decay", 1, 300, 200, "bf16", 2)[0]
    want = spec.orthogonalize(G)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = spec.orthogonalize(G)
    s.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = spec.orthogonalize(G)
    for k in range(4):
        G.copy_(_update("flat", 1, 300, 200, "bf16", 20 + k)[0])
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, spec.orthogonalize(G)), k


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m,n", [(65, 90), (300, 200)])
def test_norms_at_the_ends_of_the_range(spec, dtype, m, n):
    """1 / |G|_F need not be an f32: a zero G is zero with eps = 0 too, subnormal updates are not infinite, and a
    power of two that no element overflows or underflows by changes no bit."""
    import torch
    print_case("orthogonalize_norms", m=m, n=n, dtype=dtype)
    G = _update("flat", 1, m, n, dtype, 4)[0].clamp(-3.9, 3.9)
    zero = torch.zeros_like(G)
    for eps in (0.0, 1e-300, 1e-40):
        assert not spec.orthogonalize(zero, eps=eps).any(), eps
    O = spec.orthogonalize(G, eps=0.0)
    three = spec.orthogonalize(torch.stack([G, zero, G]), eps=0.0)
    assert torch.equal(three[0], O) and torch.equal(three[2], O) and not three[1].any()
    assert torch.equal(spec.orthogonalize((G.double() * 2.0 ** 125).to(G.dtype), eps=0.0), O)
    for f in (2.0 ** -120, 2.0 ** (-128 if dtype == "bf16" else -140)):
        small = (G.double() * f).to(G.dtype)  # (what is left of its bits is the input)
        assert _off(spec.orthogonalize(small, eps=0.0), _ref(small, [MUON] * 5, eps=0.0)) <= LIMIT[dtype], f
