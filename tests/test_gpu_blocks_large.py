"""Rows shorter than one access, matrices taken a piece at a time, addresses past 32 bits:
the residual blocks' operators where their smaller tests do not reach."""
import pytest

from gpu_util import print_case

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def spec():
    import torch
    import weights_bf16_fp32_amd as spec
    assert torch.cuda.is_available()
    spec.lib()
    return spec


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [2, 3, 4, 5, 6, 7, 8, 9, 15])
def test_short_rows(spec, dtype, d):
    """Storage, products and norms of rows of a few values, each row followed by NaN."""
    import torch
    import test_gpu_block_norm as bn
    import test_gpu_mx as mx
    print_case("short rows", dtype=dtype, d=d)
    g = mx._gen(d)
    for fmt in ("int8", "fp4"):
        x = mx._strided(mx._mixed(g, 19, d).to(mx._dt(dtype)), 1, 1)
        m = spec.mx_quantize(x, mx._fmt(spec, fmt))
        assert mx._same(mx._values(spec, m), mx._stored(x, fmt)[0])
    w = spec.mx_quantize(torch.randn(33, d, generator=g, device="cuda"), spec.MX_FP4)
    for T in (3, 70):
        x = mx._strided(torch.randn(T, d, generator=g, device="cuda").to(mx._dt(dtype)), 1, 1)
        mx._close(spec.mx_linear(x, w), x.double(), mx._values(spec, w), dtype)
        dy = mx._strided(torch.randn(T, 5, generator=g, device="cuda").to(mx._dt(dtype)), 1, 1)
        x8 = spec.mx_quantize(x, spec.MX_INT8)
        mx._close(spec.mx_weight_grad(dy, x8), dy.double().t().contiguous(), mx._values(spec, x8).t().contiguous(), dtype)
    c = bn.Case(21, d, dtype, True, 5, pad=1)
    out = spec.block_norm(c.h, c.y, eps=bn.EPS, **c.args)
    bn.check_forward(c, out)
    h2, _, r_post, r_pre = out
    bn.check_grad(c, c.y.double(), h2.double(), r_post, r_pre, spec.block_norm_grad(c.dx, c.dout, h2, c.y, r_pre, r_post, **c.args))


def test_products_in_pieces(spec):
    """More rows of X than one launch takes, more columns of a long X than are unpacked at a time."""
    import torch
    import test_gpu_mx as mx
    g = mx._gen(1)
    T, N, K = 66000, 70, 96
    print_case("mx pieces", T=T, N=N, K=K)
    x = torch.randn(T, K, generator=g, device="cuda").bfloat16()
    w, xq = spec.mx_quantize(torch.randn(N, K, generator=g, device="cuda"), spec.MX_FP4), spec.mx_quantize(x, spec.MX_FP4)
    mx._close(spec.mx_linear(x, w), x.double(), mx._values(spec, w), "bf16")
    mx._close(spec.mx_product(xq, w), mx._values(spec, xq), mx._values(spec, w), "bf16")
    T, N, K = 700000, 9, 300
    print_case("mx pieces", T=T, N=N, K=K)
    x8 = spec.mx_quantize(torch.randn(T, K, generator=g, device="cuda"), spec.MX_INT8)
    dy = torch.randn(T, N, generator=g, device="cuda").bfloat16()
    assert spec.mx_weight_grad_workspace(T, N, K, torch.bfloat16) < 2 * T * K * 2  # (not all of X at once)
    mx._close(spec.mx_weight_grad(dy, x8), dy.double().t().contiguous(), mx._values(spec, x8).t().contiguous(), "bf16")


@pytest.mark.parametrize("dtype,a,b,k", [
    ("bf16", 70, 80, 20), ("bf16", 70, 80, 666), ("bf16", 205, 4242, 2000), ("bf16", 915, 2239, 16), ("bf16", 71, 5724, 1957),
    ("bf16", 2899, 3601, 16), ("bf16", 4096, 2047, 4200), ("f32", 70, 81, 16), ("f32", 70, 81, 356), ("f32", 2524, 202, 16),
    ("f32", 2895, 85, 803), ("f32", 1706, 1241, 16), ("f32", 1327, 1595, 527), ("f32", 2925, 2849, 16), ("f32", 710, 2806, 774)])
def test_products_of_every_tile(spec, dtype, a, b, k):
    """Tiles of all sizes, with k whole and in shares: b rows of X by a of W, and as a weight gradient of b x a."""
    import torch
    import test_gpu_mx as mx
    print_case("mx tiles", dtype=dtype, a=a, b=b, k=k)
    g = mx._gen(a + b + k)
    w = spec.mx_quantize(torch.randn(a, k, generator=g, device="cuda"), spec.MX_FP4)
    x = torch.randn(b, k, generator=g, device="cuda").to(mx._dt(dtype))
    mx._close(spec.mx_linear(x, w), x.double(), mx._values(spec, w), dtype)
    x8 = spec.mx_quantize(torch.randn(k, a, generator=g, device="cuda"), spec.MX_INT8)
    dy = torch.randn(k, b, generator=g, device="cuda").to(mx._dt(dtype))
    mx._close(spec.mx_weight_grad(dy, x8), dy.double().t().contiguous(), mx._values(spec, x8).t().contiguous(), dtype)


def test_norms_past_32_bits(spec):
    """Rows past 2^32 bytes and 2^31 elements."""
    import torch
    n, d = 270000, 8192
    print_case("block_norm past 32 bits", n=n, d=d)
    h = torch.zeros((n, d), dtype=torch.bfloat16, device="cuda")
    at = [0, 1, n // 2, n - 2, n - 1]
    rows = torch.randn(len(at), d, device="cuda").bfloat16()
    h[at] = rows
    w = torch.randn(d, device="cuda").bfloat16()
    small = spec.block_norm(rows, rows, w_post=w, w_pre=w, gate=w)
    big = spec.block_norm(h, h, w_post=w, w_pre=w, gate=w)
    for a, b in zip(small, big):
        assert torch.equal(a, b[at])
    assert not big[0][2].any() and not big[1][n - 3].any()
    gs = spec.block_norm_grad(rows, rows, small[0], rows, small[3], small[2], w_post=w, w_pre=w, gate=w)
    gb = spec.block_norm_grad(h, h, big[0], h, big[3], big[2], w_post=w, w_pre=w, gate=w)
    assert torch.equal(gs[0], gb[0][at]) and torch.equal(gs[1], gb[1][at])
    for a, b in zip(gs[2:], gb[2:]):  # five rows count; sums in another order
        assert bool(((a - b).abs() <= 16 * U * (a.abs() + 5 * a.abs().amax())).all())
