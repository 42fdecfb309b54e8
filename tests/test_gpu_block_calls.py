"""Calls of the residual blocks' operators at the ends of their documented ranges: no rows, parts left
out, values that leave f32's range."""
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


@pytest.mark.parametrize("N,K", [(70, 64), (70, 4096), (1000, 14336)])
def test_product_without_rows(spec, N, K):
    import torch
    print_case("mx_product", T=0, N=N, K=K)
    w = spec.mx_quantize(torch.randn(N, K, device="cuda"), spec.MX_FP4)
    none = spec.mx_quantize(torch.empty(0, K, device="cuda"), spec.MX_FP4)
    for dt in (torch.bfloat16, torch.float32):
        y = spec.mx_product(none, w, dt)
        assert y.shape == (0, N) and y.dtype == dt
        assert spec.mx_linear(torch.empty(0, K, dtype=dt, device="cuda"), w).shape == (0, N)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("post", [True, False])
def test_vector_gate_without_rows(spec, dtype, post):
    """The gradient of a gate [d] is a sum over the rows: without rows zeros of [d], as the weights' are."""
    import torch
    print_case("block_norm_grad", n=0, dtype=dtype, post=post)
    dt, d = torch.bfloat16 if dtype == "bf16" else torch.float32, 65
    e, w = torch.empty(0, d, dtype=dt, device="cuda"), torch.randn(d, device="cuda").to(dt)
    args = dict(post=post, w_post=w if post else None, w_pre=w, gate=w)
    h, x, r_post, r_pre = spec.block_norm(e, e, **args)
    dh, dy, dw_post, dw_pre, dgate = spec.block_norm_grad(e, e, h, e, r_pre, r_post, **args)
    assert dh.shape == dy.shape == (0, d)
    for g in (dw_pre, dgate) + ((dw_post,) if post else ()):
        assert g.shape == (d,) and g.dtype == torch.float32 and not g.any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_alone_has_no_scales(spec, dtype):
    """Without a block the norm is that of H: alpha and beta scale neither it nor its gradient."""
    import torch
    print_case("block_norm alone", dtype=dtype)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    h, dx, dout = (torch.randn(19, 100, generator=g, device="cuda").to(dt) for _ in range(3))
    w = torch.randn(100, generator=g, device="cuda").to(dt)
    scales = dict(alpha=0.5, beta=3.0)
    _, x, _, r = spec.block_norm(h, w_pre=w)
    _, again, _, r2 = spec.block_norm(h, w_pre=w, **scales)
    assert torch.equal(x, again) and torch.equal(r, r2)
    for a, b in ((dx, dout), (dx, None), (None, dout)):
        want = spec.block_norm_grad(a, b, h, None, r, w_pre=w)
        got = spec.block_norm_grad(a, b, h, None, r, w_pre=w, **scales)
        for s, t in zip(want, got):
            assert (s is None and t is None) or torch.equal(s, t)


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_weight_of_an_absent_gradient(spec, bad):
    """Without dX nothing comes through the second norm, whatever its weight holds."""
    import torch
    print_case("block_norm_grad without dX", bad=bad)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    for d in (5, 100, 9000):
        h, y, dout = (torch.randn(7, d, generator=g, device="cuda") for _ in range(3))
        w = torch.randn(d, generator=g, device="cuda")
        odd = w.clone()
        odd[d // 2] = bad
        _, _, r_post, r_pre = spec.block_norm(h, y, w_post=w, w_pre=w)
        args = dict(w_post=w, gate=w, alpha=0.75)
        want = spec.block_norm_grad(None, dout, h, y, r_pre, r_post, w_pre=w, **args)
        got = spec.block_norm_grad(None, dout, h, y, r_pre, r_post, w_pre=odd, **args)
        assert torch.equal(want[0], 0.75 * dout) and got[3] is None
        for s, t in zip(want, got):
            assert (s is None and t is None) or torch.equal(s, t)


@pytest.mark.parametrize("d", [3, 100, 1000, 4096, 9000])
def test_norm_alone_of_infinities(spec, d):
    """The mean square of a row with an infinity is infinite and its factor zero: zeros beside the
    infinity, NaN (0 inf) at it.  A row with NaN is NaN."""
    import torch
    print_case("block_norm alone of infinities", d=d)
    for dt in (torch.bfloat16, torch.float32):
        g = torch.Generator(device="cuda")
        g.manual_seed(d)
        h = torch.randn(6, d, generator=g, device="cuda").to(dt)
        _, clean, _, r = spec.block_norm(h)
        h[1, 0], h[3, d - 1], h[4, d // 2] = float("inf"), -float("inf"), float("nan")
        _, x, _, r2 = spec.block_norm(h)
        assert torch.equal(x[[0, 2, 5]], clean[[0, 2, 5]]) and torch.equal(r2[[0, 2, 5]], r[[0, 2, 5]])
        assert r2[1] == 0 and r2[3] == 0 and r2[4].isnan() and x[4].isnan().all()
        assert x[1, 0].isnan() and not x[1, 1:].any() and x[3, d - 1].isnan() and not x[3, :d - 1].any()


@pytest.mark.parametrize("d,v,eps", [(1, 1e19, 3e38), (100, 3e19, 3e38), (1000, 1e18, 1e38), (5000, 2e19, 1e37), (100, 1e25, 1e38),
                                     (16384, 1e19, 3.3e38)])
def test_large_eps_beside_large_values(spec, d, v, eps):
    """eps counts as far as f32 holds it, where sums of squares or they and eps leave f32's range too.
    r within (d / 2 + 8) u: half of the sum's error, the mean's, the sum's with eps, the root's."""
    import torch
    print_case("block_norm eps", d=d, v=v, eps=eps)
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    h = (v * (1 + torch.rand(5, d, generator=g, device="cuda")))
    eps32 = torch.tensor(eps).double().item()
    hd = h.double()
    want = ((hd * hd).mean(1) + eps32).rsqrt()
    rel = (d / 2 + 8) * U
    _, x, _, r = spec.block_norm(h, eps=eps)
    assert bool(((r.double() - want).abs() <= rel * want).all())
    assert bool(((x.double() - hd * want[:, None]).abs() <= (rel + 3 * U) * (hd * want[:, None])).all())
    _, _, r_post, _ = spec.block_norm(torch.zeros_like(h), h, eps=eps)
    assert bool(((r_post.double() - want).abs() <= rel * want).all())
