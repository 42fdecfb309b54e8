"""Products of few rows with every number of row tiles to a workgroup: matrices of many rows."""
import pytest

from gpu_util import print_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,N,K", [(1, 6656, 96), (17, 6657, 300), (40, 8191, 257), (3, 13312, 544), (20, 13313, 64), (64, 13400, 100)])
def test_linear_of_many_columns(dtype, T, N, K):
    """Against float64: sums of K products in f32 and one rounding (as in test_gpu_mx.py)."""
    import torch
    import weights_bf16_fp32_amd as spec
    print_case("mx_linear", dtype=dtype, T=T, N=N, K=K)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    x = torch.randn(T, K, generator=g, device="cuda").to(dt)
    w = spec.mx_quantize(torch.randn(N, K, generator=g, device="cuda"), spec.MX_FP4)
    y = spec.mx_linear(x, w)
    wv = spec.mx_dequantize(w, torch.float32).double()
    want, mag = x.double() @ wv.t().contiguous(), x.double().abs() @ wv.abs().t().contiguous()
    assert bool(((y.double() - want).abs() <= (K + 3) * 2.0 ** -24 * 1.01 * mag + torch.finfo(dt).eps / 2 * want.abs()).all())
