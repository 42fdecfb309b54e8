"""The block norms' entry points with every output wanted by itself, with one matrix stored in 8 bits
and the other not, and with gate rows of which a worker has several: each output as it is when all
are wanted."""
import ctypes

import pytest

from gpu_util import print_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def spec():
    import torch
    import weights_bf16_fp32_amd as spec
    assert torch.cuda.is_available()
    spec.lib()
    return spec


def _same(a, b):
    import torch
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def _call(spec, f, *args):
    import torch
    assert f(spec._stream(), *args) == 0
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,d", [(5, 3), (70, 100), (9, 1000), (4, 4097), (3, 9000)])
@pytest.mark.parametrize("post", [1, 0])
def test_one_output_at_a_time(spec, dtype, n, d, post):
    import torch
    import test_gpu_block_norm as bn
    print_case("spec_block_norm", dtype=dtype, n=n, d=d, post=post)
    c = bn.Case(n, d, dtype, bool(post), 2)
    L, t = spec.lib(), spec._dt(c.h)
    b = spec.Block(n, d, t, post, c.alpha, c.beta, bn.EPS, c.w_post.data_ptr() if post else None, c.w_pre.data_ptr(),
                   c.gate.data_ptr(), d, 2)
    h2, x, r_post, r_pre = spec.block_norm(c.h, c.y, eps=bn.EPS, **c.args)
    matrix = lambda: torch.full((n, d), 7.0, dtype=c.dt, device="cuda")  # noqa: E731
    vector = lambda: torch.full((n,), 7.0, device="cuda")  # noqa: E731
    mx = lambda m: ctypes.byref(spec._mx(m, n, d))  # noqa: E731
    base = [b, c.y.data_ptr(), d, c.h.data_ptr(), d, None, d, None, d, None, None, None, None, None]
    for at, make, want in ((5, matrix, h2), (7, matrix, x), (9, vector, r_post), (10, vector, r_pre)):
        if want is None:
            continue
        got = make()
        _call(spec, L.spec_block_norm, *[got.data_ptr() if i == at else a for i, a in enumerate(base)])
        assert _same(got, want), at
    for at, want in ((11, c.y), (12, h2), (13, x)):
        got, q = spec.mx_empty(n, d, spec.MX_INT8), spec.mx_quantize(want, spec.MX_INT8)
        _call(spec, L.spec_block_norm, *[mx(got) if i == at else a for i, a in enumerate(base)])
        assert _same(got.q, q.q) and _same(got.s, q.s), at
    _call(spec, L.spec_block_norm, *base)  # nothing wanted
    # the norm alone, its factor and its 8 bits
    want = spec.block_norm(c.h, w_pre=c.w_pre, eps=bn.EPS)
    got, q = vector(), spec.mx_empty(n, d, spec.MX_INT8)
    _call(spec, L.spec_block_norm, b, None, 0, c.h.data_ptr(), d, None, 0, None, 0, None, got.data_ptr(), None, None, mx(q))
    assert _same(got, want[3]) and _same(q.q, spec.mx_quantize(want[1], spec.MX_INT8).q)

    got = spec.block_norm_grad(c.dx, c.dout, h2, c.y, r_pre, r_post, **c.args)
    size = ctypes.c_size_t()
    assert L.spec_block_norm_grad_workspace(b, size) == 0
    ws = torch.empty(size.value, dtype=torch.uint8, device="cuda")
    base = [b, c.y.data_ptr(), d, None, h2.data_ptr(), d, None, r_post.data_ptr() if post else None, r_pre.data_ptr(),
            c.dout.data_ptr(), d, c.dx.data_ptr(), d, None, d, None, d, None, None, None, ws.data_ptr(), size.value]
    for at, want in ((13, got[0]), (15, got[1]), (17, got[2]), (18, got[3]), (19, got[4])):
        if want is None:
            continue
        out = torch.full(want.shape, 7.0, dtype=want.dtype, device="cuda")
        ws.fill_(0xFF)
        _call(spec, L.spec_block_norm_grad, *[out.data_ptr() if i == at else a for i, a in enumerate(base)])
        assert _same(out, want), at
    _call(spec, L.spec_block_norm_grad, *base)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,d,rows", [(40, 100, 7), (700, 8200, 1), (1100, 2050, 1), (600, 8193, 2), (3000, 600, 1), (5000, 5, 1),
                                      (2500, 1025, 1 << 40)])
@pytest.mark.parametrize("y8,h8", [(True, False), (False, True)])
def test_mixed_storage_and_gate_rows(spec, dtype, n, d, rows, y8, h8):
    """Y or Hout stored in 8 bits; a gate of more rows than the matrices need, of which the rest does not count."""
    import torch
    import test_gpu_block_norm as bn
    print_case("block_norm_grad", dtype=dtype, n=n, d=d, rows=rows, y8=y8, h8=h8)
    c = bn.Case(n, d, dtype, True, min(rows, n))
    c.rows = rows
    gates = c.gate.shape[0]
    c.gate = torch.cat((c.gate, torch.full((3, d), float("nan"), dtype=c.dt, device="cuda")))
    h2, x, r_post, r_pre = spec.block_norm(c.h, c.y, eps=bn.EPS, **c.args)
    bn.check_forward(c, (h2, x, r_post, r_pre))
    y, h = (spec.mx_quantize(t, spec.MX_INT8) if q else t for t, q in ((c.y, y8), (h2, h8)))
    yv, hv = (spec.mx_dequantize(t, torch.float32).double() if q else t.double() for t, q in ((y, y8), (h, h8)))
    got = spec.block_norm_grad(c.dx, c.dout, h, y, r_pre, r_post, **c.args)
    assert got[4].shape == (gates, d)
    c.rows = min(rows, n)  # (the bound of a gate row's sum counts its rows)
    bn.check_grad(c, yv, hv, r_post, r_pre, got)
