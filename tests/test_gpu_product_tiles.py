"""The products with microscaled matrices on every tile that they choose, with the sums' dimension whole
and in shares, at sizes that end inside tiles, steps and groups of scales.

The operands are small whole numbers of a unit, with scales of two sizes, so that every sum is a whole
number below 2^24 units: exact in f32 in any order.  The results are compared for equality.  Each case
names the tile and whether there are shares, as spec_mx_plan reports them: where the choice
changes, the case has to move, not to test another tile."""
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


def _dt(name):
    import torch
    return torch.bfloat16 if name == "bf16" else torch.float32


class Numbers:
    """Operands of whole numbers from a seed."""

    def __init__(self, spec, *seed):
        import torch
        self.spec = spec
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(sum(s << 8 * i for i, s in enumerate(seed)) % (1 << 60))

    def ints(self, lo, hi, *shape):
        import torch
        return torch.randint(lo, hi + 1, shape, generator=self.g, device="cuda")

    def storage(self, rows, cols, fmt, top, byte):
        """(storage, values in units): whole numbers up to `top` units, scales of one or two units."""
        import torch
        nb = -(-cols // 32)
        lq, ls = self.spec._mx_rows(fmt, cols)
        q = self.ints(-top, top, rows, nb * 32).short()
        q[:, cols:] = 0
        b = self.ints(0, 1, rows, nb)
        s = torch.zeros(rows, ls, dtype=torch.uint8, device="cuda")
        s[:, :nb] = byte + b
        values = (q.view(rows, nb, 32) << b[:, :, None].short()).view(rows, nb * 32)[:, :cols]
        if fmt == self.spec.MX_INT8:
            codes = q.to(torch.int8).view(torch.uint8)
        else:  # units of 1/2: 0, 1, 2, 3, 4, 6, 8, 12 of them, by index
            index, units = q.abs(), torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], dtype=torch.int16, device="cuda")
            codes = (index + 8 * (q < 0)).to(torch.uint8)
            codes = (codes[:, 0::2] | codes[:, 1::2] << 4)
            signed = torch.where(q < 0, -units[index.long()], units[index.long()])
            values = (signed.view(rows, nb, 32) << b[:, :, None].short()).view(rows, nb * 32)[:, :cols]
        assert codes.shape[1] == lq
        return self.spec.Mx(codes.contiguous(), s, cols, fmt), values

    def fp4(self, rows, cols, top=7):
        return self.storage(rows, cols, self.spec.MX_FP4, top, 127)

    def int8(self, rows, cols):
        return self.storage(rows, cols, self.spec.MX_INT8, 127, 133)


def _product(a, b, unit, dt):
    """a b^T times a unit, rounded once."""
    want = a.double() @ b.double().t().contiguous()
    assert want.abs().max() < 1 << 24
    return (want * unit).float().to(dt)


def _on(spec, op, T, N, K, dt, edge, split):
    e, w = spec.mx_plan(op, T, N, K, dt)
    assert (e, w > 1) == (edge, split), (e, w)


# a rows of W (or columns of dW) by b rows of X (or rows of dW), k summed
TILES = [("bf16", 256, False, 1601, 5459, 33), ("bf16", 256, False, 4090, 4001, 1001), ("bf16", 256, False, 2901, 3601, 72),
         ("bf16", 256, True, 5709, 411, 2323), ("bf16", 256, True, 4096, 2047, 6001), ("bf16", 192, False, 917, 2239, 17),
         ("bf16", 192, True, 73, 5724, 1957), ("bf16", 128, True, 205, 4243, 2001), ("bf16", 64, False, 71, 81, 21),
         ("bf16", 64, True, 71, 81, 667), ("f32", 256, False, 7257, 1195, 35), ("f32", 256, False, 4091, 4093, 700),
         ("f32", 256, True, 1735, 2437, 681), ("f32", 192, False, 2925, 2849, 17), ("f32", 192, True, 711, 2807, 775),
         ("f32", 128, False, 1707, 1241, 17), ("f32", 128, True, 1327, 1595, 527), ("f32", 64, False, 2525, 203, 17),
         ("f32", 64, True, 2895, 85, 803), ("f32", 32, False, 71, 81, 17), ("f32", 32, True, 71, 81, 357)]


@pytest.mark.parametrize("dtype,edge,split,a,b,k", TILES)
def test_linear(spec, dtype, edge, split, a, b, k):
    import torch
    print_case("mx_linear", dtype=dtype, T=b, N=a, K=k, edge=edge, split=split)
    _on(spec, spec.MX_OP_LINEAR, b, a, k, _dt(dtype), edge, split)
    n = Numbers(spec, a, b, k)
    w, wv = n.fp4(a, k)
    x = n.ints(-3, 3, b, k)
    assert torch.equal(spec.mx_linear(x.to(_dt(dtype)), w), _product(x, wv, 0.5, _dt(dtype)))


@pytest.mark.parametrize("dtype,edge,split,a,b,k", TILES)
def test_weight_grad(spec, dtype, edge, split, a, b, k):
    import torch
    print_case("mx_weight_grad", dtype=dtype, T=k, N=b, K=a, edge=edge, split=split)
    _on(spec, spec.MX_OP_WEIGHT_GRAD, k, b, a, _dt(dtype), edge, split)
    n = Numbers(spec, a, b, k)
    x, xv = n.int8(k, a)
    dy = n.ints(-2, 2, k, b)
    got = spec.mx_weight_grad(dy.to(_dt(dtype)), x)
    assert torch.equal(got, _product(dy.t(), xv.t(), 1.0, _dt(dtype)))
    # on top of what is there
    dw = n.ints(-100, 100, b, a)
    got = spec.mx_weight_grad(dy.to(_dt(dtype)), x, beta=2.0, dW=dw.to(_dt(dtype)))
    want = dy.double().t().contiguous() @ xv.double() + 2 * dw.double()
    assert torch.equal(got, want.float().to(_dt(dtype)))


@pytest.mark.parametrize("edge,split,T,N,K", [
    (256, False, 3141, 3877, 34), (256, False, 3141, 3877, 257), (256, False, 3145, 3901, 700), (256, False, 3200, 3950, 1500),
    (256, False, 3333, 3999, 2111), (256, False, 3841, 4096, 4097), (128, False, 333, 5491, 44), (128, False, 333, 5491, 700),
    (128, False, 2100, 1701, 2500), (128, False, 1701, 2101, 1029), (64, False, 4345, 33, 45), (64, False, 333, 1001, 1001),
    (64, True, 36, 2091, 2183), (64, True, 500, 501, 6001), (32, False, 35, 33, 45), (32, True, 33, 33, 2099),
    (32, True, 70, 71, 6001)])
def test_product(spec, edge, split, T, N, K):
    import torch
    print_case("mx_product", T=T, N=N, K=K, edge=edge, split=split)
    n = Numbers(spec, T, N, K)
    (x, xv), (w, wv) = n.fp4(T, K, 3), n.fp4(N, K)
    for dt in (torch.float32, torch.bfloat16):
        _on(spec, spec.MX_OP_PRODUCT, T, N, K, dt, edge, split)
        assert torch.equal(spec.mx_product(x, w, dt), _product(xv, wv, 0.25, dt))


@pytest.mark.parametrize("edge,split,T,N,K", [(256, False, 3145, 3901, 1500), (128, False, 2100, 1701, 1029), (64, False, 333, 1001, 1001),
                                              (64, True, 500, 501, 6001), (32, True, 70, 71, 6001)])
def test_nan_blocks_of_product(spec, edge, split, T, N, K):
    """A block of NaN anywhere along a row reaches that row's results and no other's."""
    import torch
    print_case("mx_product of NaN", T=T, N=N, K=K, edge=edge, split=split)
    _on(spec, spec.MX_OP_PRODUCT, T, N, K, torch.float32, edge, split)
    n = Numbers(spec, T, N, K)
    (x, xv), (w, wv) = n.fp4(T, K, 3), n.fp4(N, K)
    want = _product(xv, wv, 0.25, torch.float32)
    nb = -(-K // 32)
    for m, rows in ((x, T), (w, N)):
        for block in (0, 1, nb // 2, nb - 2, nb - 1):
            row = int(n.ints(0, rows - 1, 1))
            m.s[row, block] = 255
            if m is x:
                want[row] = float("nan")
            else:
                want[:, row] = float("nan")
    got = spec.mx_product(x, w, torch.float32)
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(), want.nan_to_num())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_linear_in_pieces_of_w(spec, dtype):
    """Rows of W so long that they are unpacked a piece at a time, the last of them ragged: the longest K."""
    import torch
    T, N, K = 67, 301, 1 << 20
    print_case("mx_linear pieces", dtype=dtype, T=T, N=N, K=K)
    assert spec.mx_linear_workspace(T, N, K, _dt(dtype)) < N * K * _dt(dtype).itemsize + T * K * 4
    n = Numbers(spec, T, N)
    w, wv = n.fp4(N, K, 2)  # products of at most 4 units: 2^22 of them
    x = n.ints(-1, 1, T, K)
    assert torch.equal(spec.mx_linear(x.to(_dt(dtype)), w), _product(x, wv, 0.5, _dt(dtype)))


def test_product_in_pieces_of_x(spec):
    """More rows of X than one launch takes: the first piece with k whole, the last, of few rows, in shares."""
    import torch
    T, N, K = 65536 + 5, 70, 4097
    print_case("mx_product pieces", T=T, N=N, K=K)
    assert spec.mx_plan(spec.MX_OP_PRODUCT, T, N, K, torch.float32)[1] == 1
    assert spec.mx_plan(spec.MX_OP_PRODUCT, 5, N, K, torch.float32)[1] > 1
    n = Numbers(spec, T, N)
    (x, xv), (w, wv) = n.fp4(T, K, 3), n.fp4(N, K)
    assert torch.equal(spec.mx_product(x, w, torch.float32), _product(xv, wv, 0.25, torch.float32))
