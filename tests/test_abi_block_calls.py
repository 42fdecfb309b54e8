"""Calls of the residual blocks' operators at the ends of their documented ranges, as far as the host
decides them (no GPU needed)."""
import ctypes
import os

import pytest

import weights_bf16_fp32_amd as spec


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(spec.LIB_PATH):
        from weights_bf16_fp32_amd import build
        build.build()
    return spec.lib()


def test_no_workspace_is_empty(L):
    """A workspace of no bytes has no address, which the entry points refuse: every size asks for some."""
    b = ctypes.c_size_t()
    for T in (0, 1, 5, 64, 65, 70000):
        for N in (1, 70, 1000, 16384):
            for K in (1, 64, 2049, 4096, 1 << 20):
                assert L.spec_mx_product_workspace(T, N, K, b) == 0 and b.value > 0, (T, N, K)
                for t in (spec.BF16, spec.F32):
                    assert L.spec_mx_linear_workspace(T, N, K, t, b) == 0 and b.value > 0, (T, N, K)
                    assert L.spec_mx_weight_grad_workspace(T, N, K, t, b) == 0 and b.value > 0, (T, N, K)


def test_product_without_rows(L):
    """T = 0 has nothing to do, whatever the other sizes: what the query asks for is enough."""
    at = 1 << 20  # an aligned address; never dereferenced, because nothing is launched
    b = ctypes.c_size_t()
    for N, K in ((70, 64), (70, 4096), (1, 1 << 20), (14336, 4096)):
        lq, ls = spec._mx_rows(spec.MX_FP4, K)
        X, W = spec.MxMatrix(None, None, lq, ls, spec.MX_FP4), spec.MxMatrix(at, at, lq, ls, spec.MX_FP4)
        assert L.spec_mx_product_workspace(0, N, K, b) == 0
        ws = at if b.value else None
        assert L.spec_mx_product(None, X, W, 0, N, K, None, spec.BF16, N, ws, b.value) == 0, (N, K)


def test_outputs_that_no_call_writes(L):
    """Without Y there is no sum and no gradient of Y: what is passed to receive them is refused."""
    import torch
    X = torch.zeros(4, 64)
    m = spec.mx_empty(4, 64, spec.MX_INT8, device="cpu")
    for kw in (dict(Hout=X), dict(y8=m), dict(h8=m), dict(Hout=X, x8=m)):
        with pytest.raises(spec.SpecError, match="without Y"):
            spec.block_norm(X, **kw)
    for args in ((X, None), (None, X), (X, X)):
        with pytest.raises(spec.SpecError, match="without Y"):
            spec.block_norm_grad(*args, X, None, torch.zeros(4), dY=X)


def test_workspace_is_its_bytes(L):
    """A workspace counts with the bytes that it has: one byte expanded to a thousand is refused."""
    import torch
    ws = torch.zeros(1000, dtype=torch.uint8)
    at = spec._scratch(ws, 1000, -1)
    assert at[:2] == (ws.data_ptr(), 1000)
    assert spec._scratch(ws.view(torch.float32), 1000, -1)[1] == 1000
    for bad in (ws[:1].expand(1000), ws[::2], ws.view(10, 100)[:, :50]):
        with pytest.raises(spec.SpecError, match="contiguous"):
            spec._scratch(bad, 500, -1)


def test_plan(L):
    """The query of a product's tile and shares: its refusals, and answers that the products can take."""
    import torch
    e, w = ctypes.c_int32(), ctypes.c_int32()
    ok = (100, 1000, 500, spec.BF16)
    assert L.spec_mx_plan(3, *ok, e, w) == -2 and L.spec_mx_plan(-1, *ok, e, w) == -2
    assert L.spec_mx_plan(0, 100, 1000, 500, spec.F64, e, w) == -2
    assert L.spec_mx_plan(0, *ok, None, w) == -1 and L.spec_mx_plan(0, *ok, e, None) == -1
    for T, N, K in ((-1, 1, 1), ((1 << 22) + 1, 1, 1), (1, 0, 1), (1, 1, 0), (1, (1 << 20) + 1, 1), (1, 1, (1 << 20) + 1)):
        assert L.spec_mx_plan(1, T, N, K, spec.F32, e, w) == -1
    for op in (spec.MX_OP_LINEAR, spec.MX_OP_PRODUCT, spec.MX_OP_WEIGHT_GRAD):
        for dt in (torch.bfloat16, torch.float32):
            for T in (0, 1, 64, 65, 3000, 70000, 1 << 22):
                for N, K in ((1, 1), (1000, 1000), (1 << 20, 33), (33, 1 << 20)):
                    edge, shares = spec.mx_plan(op, T, N, K, dt)
                    assert edge in ((16,) if op == spec.MX_OP_LINEAR and T <= 64 else (32, 64, 128, 192, 256))
                    assert 1 <= shares <= 64
