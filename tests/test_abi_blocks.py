"""The entry points of a student's residual blocks reject bad arguments on the host before
anything is enqueued (no GPU needed: every call here fails validation, or has no
rows and nothing to do), and their size queries answer."""
import ctypes

import pytest

import weights_bf16_fp32_amd as spec

EINVAL, EUNSUPPORTED, EWORKSPACE = -1, -2, -3
FAKE = 1 << 20  # an aligned non-null address; never dereferenced because validation fails first
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    import os
    if not os.path.exists(spec.LIB_PATH):
        from weights_bf16_fp32_amd import build
        build.build()
    return spec.lib()


def _with(ok, **changes):
    a = dict(ok)
    a.update(changes)
    return list(a.values())


def _mx(q=FAKE, s=FAKE, ldq=1024, lds=32, fmt=spec.MX_FP4):
    return ctypes.byref(spec.MxMatrix(q, s, ldq, lds, fmt))


BAD_MX = (dict(q=None), dict(s=None), dict(q=FAKE + 8), dict(s=FAKE + 1), dict(ldq=1000), dict(lds=24), dict(ldq=16),
          dict(lds=0), dict(ldq=1 << 23), dict(lds=1 << 23))


def test_row_bytes(L):
    a, b = ctypes.c_int64(), ctypes.c_int64()
    for cols, codes8, codes4, scales in ((1, 32, 16, 16), (32, 32, 16, 16), (33, 64, 32, 16), (512, 512, 256, 16),
                                         (513, 544, 272, 32), (1 << 20, 1 << 20, 1 << 19, 1 << 15)):
        for fmt, codes in ((spec.MX_INT8, codes8), (spec.MX_FP4, codes4)):
            assert L.spec_mx_row_bytes(fmt, cols, a, b) == 0 and (a.value, b.value) == (codes, scales)
            assert spec._mx_rows(fmt, cols) == (codes, scales)
    for cols in (0, -1, (1 << 20) + 1):
        assert L.spec_mx_row_bytes(spec.MX_INT8, cols, a, b) == EINVAL
    assert L.spec_mx_row_bytes(spec.MX_INT8, 5, None, b) == EINVAL
    assert L.spec_mx_row_bytes(2, 5, a, b) == EUNSUPPORTED


def test_mx_storage_validation(L):
    ok = dict(stream=None, X=FAKE, t=spec.BF16, rows=10, cols=1000, ldx=1000, out=_mx())
    bads = (dict(X=None), dict(X=FAKE + 1), dict(rows=-1), dict(rows=1 << 31), dict(cols=0), dict(cols=(1 << 20) + 1),
            dict(ldx=999), dict(out=None))
    for bad in bads:
        assert L.spec_mx_quantize(*_with(ok, **bad)) == EINVAL, bad
    for mx in BAD_MX:
        assert L.spec_mx_quantize(*_with(ok, out=_mx(**mx))) == EINVAL, mx
        assert L.spec_mx_dequantize(None, _mx(**mx), 10, 1000, FAKE, spec.BF16, 1000) == EINVAL, mx
    assert L.spec_mx_quantize(*_with(ok, out=_mx(ldq=512, fmt=spec.MX_INT8))) == EINVAL  # INT8 rows are longer
    for bad in (dict(t=spec.F64), dict(out=_mx(fmt=2)), dict(out=_mx(fmt=-1))):
        assert L.spec_mx_quantize(*_with(ok, **bad)) == EUNSUPPORTED, bad
    assert L.spec_mx_quantize(*_with(ok, rows=0, X=None, out=_mx(q=None, s=None))) == 0
    assert L.spec_mx_dequantize(None, _mx(), 10, 1000, FAKE, spec.I32, 1000) == EUNSUPPORTED
    for args in ((None, 10, 1000, FAKE, spec.F32, 1000), (_mx(), 10, 1000, None, spec.F32, 1000),
                 (_mx(), 10, 1000, FAKE + 2, spec.F32, 1000), (_mx(), 10, 1000, FAKE, spec.F32, 999)):
        assert L.spec_mx_dequantize(None, *args) == EINVAL


def _queries(L):
    b = ctypes.c_size_t()
    return b, ((L.spec_mx_linear_workspace, (spec.BF16,)), (L.spec_mx_product_workspace, ()),
               (L.spec_mx_weight_grad_workspace, (spec.F32,)))


def test_product_workspaces(L):
    b, queries = _queries(L)
    for f, t in queries:
        for T, N, K in ((0, 1, 1), (1, 1, 1), (8192, 14336, 4096), (1 << 22, 32, 32), (1, 1 << 20, 1 << 20)):
            assert f(T, N, K, *t, b) == 0 and 0 < b.value < 1 << 42
        for T, N, K in ((-1, 1, 1), ((1 << 22) + 1, 1, 1), (1, 0, 1), (1, 1, 0), (1, (1 << 20) + 1, 1), (1, 1, (1 << 20) + 1)):
            assert f(T, N, K, *t, b) == EINVAL
        assert f(1, 1, 1, *t, None) == EINVAL
    assert L.spec_mx_linear_workspace(1, 1, 1, spec.F64, b) == EUNSUPPORTED


def test_linear_validation(L):
    ok = dict(stream=None, X=FAKE, t=spec.BF16, T=10, N=100, K=1000, ldx=1000, W=_mx(), Y=FAKE, ldy=100, ws=FAKE,
              ws_bytes=1 << 40)
    f = L.spec_mx_linear
    for bad in (dict(X=None), dict(Y=None), dict(W=None), dict(ldx=999), dict(ldx=1 << 21), dict(ldy=99), dict(T=-1),
                dict(N=0), dict(K=0), dict(X=FAKE + 1), dict(Y=FAKE + 1), dict(ws=FAKE + 128)):
        assert f(*_with(ok, **bad)) == EINVAL, bad
    for mx in BAD_MX:
        assert f(*_with(ok, W=_mx(**mx))) == EINVAL, mx
    for bad in (dict(t=spec.F64), dict(W=_mx(fmt=spec.MX_INT8)), dict(W=_mx(fmt=7))):
        assert f(*_with(ok, **bad)) == EUNSUPPORTED, bad
    for bad in (dict(ws=None), dict(ws_bytes=100)):
        assert f(*_with(ok, **bad)) == EWORKSPACE, bad
    assert f(*_with(ok, T=0, X=None, Y=None)) == 0


def test_product_validation(L):
    ok = dict(stream=None, X=_mx(), W=_mx(), T=10, N=100, K=1000, Y=FAKE, yt=spec.BF16, ldy=100, ws=FAKE, ws_bytes=1 << 40)
    f = L.spec_mx_product
    for bad in (dict(X=None), dict(W=None), dict(Y=None), dict(ldy=99), dict(Y=FAKE + 1), dict(T=-1), dict(K=(1 << 20) + 1),
                dict(ws=FAKE + 8)):
        assert f(*_with(ok, **bad)) == EINVAL, bad
    for mx in BAD_MX:
        assert f(*_with(ok, X=_mx(**mx))) == EINVAL and f(*_with(ok, W=_mx(**mx))) == EINVAL, mx
    for bad in (dict(yt=spec.F64), dict(X=_mx(fmt=spec.MX_INT8)), dict(W=_mx(fmt=spec.MX_INT8))):
        assert f(*_with(ok, **bad)) == EUNSUPPORTED, bad
    for bad in (dict(ws=None), dict(ws_bytes=100)):
        assert f(*_with(ok, **bad)) == EWORKSPACE, bad
    assert f(*_with(ok, T=0, Y=None)) == 0


def test_weight_grad_validation(L):
    i8 = dict(fmt=spec.MX_INT8)
    ok = dict(stream=None, dY=FAKE, t=spec.BF16, T=10, N=100, K=1000, ldy=100, X=_mx(**i8), beta=0.0, dW=FAKE, lddw=1000,
              ws=FAKE, ws_bytes=1 << 40)
    f = L.spec_mx_weight_grad
    for bad in (dict(dY=None), dict(dW=None), dict(X=None), dict(ldy=99), dict(ldy=1 << 21), dict(lddw=999), dict(T=-1),
                dict(beta=NAN), dict(beta=1e39), dict(dY=FAKE + 1), dict(dW=FAKE + 1), dict(ws=FAKE + 16)):
        assert f(*_with(ok, **bad)) == EINVAL, bad
    for mx in BAD_MX:
        assert f(*_with(ok, X=_mx(**{**i8, **mx}))) == EINVAL, mx
    for bad in (dict(t=spec.F64), dict(X=_mx())):
        assert f(*_with(ok, **bad)) == EUNSUPPORTED, bad
    for bad in (dict(ws=None), dict(ws_bytes=100)):
        assert f(*_with(ok, **bad)) == EWORKSPACE, bad


def _block(**kw):
    b = dict(n=10, d=100, t=spec.BF16, post=1, alpha=1.0, beta=1.0, eps=1e-6, w_post=FAKE, w_pre=FAKE, gate=FAKE, ldg=100,
             gate_rows=4)
    b.update(kw)
    return ctypes.byref(spec.Block(*b.values()))


BAD_BLOCK = (dict(n=-1), dict(n=1 << 31), dict(d=0), dict(d=16385), dict(alpha=NAN), dict(beta=1e39), dict(eps=0.0),
             dict(eps=-1.0), dict(eps=1e-39), dict(eps=NAN), dict(eps=INF), dict(w_post=FAKE + 1), dict(w_pre=FAKE + 1),
             dict(gate=FAKE + 1), dict(post=0), dict(ldg=99), dict(gate_rows=0))


def test_block_norm_validation(L):
    i8 = dict(fmt=spec.MX_INT8)
    ok = dict(stream=None, b=_block(), Y=FAKE, ldy=100, H=FAKE, ldh=100, Hout=FAKE, ldo=100, X=FAKE, ldx=100, r_post=FAKE,
              r_pre=FAKE, y8=_mx(**i8), h8=_mx(**i8), x8=_mx(**i8))
    f = L.spec_block_norm
    for bad in BAD_BLOCK:
        assert f(*_with(ok, b=_block(**bad))) == EINVAL, bad
    for bad in (dict(b=None), dict(H=None), dict(ldy=99), dict(ldh=99), dict(ldo=99), dict(ldx=99), dict(Y=FAKE + 1),
                dict(X=FAKE + 1), dict(r_post=FAKE + 2), dict(r_pre=FAKE + 1), dict(Y=None), dict(Y=None, Hout=None),
                dict(Y=None, Hout=None, r_post=None, y8=None), dict(b=_block(post=0, w_post=None))):
        assert f(*_with(ok, **bad)) == EINVAL, bad
    for k in ("y8", "h8", "x8"):
        for mx in BAD_MX:
            assert f(*_with(ok, **{k: _mx(**{**i8, **mx})})) == EINVAL, (k, mx)
        assert f(*_with(ok, **{k: _mx()})) == EUNSUPPORTED
    assert f(*_with(ok, b=_block(t=spec.F64))) == EUNSUPPORTED
    assert f(*_with(ok, b=_block(n=0))) == 0


def test_block_norm_grad_validation(L):
    i8 = dict(fmt=spec.MX_INT8)
    ok = dict(stream=None, b=_block(), Y=FAKE, ldy=100, y8=None, Hout=FAKE, ldo=100, h8=None, r_post=FAKE, r_pre=FAKE,
              dHout=FAKE, lddo=100, dX=FAKE, lddx=100, dH=FAKE, lddh=100, dY=FAKE, lddy=100, dw_post=FAKE, dw_pre=FAKE,
              dgate=FAKE, ws=FAKE, ws_bytes=1 << 40)
    f = L.spec_block_norm_grad
    b = ctypes.c_size_t()
    for bad in BAD_BLOCK:
        assert f(*_with(ok, b=_block(**bad))) == EINVAL, bad
        assert L.spec_block_norm_grad_workspace(_block(**bad), b) == EINVAL
    for bad in (dict(b=None), dict(ldy=99), dict(ldo=99), dict(lddo=99), dict(lddx=99), dict(lddh=99), dict(lddy=99),
                dict(Hout=None), dict(r_pre=None), dict(r_post=None), dict(Y=None), dict(Y=None, dY=None),
                dict(Y=None, dY=None, dw_post=None), dict(dX=None), dict(b=_block(post=0, w_post=None)),
                dict(b=_block(gate=None)), dict(dH=FAKE + 1), dict(dw_pre=FAKE + 2), dict(dgate=FAKE + 1),
                dict(ws=FAKE + 4)):
        assert f(*_with(ok, **bad)) == EINVAL, bad
    for k in ("y8", "h8"):
        for mx in BAD_MX:
            assert f(*_with(ok, **{k: _mx(**{**i8, **mx})})) == EINVAL, (k, mx)
        assert f(*_with(ok, **{k: _mx()})) == EUNSUPPORTED
    assert f(*_with(ok, b=_block(t=spec.F64))) == EUNSUPPORTED
    for bad in (dict(ws=None), dict(ws_bytes=100)):
        assert f(*_with(ok, **bad)) == EWORKSPACE, bad
    assert L.spec_block_norm_grad_workspace(_block(), None) == EINVAL
    for n, d, rows in ((0, 1, 1), (1, 16384, 1), (1 << 30, 4096, 1), (16384, 4096, 7), (16384, 4096, 1 << 40)):
        assert L.spec_block_norm_grad_workspace(_block(n=n, d=d, ldg=d, gate_rows=rows), b) == 0 and 0 < b.value < 1 << 36


def test_binding_refuses(L):
    """What the binding itself looks at: formats, shapes, types, devices."""
    import torch
    X = torch.zeros(4, 64)
    m = spec.mx_empty(4, 64, spec.MX_FP4, device="cpu")
    calls = [(lambda: spec.mx_quantize(X, 5), -2), (lambda: spec.mx_quantize(X, spec.MX_INT8, out=m), -1),
             (lambda: spec.mx_quantize(X, spec.MX_FP4), -1),  # not on a GPU
             (lambda: spec.mx_dequantize(m), -1), (lambda: spec.mx_linear(X, m), -1), (lambda: spec.mx_linear(X, X), -1),
             (lambda: spec.mx_linear(X[:, :32], m), -1), (lambda: spec.mx_quantize(X.t(), spec.MX_FP4), -1),
             (lambda: spec.mx_product(m, m._replace(cols=32)), -1),
             (lambda: spec.mx_product(m, m._replace(q=m.q[:, :16])), -1),
             (lambda: spec.mx_product(m._replace(s=m.s.int()), m), -1),
             (lambda: spec.mx_weight_grad(X[:2], m), -1), (lambda: spec.mx_empty(3, 0, spec.MX_FP4, device="cpu"), -1),
             (lambda: spec.block_norm(X, X), -1), (lambda: spec.block_norm(X, X, w_post=torch.zeros(63)), -1),
             (lambda: spec.block_norm(X, X, gate=torch.zeros(1, 64), gate_rows=3), -1),
             (lambda: spec.block_norm(X, X, gate=torch.zeros(1, 64), gate_rows=0), -1),
             (lambda: spec.block_norm(X, X, gate=torch.zeros(64, dtype=torch.bfloat16)), -1),
             (lambda: spec.block_norm(X.int()), -2),
             (lambda: spec.block_norm_grad(None, None, X, X, None), -1)]
    for i, (f, status) in enumerate(calls):
        with pytest.raises(spec.SpecError) as e:
            f()
        assert e.value.status == status, i
