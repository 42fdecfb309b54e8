"""The training entry points reject bad arguments on the host before anything is
enqueued (no GPU needed: every call here fails validation), and their workspace
queries answer."""
import ctypes

import pytest

import weights_bf16_fp32_amd as spec

EINVAL, EUNSUPPORTED, EWORKSPACE = -1, -2, -3
FAKE = 1 << 20  # an aligned non-null address; never dereferenced because validation fails first


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


def test_embed_validation(L):
    ok = dict(stream=None, E=FAKE, t=spec.BF16, V=100, d=64, lde=64, ids=FAKE, idt=spec.I64, n=10, scale=1.0, Y=FAKE,
              ldy=64)
    f = L.spec_embed
    for bad in (dict(E=None), dict(ids=None), dict(Y=None), dict(V=0), dict(d=0), dict(n=-1), dict(lde=63),
                dict(ldy=63), dict(E=FAKE + 1), dict(Y=FAKE + 1), dict(ids=FAKE + 4), dict(V=1 << 31), dict(n=1 << 31),
                dict(d=(1 << 20) + 1), dict(scale=float("nan")), dict(scale=float("inf"))):
        assert f(*_with(ok, **bad)) == EINVAL, bad
    for bad in (dict(t=spec.F64), dict(t=7), dict(idt=spec.F32)):
        assert f(*_with(ok, **bad)) == EUNSUPPORTED, bad
    assert f(*_with(ok, idt=spec.I32, ids=FAKE + 2)) == EINVAL


def test_embed_grad_validation(L):
    ok = dict(stream=None, dY=FAKE, yt=spec.BF16, n=10, V=100, d=64, ldy=64, ids=FAKE, idt=spec.I64, scale=1.0,
              beta=0.0, dE=FAKE, et=spec.BF16, ldd=64, ws=FAKE, ws_bytes=1 << 30)
    f = L.spec_embed_grad
    for bad in (dict(dY=None), dict(dE=None), dict(ids=None), dict(ldy=63), dict(ldd=1), dict(n=-1), dict(V=0),
                dict(d=0), dict(dE=FAKE + 1), dict(scale=float("nan")), dict(beta=float("nan")), dict(ws=FAKE + 128)):
        assert f(*_with(ok, **bad)) == EINVAL, bad
    for bad in (dict(yt=spec.F32), dict(et=spec.F64), dict(yt=spec.F64, et=spec.F64), dict(beta=0.5), dict(idt=0)):
        assert f(*_with(ok, **bad)) == EUNSUPPORTED, bad
    for bad in (dict(ws=None), dict(ws_bytes=16)):
        assert f(*_with(ok, **bad)) == EWORKSPACE, bad


XENT = dict(stream=None, H=FAKE, W=FAKE, t=spec.BF16, T=10, V=100, d=64, ldh=64, ldw=64, target=FAKE, tt=spec.I64,
            scale=1.0)


@pytest.mark.parametrize("grad", [False, True])
def test_linear_xent_validation(L, grad):
    if grad:
        f = L.spec_linear_xent_grad
        ok = dict(XENT, lse=FAKE, dloss=FAKE, beta=0.0, dH=FAKE, lddh=64, dW=FAKE, lddw=64, ws=FAKE, ws_bytes=1 << 40)
        own = (dict(lse=None), dict(dloss=None), dict(dH=None), dict(dW=None), dict(lddh=63), dict(lddw=63),
               dict(beta=float("inf")), dict(dloss=FAKE + 2), dict(dW=FAKE + 1))
    else:
        f = L.spec_linear_xent
        ok = dict(XENT, loss=FAKE, lse=FAKE, ws=FAKE, ws_bytes=1 << 40)
        own = (dict(loss=None), dict(lse=None), dict(loss=FAKE + 2))
    for bad in own + (dict(H=None), dict(W=None), dict(target=None), dict(T=-1), dict(T=(1 << 22) + 1), dict(V=0),
                      dict(d=0), dict(ldh=63), dict(ldw=63), dict(ldw=1 << 21), dict(H=FAKE + 1), dict(W=FAKE + 1),
                      dict(scale=float("nan")), dict(ws=FAKE + 64)):
        assert f(*_with(ok, **bad)) == EINVAL, bad
    for bad in (dict(t=spec.F64), dict(tt=spec.F32)):
        assert f(*_with(ok, **bad)) == EUNSUPPORTED, bad
    for bad in (dict(ws=None), dict(ws_bytes=100)):
        assert f(*_with(ok, **bad)) == EWORKSPACE, bad


def test_orthogonalize_validation(L):
    co = (ctypes.c_double * 3)(3.4445, -4.7750, 2.0315)
    ok = dict(stream=None, G=FAKE, t=spec.BF16, batch=2, m=64, n=32, ldg=32, sg=2048, coeffs=co, steps=1, eps=1e-7,
              scale=1.0, O=FAKE, ldo=32, so=2048, ws=FAKE, ws_bytes=1 << 40)
    f = L.spec_orthogonalize
    wild, nan = (ctypes.c_double * 3)(3.0, 1e6, 1.0), (ctypes.c_double * 3)(3.0, float("nan"), 1.0)
    for bad in (dict(G=None), dict(O=None), dict(coeffs=None), dict(batch=0), dict(batch=65536), dict(m=0), dict(n=0),
                dict(ldg=31), dict(ldo=31), dict(sg=2047), dict(so=2047), dict(steps=0), dict(steps=33), dict(eps=-1.0),
                dict(eps=float("nan")), dict(scale=float("inf")), dict(coeffs=nan), dict(coeffs=wild), dict(G=FAKE + 1),
                dict(ws=FAKE + 8), dict(m=65537), dict(m=40000, n=40000, ldg=40000, ldo=40000, batch=1)):
        assert f(*_with(ok, **bad)) == EINVAL, bad
    assert f(*_with(ok, t=spec.F64)) == EUNSUPPORTED
    for bad in (dict(ws=None), dict(ws_bytes=100)):
        assert f(*_with(ok, **bad)) == EWORKSPACE, bad


def test_factors_beyond_f32(L):
    """Factors are applied in f32: 1e39 would make NaN of a zero there (and is no f32), 3e38 is one."""
    three = ctypes.c_double * 3
    for x, status in ((1e39, EINVAL), (-1e39, EINVAL), (1e308, EINVAL), (3e38, EWORKSPACE), (-3e38, EWORKSPACE)):
        assert L.spec_embed(None, FAKE, spec.F32, 100, 64, 64, FAKE, spec.I64, 0, x, FAKE, 64) == (
            EINVAL if status == EINVAL else 0)  # (no position: nothing is enqueued)
        assert L.spec_embed_grad(None, FAKE, spec.F32, 10, 100, 64, 64, FAKE, spec.I64, x, 0.0, FAKE, spec.F32, 64, None,
                                 0) == status
        xent = dict(XENT, t=spec.F32, scale=x)
        assert L.spec_linear_xent(*xent.values(), FAKE, FAKE, None, 0) == status
        assert L.spec_linear_xent_grad(*xent.values(), FAKE, FAKE, 0.0, FAKE, 64, FAKE, 64, None, 0) == status
        xent["scale"] = 1.0
        assert L.spec_linear_xent_grad(*xent.values(), FAKE, FAKE, x, FAKE, 64, FAKE, 64, None, 0) == status
        for co, scale in ((three(3.4445, -4.7750, 2.0315), x), (three(x, -4.7750, 2.0315), 1.0)):
            assert L.spec_orthogonalize(None, FAKE, spec.F32, 1, 64, 32, 32, 2048, co, 1, 1e-7, scale, FAKE, 32, 2048,
                                        None, 0) == status


def test_orthogonalize_strides_past_64_bits(L):
    """64 rows of 2^62 elements do not fit a stride of 0, though 64 * 2^62 is 0 in 64 bits."""
    co = (ctypes.c_double * 3)(3.4445, -4.7750, 2.0315)
    for ldg, sg, ldo, so in ((1 << 62, 0, 32, 2048), (32, 2048, 1 << 62, 0), (32, -2048, 32, 2048)):
        assert L.spec_orthogonalize(None, FAKE, spec.BF16, 2, 64, 32, ldg, sg, co, 1, 1e-7, 1.0, FAKE, ldo, so, None,
                                    0) == EINVAL


@pytest.mark.parametrize("c", [0.0, 1e-15, -1e-15, 1e-18, 1e-300, 1e-6, -1e-6])
def test_orthogonalize_bound_with_a_small_quintic_term(L, c):
    """40 s - 40 s^3 + c s^5 reaches 15.4 at s = 1 / sqrt(3) and is c at s = 1: past what f16 steps hold, whatever c;
    2 s - 2 s^3 + c s^5 reaches 0.77 and is taken (up to the missing workspace)."""
    for ab, status in ((40.0, EINVAL), (2.0, EWORKSPACE)):
        co = (ctypes.c_double * 6)(ab, -ab, c, 3.0, -3.0, 1.0)
        assert L.spec_orthogonalize(None, FAKE, spec.BF16, 1, 64, 32, 32, 2048, co, 2, 1e-7, 1.0, FAKE, 32, 2048, None,
                                    0) == status


def test_workspace_queries(L):
    import torch
    b = ctypes.c_size_t(0)
    assert L.spec_embed_grad_workspace(10, 100, 64, None) == EINVAL
    assert L.spec_embed_grad_workspace(-1, 100, 64, ctypes.byref(b)) == EINVAL
    assert L.spec_linear_xent_workspace(10, 100, 64, spec.F64, ctypes.byref(b)) == EUNSUPPORTED
    assert L.spec_linear_xent_grad_workspace(10, 0, 64, spec.F32, ctypes.byref(b)) == EINVAL
    assert L.spec_orthogonalize_workspace(1, 0, 64, spec.F32, ctypes.byref(b)) == EINVAL
    assert L.spec_orthogonalize_workspace(1, 64, 64, spec.F64, ctypes.byref(b)) == EUNSUPPORTED
    # no workspace holds the T x V logits: at 8192 x 131072 they would be 2 GiB in bf16 alone
    assert 0 < spec.linear_xent_workspace(8192, 131072, 4096, torch.bfloat16) < 1 << 29
    assert 0 < spec.linear_xent_grad_workspace(8192, 131072, 4096, torch.bfloat16) < 1 << 30
    assert spec.embed_grad_workspace(0, 1, 1) > 0 and spec.orthogonalize_workspace(1, 1, 1, torch.float32) > 0


def test_binding_refuses_before_the_library():
    import torch
    E, ids = torch.zeros(10, 8), torch.zeros(3, dtype=torch.int64)
    for call, status in (
            (lambda: spec.embed(E, ids), EINVAL),  # not on the GPU
            (lambda: spec.embed(E, ids.float()), EUNSUPPORTED),
            (lambda: spec.embed(E.t(), ids), EINVAL),  # inner dimension strided
            (lambda: spec.embed_grad(torch.zeros(4, 8), ids, 10), EINVAL),  # one id per row
            (lambda: spec.embed_grad(torch.zeros(3, 8), ids, 10, beta=1.0), EINVAL),  # beta without dE
            (lambda: spec.linear_xent(E, torch.zeros(5, 9), ids), EINVAL),
            (lambda: spec.linear_xent(E, torch.zeros(5, 8, dtype=torch.bfloat16), ids), EINVAL),
            (lambda: spec.orthogonalize(torch.zeros(4)), EINVAL),
            (lambda: spec.orthogonalize(torch.zeros(4, 4).t()[:, ::2]), EINVAL)):
        with pytest.raises(spec.SpecError) as e:
            call()
        assert e.value.status == status
