"""Embedding lookup, its gradient, and the vocabulary cross entropy with its
gradients against their definitions in float64.

Bounds.  u = 2^-24 (f32), r = the output type's unit roundoff (2^-8 bf16, 2^-24 f32).
A sum of m products accumulated in f32, in any order, is off by at most
(m + 2) u sum|terms|; exp and log of the device are taken as good to 2^-21
relative (arguments below 2^7 round by 2^-17 at most, absolutely)."""
import math

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


def _dt(name):
    import torch
    return torch.bfloat16 if name == "bf16" else torch.float32


def _r(name):
    import torch
    return torch.finfo(_dt(name)).eps / 2


def _gen(seed):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    import torch
    return torch.randn(*shape, generator=g, device="cuda")


def _strided(x, pad, shift=0):
    """x with rows `pad` elements further apart, its first element `shift` elements into the buffer."""
    import torch
    n, d = x.shape
    buf = torch.full((n * (d + pad) + shift,), float("nan"), dtype=x.dtype, device=x.device)
    y = torch.as_strided(buf, (n, d), (d + pad, 1), shift)
    y.copy_(x)
    return y


# ---------------------------------------------------------------- lookup

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,V,d,pad,shift,idt", [
    (1, 1, 1, 0, 0, "i64"), (1, 1000, 4096, 0, 0, "i32"), (5, 17, 8, 0, 0, "i64"), (63, 257, 1000, 8, 0, "i32"),
    (130, 50, 333, 3, 0, "i64"), (67, 99, 64, 0, 1, "i64"), (1025, 31, 4104, 0, 0, "i64"), (0, 10, 16, 0, 0, "i64")])
def test_embed(spec, dtype, n, V, d, pad, shift, idt):
    import torch
    print_case("embed", n=n, V=V, d=d, pad=pad, dtype=dtype)
    g = _gen(n + d)
    E = _strided(_randn(g, V, d).to(_dt(dtype)), pad, shift)
    ids = torch.randint(-2, V + 2, (n,), generator=g, device="cuda")  # some outside on both sides
    scale = math.sqrt(d)
    Y = spec.embed(E, ids.to(torch.int32 if idt == "i32" else torch.int64), scale=scale)
    ok = (ids >= 0) & (ids < V)
    # one product in f32 and one rounding: exact
    want = (E[ids.clamp(0, V - 1)].float() * torch.tensor(scale, dtype=torch.float32, device="cuda")).to(_dt(dtype))
    want = torch.where(ok[:, None], want, torch.zeros_like(want))
    assert Y.dtype == _dt(dtype) and torch.equal(Y, want)


def test_embed_into_strided_rows_and_past_32_bits(spec):
    import torch
    V, d = 270000, 8192  # 4.4 GB: the last rows lie past 2^32 bytes and 2^31 elements
    E = torch.empty((V, d), dtype=torch.bfloat16, device="cuda")
    E[0] = 1.0
    E[V - 3:] = torch.arange(3, device="cuda")[:, None].to(torch.bfloat16) + 5.0
    ids = torch.tensor([V - 1, 0, V - 3, V], device="cuda")
    out = torch.full((4, d + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    spec.embed(E, ids, scale=2.0, out=out[:, :d])
    assert [out[i, :d].unique().tolist() for i in range(4)] == [[14.0], [2.0], [10.0], [0.0]]
    assert bool((out[:, d:] == 7.0).all())


# ---------------------------------------------------------------- lookup's gradient

def _grad_ref(dY, ids, V, scale):
    """(sums, sums of magnitudes, counts) in float64."""
    import torch
    ok = (ids >= 0) & (ids < V)
    out, mag = (torch.zeros(V, dY.shape[1], dtype=torch.float64, device="cuda") for _ in range(2))
    rows = dY[ok].double()
    out.index_add_(0, ids[ok], rows)
    mag.index_add_(0, ids[ok], rows.abs())
    return out * scale, mag * abs(scale), torch.bincount(ids[ok], minlength=V).double()


@pytest.mark.parametrize("types", ["bf16-bf16", "bf16-f32", "f32-f32"])
@pytest.mark.parametrize("n,V,d,pad,kind", [
    (1, 1, 1, 0, "any"), (1, 50021, 1000, 0, "any"), (31, 7, 64, 0, "any"), (32, 7, 64, 4, "one"),
    (33, 1, 100, 0, "one"), (257, 65536, 333, 0, "any"), (1000, 40, 72, 8, "any"), (4099, 3, 260, 0, "one"),
    (5000, 131072, 128, 0, "zipf"), (2048, 1023, 1024, 0, "zipf"), (2049, 1024, 2056, 0, "zipf"), (64, 9, 16, 0, "none"),
    (0, 9, 16, 0, "none"), (70000, 300, 8, 0, "zipf")])
def test_embed_grad(spec, types, n, V, d, pad, kind):
    import torch
    print_case("embed_grad", n=n, V=V, d=d, kind=kind, types=types)
    yt, et = types.split("-")
    g = _gen(n + V)
    dY = _strided(_randn(g, n, d).to(_dt(yt)), pad) if n else torch.zeros((0, d), dtype=_dt(yt), device="cuda")
    if kind == "one":  # one long segment
        ids = torch.full((n,), V - 1, device="cuda")
    elif kind == "none":
        ids = torch.full((n,), -1, device="cuda")
    elif kind == "zipf":
        u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
        ids = (torch.exp(u * math.log(V + 1)) - 1).long().clamp(0, V - 1)
        ids = torch.where(torch.rand(n, generator=g, device="cuda") < 0.05, ids * 0 - 100, ids)
    else:
        ids = torch.randint(-1, V + 1, (n,), generator=g, device="cuda")
    out = ids[(ids < 0) | (ids >= V)].shape[0]
    if out:  # what stands in a row without a token reaches nothing
        dY[(ids < 0) | (ids >= V)] = float("nan")
    scale = 0.37
    dE = spec.embed_grad(dY, ids, V, scale=scale, dE=torch.full((V, d), float("nan"), dtype=_dt(et), device="cuda"))
    want, mag, cnt = _grad_ref(torch.nan_to_num(dY), ids, V, scale)
    bound = (cnt[:, None] + 3) * U * mag + _r(et) * want.abs() + 1e-38
    assert bool(((dE.double() - want).abs() <= bound * 1.01).all())
    assert torch.equal(dE, spec.embed_grad(dY, ids.int(), V, scale=scale, dE=torch.empty_like(dE)))  # every run the same
    # added to what is there, rows without a token untouched
    base = _randn(g, V, d).to(_dt(et))
    acc = spec.embed_grad(dY, ids, V, scale=scale, beta=1.0, dE=base.clone())
    total = want + base.double()
    bound = (cnt[:, None] + 3) * U * (mag + base.double().abs()) + _r(et) * total.abs() + 1e-38
    assert bool(((acc.double() - total).abs() <= bound * 1.01).all())
    assert torch.equal(acc[cnt == 0], base[cnt == 0])


def test_embed_grad_is_the_difference_quotient(spec):
    """The lookup is linear in the table: (f(E + h D) - f(E - h D)) / 2h = <dE, D> for f = <C, Y>."""
    import torch
    g = _gen(5)
    V, d, n = 97, 40, 300
    E, D, C = _randn(g, V, d), _randn(g, V, d), _randn(g, n, d)
    ids = torch.randint(-1, V, (n,), generator=g, device="cuda")
    f = lambda X: (C.double() * spec.embed(X, ids, scale=3.0).double()).sum()  # noqa: E731
    dE = spec.embed_grad(C, ids, V, scale=3.0).double()
    quotient = (f(E + D) - f(E - D)) / 2
    slack = n * d * 16 * U * 3.0 * 4.0 * 4.0  # every product below 4 sigma on each side
    assert abs(quotient - (dE * D.double()).sum()) <= slack


# ---------------------------------------------------------------- cross entropy

def _xent_ref(H, W, target, scale, dloss=None):
    """loss, lse, dH, dW in float64, and the bounds of the kernels' errors."""
    import torch
    T, V, d = H.shape[0], W.shape[0], W.shape[1]
    name = "bf16" if H.dtype == torch.bfloat16 else "f32"
    r = _r(name)
    ok = (target >= 0) & (target < V)
    Hd = torch.where(ok[:, None], H.double(), 0.0)
    Wd = W.double()
    z = scale * Hd @ Wd.t()
    ez = (d + 3) * U * abs(scale) * (Hd.abs() @ Wd.abs().t())  # of a logit
    lse = torch.logsumexp(z, 1)
    span = (lse[:, None] - z).clamp(min=0)
    # exponentials: device exp and its argument's rounding; sums of at most V terms, 64 + 64 + V / 8192 in a row
    ee = 2.0 ** -20 + 4 * U * (span + z.abs())
    p = torch.exp(z - lse[:, None])
    el = (p * (ez + ee)).sum(1) + (160 + V / 8192) * U + 2.0 ** -20 + 4 * U * lse.abs()
    tgt = target.clamp(0, V - 1)[:, None]
    zt, ezt = z.gather(1, tgt)[:, 0], ez.gather(1, tgt)[:, 0]
    out = dict(loss=torch.where(ok, lse - zt, 0.0), lse=torch.where(ok, lse, 0.0))
    bound = dict(loss=torch.where(ok, el + ezt + 4 * U * (lse.abs() + zt.abs()), 0.0), lse=torch.where(ok, el, 0.0))
    if dloss is not None:
        w = torch.where(ok, dloss.double(), 0.0)[:, None] * scale
        hot = torch.zeros_like(z).scatter_(1, tgt, 1.0)
        G = (p - hot) * w
        eG = w.abs() * p * (ez + ee + el[:, None]) + (r + 4 * U) * G.abs() + 4 * U * w.abs() * (p + hot)
        out["dH"], out["dW"] = G @ Wd, G.t() @ Hd
        bound["dH"] = eG @ Wd.abs() + (V + 64) * U * (G.abs() @ Wd.abs()) + r * out["dH"].abs()
        bound["dW"] = eG.t() @ Hd.abs() + (T + 3) * U * (G.abs().t() @ Hd.abs()) + r * out["dW"].abs()
    return out, bound


def _within(got, want, bound, what):
    d = (got.double() - want).abs()
    assert bool((d <= 1.05 * bound + 1e-37).all()), f"{what}: {(d / (bound + 1e-37)).max().item():.3g} times the bound"


CASES = [  # T, V, d, padding of H's and W's rows, their shift, scale
    (1, 1, 1, 0, 0, 1.0), (1, 1000, 64, 0, 0, 1.0), (3, 129, 8, 0, 0, 0.5), (16, 4099, 256, 0, 0, 1.0),
    (63, 127, 33, 0, 0, 2.0), (129, 257, 100, 4, 0, 1.0), (200, 1000, 1000, 8, 0, 1.0), (257, 513, 72, 0, 1, 1.0),
    (300, 2500, 136, 24, 0, -0.7), (2, 70000, 40, 0, 0, 1.0), (515, 3, 512, 0, 0, 1.0), (128, 128, 64, 0, 0, 1.0),
    (256, 256, 128, 0, 0, 1.0), (513, 5000, 320, 0, 0, 1.0)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("masked", ["none", "some", "odd"])
@pytest.mark.parametrize("T,V,d,pad,shift,scale", CASES)
def test_linear_xent(spec, dtype, masked, T, V, d, pad, shift, scale):
    import torch
    print_case("linear_xent", T=T, V=V, d=d, pad=pad, shift=shift, dtype=dtype, masked=masked)
    g = _gen(T * 7 + V + d)
    H = _strided(_randn(g, T, d).to(_dt(dtype)), pad, shift)
    W = _strided((_randn(g, V, d) * (2.0 / math.sqrt(d))).to(_dt(dtype)), pad, shift)
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    if masked == "some":
        target = torch.where(torch.rand(T, generator=g, device="cuda") < 0.4, target * 0 - 100, target)
    elif masked == "odd":
        target[::2] = V  # past the vocabulary
    off = (target < 0) | (target >= V)
    if bool(off.any()):
        H[off] = float("nan")  # what a masked row holds reaches nothing
    dloss = torch.rand(T, generator=g, device="cuda") / T
    want, bound = _xent_ref(torch.nan_to_num(H), W, target, scale, dloss)
    loss, lse = spec.linear_xent(H, W, target, scale=scale)
    _within(loss, want["loss"], bound["loss"], "loss")
    _within(lse, want["lse"], bound["lse"], "lse")
    assert bool((loss[off] == 0).all()) and bool((lse[off] == 0).all())
    dW0 = torch.full((V, d), float("nan"), dtype=H.dtype, device="cuda")
    dH, dW = spec.linear_xent_grad(H, W, target.int(), lse, dloss, scale=scale, dW=dW0)
    _within(dH, want["dH"], bound["dH"], "dH")
    _within(dW, want["dW"], bound["dW"], "dW")
    assert bool((dH[off] == 0).all())
    again = spec.linear_xent_grad(H, W, target, lse, dloss, scale=scale)
    assert torch.equal(dH, again[0]) and torch.equal(dW, again[1])
    # accumulated into what is there, in rows further apart than d
    base = _strided(_randn(g, V, d).to(_dt(dtype)), 5)
    total = want["dW"] - 0.5 * base.double()
    more = bound["dW"] + (_r(dtype) + 4 * U) * (total.abs() + base.double().abs())
    _, acc = spec.linear_xent_grad(H, W, target, lse, dloss, scale=scale, beta=-0.5, dW=base)
    _within(acc, total, more, "accumulated dW")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_linear_xent_pieces(spec, dtype):
    """Enough rows that the vocabulary is taken in several pieces, the last one ragged."""
    import torch
    T, V, d = (20000, 9001, 64) if dtype == "bf16" else (10500, 9001, 64)
    print_case("linear_xent_pieces", T=T, V=V, d=d, dtype=dtype)
    g = _gen(11)
    H, W = _randn(g, T, d).to(_dt(dtype)), (_randn(g, V, d) * 0.3).to(_dt(dtype))
    target = torch.randint(-1, V, (T,), generator=g, device="cuda")
    dloss = torch.full((T,), 1.0 / T, device="cuda")
    want, bound = _xent_ref(H, W, target, 1.0, dloss)
    loss, lse = spec.linear_xent(H, W, target)
    dH, dW = spec.linear_xent_grad(H, W, target, lse, dloss)
    for k, x in (("loss", loss), ("lse", lse), ("dH", dH), ("dW", dW)):
        _within(x, want[k], bound[k], k)


def test_linear_xent_without_targets(spec):
    import torch
    g = _gen(3)
    W = _randn(g, 300, 64).bfloat16()
    for T in (0, 70):
        H = torch.full((T, 64), float("inf"), dtype=torch.bfloat16, device="cuda")
        target = torch.full((T,), -100, dtype=torch.int64, device="cuda")
        loss, lse = spec.linear_xent(H, W, target)
        base = _randn(g, 300, 64).bfloat16()
        dH, dW = spec.linear_xent_grad(H, W, target, lse, torch.full((T,), float("nan"), device="cuda"), beta=2.0,
                                       dW=base.clone())
        assert not loss.any() and not lse.any() and not dH.any()
        assert torch.equal(dW, (base.float() * 2).bfloat16())
        assert not spec.linear_xent_grad(H, W, target, lse, torch.ones(T, device="cuda"))[1].any()


def test_linear_xent_extremes(spec):
    """Large logits neither overflow nor lose the loss; a row with NaN or inf says so and leaves the others alone."""
    import torch
    g = _gen(4)
    T, V, d = 40, 1000, 64
    H, W = _randn(g, T, d), _randn(g, V, d)
    H[0] = 200.0 * W[7]  # one logit far above the rest: exp of the difference is zero in f32
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    target[0] = 7
    target[1], H[1] = 3, -300.0 * W[3]  # the target far below the rest
    want, bound = _xent_ref(H, W, target, 1.0)
    loss, lse = spec.linear_xent(H, W, target)
    _within(loss, want["loss"], bound["loss"], "loss")
    _within(lse, want["lse"], bound["lse"], "lse")
    H[5, 0], H[6, 0] = float("nan"), float("inf")
    loss2, lse2 = spec.linear_xent(H, W, target)
    bad = torch.zeros(T, dtype=torch.bool, device="cuda")
    bad[5:7] = True
    assert bool(loss2[bad].isnan().all()) and bool(lse2[bad].isnan().all())
    assert torch.equal(loss2[~bad], loss[~bad]) and torch.equal(lse2[~bad], lse[~bad])
    # a vocabulary entry of the most negative value: its logits are -inf or the least number, others stand
    W2 = torch.full_like(W[:2], torch.finfo(torch.float32).min)
    Hp = H.abs().nan_to_num(1.0, 1.0)
    l3, s3 = spec.linear_xent(Hp, torch.cat([W, W2]), target)
    l4, s4 = spec.linear_xent(Hp, W, target)
    assert bool(torch.isfinite(l3).all())
    tiny = 64 * U * (s4.abs() + (Hp @ W.t()).abs().max(1).values)
    assert bool(((l3 - l4).abs() <= tiny).all()) and bool(((s3 - s4).abs() <= tiny).all())


def test_linear_xent_gradient_is_the_difference_quotient(spec):
    """Central differences of the summed loss along random directions, f32."""
    import torch
    g = _gen(6)
    T, V, d = 50, 300, 32
    H, W = _randn(g, T, d), _randn(g, V, d) * 0.3
    target = torch.randint(-1, V, (T,), generator=g, device="cuda")
    dloss = torch.rand(T, generator=g, device="cuda")
    _, lse = spec.linear_xent(H, W, target, scale=0.8)
    dH, dW = spec.linear_xent_grad(H, W, target, lse, dloss, scale=0.8)
    f = lambda h, w: (spec.linear_xent(h, w, target, scale=0.8)[0].double() * dloss.double()).sum().item()  # noqa: E731
    step = 2.0 ** -6
    for dirH, dirW in ((_randn(g, T, d), torch.zeros_like(W)), (torch.zeros_like(H), _randn(g, V, d) * 0.3)):
        quotient = (f(H + step * dirH, W + step * dirW) - f(H - step * dirH, W - step * dirW)) / (2 * step)
        slope = ((dH.double() * dirH.double()).sum() + (dW.double() * dirW.double()).sum()).item()
        # third derivative of a row's loss along a direction that moves its logits by at most m: |third central
        # moment| <= m^3; rounding of T losses below 16, each good to 2^-18
        m = 0.8 * ((dirH @ W.t()).abs().max(1).values + (H @ dirW.t()).abs().max(1).values).double()
        slack = (dloss.double() * m ** 3).sum().item() * step ** 2 / 6 + T * 2.0 ** -18 / step
        assert abs(quotient - slope) <= slack


def test_on_another_stream(spec):
    """Every call goes to the current stream and orders with what is there."""
    import torch
    g = _gen(8)
    T, V, d = 300, 2000, 256
    H, W = _randn(g, T, d).bfloat16(), _randn(g, V, d).bfloat16()
    ids = torch.randint(-1, V, (T,), generator=g, device="cuda")
    dl = torch.rand(T, generator=g, device="cuda")

    def all_of_it():
        loss, lse = spec.linear_xent(H * 0.1, W, ids)
        dH, dW = spec.linear_xent_grad(H * 0.1, W, ids, lse, dl)
        X = spec.embed(W, ids, scale=2.0)
        spec.embed_grad(dH, ids, V, beta=1.0, dE=dW)
        return loss, lse, dH, dW, X
    want = [x.clone() for x in all_of_it()]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = all_of_it()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_graph_capture_replays(spec):
    """The calls record into a HIP graph (no clears by the runtime among them) and replay on new inputs."""
    import torch
    g = _gen(9)
    T, V, d = 130, 1500, 128
    H, W = _randn(g, T, d).bfloat16(), (_randn(g, V, d) * 0.2).bfloat16()
    ids = torch.randint(-1, V, (T,), generator=g, device="cuda")
    dl = torch.rand(T, generator=g, device="cuda")

    def step():
        loss, lse = spec.linear_xent(H, W, ids)
        dH, dW = spec.linear_xent_grad(H, W, ids, lse, dl)
        return loss, dH, spec.embed_grad(dH, ids, V, beta=1.0, dE=dW), spec.embed(W, ids)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(4):
        H.copy_(_randn(g, T, d))
        ids.copy_(torch.randint(-1, V, (T,), generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in out]
        assert all(torch.equal(a, b) for a, b in zip(got, step())), k


def test_linear_xent_past_32_bits(spec):
    """A head of 4.4 GB: rows at its end are read and written at the right places."""
    import torch
    V, d, T = 270000, 8192, 3
    print_case("linear_xent_past_32_bits", T=T, V=V, d=d)
    g = _gen(10)
    W = torch.zeros((V, d), dtype=torch.bfloat16, device="cuda")
    H = _randn(g, T, d).bfloat16()
    W[V - 2:] = (_randn(g, 2, d) / 100).bfloat16()
    target = torch.tensor([V - 1, 5, V - 2], device="cuda")
    loss, lse = spec.linear_xent(H, W, target)
    z2 = H.double() @ W[V - 2:].double().t()
    want = torch.log(torch.exp(z2).sum(1) + (V - 2))
    zt = torch.stack([z2[0, 1], z2[1, 0] * 0, z2[2, 0]])
    assert bool(((lse - want).abs() <= 1e-5 * want).all()) and bool(((loss - (want - zt)).abs() <= 1e-4).all())
    dl = torch.tensor([1.0, 2.0, 3.0], device="cuda")
    dH, dW = spec.linear_xent_grad(H, W, target, lse, dl)
    p2 = torch.exp(z2 - want[:, None])
    g2 = p2 - torch.tensor([[0.0, 1.0], [0.0, 0.0], [1.0, 0.0]], device="cuda")
    g2 = g2 * dl.double()[:, None]
    refW, refH = g2.t() @ H.double(), g2 @ W[V - 2:].double()
    lim = 2.0 ** -7  # a rounding of G and one of the result, each 2^-8 of terms of one size
    assert bool(((dW[V - 2:].double() - refW).abs() <= lim * (g2.abs().t() @ H.double().abs())).all())
    assert bool(((dH.double() - refH).abs() <= lim * (g2.abs() @ W[V - 2:].double().abs()) + 1e-30).all())
    row = (torch.exp(-want) * dl)[None, :] @ H.double()  # rows of no token and zero weights: all alike
    assert bool(((dW[100].double() - row[0]).abs() <= lim * row.abs().max() + 1e-7).all())
    assert torch.equal(dW[100], dW[V // 2]) and torch.equal(dW[100], dW[V - 3])
