"""Sizes whose work items do not fit one launch (a grid holds fewer than 2^32
threads per dimension): the training operators take them all the same."""
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


def test_embed_of_many_positions(spec):
    import torch
    n, V = (1 << 26) + 5, 300
    print_case("embed_many", n=n, V=V, d=1)
    E = torch.randn(V, 1, device="cuda").bfloat16()
    ids = torch.arange(n, dtype=torch.int32, device="cuda") % (V + 1)  # V: no row
    Y = spec.embed(E, ids)
    want = torch.cat([E[:, 0], torch.zeros(1, dtype=torch.bfloat16, device="cuda")])[ids.long()]
    assert torch.equal(Y[:, 0], want)


def test_embed_grad_of_many_rows(spec):
    """More rows of zeros than one launch writes."""
    import torch
    V = (1 << 30) + (1 << 25)
    print_case("embed_grad_many_rows", n=3, V=V, d=1)
    dE = torch.full((V, 1), float("nan"), dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([V - 1, 5, V - 1], device="cuda")
    spec.embed_grad(torch.tensor([[1.0], [2.0], [4.0]], device="cuda").bfloat16(), ids, V, dE=dE)
    assert dE[V - 1].item() == 5.0 and dE[5].item() == 2.0 and torch.count_nonzero(dE).item() == 2


def test_embed_grad_of_many_positions(spec):
    """More shares of positions than one launch adds or joins; integers, so the sums are exact."""
    import torch
    V = 1024
    k = (1 << 19) + 8  # positions of every row
    n = k * V
    print_case("embed_grad_many_positions", n=n, V=V, d=1)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    dY = torch.randint(-1, 2, (k, V), generator=g, device="cuda", dtype=torch.int8)
    want = dY.sum(0, dtype=torch.int64)
    ids = torch.arange(n, dtype=torch.int32, device="cuda") % V
    dE = spec.embed_grad(dY.view(n, 1).bfloat16(), ids, V, dE=torch.full((V, 1), float("nan"), device="cuda"))
    assert torch.equal(dE[:, 0].long(), want)


def test_linear_xent_of_many_tiles(spec):
    """2^23 and more tiles of 256 x 256 logits; the rows repeat, so a few stand for all."""
    import torch
    T, V, d, k = 1 << 16, (1 << 23) + 300, 8, 16
    print_case("linear_xent_many_tiles", T=T, V=V, d=d)
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    W = torch.randn(V, d, generator=g, device="cuda").bfloat16()
    few = torch.randn(k, d, generator=g, device="cuda").bfloat16()
    tgt = torch.randint(0, V, (k,), generator=g, device="cuda")
    tgt[0], tgt[1], tgt[2] = V - 1, 0, -1
    loss, lse = spec.linear_xent(few.repeat(T // k, 1), W, tgt.repeat(T // k))
    z = few.double() @ W.double().t()
    want = torch.where(tgt >= 0, torch.logsumexp(z, 1), 0.0)
    want_loss = torch.where(tgt >= 0, want - z.gather(1, tgt.clamp(min=0)[:, None])[:, 0], 0.0)
    # in units of 2^-24: (160 + V / 8192) for the sums, 16 for exp and log, 4 lse for its rounding, and (d + 3)
    # |h| |w| < 1000 for a logit, in the lse and in the loss; together below 2^12
    tol = 2.0 ** -12
    assert ((lse.view(-1, k).double() - want).abs().max() <= tol) and ((loss.view(-1, k).double() - want_loss).abs().max() <= tol)
    assert bool((lse.view(-1, k)[:, 2] == 0).all()) and bool((loss.view(-1, k)[:, 2] == 0).all())


def test_linear_xent_grad_without_rows(spec):
    """No row at all: dW is scaled, however many rows it has."""
    import torch
    V = (1 << 24) + 3
    print_case("linear_xent_grad_without_rows", V=V, d=1)
    W = torch.zeros(V, 1, dtype=torch.bfloat16, device="cuda")
    dW = (torch.arange(V, device="cuda") % 100).bfloat16()[:, None]
    none = torch.zeros(0, device="cuda")
    got = spec.linear_xent_grad(W[:0], W, none.long(), none, none, beta=2.0, dW=dW.clone())[1]
    assert torch.equal(got, dW * 2)
