"""The ways that the training operators take at larger sizes, against the same
float64 definitions and bounds as at the smaller ones: sorts of several passes,
large tiles of dH, heads with unaligned rows in several pieces."""
import pytest

import test_gpu_embed_xent as base
from gpu_util import print_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def spec():
    import torch
    import weights_bf16_fp32_amd as spec
    assert torch.cuda.is_available()
    spec.lib()
    return spec


# one workgroup's sort in its longest form; two and three passes of the others'
@pytest.mark.parametrize("types", ["bf16-bf16", "bf16-f32", "f32-f32"])
@pytest.mark.parametrize("n,V,d", [(12000, 131072, 24), (16384, 50021, 16), (16385, 50021, 16), (20001, 131072, 40),
                                   (17000, 1100000, 8)])
def test_embed_grad_sorts(spec, types, n, V, d):
    base.test_embed_grad(spec, types, n, V, d, 0, "zipf")


@pytest.mark.parametrize("n,V", [(4096, 131072), (16384, 131072), (20480, 1000), (20480, 131072), (40960, 1100000)])
def test_embed_grad_adds_in_order_of_position(spec, n, V):
    """Four positions per token, 2^24, 1, 1, -2^24 in this order: f32 sums to 0 in it and to 1 or 2 in others.
    (Tokens of four do not cross the shares of 8 or 32 positions.)"""
    import torch
    print_case("embed_grad_order", n=n, V=V)
    g = base._gen(n + V)
    k = min(n // 4, V // 2)
    tokens = torch.randperm(V, generator=g, device="cuda")[:k]
    ids = torch.full((n,), -1, device="cuda")
    place = torch.randperm(n, generator=g, device="cuda")[:4 * k].view(k, 4).sort(1).values  # of each token, in order
    ids[place.view(-1)] = tokens.repeat_interleave(4)
    dY = torch.zeros(n, 8, device="cuda")
    dY[place.view(-1)] = torch.tensor([2.0 ** 24, 1.0, 1.0, -2.0 ** 24], device="cuda").repeat(k)[:, None]
    assert not spec.embed_grad(dY, ids, V).any()
    assert spec.embed_grad(dY.flip(0), ids.flip(0), V)[tokens].eq(2.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,d,pad,shift", [
    (64, 700, 96, 0, 0), (65, 700, 96, 0, 0),  # either side of the tiles for few rows
    (4100, 1500, 2056, 0, 0),                  # dH in 256 x 256 tiles, the last round split along the vocabulary
    (5, 140001, 1001, 0, 0),                   # W copied in pieces, few rows
    (20000, 9001, 63, 0, 0),                   # and many
    (9000, 20000, 64, 0, 1)])                  # rows of whole 16 bytes that do not begin at them
def test_linear_xent_paths(spec, dtype, T, V, d, pad, shift):
    base.test_linear_xent(spec, dtype, "some", T, V, d, pad, shift, 1.0)
