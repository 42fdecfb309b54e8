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
