"""The training operators together, as examples/student_step.py runs them: one
step against float64 autograd, and a training run that learns."""
import importlib.util
import os

import pytest

from gpu_util import print_case

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def student():
    import torch
    import weights_bf16_fp32_amd as spec
    assert torch.cuda.is_available()
    spec.lib()
    f = importlib.util.spec_from_file_location("student_step", os.path.join(ROOT, "examples", "student_step.py"))
    m = importlib.util.module_from_spec(f)
    f.loader.exec_module(m)
    return m


def test_one_step_is_autograds(student):
    """Table, hidden states and layer in f32: every gradient of a step within 1e-5 of float64 autograd in norm
    (products of up to 700 terms in f32: 700 * 2^-24 is 4e-5 at worst, a tenth of it in practice)."""
    import torch
    import weights_bf16_fp32_amd as spec
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    V, k, T, scale = 700, 48, 500, 48 ** 0.5
    print_case("student_step", V=V, k=k, T=T)
    table = torch.randn(V, k, generator=g, device="cuda") / k ** 0.5
    layer = torch.randn(k, k, generator=g, device="cuda") / k ** 0.5
    ids = torch.randint(-1, V, (T,), generator=g, device="cuda")
    target = torch.randint(-1, V, (T,), generator=g, device="cuda")
    dloss = (target >= 0).float() / (target >= 0).sum()
    x = spec.embed(table, ids, scale=scale)
    h = x @ layer.t()
    loss, lse = spec.linear_xent(h, table, target)
    dh, dtable = spec.linear_xent_grad(h, table, target, lse, dloss)
    spec.embed_grad(dh @ layer, ids, V, scale=scale, beta=1.0, dE=dtable)
    dlayer = dh.t() @ x
    t, w = table.double().requires_grad_(), layer.double().requires_grad_()
    xr = torch.where((ids >= 0)[:, None], t[ids.clamp(min=0)] * scale, 0.0)
    total = (torch.nn.functional.cross_entropy(xr @ w.t() @ t.t(), target, ignore_index=-1, reduction="none") * dloss).sum()
    total.backward()
    assert abs((loss * dloss).sum().item() - total.item()) <= 1e-5 * total.item()
    for got, want in ((dtable, t.grad), (dlayer, w.grad)):
        assert torch.linalg.vector_norm(got.double() - want) <= 1e-5 * torch.linalg.vector_norm(want)


def test_training_learns_and_repeats(student):
    losses = student.train(steps=40, log=lambda s: None)
    assert losses[-1] < 0.5 * losses[0] and all(x == x for x in losses)
    assert losses == student.train(steps=40, log=lambda s: None)  # no step depends on the order of additions
