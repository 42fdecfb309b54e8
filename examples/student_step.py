"""A layer compressed to the signal subspace of its activations, and trained there.

The covariance of the teacher's activations, its leading eigenvectors P, the
projected layer W' = P^T W P and table E' = E P ("Random matrix theory spectral
methods" page, section 4.1) come from the spectral path.  The student then takes
training steps on a next-token task: lookup, layer, cross entropy of the tied
head, both gradients into one table, and an orthogonalised update of the layer.

    python examples/student_step.py [steps]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import weights_bf16_fp32_amd as spec  # noqa: E402


def teacher(V, d, g):
    """A table whose rows lie near a 32-dimensional subspace, and a layer."""
    basis = torch.linalg.qr(torch.randn(d, 32, generator=g, device="cuda"))[0]
    E = torch.randn(V, 32, generator=g, device="cuda") @ basis.t() + 0.05 * torch.randn(V, d, generator=g, device="cuda")
    return E, torch.eye(d, device="cuda") + 0.1 * torch.randn(d, d, generator=g, device="cuda") / d ** 0.5


def project(E, W, k=32):
    """(P, W', E'): the k leading eigenvectors of the rows' covariance, the layer and the table on them."""
    V, d = E.shape
    C = torch.zeros(d, d, device="cuda")
    spec.cov_accumulate(E.bfloat16(), C, alpha=1.0 / V)
    P = spec.eigh_large(C, k)[1]
    Wp, _ = spec.project_weight(W, P)
    return P, Wp, E @ P


def train(steps=60, V=500, d=256, T=4096, lr=0.02, log=print):
    """Losses of `steps` steps; the targets follow a fixed successor of each token, a tenth of
    them anything, and the first positions of every row of 64 are a prompt without targets."""
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    E, W = teacher(V, d, g)
    P, Wp, table = project(E, W)
    k = Wp.shape[0]
    layer = Wp.bfloat16()
    table = (table / table.norm(dim=1, keepdim=True)).bfloat16()
    successor = torch.randperm(V, generator=g, device="cuda")
    moment, scale, losses = torch.zeros(k, k, device="cuda"), k ** 0.5, []
    for step in range(steps):
        ids = torch.randint(0, V, (T,), generator=g, device="cuda")
        noise = torch.rand(T, generator=g, device="cuda") < 0.1
        target = torch.where(noise, torch.randint(0, V, (T,), generator=g, device="cuda"), successor[ids])
        target[torch.arange(T, device="cuda") % 64 < 8] = -1
        dloss = (target >= 0).float() / (target >= 0).sum()

        x = spec.embed(table, ids, scale=scale)                                  # [T, k]
        h = x @ layer.t()
        loss, lse = spec.linear_xent(h, table, target)
        dh, dtable = spec.linear_xent_grad(h, table, target, lse, dloss)
        dx = dh @ layer
        spec.embed_grad(dx, ids, V, scale=scale, beta=1.0, dE=dtable)            # the tied table's other half
        moment = 0.9 * moment + (dh.t() @ x).float()
        update = spec.orthogonalize(moment.bfloat16(), scale=lr)
        layer = (layer.float() - update.float()).bfloat16()
        table = (table.float() - 20.0 * lr * dtable.float() * V ** 0.5).bfloat16()

        losses.append((loss * dloss).sum().item())
        if step % 10 == 0 or step == steps - 1:
            log(f"step {step:3d}  loss {losses[-1]:.4f}")
    return losses


if __name__ == "__main__":
    train(int(sys.argv[1]) if len(sys.argv) > 1 else 60)
