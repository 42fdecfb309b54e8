"""A student of residual blocks: trained with its activations stored in 8 bits, scored from
its layers in 4.

Each block norms the residual stream, takes the norm through a layer, norms the
result, gates it and adds it to the stream; the tied head reads the last norm.  The
forward pass keeps, per block, the layer's input, its output and the new stream as
MX_INT8 (a little over a byte per value); the gradients of the norms and of the layers are
formed from those.  (The layers themselves, in bf16 while training, are random at first
and multiplied by torch.)  At the end they are packed into MX_FP4 and the same tokens
scored with them.

    python examples/residual_student.py [steps]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import weights_bf16_fp32_amd as spec  # noqa: E402

ALPHA, BETA = 1.0, 0.5  # residual scales: h <- ALPHA h + BETA gate norm(z)


def student(V=400, k=128, blocks=2, dtype=torch.bfloat16, seed=0):
    """Parameters: a tied table, and per block a layer, two norm weights and a gate."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")
    p = {"table": randn(V, k) / k ** 0.5, "first": 1 + 0.1 * randn(k)}
    for i in range(blocks):
        p[f"layer{i}"] = randn(k, k) / k ** 0.5
        p[f"post{i}"], p[f"pre{i}"], p[f"gate{i}"] = (1 + 0.1 * randn(k) for _ in range(3))
    return {n: t.to(dtype) for n, t in p.items()}


def block(p, i):
    return dict(w_post=p[f"post{i}"], w_pre=p[f"pre{i}"], gate=p[f"gate{i}"], alpha=ALPHA, beta=BETA)


def forward(p, ids, target, stored8=True, packed=None):
    """(losses, lse, what the backward pass needs); with `packed` layers (MX_FP4) they are used instead."""
    k = p["table"].shape[1]
    blocks = sum(n.startswith("layer") for n in p)
    h = spec.embed(p["table"], ids, scale=k ** 0.5)
    kept = []

    def store(t):
        return spec.mx_quantize(t, spec.MX_INT8) if stored8 else t

    def room():
        return spec.mx_empty(h.shape[0], k, spec.MX_INT8) if stored8 else None
    x8 = room()
    _, x, _, r = spec.block_norm(h, w_pre=p["first"], x8=x8)
    first = (store(h), r)
    for i in range(blocks):
        z = spec.mx_linear(x, packed[i]) if packed else x @ p[f"layer{i}"].t()
        z8, h8, next8 = room(), room(), room()  # filled by the pass that has the values in hand
        xin = x8 if stored8 else x
        h, x, r_post, r_pre = spec.block_norm(h, z, y8=z8, h8=h8, x8=next8, **block(p, i))
        kept.append((xin, z8 if stored8 else z, h8 if stored8 else h, r_post, r_pre))
        x8 = next8
    loss, lse = spec.linear_xent(x, p["table"], target)
    return loss, lse, (first, kept, x)


def backward(p, ids, target, lse, dloss, state):
    """Gradients of sum(dloss * loss), by parameter."""
    (h0, r0), kept, x = state
    V, k = p["table"].shape
    g = {}
    dx, g["table"] = spec.linear_xent_grad(x, p["table"], target, lse, dloss)
    dh = None
    for i in reversed(range(len(kept))):
        xin, z, h, r_post, r_pre = kept[i]
        dh, dz, g[f"post{i}"], g[f"pre{i}"], g[f"gate{i}"] = spec.block_norm_grad(dx, dh, h, z, r_pre, r_post, **block(p, i))
        g[f"layer{i}"] = spec.mx_weight_grad(dz, xin) if isinstance(xin, spec.Mx) else dz.t() @ xin
        dx = dz @ p[f"layer{i}"]
    dh, _, _, g["first"], _ = spec.block_norm_grad(dx, dh, h0, None, r0, w_pre=p["first"])
    spec.embed_grad(dh, ids, V, scale=k ** 0.5, beta=1.0, dE=g["table"])
    return g


def train(steps=40, V=400, k=128, T=2048, lr=0.02, log=print):
    """(losses of the steps, loss of the last batch, and its loss with the layers in 4 bits)."""
    p = student(V, k)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    successor = torch.randperm(V, generator=g, device="cuda")
    moments = {n: torch.zeros_like(t, dtype=torch.float32) for n, t in p.items()}
    losses = []
    for step in range(steps):
        ids = torch.randint(0, V, (T,), generator=g, device="cuda")
        target = successor[ids]
        target[torch.arange(T, device="cuda") % 64 < 8] = -1
        dloss = (target >= 0).float() / (target >= 0).sum()
        loss, lse, state = forward(p, ids, target)
        grads = backward(p, ids, target, lse, dloss, state)
        for n, m in moments.items():
            m.mul_(0.9).add_(grads[n].float())
            if n.startswith("layer"):
                update = spec.orthogonalize(m.bfloat16(), scale=lr).float()
            else:
                update = m * (20 * lr * V ** 0.5 if n == "table" else lr)
            p[n] = (p[n].float() - update).to(p[n].dtype)
        losses.append((loss * dloss).sum().item())
        if step % 10 == 0 or step == steps - 1:
            log(f"step {step:3d}  loss {losses[-1]:.4f}")
    packed = [spec.mx_quantize(p[f"layer{i}"], spec.MX_FP4) for i in range(2)]
    ends = [(forward(p, ids, target, stored8=False, packed=w)[0] * dloss).sum().item() for w in (None, packed)]
    log(f"loss {ends[0]:.4f}, with the layers in 4 bits {ends[1]:.4f}")
    return losses, *ends


if __name__ == "__main__":
    train(int(sys.argv[1]) if len(sys.argv) > 1 else 40)
