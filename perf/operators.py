"""Workloads of the operators that a student's training step is made of, at
sizes from a single decode step to a full training batch, with their plain
forms in float32 torch operations and their definitions in float64.

A layer compressed to the signal subspace of its activations is trained on
(embedding lookup -> layers -> softmax cross entropy over the vocabulary), and
its matrices are updated with orthogonalised gradients:

  embed          Y[i] = scale * E[ids[i]]                      (a zero row where ids[i] is no row of E)
  embed_grad     dE[v] = scale * sum of dY[i] over ids[i] = v
  xent           z = scale * H W^T,  lse_t = log sum_v exp z_tv,  loss_t = lse_t - z_t,target
                 (both 0 in a row whose target is no vocabulary entry)
  xent_step      the same, and for weights dloss_t on the rows' losses the gradients
                 G = dloss_t (softmax(z_t) - onehot(target_t)),  dH = scale G W,  dW = scale G^T H
  orthogonalize  X <- G / (|G|_F + eps), then `steps` times A = X X^T, X <- a X + (b A + c A^2) X
                 (on the shorter side of G), each step one factor on every singular value
"""
import math
import random

import torch

own = False

COEFFS = (3.4445, -4.7750, 2.0315)
EPS = 1e-7


def _case(name, **kw):
    return dict(name=name, **kw)


def listed():
    return [
        # one decode step of 8 sequences: latency
        _case("embed_decode", op="embed", n=8, V=65536, d=4096, dtype="bf16", pad=0.0),
        # packed prompts of 8192 tokens, some of them padding
        _case("embed_prompt", op="embed", n=8192, V=65536, d=4096, dtype="bf16", pad=0.03),
        # a narrow student in f32, odd vocabulary and row length
        _case("embed_grad_student", op="embed_grad", n=2047, V=50021, d=1000, dtype="f32", pad=0.03),
        # a training batch into the whole table's gradient; frequent tokens make long segments
        _case("embed_grad_train", op="embed_grad", n=16384, V=131072, d=4096, dtype="bf16", pad=0.03),
        # log-probabilities of the next token of 8 sequences: latency, bound by reading W
        _case("xent_score", op="xent", n=8, V=65536, d=4096, dtype="bf16", pad=0.0),
        # perplexity of an evaluation batch, the prompt half of every row not counted; odd sizes
        _case("xent_eval", op="xent", n=2047, V=50021, d=1000, dtype="bf16", pad=0.5),
        # a small student's step in f32
        _case("xent_step_f32", op="xent_step", n=509, V=32768, d=512, dtype="f32", pad=0.1),
        # a training step's head, a quarter of the tokens being prompt
        _case("xent_step_train", op="xent_step", n=8192, V=131072, d=4096, dtype="bf16", pad=0.25),
        # one projected layer of 256 x 256: latency
        _case("ortho_student", op="orthogonalize", batch=1, m=256, n=256, dtype="bf16"),
        # several layers of one odd shape, f32
        _case("ortho_odd", op="orthogonalize", batch=3, m=333, n=1000, dtype="f32"),
        # an attention projection
        _case("ortho_qproj", op="orthogonalize", batch=1, m=4096, n=4096, dtype="bf16"),
        # a feed-forward matrix, taller than wide
        _case("ortho_ffn", op="orthogonalize", batch=1, m=14336, n=4096, dtype="bf16"),
    ]


def _logu(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    """A size in [lo, hi], uniform in its logarithm: any odd number, or a power of two."""
    if rng.random() < 0.4:
        return 1 << rng.randint(max(0, math.ceil(math.log2(lo))), math.floor(math.log2(hi)))
    return min(hi, _logu(rng, lo, hi) | 1)


def draw(rng: random.Random):
    op = rng.choice(("embed", "embed_grad", "xent", "xent_step", "orthogonalize"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    if op == "orthogonalize":
        m, n = _size(rng, 32, 4096), _size(rng, 32, 8192)
        if rng.random() < 0.5:
            m, n = n, m
        if dtype == "f32":  # the f32 products run at a sixteenth of the bf16 rate
            m, n = min(m, 2048), min(n, 2048)
        batch = rng.choice((1, 1, 2, 5)) if m * n <= 1 << 20 else 1
        return dict(op=op, batch=batch, m=m, n=n, dtype=dtype)
    pad = rng.choice((0.0, 0.03, 0.25, 0.5))
    if op in ("embed", "embed_grad"):
        n, V, d = _size(rng, 1, 16384), _size(rng, 1000, 131072), _size(rng, 64, 4096)
        return dict(op=op, n=n, V=V, d=d, dtype=dtype, pad=pad)
    n, V, d = _size(rng, 1, 8192), _size(rng, 1000, 131072), _size(rng, 64, 4096)
    if dtype == "f32":
        n, d = min(n, 2048), min(d, 1024)
    return dict(op=op, n=n, V=V, d=d, dtype=dtype, pad=pad)


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _ids(case, g, dev):
    """Token ids as text has them: frequencies fall as one over the rank (ranks
    scattered over the vocabulary), and `pad` of the positions hold none (-1), in
    runs as padding and prompts come."""
    n, V = case["n"], case["V"]
    u = torch.rand(n, generator=g, device=dev, dtype=torch.float64)
    rank = (torch.exp(u * math.log(V + 1)) - 1).long().clamp_(0, V - 1)
    ids = (rank * 40503 + 12345) % V
    period = min(n, 256)
    off = torch.randint(period, (1,), generator=g, device=dev)
    masked = (torch.arange(n, device=dev) + off) % period < int(case["pad"] * period)
    return torch.where(masked, torch.full_like(ids, -1), ids)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = _dtype(case)
    op = case["op"]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    if op == "orthogonalize":
        b, m, n = case["batch"], case["m"], case["n"]
        # a gradient dY^T X over a batch of tokens: features of falling variance, mixed, and
        # tokens of unequal weight
        tok = 1024
        lo = min(m, n)

        def features(k):
            f = randn(b, tok, k) * torch.arange(1, k + 1, device=dev).float().rsqrt()
            return torch.matmul(f, randn(b, k, k) / math.sqrt(k)) if k <= 4096 else f
        w = torch.exp(randn(b, tok, 1))
        G = torch.matmul((features(m) * w).transpose(1, 2).contiguous(), features(n))
        G = G / tok + randn(b, m, n) * (0.05 / math.sqrt(lo * tok))
        G = G.to(dt)
        return dict(op=op, G=G if b > 1 else G[0])
    n, V, d = case["n"], case["V"], case["d"]
    ids = _ids(case, g, dev)
    if op == "embed":
        return dict(op=op, E=(randn(V, d) * 0.02).to(dt), ids=ids, scale=math.sqrt(d))
    if op == "embed_grad":
        return dict(op=op, dY=(randn(n, d) * 1e-3).to(dt), ids=ids, V=V, scale=math.sqrt(d))
    # hidden states of unit variance; a part of each row points at its target's row of W, so
    # that targets range from hardly to almost certainly predicted
    W = randn(V, d) / math.sqrt(d)
    H = randn(n, d) * 1.5
    H = H + W[ids.clamp(min=0)] * (torch.rand(n, 1, generator=g, device=dev) * 16.0)
    valid = ids >= 0
    dloss = torch.where(valid, 1.0, 0.0) / valid.sum().clamp(min=1)
    return dict(op=op, H=H.to(dt), W=W.to(dt), target=ids, dloss=dloss.float(), scale=1.0)


def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    import weights_bf16_fp32_amd as spec
    op = s["op"]
    if op == "embed":
        return spec.embed(s["E"], s["ids"], scale=s["scale"])
    if op == "embed_grad":
        return spec.embed_grad(s["dY"], s["ids"], s["V"], scale=s["scale"])
    if op == "orthogonalize":
        return spec.orthogonalize(s["G"], coeffs=[COEFFS] * 5, eps=EPS)
    loss, lse = spec.linear_xent(s["H"], s["W"], s["target"], scale=s["scale"])
    if op == "xent":
        return {"loss": loss, "lse": lse}
    dH, dW = spec.linear_xent_grad(s["H"], s["W"], s["target"], lse, s["dloss"], scale=s["scale"])
    return {"loss": loss, "lse": lse, "dH": dH, "dW": dW}


def _plain(s):
    op = s["op"]
    if op == "embed":
        ids = s["ids"]
        rows = s["E"][ids.clamp(min=0)].float() * s["scale"]
        return torch.where((ids >= 0)[:, None], rows, torch.zeros((), device=rows.device)).to(s["E"].dtype)
    if op == "embed_grad":
        ids, dY = s["ids"], s["dY"]
        sums = torch.zeros(s["V"] + 1, dY.shape[1], device=dY.device)  # the last row takes what has no token
        sums.index_add_(0, torch.where(ids >= 0, ids, s["V"]), dY.float())
        return (sums[:-1] * s["scale"]).to(dY.dtype)
    if op == "orthogonalize":
        G = s["G"]
        tall = G.shape[-2] > G.shape[-1]
        X = G.float().transpose(-1, -2) if tall else G.float()
        X = X / ((X * X).sum(dim=(-2, -1), keepdim=True).sqrt() + EPS)
        a, b, c = COEFFS
        for _ in range(5):
            A = torch.matmul(X, X.transpose(-1, -2))
            X = a * X + torch.matmul(b * A + c * torch.matmul(A, A), X)
        return (X.transpose(-1, -2) if tall else X).to(G.dtype).contiguous()
    target, scale = s["target"], s["scale"]
    valid = target >= 0
    tgt = target.clamp(min=0)[:, None]
    H = torch.where(valid[:, None], s["H"].float(), 0.0)
    W = s["W"].float()
    z = torch.matmul(H, W.t()) * scale
    top = z.max(dim=1, keepdim=True).values
    lse = top + torch.log(torch.exp(z - top).sum(dim=1, keepdim=True))
    loss = torch.where(valid, (lse - z.gather(1, tgt))[:, 0], 0.0)
    if op == "xent":
        return {"loss": loss, "lse": torch.where(valid, lse[:, 0], 0.0)}
    P = torch.exp(z - lse)
    del z
    P.scatter_add_(1, tgt, torch.full_like(lse, -1.0))
    P *= (torch.where(valid, s["dloss"], 0.0) * scale)[:, None]
    dH, dW = torch.matmul(P, W), torch.matmul(P.t(), H)
    return {"loss": loss, "lse": torch.where(valid, lse[:, 0], 0.0), "dH": dH.to(s["H"].dtype),
            "dW": dW.to(s["W"].dtype)}


def _valid(case):
    """Positions that hold a token, up to where their runs begin."""
    period = min(case["n"], 256)
    return case["n"] * (period - int(case["pad"] * period)) / period


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op == "orthogonalize":
        b, r, s = case["batch"], min(case["m"], case["n"]), max(case["m"], case["n"])
        # of the symmetric products A and A^2 half the entries
        return {"bytes": b * 2 * r * s * es, "flops": b * 5 * (r * r * s + r * r * r + 2 * r * r * s)}
    n, V, d, t = case["n"], case["V"], case["d"], _valid(case)
    if op == "embed":
        return {"bytes": (min(t, V) + n) * d * es + n * 8, "flops": t * d}
    if op == "embed_grad":
        return {"bytes": (t + V) * d * es + n * 8, "flops": 2 * t * d}
    if op == "xent":
        return {"bytes": (t + V) * d * es + n * 16, "flops": 2 * t * V * d}
    return {"bytes": (t + n + 2 * V) * d * es + n * 20, "flops": 6 * t * V * d}


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "embed":
        E = torch.cat([s["E"].double(), torch.zeros_like(s["E"][:1]).double()])  # -1 is the zero row
        return E[s["ids"]] * s["scale"]
    if op == "embed_grad":
        # rows in order of their token, running sums, and their differences at the segments' ends
        order = torch.argsort(s["ids"], stable=True)
        sums = torch.cat([torch.zeros_like(s["dY"][:1]).double(), torch.cumsum(s["dY"].double()[order], 0)])
        ends = torch.searchsorted(s["ids"][order], torch.arange(s["V"] + 1, device=order.device))
        return (sums[ends[1:]] - sums[ends[:-1]]) * s["scale"]
    if op == "orthogonalize":
        # in the Gram matrix alone: every step multiplies X by a polynomial of A from the left
        G = s["G"].double()
        if G.dim() == 2:
            G = G[None]
        if G.shape[1] > G.shape[2]:
            O = _exact_ortho(G.transpose(1, 2).contiguous()).transpose(1, 2).contiguous()
        else:
            O = _exact_ortho(G)
        return O if case["batch"] > 1 else O[0]
    H, W = s["H"].double().requires_grad_(), s["W"].double().requires_grad_()
    z = torch.nn.functional.linear(H, W) * s["scale"]
    lse = torch.logsumexp(z, 1)
    loss = torch.nn.functional.cross_entropy(z, s["target"], ignore_index=-1, reduction="none")
    out = {"loss": loss.detach(), "lse": torch.where(s["target"] >= 0, lse, 0.0).detach()}
    if op == "xent_step":
        out["dH"], out["dW"] = torch.autograd.grad((loss * s["dloss"].double()).sum(), (H, W))
    return out


def _exact_ortho(G):
    nrm = torch.linalg.vector_norm(G, dim=(1, 2), keepdim=True) + EPS
    A = torch.matmul(G, G.transpose(1, 2).contiguous()) / nrm ** 2
    eye = torch.eye(G.shape[1], device=G.device, dtype=G.dtype).expand_as(A)
    Q = eye
    for _ in range(5):
        P = COEFFS[0] * eye + COEFFS[1] * A + COEFFS[2] * torch.matmul(A, A)
        Q, A = torch.matmul(P, Q), torch.matmul(torch.matmul(P, A), P)
    return torch.matmul(Q, G) / nrm
