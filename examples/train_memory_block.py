"""Trains one residual block around the memory scan, then decodes with it.

    n = LN(x);  r | g | k | v = n W_in;  u = gated recurrence of r with retention sigmoid(g + 3)
    q, k l2-normalised per head;  z = Titans memory scan from a learned W0
    y = x + LN_head(z) W_o

The task is associative recall: every token carries a key and a value, every fourth asks for the
value that came with an earlier key.  Matrices (W_in, W_o and every head's W0) are updated by the
orthogonalised momentum, vectors by plain momentum.  Decoding continues a prefix token by token
from the recurrence's and the memory's state and is compared with the full pass.

    python examples/train_memory_block.py [steps]
"""
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import test_neural_memory_gb300 as ttm  # noqa: E402

B, T, H, d, CHUNK = 4, 256, 4, 64, 64
D = H * d
BF16 = torch.bfloat16


class LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, b):
        y, mean, rstd = ttm.layer_norm_fwd(x, w, b)
        ctx.save_for_backward(x, mean, rstd, w)
        return y

    @staticmethod
    def backward(ctx, dy):
        x, mean, rstd, w = ctx.saved_tensors
        g = ttm.layer_norm_bwd(dy.contiguous(), x, mean, rstd, w)
        return g["dx"], g["dw"], g["db"]


class Recurrence(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, g):
        h, last = ttm.glr_fwd(x, g)
        ctx.save_for_backward(g, h)
        return h, last

    @staticmethod
    def backward(ctx, dh, dlast):
        g, h = ctx.saved_tensors
        out = ttm.glr_bwd(g, h, dh.contiguous(), dh_last=dlast.contiguous(), want_dh0=False)
        return out["dx"], out["dg"]


class Memory(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, theta, eta, alpha, W0):
        z, W, S = ttm.titans_fwd(q, k, v, theta, W0, CHUNK, eta=eta, alpha=alpha, w0_shared=True)
        ctx.save_for_backward(q, k, v, theta, eta, alpha, W0)
        ctx.mark_non_differentiable(W, S)
        return z, W, S

    @staticmethod
    def backward(ctx, dz, _dW, _dS):
        q, k, v, theta, eta, alpha, W0 = ctx.saved_tensors
        g = ttm.titans_bwd(q, k, v, theta, W0, CHUNK, dz.contiguous(), eta=eta, alpha=alpha, w0_shared=True,
                           want_gates=False, want_dS0=False)
        return g["dq"], g["dk"], g["dv"], None, None, None, g["dW0"]


def parameters(gen):
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    p = dict(W_in=rand(D, 4 * D) / D ** 0.5, W_o=rand(D, D) / D ** 0.5, W0=0.02 * rand(1, H, d, d),
             w1=torch.ones(D, device="cuda"), b1=torch.zeros(D, device="cuda"),
             w2=torch.ones(d, device="cuda"), b2=torch.zeros(d, device="cuda"))
    return {k: v.requires_grad_() for k, v in p.items()}


def gates(n):
    """The memory's step, momentum and forgetting, constant here."""
    full = lambda v: torch.full((B, H, n), v, device="cuda")  # noqa: E731
    return full(0.05), full(0.6), full(0.005)


def heads(t):
    return t.unflatten(-1, (H, d)).transpose(1, 2).contiguous()


def project(p, x):
    """r, g (columns of one projection), k, v of the normed input."""
    proj = LayerNorm.apply(x, p["w1"], p["b1"]) @ p["W_in"].to(BF16)
    r, g, k, v = proj.split(D, dim=-1)
    return r, F.logsigmoid(g + 3), k, v


def unit(t):
    return F.normalize(t.float(), dim=-1).to(BF16)


def read_out(p, x, z):
    z = LayerNorm.apply(z, p["w2"], p["b2"])
    return x + z.transpose(1, 2).reshape(x.shape) @ p["W_o"].to(BF16)


def block(p, x):
    """y and the states (recurrence, memory, momentum) after the last token."""
    r, g, k, v = project(p, x)
    u, last = Recurrence.apply(r, g)
    theta, eta, alpha = gates(x.shape[1])
    z, W, S = Memory.apply(unit(heads(u)), unit(heads(k)), heads(v), theta, eta, alpha, p["W0"])
    return read_out(p, x, z), (last, W, S)


def batch(gen, keys, values):
    """Tokens of a key and its value, every fourth one of an earlier key alone; the targets."""
    pick = torch.randint(0, len(keys), (B, T), generator=gen, device="cuda")
    ask = torch.arange(T, device="cuda") % 4 == 3
    pick[:, ask] = pick[:, torch.nonzero(ask)[:, 0] - 2]
    x = keys[pick] + torch.where(ask[None, :, None], 0.0, values[pick])
    return x.to(BF16), values[pick], ask


def train(steps, lr=0.02, momentum=0.9, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    keys = torch.randn((64, D), generator=gen, device="cuda")
    values = torch.randn((64, D), generator=gen, device="cuda")
    p = parameters(gen)
    buf = {k: torch.zeros_like(v) for k, v in p.items()}
    losses = []
    for _ in range(steps):
        x, target, ask = batch(gen, keys, values)
        y, _ = block(p, x)
        loss = F.mse_loss(y[:, ask].float(), target[:, ask])
        grads = torch.autograd.grad(loss, list(p.values()))
        with torch.no_grad():
            for (name, w), g in zip(p.items(), grads):
                m = buf[name].mul_(momentum).add_(g)
                if w.dim() > 1:     # one singular value of the update is about one: scale by the shape
                    rows, cols = w.shape[-2:]
                    w.sub_(ttm.orthogonalize(m.contiguous()), alpha=lr * max(1, rows / cols) ** 0.5)
                else:
                    w.sub_(m, alpha=lr)
        losses.append(loss.detach())
    return p, [float(v) for v in losses], (gen, keys, values)


@torch.no_grad()
def decode(p, x, start):
    """Continues the prefix x[:, :start] (whole chunks) by the tokens after it, one at a time."""
    _, (state, W, S) = block(p, x[:, :start].contiguous())
    Wc, pos, out = None, 0, []
    for t in range(start, x.shape[1]):
        now = x[:, t:t + 1].contiguous()
        r, g, k, v = project(p, now)
        u = ttm.glr_step(r, g, state)
        theta, eta, alpha = gates(1)
        z, Wc, pos = ttm.titans_step(unit(heads(u)), unit(heads(k)), heads(v), theta, W, CHUNK, pos, eta=eta,
                                     alpha=alpha, S=S, Wc=Wc)
        out.append(read_out(p, now, z))
    return torch.cat(out, 1)


def main(steps=60):
    p, losses, (gen, keys, values) = train(steps)
    x, _, _ = batch(gen, keys, values)
    with torch.no_grad():
        full, _ = block(p, x)
    tail = decode(p, x, T - CHUNK)
    off = float((tail.float() - full[:, T - CHUNK:].float()).norm() / full[:, T - CHUNK:].float().norm())
    assert ttm.device_status() == ttm.OK
    return losses, off


if __name__ == "__main__":
    losses, off = main(int(sys.argv[1]) if len(sys.argv) > 1 else 60)
    print(f"loss {losses[0]:.3f} -> {losses[-1]:.3f} in {len(losses)} steps; "
          f"decoding differs from the full pass by {off:.1e}")
