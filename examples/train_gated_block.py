"""Trains a language-model-like layer around the memory scan, then decodes with it.

    n = LN(x);  q | k | v = SiLU(short causal convolution of n W_qkv);  q, k l2-normalised per head
    z = Titans memory scan from a learned W0;  s = x + LN_head(z) W_o
    y = s + (SiLU(m W_g) * (m W_u)) W_d,  m = LN(s)

Rows are packed: two documents each, which the convolution keeps apart.  Weights are fp32; the products read bf16
copies, which the optimiser writes with its step.  AdamW takes everything but every head's W0, whose update
is the orthogonalised momentum.  The task is that of train_memory_block.py: recall of the value that
came with a key.  Decoding continues a prefix token by token from the convolution's, the memory's and the momentum's state and is
compared with the full pass.

    python examples/train_gated_block.py [steps]
"""
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import test_neural_memory_gb300 as ttm  # noqa: E402

B, T, H, d, CHUNK, TAPS = 4, 256, 4, 64, 64, 4
D, HIDDEN = H * d, 2 * H * d
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


class CausalConv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, doc):
        y, state = ttm.causal_conv_fwd(x, w, doc=doc)
        ctx.save_for_backward(x, w, doc)
        ctx.mark_non_differentiable(state)
        return y, state

    @staticmethod
    def backward(ctx, dy, _dstate):
        x, w, doc = ctx.saved_tensors
        g = ttm.causal_conv_bwd(dy.contiguous(), x, w, doc=doc)
        return g["dx"], g["dw"], None


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


class GatedFeedForward(torch.autograd.Function):
    """x + block(m), the weights' gradients in bf16, as their copies are."""
    @staticmethod
    def forward(ctx, m, W_in, W_out, x):
        y, gu = ttm.gated_ffn_fwd(m, W_in, W_out, residual=x)
        ctx.save_for_backward(m, gu, W_in, W_out)
        return y

    @staticmethod
    def backward(ctx, dy):
        m, gu, W_in, W_out = ctx.saved_tensors
        dy = dy.contiguous()
        g = ttm.gated_ffn_bwd(dy, m, gu, W_in, W_out)
        return g["dx"], g["dW_in"], g["dW_out"], dy


MATRICES = ("W_qkv", "W_o", "W_in", "W_down")     # those with a bf16 copy


def parameters(gen):
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    ones, zeros = (lambda n: torch.ones(n, device="cuda")), (lambda n: torch.zeros(n, device="cuda"))
    return dict(W_qkv=rand(D, 3 * D) / D ** 0.5, W_o=rand(D, D) / D ** 0.5, W_in=rand(D, 2 * HIDDEN) / D ** 0.5,
                W_down=rand(HIDDEN, D) / HIDDEN ** 0.5, taps=rand(3 * D, TAPS) / TAPS ** 0.5, W0=0.02 * rand(1, H, d, d),
                w1=ones(D), b1=zeros(D), w2=ones(d), b2=zeros(d), w3=ones(D), b3=zeros(D))


def leaves(p):
    """What a pass differentiates: the bf16 copies of the matrices, the other parameters themselves."""
    return {k: (v.to(BF16) if k in MATRICES else v).detach().requires_grad_() for k, v in p.items()}


def gates(n):
    """The memory's step, momentum and forgetting, constant here."""
    full = lambda v: torch.full((B, H, n), v, device="cuda")  # noqa: E731
    return full(0.05), full(0.6), full(0.005)


def heads(t):
    return t.unflatten(-1, (H, d)).transpose(1, 2).contiguous()


def unit(t):
    return F.normalize(t.float(), dim=-1).to(BF16)


def qkv(c):
    q, k, v = c.split(D, dim=-1)
    return unit(heads(q)), unit(heads(k)), heads(v)


def read_out(p, x, z):
    z = LayerNorm.apply(z, p["w2"], p["b2"])
    s = x + z.transpose(1, 2).reshape(x.shape) @ p["W_o"]
    return GatedFeedForward.apply(LayerNorm.apply(s, p["w3"], p["b3"]), p["W_in"], p["W_down"], s)


def block(p, x, doc=None):
    """y and the states (convolution, memory, momentum) after the last token."""
    proj = LayerNorm.apply(x, p["w1"], p["b1"]) @ p["W_qkv"]
    c, last = CausalConv.apply(proj, p["taps"], doc)
    q, k, v = qkv(c)
    theta, eta, alpha = gates(x.shape[1])
    z, W, S = Memory.apply(q, k, v, theta, eta, alpha, p["W0"])
    return read_out(p, x, z), (last, W, S)


def batch(gen, keys, values):
    """Tokens of a key and its value, every fourth one of an earlier key alone; the targets; a border in each row."""
    pick = torch.randint(0, len(keys), (B, T), generator=gen, device="cuda")
    ask = torch.arange(T, device="cuda") % 4 == 3
    pick[:, ask] = pick[:, torch.nonzero(ask)[:, 0] - 2]
    x = keys[pick] + torch.where(ask[None, :, None], 0.0, values[pick])
    border = torch.randint(1, T, (B, 1), generator=gen, device="cuda")
    doc = (torch.arange(T, device="cuda") >= border).to(torch.int32)
    return x.to(BF16), values[pick], ask, doc


def train(steps, lr=3e-3, momentum=0.9, bits=8, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    keys = torch.randn((64, D), generator=gen, device="cuda")
    values = torch.randn((64, D), generator=gen, device="cuda")
    p = parameters(gen)
    used = leaves(p)
    names = [k for k in p if k != "W0"]
    state = ttm.adamw_state([p[k] for k in names], bits=bits)
    buf = torch.zeros_like(p["W0"])
    losses = []
    for _ in range(steps):
        x, target, ask, doc = batch(gen, keys, values)
        y, _ = block(used, x, doc)
        loss = F.mse_loss(y[:, ask].float(), target[:, ask])
        grads = dict(zip(used, torch.autograd.grad(loss, list(used.values()))))
        with torch.no_grad():
            # one scale for all gradients, on the device: their norm is clipped at 1
            norm = torch.stack([g.float().norm() for g in grads.values()]).norm()
            ttm.adamw_step([p[k] for k in names], [grads[k].contiguous() for k in names], state, lr=lr, weight_decay=0.01,
                           grad_scale=(1 / norm.clamp_min(1.0)).reshape(()),
                           copies=[used[k] if k in MATRICES else None for k in names])
            p["W0"].sub_(ttm.orthogonalize(buf.mul_(momentum).add_(grads["W0"])), alpha=lr)
            for k in names:
                if k not in MATRICES:
                    used[k].copy_(p[k])
            used["W0"].copy_(p["W0"])
        losses.append(loss.detach())
    return used, [float(v) for v in losses], (gen, keys, values)


@torch.no_grad()
def decode(p, x, start):
    """Continues the prefix x[:, :start] (whole chunks) by the tokens after it, one at a time."""
    _, (last, W, S) = block(p, x[:, :start].contiguous())
    Wc, pos, out = None, 0, []
    for t in range(start, x.shape[1]):
        now = x[:, t:t + 1].contiguous()
        proj = LayerNorm.apply(now, p["w1"], p["b1"]) @ p["W_qkv"]
        q, k, v = qkv(ttm.causal_conv_step(proj, p["taps"], last))
        theta, eta, alpha = gates(1)
        z, Wc, pos = ttm.titans_step(q, k, v, theta, W, CHUNK, pos, eta=eta, alpha=alpha, S=S, Wc=Wc)
        out.append(read_out(p, now, z))
    return torch.cat(out, 1)


def main(steps=60):
    p, losses, (gen, keys, values) = train(steps)
    x, _, _, _ = batch(gen, keys, values)
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
