"""Fine-tunes one transformer block over frozen 4-bit projections: the norms around its two halves, causal
attention over packed samples, low-rank adapters on the projections, and an 8-bit AdamW step.

    python examples/train_block.py [--steps 40] [--tokens 2048] [--hidden 1024]

Everything but the rotary embedding and the activation of the feed-forward half runs in the library's
kernels.  The block learns to reproduce the output of a second block whose adapters are set at random."""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_nf4_quantized_linear_gb300 as nf4  # noqa: E402


class Adapted(torch.nn.Module):
    """Frozen 4-bit weights that share an input, each with a rank-r adapter."""

    def __init__(self, hidden, outs, rank, g):
        super().__init__()
        self.ws = [nf4.quantize(torch.randn(n, hidden, generator=g, device="cuda") * 0.02) for n in outs]
        self.down = torch.nn.ParameterList(torch.randn(rank, hidden, generator=g, device="cuda").bfloat16() * hidden ** -0.5
                                           for _ in outs)
        self.up = torch.nn.ParameterList(torch.zeros(n, rank, device="cuda", dtype=torch.bfloat16) for n in outs)

    def forward(self, x):
        frozen = nf4.nf4_linear_multi(x, self.ws) if len(self.ws) > 1 else (nf4.nf4_linear(x, self.ws[0]),)
        return [y + (x @ a.T) @ b.T for y, a, b in zip(frozen, self.down, self.up)]


def rotary(x, pos):
    """Position rotation of [T, heads, D]; pos [T] counts from each sample's start."""
    half = x.shape[-1] // 2
    freq = 10000.0 ** (-torch.arange(half, device=x.device, dtype=torch.float32) / half)
    ang = pos[:, None, None] * freq
    a, b = x.float().split(half, -1)
    return torch.cat([a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()], -1).to(x.dtype)


class Block(torch.nn.Module):
    def __init__(self, hidden, heads, kv_heads, rank, seed):
        super().__init__()
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.heads, self.kv, self.dim = heads, kv_heads, hidden // heads
        self.qkv = Adapted(hidden, [hidden, kv_heads * self.dim, kv_heads * self.dim], rank, g)
        self.o = Adapted(hidden, [hidden], rank, g)
        self.gate_up = Adapted(hidden, [4 * hidden, 4 * hidden], rank, g)
        self.down = Adapted(4 * hidden, [hidden], rank, g)
        self.gains = torch.nn.ParameterList(torch.ones(hidden, device="cuda") for _ in range(4))
        self.branch = torch.nn.ParameterList(torch.full((hidden,), 0.5, device="cuda") for _ in range(2))

    def forward(self, x, cu, pos):
        before, after_attn, between, after_mlp = self.gains
        x, h = nf4.nf4_norm_residual(x, w_pre=before)
        q, k, v = (t.view(t.shape[0], -1, self.dim) for t in self.qkv(h))
        a = nf4.nf4_attention(rotary(q, pos), rotary(k, pos), v, cu)
        x, h = nf4.nf4_norm_residual(self.o(a.flatten(1))[0], x, w_post=after_attn, gate=self.branch[0], w_pre=between)
        gate, up = self.gate_up(h)
        y = self.down(torch.nn.functional.silu(gate) * up)[0]
        return nf4.nf4_norm_residual(y, x, w_post=after_mlp, gate=self.branch[1])[0]


def train(steps=40, tokens=2048, hidden=1024, rank=16, seed=0, lr=1e-3):
    """Runs the steps and returns the losses."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    args = (hidden, hidden // 64, max(1, hidden // 256), rank, seed)
    block, target = Block(*args), Block(*args)
    with torch.no_grad():
        for name, p in target.named_parameters():
            if ".up." in name:
                p.copy_(0.02 * torch.randn(p.shape, generator=g, device="cuda"))
    opt = nf4.NF4AdamW(block.parameters(), lr=lr, weight_decay=0.0, state_bits=8)
    # packed samples of uneven length, the last tenth of the rows padding
    cuts = [0, tokens // 8, tokens // 2, tokens - tokens // 10]
    cu = torch.tensor(cuts, dtype=torch.int32, device="cuda")
    pos = torch.cat([torch.arange(b - a) for a, b in zip(cuts, cuts[1:] + [tokens])]).to("cuda")
    losses = []
    for _ in range(steps):
        x = torch.randn(tokens, hidden, generator=g, device="cuda").bfloat16()
        with torch.no_grad():
            want = target(x, cu, pos)
        loss = (block(x, cu, pos) - want)[:cuts[-1]].float().square().mean()
        loss.backward()
        norm = torch.nn.utils.get_total_norm([p.grad for p in block.parameters()])
        opt.step(grad_scale=(1.0 / norm.clamp(min=1.0)).float().reshape(1))
        opt.zero_grad(set_to_none=True)
        losses.append(loss.item())
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=40)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--hidden", type=int, default=1024)
    a = ap.parse_args()
    for i, loss in enumerate(train(a.steps, a.tokens, a.hidden)):
        print(f"step {i:3d}  loss {loss:.5f}")
