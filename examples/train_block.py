"""One pre-norm transformer block trained on this library alone: layer norms, the four linear layers in NVFP4
(fused QKV projection, attention output, MLP up and down with the squared ReLU between them), attention over packed
documents, and AdamW with 8-bit states, on fp32 master weights.

    python examples/train_block.py [--steps 30] [--tokens 1024] [--hidden 512]

fits the block to a fixed random map and prints the loss."""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import nvfp4_bit_quantized_gb300 as nv  # noqa: E402

HEAD = 64


class Linear:
    """y = x W^T in NVFP4: the recipe's three GEMMs on one 2D-quantized weight a step."""

    def __init__(self, n, k, gen):
        self.weight = torch.randn(n, k, generator=gen, device="cuda") * k ** -0.5

    def quantize(self):
        self.q = nv.quantize_weight(self.weight)

    def forward(self, x, rht_seed):
        row, self.col = nv.quantize_dual(x, nv.RNE, nv.RNE, rht=True, rht_seed=rht_seed)
        return nv.gemm(row, self.q, torch.bfloat16)

    def backward(self, dy, rht_seed, sr_seed, sr_offset):
        row, col = nv.quantize_dual(dy, nv.SR, nv.SR, rht=True, rht_seed=rht_seed, sr_seed=sr_seed, sr_offset=sr_offset)
        return nv.gemm(row, self.q.transposed(), torch.bfloat16), nv.gemm(col, self.col, torch.bfloat16)


class Block:
    def __init__(self, hidden, kv_heads, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.heads, self.kv = hidden // HEAD, kv_heads
        self.qkv = Linear((self.heads + 2 * kv_heads) * HEAD, hidden, gen)
        self.proj = Linear(hidden, hidden, gen)
        self.up, self.down = Linear(4 * hidden, hidden, gen), Linear(hidden, 4 * hidden, gen)
        self.linears = [self.qkv, self.proj, self.up, self.down]
        self.norms = [(torch.ones(hidden, device="cuda"), torch.zeros(hidden, device="cuda")) for _ in range(3)]

    def parameters(self):
        return [x.weight for x in self.linears] + [t for wb in self.norms for t in wb]

    def mlp(self, y, seed):
        """down(relu(up(y))^2): the activation is applied as its quantizer loads the up projection."""
        self.hidden = self.up.forward(y, seed)
        act, self.act_t = nv.quantize_dual(self.hidden, nv.RNE, nv.RNE, rht=True, rht_seed=seed, pre="sqrelu")
        return nv.gemm(act, self.down.q, torch.bfloat16)

    def mlp_backward(self, dz, seed):
        row, col = nv.quantize_dual(dz, nv.SR, nv.SR, rht=True, rht_seed=seed, sr_seed=seed, sr_offset=0)
        dhidden = nv.gemm_sqrelu_backward(row, self.down.q.transposed(), self.hidden)
        ddown = nv.gemm(col, self.act_t, torch.bfloat16)
        dy, dup = self.up.backward(dhidden, seed, seed, 1)
        return dy, dup, ddown

    def step(self, x, target, cu, seed):
        """Loss, and the gradients in the order of :meth:`parameters`."""
        T, H, K = x.shape[0], self.heads, self.kv
        for lin in self.linears:
            lin.quantize()
        (w1, b1), (w2, b2), (w3, b3) = self.norms
        # forward
        y1, m1, r1, _ = nv.layer_norm_forward(x, w1, b1)
        qkv = self.qkv.forward(y1, seed).view(T, H + 2 * K, HEAD)
        q, k, v = qkv[:, :H], qkv[:, H:H + K], qkv[:, H + K:]
        out, lse = nv.attention_forward(q, k, v, causal=True, cu_q=cu)
        o = self.proj.forward(out.view(T, -1), seed)
        y2, m2, r2, h2 = nv.layer_norm_forward(o, w2, b2, residual=x)
        z = self.mlp(y2, seed)
        y3, m3, r3, h3 = nv.layer_norm_forward(z, w3, b3, residual=h2)
        diff = y3.float() - target
        loss = diff.square().mean()
        # backward
        dy3 = (diff * (2 / diff.numel())).bfloat16()
        dz, dw3, db3 = nv.layer_norm_backward(dy3, h3, w3, m3, r3)              # reaches z and h2
        dy2, dwup, ddown = self.mlp_backward(dz, seed)
        do, dw2, db2 = nv.layer_norm_backward(dy2, h2, w2, m2, r2, dh=dz)       # reaches o and x
        dout, dproj = self.proj.backward(do, seed, seed, 2)
        dqkv = torch.empty_like(qkv)
        nv.attention_backward(dout.view(T, H, HEAD), q, k, v, out, lse, causal=True, cu_q=cu, dq=dqkv[:, :H],
                              dk=dqkv[:, H:H + K], dv=dqkv[:, H + K:])
        dy1, dwqkv = self.qkv.backward(dqkv.view(T, -1), seed, seed, 3)
        dx, dw1, db1 = nv.layer_norm_backward(dy1, x, w1, m1, r1, dh=do)        # what a block below would receive
        return loss, [dwqkv, dproj, dwup, ddown, dw1, db1, dw2, db2, dw3, db3], dx


def train(steps=30, tokens=1024, hidden=512, kv_heads=2, bits=8, lr=2e-3):
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(tokens, hidden, generator=gen, device="cuda").bfloat16()
    target = torch.randn(hidden, hidden, generator=gen, device="cuda") * hidden ** -0.5
    target = x.float() @ target
    cu = torch.tensor([0, tokens // 5, tokens // 2, tokens], dtype=torch.int32, device="cuda")   # three documents
    block = Block(hidden, kv_heads)
    params = block.parameters()
    opt = nv.AdamW(params, bits=bits, weight_decay=[0.01 if p.dim() > 1 else 0.0 for p in params])
    losses = []
    for t in range(steps):
        loss, grads, _ = block.step(x, target, cu, seed=t)
        opt.step(grads, lr=lr, betas=(0.9, 0.95), sr_seed=17)
        losses.append(loss)
    assert nv.status_query() == 0
    return [v.item() for v in losses]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--tokens", type=int, default=1024)
    ap.add_argument("--hidden", type=int, default=512)
    ap.add_argument("--bits", type=int, choices=(8, 32), default=8)
    a = ap.parse_args()
    for t, v in enumerate(train(a.steps, a.tokens, a.hidden, bits=a.bits)):
        print(f"step {t:3d}  loss {v:.4f}")
