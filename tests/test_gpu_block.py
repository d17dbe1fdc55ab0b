"""The example's transformer block: with linear layers computed in float32, its gradients against autograd of the same block
(the norms, the attention and the joints between them are then all that differs); and training in NVFP4 that lowers the loss,
with states in 8 and in 32 bits."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def ex():
    import __graft_entry__
    __graft_entry__.build()
    import train_block
    train_block.nv.reset_status()
    return train_block


def dense_block(block, x, target, cu):
    """Loss of the block with exact linear layers, for autograd."""
    F, H, K, D = torch.nn.functional, block.heads, block.kv, 64
    T, C = x.shape
    (w1, b1), (w2, b2), (w3, b3) = block.norms
    qkv = (F.layer_norm(x, (C,), w1, b1) @ block.qkv.weight.T).view(T, H + 2 * K, D)
    q, k, v = qkv[:, :H].transpose(0, 1), qkv[:, H:H + K].transpose(0, 1), qkv[:, H + K:].transpose(0, 1)
    k, v = k.repeat_interleave(H // K, 0), v.repeat_interleave(H // K, 0)
    pos = torch.arange(T, device="cuda")
    doc = torch.searchsorted(cu[1:].long(), pos, right=True)
    seen = (doc[:, None] == doc[None]) & (pos[None] <= pos[:, None])
    p = torch.softmax((q @ k.transpose(1, 2) * D ** -0.5).masked_fill(~seen, float("-inf")), -1)
    o = (p @ v).transpose(0, 1).reshape(T, C) @ block.proj.weight.T
    h2 = o + x
    a = torch.relu(F.layer_norm(h2, (C,), w2, b2) @ block.up.weight.T).square()
    return (F.layer_norm(a @ block.down.weight.T + h2, (C,), w3, b3) - target).square().mean()


def float32_block(ex, hidden, kv_heads):
    """The example's block with its linear layers and MLP in float32 products of the bf16 activations."""
    class Exact(ex.Linear):
        def quantize(self):
            pass

        def forward(self, x, seed):
            self.x = x
            return (x.float() @ self.weight.T).bfloat16()

        def backward(self, dy, *seeds):
            return (dy.float() @ self.weight).bfloat16(), dy.float().T @ self.x.float()

    class Block(ex.Block):
        def mlp(self, y, seed):
            self.hidden = self.up.forward(y, seed)
            return self.down.forward(torch.relu(self.hidden.float()).square().bfloat16(), seed)

        def mlp_backward(self, dz, seed):
            da, ddown = self.down.backward(dz)
            dy, dup = self.up.backward((da.float() * 2 * torch.relu(self.hidden.float())).bfloat16())
            return dy, dup, ddown

    block = Block(hidden, kv_heads)
    for lin in block.linears:
        lin.__class__ = Exact
    return block


def test_gradients_of_the_block_are_autograds(ex):
    """Every tensor that passes from one operator to the next is rounded to bf16 (2^-8 at most, 2^-9 in the mean); a gradient has
    some 20 such roundings behind it, independent: about sqrt(20) 2^-9 = 0.9 % of its norm, and less than 20 2^-8 = 8 % at the
    very most.  A wrong sign, mask or residual branch changes it by more."""
    torch.manual_seed(0)
    x = torch.randn(512, 256, device="cuda").bfloat16()
    target = torch.randn(512, 256, device="cuda")
    cu = torch.tensor([0, 100, 300, 512], dtype=torch.int32, device="cuda")
    block = float32_block(ex, 256, 2)
    loss, grads, dx = block.step(x, target, cu, seed=5)
    params = block.parameters()
    xf = x.float().requires_grad_()
    for p in params:
        p.requires_grad_()
    want = dense_block(block, xf, target, cu)
    exact = torch.autograd.grad(want, params + [xf])
    assert abs(loss.item() / want.item() - 1) < 0.08
    for i, (g, e) in enumerate(zip(grads + [dx], exact)):
        off = ((g.float() - e).norm() / e.norm()).item()
        assert off < 0.08, (i, off)


@pytest.mark.parametrize("bits", [8, 32])
def test_training_lowers_the_loss(ex, bits):
    losses = ex.train(steps=25, tokens=512, hidden=256, bits=bits)
    assert all(v == v for v in losses)
    assert losses[-1] < 0.7 * losses[0], losses
