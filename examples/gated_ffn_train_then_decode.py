"""Train a gated feed-forward block, quantise it to 4 bits, decode with it.

1. Train y = W2 h(x), h = silu(x Wg^T) * (x Wu^T), on a teacher block's outputs: the forward keeps
   its checkpoint of g and u in 8 bits, the backward pass returns the gradients of x and W13.
2. Quantise W13 and W2 to 4-bit codes with a bf16 scale and a zero point per group of K.
3. Decode token by token through the 4-bit block (two launches a token, captured in a CUDA graph).

    python examples/gated_ffn_train_then_decode.py [steps]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import skinny_gemm_dequant_gb300 as ql  # noqa: E402


def quantise(w, group):
    """bf16 [N, K] -> packed codes [N, K/2], bf16 scales and uint8 zero points [N, K/group]."""
    n, k = w.shape
    v = w.float().reshape(n, k // group, group)
    low, high = v.amin(2).clamp(max=0), v.amax(2).clamp(min=0)
    scale = ((high - low) / 15).clamp(min=1e-8).to(torch.bfloat16)
    zero = torch.round(-low / scale.float()).clamp(0, 15)
    q = torch.round(v / scale.float()[..., None] + zero[..., None]).clamp(0, 15).to(torch.uint8).reshape(n, k)
    return q[:, 0::2] | (q[:, 1::2] << 4), scale, zero.to(torch.uint8)


def train(steps=120, tokens=512, hidden=512, inner=1024, lr=0.2, seed=0):
    """Returns (w13, w2, first loss, last loss)."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, gain=1.0):
        return torch.randn(*shape, device="cuda", generator=g) * gain

    t13 = normal(2 * inner, hidden, gain=hidden ** -0.5).bfloat16()
    t2 = normal(hidden, inner, gain=inner ** -0.5).bfloat16()
    m13 = t13.float() + normal(2 * inner, hidden, gain=0.5 * hidden ** -0.5)  # fp32 master weights
    m2 = t2.float() + normal(hidden, inner, gain=0.5 * inner ** -0.5)
    losses = []
    for _ in range(steps):
        x = normal(tokens, hidden).bfloat16()
        target = (ql.gated_ffn(x, t13) @ t2.t()).float()
        w13, w2 = m13.bfloat16(), m2.bfloat16()
        h, saved = ql.gated_ffn(x, w13, save="int8")
        diff = (h @ w2.t()).float() - target
        losses.append(diff.square().mean())
        dy = (diff * (2.0 / tokens)).bfloat16()  # of sum over channels, mean over tokens
        _, dw13 = ql.gated_ffn_backward(dy @ w2, x, w13, saved, need_dx=False)
        m2 -= lr * (dy.t() @ h).float()
        m13 -= lr * dw13.float()
    return m13.bfloat16(), m2.bfloat16(), float(losses[0]), float(losses[-1])


class Decoder:
    """The block on 4-bit weights for one token, bf16 [1, H] -> bf16 [1, H], as a CUDA graph.  The graph
    holds addresses only, so the weights live as long as the decoder."""

    def __init__(self, w13, w2, group=64):
        self.group = group
        self.w13, self.w2 = quantise(w13, group), quantise(w2, group)
        self.x = torch.zeros(1, w13.shape[1], dtype=torch.bfloat16, device="cuda")
        self.block()
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.y = self.block()

    def block(self):
        h = ql.gated_ffn_int4(self.x, *self.w13, group=self.group)
        return ql.qlinear_int4(h, *self.w2, group=self.group)

    def __call__(self, token):
        self.x.copy_(token)
        self.graph.replay()
        return self.y.clone()


def main(steps=120):
    w13, w2, first, last = train(steps)
    print(f"training: mean squared error {first:.4f} -> {last:.4f} in {steps} steps")
    decode = Decoder(w13, w2)
    tokens = torch.randn(16, w13.shape[1], device="cuda").bfloat16()
    got = torch.cat([decode(t[None]) for t in tokens]).float()
    want = (ql.gated_ffn(tokens, w13) @ w2.t()).float()
    off = float((got - want).norm() / want.norm())
    print(f"decode on 4-bit weights: {off:.3f} relative to the bf16 block")
    return first, last, off


if __name__ == "__main__":
    main(*(int(a) for a in sys.argv[1:2]))
