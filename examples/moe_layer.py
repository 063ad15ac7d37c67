"""A feed-forward layer of routed NVFP4 experts beside a dense NVFP4 projection.

Makes the weights' 4-bit form once, from 32-bit values, as a loader would; then, for
a batch of tokens, routes them, runs the experts and the projection, and compares the
result with the same layer in fp32 on the dequantised weights.

    python examples/moe_layer.py [tokens]
"""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import nvfp4_block_scaled_gemv_gb300 as nv  # noqa: E402


class Layer:
    """Router, experts (gate and input rows interleaved) and a dense projection."""

    def __init__(self, experts=16, top_k=4, hidden=512, inner=256, seed=0, device="cuda:0"):
        g = torch.Generator(device=device).manual_seed(seed)

        def weights(*shape):
            return torch.randn(shape, device=device, generator=g) / shape[-1] ** 0.5

        self.top_k = top_k
        self.router = weights(experts, hidden)
        self.balance = 0.02 * torch.randn(experts, device=device, generator=g)
        # the values are brought near the middle of the scales' range, and back by alpha
        self.encode_w, self.encode_x, self.encode_h = 64.0, 1.0, 4.0
        gate, up = weights(experts, inner, hidden), weights(experts, inner, hidden)
        self.w1, self.s1 = nv.quantize(torch.stack((gate, up), dim=2).flatten(1, 2), self.encode_w)
        self.w2, self.s2 = nv.quantize(weights(experts, hidden, inner), self.encode_w)
        self.wd, self.sd = nv.quantize(weights(1, hidden, hidden), self.encode_w)
        self.alpha1 = torch.full((experts,), 1 / (self.encode_w * self.encode_x), device=device)
        self.alpha2 = torch.full((experts,), 1 / (self.encode_w * self.encode_h), device=device)

    def __call__(self, x):
        """x [T, hidden] bf16 -> [T, hidden] bf16."""
        ids, weights = nv.route(x.float() @ self.router.T, self.top_k, score=nv.SCORE_SIGMOID, bias=self.balance)
        routed = nv.moe_ffn(x, ids, weights, self.w1, self.s1, self.w2, self.s2, alpha1=self.alpha1,
                            alpha2=self.alpha2, encode_x=self.encode_x, encode_h=self.encode_h)
        q, s = nv.quantize(x, self.encode_x)
        dense = nv.gemm(self.wd, q.unsqueeze(0), self.sd, s, alpha=1 / (self.encode_w * self.encode_x),
                        dtype=x.dtype)
        return routed + dense[0]

    def reference(self, x):
        """The same layer in fp32: dequantised weights, no 4-bit activations."""
        w1, w2, wd = (nv.dequantize(q, s, scale=1 / self.encode_w)
                      for q, s in ((self.w1, self.s1), (self.w2, self.s2), (self.wd, self.sd)))
        x = x.float()
        score = torch.sigmoid(x @ self.router.T)
        ids = (score + self.balance).topk(self.top_k, dim=1).indices
        weights = score.gather(1, ids)
        weights = weights / weights.sum(1, keepdim=True)
        out = x @ wd[0].T
        for e in range(self.router.shape[0]):
            t, j = (ids == e).nonzero(as_tuple=True)
            u = x[t] @ w1[e].T
            h = torch.nn.functional.silu(u[:, 0::2]) * u[:, 1::2]
            out.index_add_(0, t, weights[t, j].unsqueeze(1) * (h @ w2[e].T))
        return out


def main(tokens=64):
    layer = Layer()
    x = torch.randn(tokens, 512, device="cuda:0").bfloat16()
    got, want = layer(x).float(), layer.reference(x)
    error = ((got - want).norm() / want.norm()).item()
    print(f"{tokens} tokens: relative difference from 32-bit activations {error:.3f}")
    return error


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 64)
