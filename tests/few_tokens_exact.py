"""Layers for a few tokens whose every step is exact, so that a result can be
compared for equality: a product that is lost, repeated or taken from another
expert, strip or step shows.

x holds -1, 0 and 1, the first value 1; gates are 32 times 1, 1.5, 2, 3, 4 or 6
(their sigmoid is 1 in fp32: exp(-32) < 2^-25), up is a sum of e2m1 values
(multiples of 1/2), the weights of the sum are 1/4, 1/2 or 1 and W2 holds e2m1
values.  An activation then has at most 15 bits, and every term of out is a
multiple of 1: sums below 2^24 are exact in any order."""
from __future__ import annotations

import torch

import fp4_ref
from moe_grouped_gemm_ragged_amd import binding as gg

BF, U8, I32, F32 = torch.bfloat16, torch.uint8, torch.int32, torch.float32


class Layer:
    """Weights on the GPU (bf16 takes any multiple of 8, 4 bits of 32)."""

    def __init__(self, four, experts, hidden, inter, topk, seed=0, dev="cuda"):
        self.four, self.experts, self.hidden, self.inter = four, experts, hidden, inter
        g = torch.Generator(device=dev)
        g.manual_seed(seed)
        k13, k2 = -(-hidden // 32) * 32, -(-inter // 32) * 32

        def codes(*shape):
            return torch.randint(0, 16, shape, generator=g, device=dev, dtype=U8)
        c13 = codes(experts, 2 * inter, k13)
        gate = torch.randint(2, 8, (experts, inter), generator=g, device=dev, dtype=U8)
        c13[:, :inter] = 0
        c13[:, :inter, 0] = gate
        c2 = codes(experts, hidden, k2)
        # (so many of W2's values that a sum stays below 2^24)
        keep = 24000.0 / (topk * inter * max(hidden, 64) ** 0.5)
        if keep < 1:
            c2[torch.rand(c2.shape, generator=g, device=dev) >= keep] = 0
        grid = torch.cat([fp4_ref.GRID, -fp4_ref.GRID]).to(dev).to(BF)
        self.v13, self.v2 = grid[c13.int()], grid[c2.int()]
        self.v13[:, :inter] *= 32
        self.v13, self.v2 = self.v13[..., :hidden].contiguous(), self.v2[..., :inter].contiguous()
        if four:
            self.w13, self.w2 = fp4_ref.pack(c13), fp4_ref.pack(c2)
            raw = torch.full((experts, 2 * inter, hidden // 32), 127, dtype=U8, device=dev)
            raw[:, :inter] += 5
            self.s13 = gg.fp4_pack_scales(gg.GG_FP4_WEIGHT, raw)
            self.s2 = gg.fp4_pack_scales(gg.GG_FP4_WEIGHT, torch.full((experts, hidden, inter // 32), 127, dtype=U8, device=dev))
        else:
            self.w13, self.w2 = self.v13, self.v2

    def __call__(self, x, ids, weights=None, **kw):
        if self.four:
            return gg.fp4_moe_few_tokens(x, ids, self.w13, self.s13, self.w2, self.s2, weights, **kw)
        return gg.moe_few_tokens(x, ids, self.w13, self.w2, weights, **kw)

    def want(self, x, ids, weights=None):
        """The formula in 64 bits."""
        xd, ids = x.double(), ids.long()
        weights = torch.ones(ids.shape, device=x.device) if weights is None else weights
        out = torch.zeros(x.shape[0], self.hidden, dtype=torch.float64, device=x.device)
        size = torch.zeros_like(out)
        for e in sorted(set(ids.reshape(-1).tolist())):
            if not 0 <= e < self.experts:
                continue
            rows = (ids == e).any(-1).nonzero()[:, 0]
            share = (weights.double()[rows] * (ids[rows] == e)).sum(-1, keepdim=True)
            gate, up = (xd[rows] @ self.v13[e].double().t()).chunk(2, -1)
            v2 = self.v2[e].double().t()
            out[rows] += (share * gate * up) @ v2
            size[rows] += (share * gate * up).abs() @ v2.abs()
        assert float(size.max()) < 2.0 ** 24, "the sums would round"
        return out


def inputs(seed, tokens, hidden, ids, dev="cuda"):
    """x, the ids on the device and weights of the sum."""
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    x = torch.randint(-1, 2, (tokens, hidden), generator=g, device=dev).to(BF)
    x[:, 0] = 1
    weights = torch.exp2(-torch.randint(0, 3, ids.shape, generator=g, device=dev).float())
    return x, ids.to(dev).to(I32).contiguous(), weights


def some_experts(seed, tokens, topk, experts, drop=0.0):
    g = torch.Generator().manual_seed(seed)
    ids = torch.rand(tokens, experts, generator=g).topk(topk, dim=1).indices
    return torch.where(torch.rand(ids.shape, generator=g) < drop, -1, ids)
