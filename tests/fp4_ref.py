"""Plain fp64 forms of the 4-bit operators (rows to 4 bits and back, packed
scales, the grouped product) and the error each may show, for the tests.

Codes and scales of bf16 rows are exact: dividing by a power of two and
comparing with the borders between neighbouring e2m1 values rounds nothing, so
they are compared for equality.  A SiLU-mul row is known up to its fp32
arithmetic (layer_ref.silu_mul's slack); its codes are held to the nearest value
within that.  The product's operands are exact, and its bound is the
accumulation model of the scaled matrix instructions (parity.fp8_model_bound)
plus half a step of the output's type."""
from __future__ import annotations

import torch

from layer_ref import close, f64
from parity import fp8_model_bound

GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}     # half a step, relative to the value


def quantise(v):
    """Codes (one a value, uint8) and scale bytes of v [..., k], in 64 bits."""
    b = v.detach().cpu().double().reshape(*v.shape[:-1], -1, 32)
    bad = ~torch.isfinite(b).all(-1)
    amax = torch.where(torch.isfinite(b), b.abs(), 0.0).amax(-1)
    frac, e = torch.frexp(amax)                       # 6 = 0.75 * 2^3
    e = torch.where(amax == 0, torch.zeros_like(e), (e - 3 + (frac > 0.75).int()).clamp(min=-126))
    m = torch.where(bad[..., None], 0.0, b / torch.pow(2.0, e.double())[..., None])
    # the nearest of the grid; between two at the same distance the even code
    d = (m.abs()[..., None] - GRID).abs()
    best = d.amin(-1, keepdim=True)
    tied = d == best
    even = torch.tensor([i % 2 == 0 for i in range(8)])
    pick = torch.where((tied & even).any(-1, keepdim=True), tied & even, tied)
    code = pick.int().argmax(-1) + 8 * torch.signbit(m).int()
    code = torch.where(bad[..., None], 0, code)
    byte = torch.where(bad, 255, e + 127)
    return code.to(torch.uint8).reshape(v.shape), byte.to(torch.uint8)


def pack(codes):
    """Two codes a byte, the first in the low half."""
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def unpack(b):
    return torch.stack([b & 15, b >> 4], -1).flatten(-2)


def value(packed, scales):
    """Values of code bytes [..., k / 2] with scale bytes [..., k / 32]."""
    c = unpack(packed.cpu()).long()
    v = torch.where(c >= 8, -GRID[c & 7], GRID[c & 7])
    s = torch.where(scales.cpu() == 255, float("nan"), torch.pow(2.0, scales.cpu().double() - 127))
    return (v.reshape(*scales.shape, 32) * s[..., None]).reshape(*packed.shape[:-1], -1)


def tiles(layout, groups, rows, experts):
    """(first flattened row, rows in it) of every packed tile that has rows, by tile."""
    out, t = {}, 0
    if layout == 0:
        first = 0
        for end in groups:
            end = min(max(end, first), rows)
            for r0 in range(first, end, 256):
                out[t] = (r0, min(end, r0 + 256) - r0)
                t += 1
            first = end
        return out
    per = -(-rows // 256)
    for e in range(experts):
        active = rows if layout == 2 else min(max(groups[e], 0), rows)
        for c in range(per):
            n = min(active - 256 * c, 256)
            if n > 0:
                out[e * per + c] = (e * rows + 256 * c, n)
    return out


def packed_scales(scales, layout, groups, rows, experts, fill):
    """Scale bytes [all rows, k / 32] in the packed layout; ``fill`` in the
    tiles without rows."""
    blocks = scales.shape[-1]
    scales = scales.reshape(-1, blocks)
    stages = -(-blocks // 4)
    n = -(-rows // 256) + experts if layout == 0 else -(-rows // 256) * experts
    out = torch.full((n, stages, 1024), fill, dtype=torch.uint8)
    r = torch.arange(256)
    for t, (first, count) in tiles(layout, groups, rows, experts).items():
        out[t] = 0
        for b in range(blocks):
            q = b % 4
            at = 512 * (r // 128) + 16 * (r % 32) + 8 * (q % 2) + 4 * (q // 2) + (r // 32) % 4
            out[t, b // 4, at[:count]] = scales[first:first + count, b]
    return out.reshape(-1)


def owned(layout, groups, rows, experts):
    """Which flattened rows an expert owns, and whose they are."""
    total = rows if layout == 0 else rows * experts
    who = torch.full((total,), -1)
    if layout == 0:
        first = 0
        for g, end in enumerate(groups):
            end = min(max(end, first), rows)
            who[first:end] = g
            first = end
    else:
        for e in range(experts):
            who[e * rows:e * rows + (rows if layout == 2 else min(max(groups[e], 0), rows))] = e
    return who


def check_product(got, x, w, who, what):
    """got [rows, n] (bf16 or fp32) against x [rows, k] . w[who]^T, rows somebody owns."""
    k = x.shape[-1]
    for g in sorted(set(who.tolist()) - {-1}):
        rows = who == g
        ref, size = x[rows] @ w[g].t(), x[rows].abs() @ w[g].abs().t()
        bound = fp8_model_bound(k) * size
        close(got.cpu()[rows], ref, bound + (ref.abs() + bound) * HALF[got.dtype], f"{what}, expert {g}")


def close4(packed, scales, ref, slack, what):
    """4-bit rows of values known to within ``slack``: the scale fits the
    block's largest value, and every code is the value's nearest."""
    s = torch.pow(2.0, scales.cpu().double() - 127)
    b, room = ref.reshape(*scales.shape, 32).abs(), slack.expand_as(ref).reshape(*scales.shape, 32)
    top, least = (b + room).amax(-1), (b - room).amax(-1)
    floor = 2.0 ** -126
    assert bool((least <= 6 * s).all()), f"{what}: a scale is too small"
    zero = (least <= 0) & (s == 1)
    assert bool(((top > 3 * s) | (s == floor) | zero).all()), f"{what}: a scale is too large"
    wide = s[..., None].expand_as(b).reshape(ref.shape)
    bound = torch.maximum(0.25 * (ref.abs() + slack), 0.25 * wide) + slack
    close(value(packed, scales), f64(ref), bound, what)
