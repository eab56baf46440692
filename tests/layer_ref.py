"""Plain fp64 forms of the layer steps around the grouped GEMM (norm, 8-bit
rows, combine gradient, SiLU-mul and their gradients, dW from 8-bit rows) and
the error each may show, for the tests.

Every bound is the sum of two parts: half a step of the output's type
(relative 2^-8 for bf16, 2^-24 for fp32; for e4m3 2^-4, or 2^-10 of the scale
below its smallest normal value), and the fp32 arithmetic before it, whose
roundings are at most 2^-24 each: a sum of L terms is off by at most
L 2^-24 sum |terms| in whatever order."""
from __future__ import annotations

import torch

U32 = 2.0 ** -24
TINY = 2.0 ** -126
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
F8 = torch.float8_e4m3fn


def f64(t):
    return None if t is None else t.detach().cpu().double()


def close(got, ref, bound, what):
    """|got - ref| <= bound element by element (and both NaN in the same places)."""
    got = f64(got)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{what}: NaN in other places"
    bad = ((got - ref).abs() > bound) & ~torch.isnan(ref)
    if bool(bad.any()):
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} out of bounds; first at {i}: got "
                             f"{got[i].item()!r} want {ref[i].item()!r} within {torch.as_tensor(bound).expand_as(ref)[i].item()!r}")


def quantise(v):
    """e4m3 codes (uint8) and E8M0 bytes of v [..., n] by the stated rule, in 64 bits."""
    b = v.double().reshape(*v.shape[:-1], -1, 128)
    ok = torch.isfinite(b)
    amax = torch.where(ok, b.abs(), 0.0).amax(-1)
    frac, e = torch.frexp(amax)                      # amax = frac 2^e, 448 = 0.875 2^9
    e = torch.where(amax == 0, torch.zeros_like(e), (e - 9 + (frac > 0.875).int()).clamp(min=-126))
    scaled = torch.where(ok, b / torch.pow(2.0, e.double())[..., None], 0.0)
    # in [-448, 448] at most 11 bits left of the fp32 rounding: v is bf16 or fp32, so the cast sees v / s itself
    codes = scaled.float().to(F8).view(torch.uint8)
    codes = torch.where(ok, codes, torch.full_like(codes, 0x7F))
    return codes.reshape(v.shape), (e + 127).to(torch.uint8)


def value(codes, scales):
    """Values of e4m3 codes [..., n] with E8M0 bytes [..., n / 128]."""
    s = torch.pow(2.0, scales.cpu().double() - 127)
    c = codes.cpu().view(F8).double()
    return (c.reshape(*scales.shape, 128) * s[..., None]).reshape(codes.shape)


def close8(codes, scales, ref, slack, what):
    """e4m3 rows of values known to within ``slack``: the scale fits the
    block's largest value, and every code is the value's nearest."""
    s = torch.pow(2.0, scales.cpu().double() - 127)
    blocks, room = ref.reshape(*scales.shape, 128).abs(), slack.expand_as(ref).reshape(*scales.shape, 128)
    top, least = (blocks + room).amax(-1), (blocks - room).amax(-1)
    live = blocks.amax(-1) > 0
    floor = 2.0 ** -126
    assert bool(((least <= 448 * s) | ~live).all()), f"{what}: a scale is too small"
    # (values within their slack of 0 may all have come out as 0, and then the scale is 1)
    zero = (least <= 0) & (s == 1)
    assert bool(((top > 224 * s) | (s == floor) | zero | ~live).all()), f"{what}: a scale is too large"
    assert bool((s[~live] == 1).all()), f"{what}: the scale of a block of zeros is not 1"
    wide = s[..., None].expand_as(blocks).reshape(ref.shape)
    close(value(codes, scales), ref, torch.maximum(2.0 ** -4 * (ref.abs() + slack), 2.0 ** -10 * wide) + slack, what)


def rmsnorm(x, residual, gamma, eps):
    h = f64(x) + (0 if residual is None else f64(residual))
    return h / torch.sqrt(h.square().mean(-1, keepdim=True) + eps) * f64(gamma), h


def rmsnorm_slack(y, n):
    # the mean of n squares: (n + 2) 2^-24 relative, half of it after the root; h, the root, the
    # reciprocal and two products
    return y.abs() * (n / 2 + 12) * U32


def rmsnorm_grad(dy, h, gamma, dh, eps):
    """dx, dgamma and their fp32 bounds."""
    d, h = f64(dy), f64(h)
    rows, n = h.shape
    rho = 1 / torch.sqrt(h.square().mean(-1, keepdim=True) + eps)
    u, p = h * rho, d * f64(gamma)
    m = (p * u).mean(-1, keepdim=True)
    extra = 0 if dh is None else f64(dh)
    dx = rho * (p - u * m) + extra
    # m: n products of four roundings each, summed; rho as in the norm
    size = rho * (p.abs() + u.abs() * (p * u).abs().mean(-1, keepdim=True)) + abs(extra)
    slack = size * (2 * n + 24) * U32
    dgamma = (d * u).sum(0)
    return dx, slack, dgamma, (d * u).abs().sum(0) * (rows + n / 2 + 16) * U32


def silu_mul(h):
    i = h.shape[-1] // 2
    g, u = h[..., :i], h[..., i:]
    a = g * torch.sigmoid(g) * u
    # exp(-g) through exp2: |g| log2(e) 2^-24 relative and two roundings; four more to a.  A sigmoid
    # below 2^-126 (fp32's smallest normal value: exp(-g) or its reciprocal leaves fp32) comes out
    # as 0, off by at most 2^-126, which g u multiplies.
    return a, a.abs() * (2 * g.abs() + 16) * U32 + TINY * (1 + (g * u).abs())


def silu_mul_grad(da, h):
    i = h.shape[-1] // 2
    g, u, d = h[..., :i], h[..., i:], da
    s = torch.sigmoid(g)
    ref = torch.cat([d * u * s * (1 + g * (1 - s)), d * g * s], -1)
    part = (2 * g.abs() + 16) * U32
    # 1 - s is off by s's own error, times g; the sum it enters is at least that large beside 1
    slack = torch.cat([(d * u * s).abs() * (1 + g.abs()) * 2 * part, (d * g * s).abs() * part], -1)
    # the same 2^-126, times what multiplies the sigmoid in each half
    return ref, slack + TINY * (1 + torch.cat([d * u * (1 + g.abs()), d * g], -1).abs())


def packed_scales(scales, ends, cap, fill=0):
    """E8M0 bytes [rows, G] of grouped rows in the packed layout, tile by
    tile; ``fill`` where no tile lies."""
    kb, tiles = scales.shape[1], -(-cap // 256) + len(ends)
    out = torch.full((tiles, kb, 256), fill, dtype=torch.uint8)
    t = first = 0
    for end in ends:
        for r0 in range(first, end, 256):
            block = scales[r0:min(end, r0 + 256)]
            out[t] = 0
            for r in range(block.shape[0]):
                out[t, :, 128 * (r // 128) + 4 * (r % 32) + (r // 32) % 4] = block[r]
            t += 1
        first = max(first, end)
    return out.reshape(-1)
