"""The 4-bit product over many tiles a workgroup, and operands past 4 GB.

With one scale for all operands every partial sum is a multiple of 1/4 below
2^16, which fp32 holds, so fp32 results are equal to the 64-bit product and a
bf16 result is its rounding: a load that arrives after its use, or a store that
overtakes another tile's, shows as a wrong value."""
import pytest
import torch

import fp4_ref as ref
from moe_grouped_gemm_ragged_amd import binding as gg
from gpu_util import device, say

pytestmark = pytest.mark.gpu
BF, U8, I32 = torch.bfloat16, torch.uint8, torch.int32
RAGGED, MASKED, WEIGHT = gg.GG_FP4_ACT_RAGGED, gg.GG_FP4_ACT_MASKED, gg.GG_FP4_WEIGHT


def values(codes):
    """fp64 values of code bytes, on their device (scale 1)."""
    grid = torch.cat([ref.GRID, -ref.GRID]).to(codes.device)
    return grid[ref.unpack(codes).long()]


def ones(layout, rows, k, experts, dev):
    return torch.full((gg.fp4_scale_bytes(layout, rows, k, experts),), 127, dtype=U8, device=dev)


def codes(g, dev, *shape):
    return torch.randint(0, 256, shape, generator=g, device=dev, dtype=U8)


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("k", [32, 128, 256, 288, 512, 640, 1024])
def test_many_tiles_a_workgroup(k, dtype):
    """More than three tiles for each compute unit: full and half heights,
    empty experts, a last column tile of 8 columns."""
    dev = device()
    g = torch.Generator(device=dev)
    g.manual_seed(k)
    sizes = [0, 1, 128, 129, 255, 256, 257, 0, 3000, 5000, 77, 12000, 640, 0, 9000, 300]
    n, e = 1544, len(sizes)
    offs = torch.tensor(sizes, device=dev).cumsum(0).to(I32)
    m = int(offs[-1]) + 5
    x, w = codes(g, dev, m, k // 2), codes(g, dev, e, n, k // 2)
    out = torch.full((m, n), 7.0, dtype=dtype, device=dev)
    say("fp4 many tiles", k, dtype)
    for _ in range(2):
        gg.fp4_forward(x, ones(RAGGED, m, k, e, dev), w, ones(WEIGHT, n, k, e, dev), offs, out=out)
    first = 0
    for i, s in enumerate(sizes):
        want = (values(x[first:first + s]) @ values(w[i]).t()).float().to(dtype)
        assert torch.equal(out[first:first + s], want), (k, i)
        first += s
    assert bool((out[first:] == 7.0).all())


@pytest.mark.parametrize("experts", [1, 63, 64, 65, 511, 512, 513, 2047, 2048])
@pytest.mark.parametrize("masked", [False, True])
def test_many_experts(experts, masked):
    """Expert counts around the wave's and the workgroup's, up to the most."""
    dev = device()
    g = torch.Generator(device=dev)
    g.manual_seed(experts)
    k, n = 64, 72
    sizes = torch.randint(0, 4, (experts,), generator=g, device=dev)
    sizes[experts // 2] = 300
    w = codes(g, dev, experts, n, k // 2)
    say("fp4 experts", experts, masked)
    if masked:
        x = codes(g, dev, experts, 300, k // 2)
        out = torch.full((experts, 300, n), 7.0, dtype=torch.float32, device=dev)
        gg.fp4_masked_forward(x, ones(MASKED, 300, k, experts, dev), w, ones(WEIGHT, n, k, experts, dev), sizes.to(I32),
                              out=out)
        ok = torch.arange(300, device=dev) < sizes[:, None]
        want = torch.matmul(values(x).float(), values(w).float().transpose(1, 2).contiguous())
        assert torch.equal(out, torch.where(ok[..., None], want, 7.0))
        back = gg.fp4_dequantize(MASKED, x, ones(MASKED, 300, k, experts, dev), sizes.to(I32),
                                 out=torch.full(x.shape[:-1] + (k,), 7.0, dtype=BF, device=dev))
        assert torch.equal(back.double(), torch.where(ok[..., None], values(x), 7.0))
        return
    offs = sizes.cumsum(0).to(I32)
    m = int(offs[-1])
    x = codes(g, dev, m, k // 2)
    out = gg.fp4_forward(x, ones(RAGGED, m, k, experts, dev), w, ones(WEIGHT, n, k, experts, dev), offs,
                         out_dtype=torch.float32)
    who = torch.repeat_interleave(torch.arange(experts, device=dev), sizes)
    want = torch.matmul(values(w).float()[who], values(x).float()[..., None])[..., 0]
    assert torch.equal(out, want)
    # and through the quantiser: these values are their own codes but for their scales
    h = (values(x) * torch.exp2((who % 7).double())[:, None]).to(BF)
    c, s = gg.fp4_quantize(RAGGED, h, offs)
    assert torch.equal(gg.fp4_dequantize(RAGGED, c, s, offs), h)


def test_rows_past_4_gb():
    """x, its codes' rows and y past 4 GB: the last rows as by themselves."""
    dev = device()
    g = torch.Generator(device=dev)
    g.manual_seed(1)
    m, k, n, tail = 1_150_000, 2048, 2048, 5000
    say("fp4 rows past 4 GB")
    x = torch.zeros(m, k, dtype=BF, device=dev)
    x[-tail:] = torch.randn(tail, k, generator=g, device=dev).to(BF)
    offs = torch.tensor([m - tail, m - tail + 100, m], dtype=I32, device=dev)
    part = offs[1:] - (m - tail)
    w = codes(g, dev, 3, n, k // 2)
    ws = torch.full((gg.fp4_scale_bytes(WEIGHT, n, k, 3),), 120, dtype=U8, device=dev)
    ws1 = torch.full((gg.fp4_scale_bytes(WEIGHT, n, k, 2),), 120, dtype=U8, device=dev)
    c, s = gg.fp4_quantize(RAGGED, x, offs)
    back = gg.fp4_dequantize(RAGGED, c, s, offs)
    y = gg.fp4_forward(c, s, w, ws, offs)
    c1, s1 = gg.fp4_quantize(RAGGED, x[-tail:].contiguous(), part.contiguous())
    assert torch.equal(c[-tail:], c1) and bool((c[:m - tail] == 0).all())
    assert torch.equal(back[-tail:], gg.fp4_dequantize(RAGGED, c1, s1, part.contiguous()))
    assert torch.equal(y[-tail:], gg.fp4_forward(c1, s1, w[1:].contiguous(), ws1, part.contiguous()))
    assert bool((y[:m - tail] == 0).all())


def test_silu_rows_past_4_gb():
    dev = device()
    g = torch.Generator(device=dev)
    g.manual_seed(2)
    m, i, tail = 1_100_000, 1024, 700
    say("fp4 silu rows past 4 GB")
    h = torch.zeros(m, 2 * i, dtype=BF, device=dev)
    h[-tail:] = torch.randn(tail, 2 * i, generator=g, device=dev).to(BF)
    offs = torch.tensor([m - tail, m], dtype=I32, device=dev)
    c, s = gg.fp4_silu_mul_rows(h, offs)
    c1, s1 = gg.fp4_silu_mul_rows(h[-tail:].contiguous(), torch.tensor([0, tail], dtype=I32, device=dev))
    assert torch.equal(c[-tail:], c1)
    # the last expert's tiles of scales: three at the end
    need = -(-tail // 256) * (i // 128) * 1024
    first = -(-(m - tail) // 256) * (i // 128) * 1024
    assert torch.equal(s[first:first + need], s1[:need])


def test_weights_past_4_gb():
    """An expert whose codes begin past 4 GB."""
    dev = device()
    g = torch.Generator(device=dev)
    g.manual_seed(3)
    e, n, k, rows = 70, 8192, 16384, 130
    say("fp4 weights past 4 GB")
    w = torch.zeros(e, n, k // 2, dtype=U8, device=dev)
    w[-1] = codes(g, dev, n, k // 2)
    x = codes(g, dev, rows, k // 2)
    offs = torch.zeros(e, dtype=I32, device=dev)
    offs[-1] = rows
    y = gg.fp4_forward(x, ones(RAGGED, rows, k, e, dev), w, ones(WEIGHT, n, k, e, dev), offs, out_dtype=torch.float32)
    one = gg.fp4_forward(x, ones(RAGGED, rows, k, 1, dev), w[-1:].contiguous(), ones(WEIGHT, n, k, 1, dev),
                         torch.tensor([rows], dtype=I32, device=dev), out_dtype=torch.float32)
    assert torch.equal(y, one)
    # its quantiser and back, at the same distance
    v = gg.fp4_dequantize(WEIGHT, w, ones(WEIGHT, n, k, e, dev))
    assert torch.equal(v[-1, -4:].double(), values(w[-1, -4:]))
    c, s = gg.fp4_quantize(WEIGHT, v)
    assert torch.equal(gg.fp4_dequantize(WEIGHT, c[-1:].contiguous(), s[-s.numel() // e:].contiguous()), v[-1:])


@pytest.mark.parametrize("four", [False, True])
def test_few_tokens_weights_past_4_gb(four):
    """Experts whose weights begin past 4 GB give what they give by themselves."""
    dev = device()
    g = torch.Generator(device=dev)
    g.manual_seed(4)
    e, h, i = (260, 4096, 2048) if four else (140, 4096, 2048)
    say("few tokens: weights past 4 GB", four)
    x = torch.randn(3, h, generator=g, device=dev).to(BF)
    ids = torch.tensor([[e - 1, 0], [e - 2, e - 1], [e - 1, 1]], dtype=I32, device=dev)
    mine = [0, 1, e - 2, e - 1]
    to = torch.tensor([[3, 0], [2, 3], [3, 1]], dtype=I32, device=dev)
    if four:
        w13, w2 = torch.zeros(e, 2 * i, h // 2, dtype=U8, device=dev), torch.zeros(e, h, i // 2, dtype=U8, device=dev)
        for j in mine:
            w13[j], w2[j] = codes(g, dev, 2 * i, h // 2), codes(g, dev, h, i // 2)

        def scales(rows, k, n):
            return torch.full((gg.fp4_scale_bytes(WEIGHT, rows, k, n),), 121, dtype=U8, device=dev)
        a = gg.fp4_moe_few_tokens(x, ids, w13, scales(2 * i, h, e), w2, scales(h, i, e))
        b = gg.fp4_moe_few_tokens(x, to, w13[mine].contiguous(), scales(2 * i, h, 4), w2[mine].contiguous(), scales(h, i, 4))
    else:
        w13, w2 = torch.zeros(e, 2 * i, h, dtype=BF, device=dev), torch.zeros(e, h, i, dtype=BF, device=dev)
        for j in mine:
            w13[j] = torch.randn(2 * i, h, generator=g, device=dev) * h ** -0.5
            w2[j] = torch.randn(h, i, generator=g, device=dev) * i ** -0.5
        a = gg.moe_few_tokens(x, ids, w13, w2)
        b = gg.moe_few_tokens(x, to, w13[mine].contiguous(), w2[mine].contiguous())
    # (the experts' order, and so the sums', is that of the slots in both)
    assert torch.equal(a, b) and bool((a != 0).any())
