"""The 4-bit operators as they are used together: a prompt's MoE layer (route ->
4-bit rows sorted by expert -> gate/up -> SiLU-mul to 4 bits -> down -> weighted
combine) with each stage checked against its fp64 form on what the stage before
wrote, the gradients of its projections through the dequantised operands, and a
decoding step's layer in two kernels against the long way on the same weights."""
import pytest
import torch

import fp4_ref as ref
import layer_ref
from layer_ref import U32
from moe_grouped_gemm_ragged_amd import binding as gg
from gpu_util import device, say

pytestmark = pytest.mark.gpu
BF, U8, I32 = torch.bfloat16, torch.uint8, torch.int32
RAGGED, WEIGHT = gg.GG_FP4_ACT_RAGGED, gg.GG_FP4_WEIGHT


def routed(g, tokens, topk, e, align):
    ids = torch.rand(tokens, e, generator=g).topk(topk, dim=1).indices.to(I32)
    ids[torch.rand(ids.shape, generator=g) < 0.05] = -1
    return ids.contiguous().cuda(), torch.rand(tokens, topk, generator=g).cuda()


@pytest.mark.parametrize("tokens,topk,e,k,i,align", [(150, 4, 8, 416, 288, 16), (1, 2, 4, 64, 32, 1), (700, 2, 3, 256, 128, 8)])
def test_layer_in_4_bits(tokens, topk, e, k, i, align):
    device()
    g = torch.Generator().manual_seed(tokens)
    x = torch.randn(tokens, k, generator=g).to(BF).cuda()
    ids, probs = routed(g, tokens, topk, e, align)
    w13 = (torch.randn(e, 2 * i, k, generator=g) * k ** -0.5).to(BF).cuda()
    w2 = (torch.randn(e, k, i, generator=g) * i ** -0.5).to(BF).cuda()
    say("layer in 4 bits", tokens, topk, e, k, i)
    w13c, w13s = gg.fp4_quantize(WEIGHT, w13)
    w2c, w2s = gg.fp4_quantize(WEIGHT, w2)
    w13v, w2v = gg.fp4_dequantize(WEIGHT, w13c, w13s), gg.fp4_dequantize(WEIGHT, w2c, w2s)
    offs, row_slot, slot_row = gg.route(ids, e, align, True)
    used = int(offs[-1])
    ends = offs.cpu().tolist()
    who = ref.owned(0, ends, used, e)

    x4, x4s = gg.fp4_gather_rows(x, row_slot, topk, offs)
    h = gg.fp4_forward(x4, x4s, w13c, w13s, offs)
    a4, a4s = gg.fp4_silu_mul_rows(h, offs)
    y = gg.fp4_forward(a4, a4s, w2c, w2s, offs)
    out = gg.combine_rows(y, slot_row, topk, probs)
    xv, av = gg.fp4_dequantize(RAGGED, x4, x4s, offs), gg.fp4_dequantize(RAGGED, a4, a4s, offs)
    torch.cuda.synchronize()

    slot = row_slot.cpu()[:used].long()
    rows = torch.where((slot >= 0)[:, None], x.cpu()[(slot // topk).clamp(min=0)].float(), 0.0)
    c, b = ref.quantise(rows)
    assert torch.equal(xv.cpu()[:used].double(), ref.value(ref.pack(c), b))
    ref.check_product(h[:used], xv.cpu()[:used].double(), w13v.cpu().double(), who, "gate/up")
    want, slack = layer_ref.silu_mul(h.cpu()[:used].double())
    # within half a step of a value of its block: a quarter of it, or of the block's scale (at most
    # amax / 3 for a block's largest value amax) where the value is below that
    block = want.abs().reshape(used, -1, 32).amax(-1, keepdim=True).expand(-1, -1, 32).reshape(want.shape)
    layer_ref.close(av[:used], want, torch.maximum(want.abs(), block / 3) / 4 + 2 * slack, "activation")
    ref.check_product(y[:used], av.cpu()[:used].double(), w2v.cpu().double(), who, "down")
    row = slot_row.cpu().long().reshape(tokens, topk)
    terms = torch.where((row >= 0)[..., None], y.cpu().double()[row.clamp(min=0)] * probs.cpu().double()[..., None], 0.0)
    total = terms.sum(1)
    layer_ref.close(out, total, (2 * topk + 2) * U32 * terms.abs().sum(1) + layer_ref.HALF[BF] * total.abs() * (1 + 2.0 ** -7),
                    "combine")

    say("layer in 4 bits: gradients of the projections")
    dy = torch.randn(y.shape, generator=g).to(BF).cuda()
    da = gg.dgrad_nk(dy, w2v, offs, out_dtype=torch.float32)
    dw = gg.wgrad_nk(av, dy, offs, out_dtype=torch.float32)
    for r in range(e):
        mine = (who == r).nonzero()[:, 0]
        d, v = dy.cpu()[mine].double(), av.cpu()[mine].double()
        wv = w2v[r].cpu().double()
        layer_ref.close(da.cpu()[mine], d @ wv, 2 * k * U32 * (d.abs() @ wv.abs()) + U32 * (d @ wv).abs(), "da")
        n = max(1, len(mine))
        layer_ref.close(dw[r], d.t() @ v, 2 * n * U32 * (d.abs().t() @ v.abs()) + U32 * (d.t() @ v).abs(), "dW")
    # and against differences of the product itself: y is linear in the activation's values, so a
    # step that 4 bits hold (a code of 1 turned into 2, in a block of its own scale) moves y by the
    # weight's column times it
    r0 = int((who >= 0).nonzero()[0, 0])
    codes = a4.clone()
    codes[r0] = 0
    codes[r0, 0] = 2
    one = gg.fp4_forward(codes, a4s, w2c, w2s, offs, out_dtype=torch.float32)[r0]
    codes[r0, 0] = 4
    two = gg.fp4_forward(codes, a4s, w2c, w2s, offs, out_dtype=torch.float32)[r0]
    step = gg.fp4_dequantize(RAGGED, codes, a4s, offs)[r0, 0].double() / 2
    unit = torch.zeros_like(dy)
    unit[r0, 3] = 1.0
    slope = gg.dgrad_nk(unit, w2v, offs, out_dtype=torch.float32)[r0, 0].double()
    assert (two - one)[3].double() / step == slope


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("tokens,topk,e,hidden,inter", [(1, 4, 8, 512, 96), (20, 4, 6, 416, 160), (64, 8, 16, 256, 96)])
def test_few_tokens_against_the_long_way(four, tokens, topk, e, hidden, inter):
    """The same layer by routing, two grouped products and the combine.  The long
    way also rounds gate/up, the activation and every expert's row to bf16."""
    device()
    g = torch.Generator().manual_seed(tokens + four)
    x = torch.randn(tokens, hidden, generator=g).to(BF).cuda()
    ids, probs = routed(g, tokens, topk, e, 1)
    w13 = (torch.randn(e, 2 * inter, hidden, generator=g) * hidden ** -0.5).to(BF).cuda()
    w2 = (torch.randn(e, hidden, inter, generator=g) * inter ** -0.5).to(BF).cuda()
    say("few tokens and the long way", four, tokens, topk, e)
    if four:
        (c13, s13), (c2, s2) = gg.fp4_quantize(WEIGHT, w13), gg.fp4_quantize(WEIGHT, w2)
        short = gg.fp4_moe_few_tokens(x, ids, c13, s13, c2, s2, probs)
        w13, w2 = gg.fp4_dequantize(WEIGHT, c13, s13), gg.fp4_dequantize(WEIGHT, c2, s2)
    else:
        short = gg.moe_few_tokens(x, ids, w13, w2, probs)
    offs, row_slot, slot_row = gg.route(ids, e, 1, False)
    h = gg.forward_nk(gg.gather_rows(x, row_slot, topk, offs), w13, offs)
    a = gg.silu_mul_rows(h, offs)
    y = gg.forward_nk(a, w2, offs)
    long = gg.combine_rows(y, slot_row, topk, probs)
    torch.cuda.synchronize()
    # the long way's roundings: h (2^-8 of each, through silu's slope of at most 1.1 and times up),
    # a and y (2^-8 each); both ways' last one, and fp32 sums beside them
    half = 2.0 ** -8
    ha, ya = h.cpu().double(), y.cpu().double()
    gate, up = ha[:, :inter].abs(), ha[:, inter:].abs()
    silu = torch.nn.functional.silu(ha[:, :inter]).abs()
    off_a = half * (1.1 * gate * up + silu * up) * 1.02 + half * silu * up
    row = slot_row.cpu().long().reshape(tokens, topk)
    who = ids.cpu().long()
    bound = torch.zeros(tokens, hidden, dtype=torch.float64)
    for t in range(tokens):
        for j in range(topk):
            if row[t, j] < 0:
                continue
            p, r = float(probs[t, j]), int(row[t, j])
            sums = 4 * (hidden + inter) * U32
            bound[t] += p * ((off_a[r] + sums * (silu[r] * up[r] + gate[r] * up[r] + 1)) @ w2[who[t, j]].cpu().double().abs().t()
                             + half * ya[r].abs())
    bound = bound + 2.1 * half * long.cpu().double().abs() + 1e-30
    layer_ref.close(short, long.cpu().double(), bound, "short against long")
