"""The few-token layer at the ends of its number range: infinite weights, the
activation's 16 bits of mantissa on its way between the two kernels, one next to
the largest fp32 value, and the 4-bit scales' ends."""
import pytest
import torch

import fp4_ref
from layer_ref import TINY, U32, close
from moe_grouped_gemm_ragged_amd import binding as gg
from gpu_util import device, say

pytestmark = pytest.mark.gpu
BF, U8, I32, F32 = torch.bfloat16, torch.uint8, torch.int32, torch.float32


class Weights:
    """[E, n, k] weights for the library and their 64-bit values, given in e2m1
    codes with a scale byte each (bf16: their values, infinite from 2^128 on)."""

    def __init__(self, four, codes, raw):
        packed = fp4_ref.pack(codes)
        bf = fp4_ref.value(packed, raw).to(BF)
        self.value = bf.double()
        self.w = packed.cuda() if four else bf.cuda()
        self.scales = gg.fp4_pack_scales(gg.GG_FP4_WEIGHT, raw.cuda()) if four else None


def layer(four, x, ids, w13, w2, weights=None, **kw):
    weights = None if weights is None else weights.cuda()
    if four:
        return gg.fp4_moe_few_tokens(x.cuda(), ids.cuda(), w13.w, w13.scales, w2.w, w2.scales, weights, **kw)
    return gg.moe_few_tokens(x.cuda(), ids.cuda(), w13.w, w2.w, weights, **kw)


def activations(x, ids, w13, weights):
    """[tokens, topk, I] weight * silu(gate) up of every slot, and the gates."""
    h = torch.matmul(w13.value[ids.long()], x.double()[:, None, :, None])[..., 0]
    gate, up = h.chunk(2, -1)
    return weights.double()[..., None] * torch.nn.functional.silu(gate) * up, gate


def random_codes(g, *shape):
    return torch.randint(0, 16, shape, generator=g, dtype=U8)


def one_hot(experts, hidden, inter, code=2):
    """W2 codes with one value a row: out[h] is activation h mod inter times it."""
    codes = torch.zeros(experts, hidden, inter, dtype=U8)
    codes[:, torch.arange(hidden), torch.arange(hidden) % inter] = code
    return codes


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("tokens", [7, 40])
def test_infinite_weights(four, dtype, tokens):
    """An infinite weight of W2 gives what the formula does: an infinity of the
    activation's sign, NaN only where infinities of both signs meet (no
    activation is 0).  Rows without one are as they were."""
    device()
    g = torch.Generator().manual_seed(tokens)
    experts, hidden, inter, topk = 6, 96, 288, 2
    w13 = Weights(four, random_codes(g, experts, 2 * inter, hidden), torch.full((experts, 2 * inter, hidden // 32), 123, dtype=U8))
    codes = random_codes(g, experts, hidden, inter)
    raw = torch.full((experts, hidden, inter // 32), 121, dtype=U8)
    clean = Weights(four, codes, raw)
    # expert, row, value, code: 6 2^127 and its negative, infinite in bf16; the rest of their blocks 0
    at = ((2, 3, 7, 7), (2, 4, 150, 15), (2, 5, 0, 7), (2, 5, 1, 15), (2, 95, 287, 7), (4, 3, 8, 15), (4, 3, 130, 7),
          (1, 10, 255, 15), (1, 11, 256, 7), (0, 20, 131, 7))
    codes = codes.clone()
    for e, r, i, _ in at:
        codes[e, r, i // 32 * 32:i // 32 * 32 + 32], raw[e, r, i // 32] = 0, 254
    for e, r, i, c in at:
        codes[e, r, i] = c
    codes[3, 40], raw[3, 40] = 7, 254
    w2 = Weights(four, codes, raw)
    assert bool(torch.isinf(w2.value).any()) and not bool(torch.isnan(w2.value).any())
    x = torch.randn(tokens, hidden, generator=g).to(BF)
    ids = torch.rand(tokens, experts, generator=g).topk(topk, dim=1).indices.to(I32)
    weights = torch.rand(tokens, topk, generator=g) + 0.1
    a, _ = activations(x, ids, w13, weights)
    assert bool((a.abs() > 1e-30).all())
    want = torch.matmul(w2.value[ids.long()], a[..., None])[..., 0].sum(1)
    say("few tokens: infinite weights", four, dtype, tokens)
    before = layer(four, x, ids, w13, clean, weights, out_dtype=dtype).cpu()
    got = layer(four, x, ids, w13, w2, weights, out_dtype=dtype).cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    inf = torch.isinf(want)
    assert int(inf.sum()) > 10 and bool(torch.isnan(want).any())
    assert torch.equal(got.double()[inf], want[inf])
    same = (w2.value == clean.value).all(-1)                # [E, hidden]: rows that were not changed
    same = same[ids.long()].all(1)
    assert torch.equal(got[same], before[same]) and bool(same.any())


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("tokens", [3, 20, 64])
def test_activation_keeps_16_bits(four, tokens):
    """x and W13 are whole multiples of 2^-4 or 1, so gate and up are exact in
    fp32 (multiples of 2^-5 below 2^9).  Each row of W2 has a single 1, so out is
    the sum of two activations: the bound is 2^-17 of each for its two bf16
    values (half a step of the second, which is at most half a step of the
    first), and the fp32 roundings."""
    device()
    g = torch.Generator().manual_seed(100 + tokens)
    experts, hidden, inter, topk = 5, 128, 96, 2
    w13 = Weights(four, random_codes(g, experts, 2 * inter, hidden), torch.full((experts, 2 * inter, hidden // 32), 123, dtype=U8))
    w2 = Weights(four, one_hot(experts, hidden, inter), torch.full((experts, hidden, inter // 32), 127, dtype=U8))
    x = torch.randint(-3, 4, (tokens, hidden), generator=g).to(BF)
    ids = torch.rand(tokens, experts, generator=g).topk(topk, dim=1).indices.to(I32)
    weights = torch.rand(tokens, topk, generator=g)
    a, gate = activations(x, ids, w13, weights)
    column = torch.arange(hidden) % inter
    want = a.sum(1)[:, column]
    # layer_ref.silu_mul's slack, the share's product, the additions over slots, halves and waves
    slack = a.abs() * (2.0 ** -17 + (2 * gate.abs() + 16 + 2 + 16) * U32) + TINY * (1 + a.abs())
    say("few tokens: activation", four, tokens)
    got = layer(four, x, ids, w13, w2, weights, out_dtype=F32)
    slack = slack.sum(1)[:, column]
    close(got, want, slack + U32 * (want.abs() + slack), "activation")


@pytest.mark.parametrize("four", [False, True])
def test_activation_next_to_fp32_max(four):
    """An activation of 2^128 - 2^118, which fp32 holds and bf16 rounds to an
    infinity, reaches out as it is: 2^28 - 2^18 after a weight of 2^-100."""
    device()
    hidden, inter = 64, 32
    codes = torch.zeros(1, 2 * inter, hidden, dtype=U8)
    codes[:, :, 0] = 2
    codes[:, inter:, 1] = 2
    w13 = Weights(four, codes, torch.full((1, 2 * inter, hidden // 32), 127 + 32, dtype=U8))
    w2 = Weights(four, one_hot(1, hidden, inter), torch.full((1, hidden, inter // 32), 27, dtype=U8))
    x = torch.zeros(2, hidden, dtype=BF)
    x[:, 0] = 2.0 ** 32
    x[0, 1] = -(2.0 ** 22)
    x[1, 1] = -(2.0 ** 31)              # (an ordinary one: 2^127)
    ids = torch.zeros(2, 1, dtype=I32)
    say("few tokens: next to fp32's largest value", four)
    got = layer(four, x, ids, w13, w2, out_dtype=F32).cpu()
    assert bool((got[0] == 2.0 ** 28 - 2.0 ** 18).all()) and bool((got[1] == 2.0 ** 27).all())


def test_scales_at_their_ends():
    """Every code with the smallest and the largest scale bytes: weights down to
    2^-128 count as they are, from 2^128 on as infinities, byte 255 as NaN."""
    device()
    hidden, inter = 192, 32
    bytes_ = torch.tensor([0, 1, 2, 3, 4, 8, 250, 251, 252, 253, 254, 255])
    code, byte = torch.arange(hidden) % 16, bytes_[torch.arange(hidden) // 16]
    codes = torch.zeros(2, hidden, inter, dtype=U8)
    codes[:, :, 0] = code
    w2 = Weights(True, codes, byte[None, :, None].expand(2, hidden, 1).to(U8).contiguous())
    # expert 0: activations of 2^100, expert 1: some 2^-61
    first = torch.zeros(2, 2 * inter, hidden, dtype=U8)
    first[:, :, 0] = 2
    raw = torch.full((2, 2 * inter, hidden // 32), 127, dtype=U8)
    raw[0], raw[1] = 127 + 50, 127 - 30
    w13 = Weights(True, first, raw)
    x = torch.zeros(2, hidden, dtype=BF)
    x[:, 0] = 1.0
    ids = torch.tensor([[0], [1]], dtype=I32)
    a, gate = activations(x, ids, w13, torch.ones(2, 1))
    want = torch.matmul(w2.value[ids.long()[:, 0]], a[:, 0, :, None])[..., 0]
    say("few tokens: scales at their ends")
    got = layer(True, x, ids, w13, w2, out_dtype=F32).cpu()
    fits = want.abs() < 2.0 ** 127
    inf = torch.isinf(w2.value[0, :, 0])
    assert bool(inf.any()) and torch.equal(got[:, inf].double(), want[:, inf])
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    got, want = got.double()[fits], want[fits]
    bound = want.abs() * (2.0 ** -17 + 40 * U32) + TINY
    assert bool(((got - want).abs() <= bound).all())
    assert bool((got[want.abs() > 2.0 ** -60] != 0).all())
