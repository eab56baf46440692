"""The few-token layer on operands whose results are exact (few_tokens_exact):
equal to the formula in 64 bits."""
import pytest
import torch

import few_tokens_exact as exact
from gpu_util import device, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("tokens,topk,experts", [(1, 1, 1), (1, 6, 9), (4, 2, 2), (5, 3, 4), (23, 4, 6), (64, 2, 3)])
@pytest.mark.parametrize("hidden,inter", [(64, 32), (160, 288), (224, 544)])
def test_every_product_counts_once(four, tokens, topk, experts, hidden, inter):
    """Both halves of a step of the down product, its waves' shares, experts of one
    to 64 tokens."""
    device()
    if not four:
        hidden, inter = hidden - 8, inter - 8
    layer = exact.Layer(four, experts, hidden, inter, topk, seed=tokens)
    x, ids, weights = exact.inputs(tokens, tokens, hidden, exact.some_experts(tokens, tokens, topk, experts))
    say("few tokens: exact", four, tokens, topk, experts, hidden, inter)
    want = layer.want(x, ids, weights)
    assert bool((want != 0).any())
    for _ in range(3):
        assert torch.equal(layer(x, ids, weights, out_dtype=torch.float32).double(), want)


def up_launch(four, slots, experts, inter):
    """Workgroups of an expert in the up kernel, the strips of each, and all strips."""
    n = -(-inter // 128) * 16 if four else -(-inter // 8)
    each = min(max(n * min(slots, experts) // 4096, 1), 4)
    return -(-n // each), each, n


def crowded(seed, tokens, topk, experts, crowd):
    """Each token's distinct experts; expert i is one of the first crowd[i] tokens' for i < len(crowd)."""
    ids = exact.some_experts(seed, tokens, topk, experts - len(crowd)) + len(crowd)
    for i, c in enumerate(crowd):
        ids[:c, i] = i
    return ids


# tokens, topk, experts, hidden, inter, tokens of the first experts: several strips a workgroup, an even
# and an odd share, with 1, 2 and 4 blocks of 16 tokens, x in LDS or not, at most 64 slots and more
STRIPS = [
    (8, 8, 64, 64, 1024, ()), (8, 8, 64, 96, 1088, (8,)), (23, 8, 128, 64, 768, (20, 16, 1)), (23, 8, 128, 64, 704, (23,)),
    (23, 8, 128, 88, 800, (9,)),
    (64, 8, 128, 64, 768, (64, 33, 17, 16, 32)), (64, 8, 100, 32, 1344, (40, 16)), (16, 8, 64, 1056, 1024, (16, 15, 13)),
    (64, 8, 512, 64, 256, (50, 16)), (64, 8, 256, 32, 544, (64, 18)),
]


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("tokens,topk,experts,hidden,inter,crowd", STRIPS)
def test_several_strips_a_workgroup(four, tokens, topk, experts, hidden, inter, crowd):
    device()
    across, each, n = up_launch(four, tokens * topk, experts, inter)
    assert each > 1 and across < n
    if four:
        hidden = -(-hidden // 32) * 32
    layer = exact.Layer(four, experts, hidden, inter, topk, seed=inter)
    x, ids, weights = exact.inputs(inter, tokens, hidden, crowded(tokens, tokens, topk, experts, crowd))
    assert all(int((ids == i).sum()) == c for i, c in enumerate(crowd))
    say("few tokens: several strips", four, tokens, experts, hidden, inter, (across, each, n))
    want = layer.want(x, ids, weights)
    for _ in range(3):
        assert torch.equal(layer(x, ids, weights, out_dtype=torch.float32).double(), want)


def test_strips_cover_the_rule():
    """The cases above take 2, 3 and 4 strips, whole shares and a last one that is
    smaller, workgroups in and past whole 32s."""
    seen = [up_launch(four, c[0] * c[1], c[2], c[4]) for c in STRIPS for four in (False, True)]
    assert {s[1] for s in seen} == {2, 3, 4}
    assert any(across * each > n for across, each, n in seen) and any(across * each == n for across, each, n in seen)
    assert any(across < 32 for across, _, _ in seen) and any(across > 32 and across % 32 for across, _, _ in seen)


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("tokens,topk,experts", [(1, 8, 16), (19, 3, 10), (20, 2, 5), (41, 1, 5), (64, 2, 7)])
@pytest.mark.parametrize("hidden", [2016, 2048, 2080, 2880, 4096])
def test_widths_around_a_strip_for_each_compute_unit(four, tokens, topk, experts, hidden):
    """4 bits: 256 strips of the down product and the next more, where workgroups
    begin to take two, up to 8 slots an expert; a last span that is not full."""
    device()
    layer = exact.Layer(four, experts, hidden, 288, topk, seed=hidden)
    x, ids, weights = exact.inputs(hidden, tokens, hidden, exact.some_experts(tokens, tokens, topk, experts, 0.1))
    say("few tokens: widths", four, tokens, experts, hidden)
    assert torch.equal(layer(x, ids, weights, out_dtype=torch.float32).double(), layer.want(x, ids, weights))


def reaching(seed, tokens, topk, reached, experts):
    """Ids that reach so many experts: each once, the other slots to the first
    of them, more than four tokens each where there are slots enough."""
    g = torch.Generator().manual_seed(seed)
    mine = torch.randperm(experts, generator=g)[:reached]
    rest = tokens * topk - reached
    crowd = max(1, min(reached, rest // 6))
    slots = torch.cat([mine, mine[torch.arange(rest) % crowd]])
    return slots[torch.randperm(slots.numel(), generator=g)].reshape(tokens, topk)


# tokens, topk, experts, reached, hidden, inter.  Down: up to 64 reached experts one list, then each wave its
# own; from 256 on whole experts a wave, below equal runs of steps that begin inside an expert.  An expert has
# inter / 128 steps in bf16 and inter / 256 in 4 bits, rounded up
REACHED = [
    (64, 8, 70, 64, 64, 544), (64, 8, 70, 65, 64, 544), (64, 8, 128, 100, 96, 288), (13, 8, 300, 97, 64, 800),
    (64, 8, 300, 255, 64, 544), (32, 8, 300, 256, 64, 288), (64, 8, 300, 256, 64, 544), (64, 8, 300, 300, 32, 800),
    (64, 8, 512, 512, 64, 288), (1, 65, 65, 65, 64, 544), (1, 512, 512, 400, 32, 288), (64, 8, 2048, 450, 32, 288),
    (64, 8, 100, 100, 2080, 288), (64, 8, 280, 257, 2080, 288),
]


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("tokens,topk,experts,reached,hidden,inter", REACHED)
def test_many_reached_experts(four, tokens, topk, experts, reached, hidden, inter):
    device()
    slots = reaching(reached, tokens, topk, reached, experts)
    assert len(set(slots.reshape(-1).tolist())) == reached
    if tokens * topk - reached > 60 and tokens > 8:
        assert max((slots == e).any(-1).sum().item() for e in range(experts)) > 4
    layer = exact.Layer(four, experts, hidden, inter, topk, seed=reached)
    x, ids, weights = exact.inputs(reached, tokens, hidden, slots)
    say("few tokens: reached experts", four, tokens, experts, reached, hidden, inter)
    want = layer.want(x, ids, weights)
    for _ in range(3):
        assert torch.equal(layer(x, ids, weights, out_dtype=torch.float32).double(), want)
