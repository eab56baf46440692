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
