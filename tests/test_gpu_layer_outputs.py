"""Every output of the layer steps' binding may be the caller's buffer: it is
returned, holds what a new tensor would, and one that does not fit is refused."""
import pytest
import torch

from moe_grouped_gemm_ragged_amd import binding as gg
from gpu_util import device, say

BF, U8 = torch.bfloat16, torch.uint8


def bf(*shape):
    return torch.zeros(*shape, dtype=BF)


I = torch.zeros(4, dtype=torch.int32)


@pytest.mark.parametrize("error,call", [
    (ValueError, lambda: gg.combine_rows_grad(bf(2, 8), bf(4, 8), I, I, I, 2, dweights=torch.zeros(2, 3))),
    (TypeError, lambda: gg.combine_rows_grad(bf(2, 8), bf(4, 8), I, I, I, 2, dweights=bf(2, 2))),
    (ValueError, lambda: gg.combine_rows_grad(bf(2, 8), bf(4, 8), I, I, I, 2, dweights=torch.zeros(2, 4)[:, ::2])),
    (ValueError, lambda: gg.combine_rows_grad(bf(2, 8), None, I, I, I, 2, with_weights=False,
                                              dweights=torch.zeros(2, 2))),
    (ValueError, lambda: gg.fp8_rmsnorm(bf(4, 128), bf(128), y_out=bf(4, 64))),
    (TypeError, lambda: gg.fp8_rmsnorm(bf(4, 128), bf(128), y_out=torch.zeros(4, 128))),
    # fitting buffers, but not on a GPU
    (ValueError, lambda: gg.fp8_rmsnorm(bf(4, 128), bf(128), y_out=bf(4, 128))),
])
def test_buffers_that_do_not_fit_are_refused(error, call):
    with pytest.raises(error):
        call()


@pytest.mark.gpu
def test_buffers_for_the_weights_gradient_and_the_bf16_norm():
    dev = device()
    g = torch.Generator(device=dev)
    g.manual_seed(3)
    ids = torch.randint(0, 5, (70, 3), generator=g, device=dev, dtype=torch.int32)
    offs, row_slot, slot_row = gg.route(ids, 5, 8, True)
    dout = torch.randn(70, 256, generator=g, device=dev).to(BF)
    y = torch.randn(row_slot.shape[0], 256, generator=g, device=dev).to(BF)
    gamma = torch.randn(256, generator=g, device=dev).to(BF)
    say("combine_rows_grad into a buffer")
    _, want = gg.combine_rows_grad(dout, y, slot_row, row_slot, offs, 3)
    mine = torch.full((70, 3), float("nan"), device=dev)
    _, dw = gg.combine_rows_grad(dout, y, slot_row, row_slot, offs, 3, dweights=mine)
    assert dw is mine and torch.equal(mine, want)
    say("fp8_rmsnorm into a buffer")
    codes, scales, _, want = gg.fp8_rmsnorm(dout, gamma, with_bf16=True)
    mine = torch.full((70, 256), float("nan"), dtype=BF, device=dev)
    got = gg.fp8_rmsnorm(dout, gamma, y_out=mine)
    assert got[3] is mine and torch.equal(mine, want)
    assert torch.equal(got[0], codes) and torch.equal(got[1], scales)
