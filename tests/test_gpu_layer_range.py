"""GPU tests of the layer steps at the ends of the number range."""
import pytest
import torch

import layer_ref as ref
from moe_grouped_gemm_ragged_amd import binding as gg
from gpu_util import device, say

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
BF_MAX = float(torch.finfo(BF).max)


def test_silu_mul_grad_of_kept_rows_beyond_fp32():
    """The largest bf16 values are kept as 2^128: gates of that size are at
    silu's limits, and up values of it give finite products."""
    dev = device()
    h = torch.zeros(12, 256)
    for i in range(12):
        h[i, :128] = (BF_MAX, -BF_MAX, 0.5)[i // 4]
        h[i, 128:] = (BF_MAX, -BF_MAX, 0.25, 0.0)[i % 4]
    h = h.to(BF).to(dev)
    da = torch.tensor([1.0, -0.5, 2.0 ** -20, 2.0 ** -120]).repeat(32).expand(12, 128).to(BF).contiguous().to(dev)
    groups = torch.tensor([12], dtype=torch.int32, device=dev)
    _, codes, scales = gg.silu_mul_rows(h, groups, keep=True)
    hv = ref.value(codes, scales)
    assert float(hv.max()) == 2.0 ** 128
    say("silu_mul_grad of kept rows beyond fp32")
    dh, act = gg.fp8_silu_mul_grad(da, codes, scales, groups, with_act=True)
    torch.cuda.synchronize()
    for got, (want, _), what in ((dh, ref.silu_mul_grad(ref.f64(da), hv), "dh"), (act, ref.silu_mul(hv), "act")):
        # the sigmoid is exactly 0 or 1 at gates of that size, and the general bounds, which grow with
        # |g|, are not needed: half a bf16 step, and what they allow at the third gate, 0.5
        got, room = ref.f64(got), want.abs() * (2.0 ** -8 + 64 * ref.U32)
        beyond = want.abs() >= 2.0 ** 128
        assert torch.equal(got[beyond], want[beyond].sign() * float("inf")), what
        ref.close(got[~beyond], want[~beyond], room[~beyond], what)
