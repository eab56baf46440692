"""GPU tests of the layer steps at the ends of the number range."""
import pytest
import torch

import layer_ref as ref
from moe_grouped_gemm_ragged_amd import binding as gg
from gpu_util import device, say

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
BF_MAX = float(torch.finfo(BF).max)


@pytest.mark.parametrize("kept", [False, True])
def test_silu_mul_grad_of_large_and_tiny_operands(kept):
    """da and up of any size against gates of any size: a product of two of
    the three factors may leave fp32 although the gradient is 0 or finite."""
    dev = device()
    sizes = torch.tensor([0.0, 1e-38, 3e-30, 1e-20, 1.0, -0.75, 1e20, -3e30, 1e38, -3.3e38], dtype=torch.float64)
    gates = torch.tensor([-3e38, -1e30, -200.0, -100.0, -87.0, -60.0, -20.0, -3.0, -1.25, -0.5, 0.0, 1e-30, 0.5, 2.5,
                          40.0, 1e30, 3e38], dtype=torch.float64)
    g, d, u = (t.reshape(-1) for t in torch.meshgrid(gates, sizes, sizes, indexing="ij"))
    width = -(-g.numel() // 128) * 128
    pad = torch.zeros(width - g.numel(), dtype=torch.float64)
    h = torch.cat([g, pad, u, pad]).to(BF).reshape(1, -1).to(dev)
    da = torch.cat([d, pad]).to(BF).reshape(1, -1).to(dev)
    if kept:
        # every value its own block's largest, so that codes and scales hold it to 4 bits
        h = h.reshape(-1, 1).expand(-1, 128).reshape(1, -1).contiguous()
        da = da.reshape(-1, 1).expand(-1, 128).reshape(1, -1).contiguous()
        codes, scales = (t.to(dev) for t in ref.quantise(h.cpu()))
        hv = ref.value(codes, scales)
    else:
        hv = ref.f64(h)
    groups = torch.ones(1, dtype=torch.int32, device=dev)
    say("silu_mul_grad of large and tiny operands", kept)
    dh = (gg.fp8_silu_mul_grad(da, codes, scales, groups) if kept else gg.silu_mul_grad(da, h, groups))
    torch.cuda.synchronize()
    want, slack = ref.silu_mul_grad(ref.f64(da), hv)
    got = ref.f64(dh)
    # beyond the largest bf16 value: an infinity of the right sign, or that value where the two lie
    # within the bounds of each other
    room = want.abs() * 2.0 ** -8 + slack
    over = want.abs() + room > BF_MAX
    assert bool((over & (want.abs() > 4e38)).any()), "no case leaves the range"
    beyond = over & (want.abs() - room > BF_MAX)
    assert bool((got[beyond] == want[beyond].sign() * float("inf")).all())
    ref.close(got[~over], want[~over], room[~over], "dh")


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
