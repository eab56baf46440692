"""GPU tests of the layer steps at the ends of the number range, and of the
norm gradient's longest sums against exact whole numbers."""
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


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_fp8_wgrad_of_every_scale_byte(masked, dtype):
    """One row an expert, all 256 codes under each of the 256 scale bytes, and
    dY 1: dW is the row itself, rounded to bf16 as it enters."""
    dev = device()
    e = 256
    codes = torch.arange(256, device=dev).to(torch.uint8).expand(e, 256).contiguous()
    scales = torch.arange(e, device=dev).to(torch.uint8)[:, None].expand(e, 2).contiguous()
    dy = torch.ones(e, 8, dtype=BF, device=dev)
    c = codes.cpu().view(torch.float8_e4m3fn).double()
    b = torch.arange(e, dtype=torch.float64)[:, None]
    want = c * torch.where(b == 255, torch.full_like(b, float("nan")), torch.pow(2.0, b - 127))
    exact = (b >= 3) & (b <= 246) & ~torch.isnan(c)
    assert torch.equal(want.to(BF).double()[exact], want[exact])
    if masked:
        groups = torch.ones(e, dtype=torch.int32, device=dev)
        packed = gg.fp8_pack_scales(gg.GG_FP8_ACT_MASKED, scales, groups, 1, 256, e)
        say("fp8_masked_wgrad of every scale byte", dtype)
        dw = gg.fp8_masked_wgrad(codes[:, None], packed, dy[:, None], groups, out_dtype=dtype)
    else:
        groups = torch.arange(1, e + 1, dtype=torch.int32, device=dev)
        packed = gg.fp8_pack_scales(gg.GG_FP8_ACT_RAGGED, scales, groups, e, 256, e)
        say("fp8_wgrad of every scale byte", dtype)
        dw = gg.fp8_wgrad(codes, packed, dy, groups, out_dtype=dtype)
    torch.cuda.synchronize()
    got, want = ref.f64(dw), want.to(BF).double()[..., None].expand(e, 256, 8)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    there = ~torch.isnan(want)
    assert torch.equal(got[there], want[there])


def test_silu_mul_grad_of_every_scale_byte():
    """Kept rows under scale bytes from 0 (2^-127) to 247 (448 2^120 leaves
    bf16), and 255, NaN."""
    dev = device()
    b = torch.tensor([*range(248), 255])
    rows = b.numel()
    codes = torch.arange(128).to(torch.uint8).repeat(rows, 2)
    codes[:, 127] = codes[:, 255] = 0x08                  # (no NaN codes)
    scales = b.to(torch.uint8)[:, None].repeat(1, 2)
    scales[:, 1] = 127
    hv = ref.value(codes, scales)
    hv[-1, :128] = float("nan")
    da = torch.full((rows, 128), 2.0 ** 100, dtype=BF)
    say("silu_mul_grad of every scale byte")
    dh = gg.fp8_silu_mul_grad(da.to(dev), codes.to(dev), scales.to(dev),
                              torch.tensor([rows], dtype=torch.int32, device=dev))
    torch.cuda.synchronize()
    want, slack = ref.silu_mul_grad(ref.f64(da), hv)
    got = ref.f64(dh)
    # (products of 2^100 and a code's 4 bits, the sigmoid being 1 at such gates: below 2^128 by a bf16
    # step or more, or not at all)
    beyond = want.abs() >= 2.0 ** 128
    assert torch.equal(got[beyond], want[beyond].sign() * float("inf"))
    want, slack = want.masked_fill(beyond, 0.0), slack.masked_fill(beyond, 0.0)
    ref.close(got.masked_fill(beyond, 0.0), want, want.abs() * 2.0 ** -8 + slack, "dh")


@pytest.mark.parametrize("rows,n", [(2 ** 31 // 8192 + 300, 8192), (2 ** 22 + 77, 8), (2 ** 20 + 5, 512), (4099, 32768),
                                    (1025, 64), (77, 1024)])
def test_dgamma_of_many_rows_is_exact(rows, n):
    """h of +-1 with eps 0 has rho 1 (n a power of two), so dgamma is the sum
    of dy h: whole numbers from 1 to 3 whose sums stay below 2^24, exact in
    fp32 in whatever order.  A row, a workgroup's share or a slice that is
    lost, repeated or added to another column shows."""
    dev = device()
    i = torch.arange(rows, device=dev, dtype=torch.int32)
    j = torch.arange(n, device=dev, dtype=torch.int32)
    h, dy = torch.empty(rows, n, dtype=BF, device=dev), torch.empty(rows, n, dtype=BF, device=dev)
    want = torch.zeros(n, dtype=torch.int64, device=dev)
    step = max(1, 2 ** 27 // n)
    for first in range(0, rows, step):
        r = i[first:first + step, None]
        sign = 1 - 2 * ((r * 5 + j * 3 + r // 7) % 2)
        term = (r * 7 + j + r // 11) % 3 + 1
        h[first:first + step] = sign.to(BF)
        dy[first:first + step] = (term * sign).to(BF)
        want += term.sum(0, dtype=torch.int64)
    assert int(want.max()) < 2 ** 24
    gamma = (j % 5 + 1).to(BF)
    say("dgamma of many rows", rows, n)
    dx, dgamma = gg.rmsnorm_grad(dy, h, gamma, eps=0.0)
    torch.cuda.synchronize()
    assert torch.equal(dgamma.double(), want.double())
    # dx = p - u mean(p u), the mean of whole numbers from 1 to 15 summed exactly: one product, one
    # difference and half a bf16 step
    pick = torch.cat([torch.arange(min(rows, 8)), torch.arange(max(rows - 8, 0), rows)]).to(dev)
    wx, _, _, _ = ref.rmsnorm_grad(dy[pick], h[pick], gamma, None, 0.0)
    ref.close(dx[pick], wx, wx.abs() * 2.0 ** -8 + 15 * 4 * ref.U32, "dx")
