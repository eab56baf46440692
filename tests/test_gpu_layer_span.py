"""GPU tests of the layer steps where an operand passes 4 GB and 2^31 elements,
or has more rows than a launch has workgroups:
the last rows (and a sample of the others) against the plain fp64 forms, or,
where the operator only moves bytes, all of them; dW from 8-bit rows against
exact integers."""
import pytest
import torch

import layer_ref as ref
from moe_grouped_gemm_ragged_amd import binding as gg
from gpu_util import device, say

pytestmark = pytest.mark.gpu
BF, U8 = torch.bfloat16, torch.uint8
N = 8192
ROWS = 2 ** 31 // N + 300


def fill(*shape):
    return torch.empty(*shape, dtype=BF, device=device()).normal_()


def sample(rows):
    """The first, the last and some other rows."""
    g = torch.Generator().manual_seed(rows)
    return torch.cat([torch.tensor([0, rows // 2]), torch.randint(0, rows, (20,), generator=g),
                      torch.arange(rows - 20, rows)]).cuda()


def test_norm_and_gradient_over_4gb():
    x, gamma = fill(ROWS, N), fill(N)
    pick = sample(ROWS)
    say("fp8_rmsnorm over 4 GB")
    codes, scales, _, y = gg.fp8_rmsnorm(x, gamma, with_bf16=True)
    want, _ = ref.rmsnorm(x[pick], None, gamma, 1e-6)
    ref.close(y[pick], want, want.abs() * 2.0 ** -8 + ref.rmsnorm_slack(want, N), "y")
    ref.close8(codes[pick], scales[pick], want, ref.rmsnorm_slack(want, N), "y8")
    del codes, scales
    say("rmsnorm_grad over 4 GB")
    dx, dgamma = gg.rmsnorm_grad(y, x, gamma)
    want, slack, _, _ = ref.rmsnorm_grad(y[pick], x[pick], gamma, None, 1e-6)
    ref.close(dx[pick], want, want.abs() * 2.0 ** -8 + slack, "dx")
    total, size = torch.zeros(N, dtype=torch.float64, device="cuda"), torch.zeros(N, dtype=torch.float64, device="cuda")
    for first in range(0, ROWS, 8192):
        h = x[first:first + 8192].double()
        t = y[first:first + 8192].double() * h / torch.sqrt(h.square().mean(-1, keepdim=True) + 1e-6)
        total += t.sum(0)
        size += t.abs().sum(0)
    # the bound of layer_ref.rmsnorm_grad, whose sum runs over all rows
    ref.close(dgamma, total.cpu(), total.cpu().abs() * 2.0 ** -24 + size.cpu() * (ROWS + N / 2 + 16) * ref.U32, "dgamma")


@pytest.mark.parametrize("rows,n", [(2 ** 22 + 77, 8), (2 ** 20 + 5, 520)])
def test_norm_of_more_rows_than_workgroups(rows, n):
    """A launch has at most 2^20 workgroups (of four rows, where rows are
    short): the last rows are a workgroup's second."""
    x, r, gamma = fill(rows, n), fill(rows, n), fill(n)
    pick = sample(rows)
    say("rmsnorm of many rows", rows, n)
    y, h = gg.rmsnorm(x, gamma, residual=r)
    want, hw = ref.rmsnorm(x[pick], r[pick], gamma, 1e-6)
    ref.close(y[pick], want, want.abs() * 2.0 ** -8 + ref.rmsnorm_slack(want, n), "y")
    ref.close(h[pick], hw, hw.abs() * (2.0 ** -8 + 2.0 ** -24), "h")
    dx, _ = gg.rmsnorm_grad(y, h, gamma)
    want, slack, _, _ = ref.rmsnorm_grad(y[pick], h[pick], gamma, None, 1e-6)
    ref.close(dx[pick], want, want.abs() * 2.0 ** -8 + slack, "dx")


def test_combine_gradient_of_more_tokens_than_workgroups():
    dev = device()
    tokens, n, e = 2 ** 20 + 33, 8, 7
    expert = torch.randint(0, e, (tokens, 1), device=dev, dtype=torch.int32)
    offs, row_slot, slot_row = gg.route(expert, e)
    dout, y = fill(tokens, n), fill(row_slot.shape[0], n)
    w = torch.rand(tokens, 1, device=dev)
    say("combine_rows_grad of many tokens")
    dy, dw = gg.combine_rows_grad(dout, y, slot_row, row_slot, offs, 1, weights=w)
    slot = row_slot[:tokens].long()
    assert int(offs[-1]) == tokens
    assert torch.equal(dy[:tokens], (dout[slot].float() * w[slot]).to(BF))
    part = y[slot_row.long()].double() * dout.double()
    want = part.sum(-1).cpu()[:, None]
    ref.close(dw, want, want.abs() * 2.0 ** -24 + part.abs().sum(-1).cpu()[:, None] * n * ref.U32, "dw")


def test_silu_rows_over_4gb():
    h, pick = fill(ROWS, N), sample(ROWS)
    offs = torch.tensor([7, 7, ROWS - 100, ROWS], dtype=torch.int32, device="cuda")
    say("fp8_silu_mul_rows over 4 GB")
    a8, a8s, kept, kept_scales = gg.fp8_silu_mul_rows(h, offs, keep=True)
    want, slack = ref.silu_mul(ref.f64(h[pick]))
    ref.close8(a8[pick], a8s[pick], want, slack, "a8")
    codes, scales = ref.quantise(h[pick].cpu())
    assert torch.equal(kept[pick].cpu(), codes) and torch.equal(kept_scales[pick].cpu(), scales)
    da = fill(ROWS, N // 2)
    for back in (None, kept_scales):
        say("silu_mul_grad over 4 GB", back is not None)
        if back is None:
            dh, act = gg.silu_mul_grad(da, h, offs, with_act=True)
            hv = ref.f64(h[pick])
        else:
            dh, act = gg.fp8_silu_mul_grad(da, kept, kept_scales, offs, with_act=True)
            hv = ref.value(codes, scales)
        want, slack = ref.silu_mul_grad(ref.f64(da[pick]), hv)
        ref.close(dh[pick], want, want.abs() * 2.0 ** -8 + slack, "dh")
        want, slack = ref.silu_mul(hv)
        ref.close(act[pick], want, want.abs() * 2.0 ** -8 + slack, "act")


def test_rows_to_experts_and_back_over_4gb():
    dev = device()
    tokens, topk, e = 2 ** 31 // N + 100, 2, 24                # 2^32 values, twice the tokens' bytes
    expert = torch.randint(0, e, (tokens, topk), device=dev, dtype=torch.int32)
    offs, row_slot, slot_row = gg.route(expert, e, 8)
    used = int(offs[-1])
    src = torch.randint(0, 256, (tokens, N), device=dev, dtype=U8)
    scales = torch.randint(1, 255, (tokens, N // 128), device=dev, dtype=U8)
    say("fp8_gather_rows over 4 GB")
    out, packed = gg.fp8_gather_rows(src, scales, row_slot, topk, offs)
    slot = row_slot[:used].long()
    for first in range(0, used, 1 << 16):
        s = slot[first:first + (1 << 16)]
        want = src[s.clamp(min=0) // topk] * (s >= 0).to(U8)[:, None]
        assert torch.equal(out[first:first + (1 << 16)][:want.shape[0]], want), first
    raw = torch.where((slot >= 0)[:, None], scales[slot.clamp(min=0) // topk],
                      torch.full((1, 1), 127, dtype=U8, device=dev))
    same = gg.fp8_pack_scales(gg.GG_FP8_ACT_RAGGED, raw.contiguous(), offs, used, N, e)
    tiles = int(((torch.diff(offs.long(), prepend=offs.new_zeros(1).long()) + 255) // 256).sum())
    assert torch.equal(packed[:tiles * (N // 128) * 256], same[:tiles * (N // 128) * 256])
    del src, out, packed, raw, same
    say("combine_rows_grad over 4 GB")
    dout, y = fill(tokens, N), fill(row_slot.shape[0], N)
    w = torch.rand(tokens, topk, device=dev)
    dy, dw = gg.combine_rows_grad(dout, y, slot_row, row_slot, offs, topk, weights=w)
    for first in range(0, used, 1 << 15):
        s = slot[first:first + (1 << 15)]
        at = s.clamp(min=0)
        # one fp32 product and its rounding to bf16: the same bits
        want = (dout[at // topk].float() * w.reshape(-1)[at][:, None] * (s >= 0)[:, None]).to(BF)
        assert bool((dy[first:first + (1 << 15)][:want.shape[0]] == want).all()), first
    pick = sample(tokens)
    rows = slot_row.reshape(tokens, topk)[pick].long()
    assert bool((rows >= 0).all())
    part = y[rows].double() * dout[pick].double()[:, None]
    want, size = part.sum(-1).cpu(), part.abs().sum(-1).cpu()
    ref.close(dw[pick], want, want.abs() * 2.0 ** -24 + size * N * ref.U32, "dw")


@pytest.mark.parametrize("masked,dtype", [(False, torch.float32), (False, BF), (True, torch.float32)])
def test_fp8_wgrad_expert_over_4gb(masked, dtype):
    """Small integers of period 3 (x: -1, 0, 1) and 5 (dY: -2 .. 2) in the
    rows: every sum is an integer below 2^24 known from the residues, so no
    row of the reduction is lost, repeated or misplaced unseen."""
    dev = device()
    k, n, rows = 256, N, 2 ** 32 // (2 * N) + 200                # dY of one expert alone passes 4 GB
    sizes = [rows] if masked else [40, rows]
    total = sum(sizes)
    code = torch.tensor([0xB8, 0, 0x38], dtype=torch.int64, device=dev)      # -1, 0, 1 in e4m3
    i, kk, j = (torch.arange(v, device=dev) for v in (total, k, n))
    x = code[(i[:, None] + kk) % 3].to(U8)
    dy = (torch.arange(5, device=dev)[:, None] * 7 + j).remainder(5).sub(2).to(BF)[i % 5]
    groups = torch.tensor(sizes if masked else [40, total], dtype=torch.int32, device=dev)
    e = len(sizes)
    layout = gg.GG_FP8_ACT_MASKED if masked else gg.GG_FP8_ACT_RAGGED
    packed = gg.fp8_pack_scales(layout, torch.full((total, k // 128), 127, dtype=U8, device=dev), groups, total, k, e)
    say("fp8_wgrad over 4 GB", masked, dtype)
    if masked:
        dw = gg.fp8_masked_wgrad(x[None], packed, dy[None], groups, out_dtype=dtype)
    else:
        dw = gg.fp8_wgrad(x, packed, dy, groups, out_dtype=dtype)
    first = 0
    for g, count in enumerate(sizes):
        want = torch.zeros(k, n, dtype=torch.int64, device=dev)
        r = torch.arange(first, first + count, device=dev)
        for c in range(15):
            xs, ds = (c + kk) % 3 - 1, (7 * (c % 5) + j) % 5 - 2
            want += int((r % 15 == c).sum()) * xs[:, None] * ds[None, :]
        assert int(want.abs().max()) < 2 ** 24
        assert torch.equal(dw[g], want.float().to(dtype)), g
        first += count
