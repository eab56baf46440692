"""One training step of an MoE layer that keeps its activations in 8 bits,
through the library alone: norm -> e4m3 rows -> sorted by expert -> fp8
gate/up -> SiLU-mul with kept rows -> fp8 down -> weighted combine, and back:
combine gradient -> dgrad and dW of the down projection -> SiLU-mul gradient
from the kept rows -> dgrad and dW of the gate/up projection from the kept
operand -> rows back to tokens -> norm gradient.  Each stage is checked
against its fp64 form on what the stage before wrote."""
import numpy as np
import pytest
import torch

import oracle
import layer_ref as ref
from moe_grouped_gemm_ragged_amd import binding as gg
from moe_grouped_gemm_ragged_amd import synth
from gpu_util import device, host, say
from parity import check, check_fp8

pytestmark = pytest.mark.gpu
BF, U8 = torch.bfloat16, torch.uint8


def weights(g, e, n, k):
    """e4m3 weights [E, n, k] with scales: (codes, bytes, packed, bf16 values)."""
    codes, scales = (t.cuda() for t in ref.quantise((torch.randn(e, n, k, generator=g, device="cuda") * 0.05).to(BF).cpu()))
    packed = gg.fp8_pack_scales(gg.GG_FP8_WEIGHT, scales, None, n, k, e)
    return codes, scales, packed, ref.value(codes, scales).to(BF).cuda()


def f32_scales(b):
    return torch.pow(2.0, b.cpu().double() - 127).float().numpy()


@pytest.mark.parametrize("tokens,topk,e,k,i", [(150, 4, 8, 384, 256), (1, 2, 4, 128, 128)])
def test_layer_step_in_8_bits(tokens, topk, e, k, i):
    dev = device()
    g = torch.Generator(device=dev)
    g.manual_seed(tokens)
    x = torch.randn(tokens, k, generator=g, device=dev).to(BF)
    r = torch.randn(tokens, k, generator=g, device=dev).to(BF)
    gamma = (1 + 0.2 * torch.randn(k, generator=g, device=dev)).to(BF)
    ids = torch.rand(tokens, e, generator=g, device=dev).topk(topk, dim=1).indices.to(torch.int32)
    probs = torch.rand(tokens, topk, generator=g, device=dev)
    dout = torch.randn(tokens, k, generator=g, device=dev).to(BF)
    dres = torch.randn(tokens, k, generator=g, device=dev).to(BF)
    w13, w13s, w13p, w13b = weights(g, e, 2 * i, k)
    w2, w2s, w2p, w2b = weights(g, e, k, i)
    eps = 1e-5

    say("layer step, forward", tokens, topk, e, k, i)
    x8, x8s, h = gg.fp8_rmsnorm(x, gamma, residual=r, eps=eps)
    offs, row_slot, slot_row = gg.route(ids.contiguous(), e, 8, True)
    xg, xgp = gg.fp8_gather_rows(x8, x8s, row_slot, topk, offs)
    gu = gg.fp8_forward(xg, xgp, w13, w13p, offs)
    a8, a8s, gu8, gu8s = gg.fp8_silu_mul_rows(gu, offs, keep=True)
    ap = gg.fp8_pack_scales(gg.GG_FP8_ACT_RAGGED, a8s, offs, a8.shape[0], i, e)
    y = gg.fp8_forward(a8, ap, w2, w2p, offs)
    out = gg.combine_rows(y, slot_row, topk, probs)
    say("layer step, backward", tokens, topk, e, k, i)
    dy, dprobs = gg.combine_rows_grad(dout, y, slot_row, row_slot, offs, topk, weights=probs)
    da = gg.dgrad_nk(dy, w2b, offs)
    dw2 = gg.fp8_wgrad(a8, ap, dy, offs)
    dgu = gg.fp8_silu_mul_grad(da, gu8, gu8s, offs)
    dw13 = gg.fp8_wgrad(xg, xgp, dgu, offs)
    dxg = gg.dgrad_nk(dgu, w13b, offs)
    dnorm = gg.combine_rows(dxg, slot_row, topk)
    dx, dgamma = gg.rmsnorm_grad(dnorm, h, gamma, dh=dres, eps=eps)
    torch.cuda.synchronize()

    used = int(offs[-1])
    slots = row_slot[:used].cpu().long()
    there = slots >= 0
    ends = offs.cpu().numpy()
    # forward
    want, hw = ref.rmsnorm(x, r, gamma, eps)
    ref.close8(x8, x8s, want, ref.rmsnorm_slack(want, k), "norm")
    ref.close(h, hw, hw.abs() * (2.0 ** -8 + 2.0 ** -24), "h")
    rows = torch.zeros(used, k, dtype=U8)
    rows[there] = x8.cpu()[slots[there] // topk]
    scales = torch.full((used, k // 128), 127, dtype=U8)
    scales[there] = x8s.cpu()[slots[there] // topk]
    assert torch.equal(xg[:used].cpu(), rows)
    f = oracle.fp8_forward(rows.numpy(), f32_scales(scales), w13.cpu().numpy(), f32_scales(w13s), ends)
    check_fp8(host(gu[:used]), f.value, f.sabs, k, "gate/up")
    hv = ref.f64(gu[:used])
    av, slack = ref.silu_mul(hv)
    ref.close8(a8[:used], a8s[:used], av, slack, "activation")
    codes, bytes_ = ref.quantise(gu[:used].cpu())
    assert torch.equal(gu8[:used].cpu(), codes) and torch.equal(gu8s[:used].cpu(), bytes_)
    f = oracle.fp8_forward(a8[:used].cpu().numpy(), f32_scales(a8s[:used]), w2.cpu().numpy(), f32_scales(w2s), ends)
    check_fp8(host(y[:used]), f.value, f.sabs, i, "down")
    c = oracle.combine_rows(host(y), slot_row.cpu().numpy(), topk, probs.cpu().numpy())
    check(host(out), c.value, c.sabs, topk, "combine")
    # backward
    d, row = ref.f64(dout), slot_row.cpu().long().reshape(tokens, topk)
    want = torch.zeros(used, k, dtype=torch.float64)
    want[there] = ref.f64(probs).reshape(-1)[slots[there]][:, None] * d[slots[there] // topk]
    ref.close(dy[:used], want, want.abs() * (2.0 ** -8 + 2.0 ** -23), "dy")
    terms = ref.f64(y)[row] * d[:, None, :]
    ref.close(dprobs, terms.sum(-1), terms.abs().sum(-1) * (k + 2) * ref.U32, "dprobs")
    f = oracle.dgrad_nk(host(dy[:used]), host(w2b), ends)
    check(host(da[:used]), f.value, f.sabs, k, "da")
    sizes = np.diff(ends, prepend=0)
    for name, got, codes, bytes_, dd in (("dW2", dw2, a8, a8s, dy), ("dW13", dw13, rows, scales, dgu)):
        v = ref.value(codes[:used].cpu(), bytes_[:used].cpu()).to(BF)
        f = oracle.wgrad(synth.bf16_bits(v), host(dd[:used]), ends)
        L = np.repeat(np.maximum(sizes, 1), got.shape[1])[:, None]
        check(host(got).reshape(-1, got.shape[2]), f.value, f.sabs, L, name)
    kept = ref.value(gu8[:used].cpu(), gu8s[:used].cpu())
    want, slack = ref.silu_mul_grad(ref.f64(da[:used]), kept)
    ref.close(dgu[:used], want, want.abs() * 2.0 ** -8 + slack, "d gate/up")
    f = oracle.dgrad_nk(host(dgu[:used]), host(w13b), ends)
    check(host(dxg[:used]), f.value, f.sabs, 2 * i, "dx grouped")
    c = oracle.combine_rows(host(dxg), slot_row.cpu().numpy(), topk)
    check(host(dnorm), c.value, c.sabs, topk, "d norm")
    wx, slack, wg, slack_g = ref.rmsnorm_grad(dnorm, h, gamma, dres, eps)
    ref.close(dx, wx, wx.abs() * 2.0 ** -8 + slack, "dx")
    ref.close(dgamma, wg, slack_g, "dgamma")


def test_masked_step_in_8_bits():
    """The same between the GEMMs on the masked layout: kept rows, the fp8
    down projection and both gradients, inactive rows untouched throughout."""
    dev = device()
    g = torch.Generator(device=dev)
    g.manual_seed(7)
    e, max_m, i, n = 6, 48, 128, 136
    masked_m = torch.tensor([0, 48, 1, 17, 33, 8], dtype=torch.int32, device=dev)
    live = torch.arange(max_m, device=dev)[None, :] < masked_m[:, None]
    gu = torch.randn(e, max_m, 2 * i, generator=g, device=dev).to(BF)
    dy = torch.randn(e, max_m, n, generator=g, device=dev).to(BF)
    gu[~live], dy[~live] = float("nan"), float("nan")
    w2, w2s, w2p, w2b = weights(g, e, n, i)
    say("masked step")
    a8, a8s, gu8, gu8s = gg.fp8_silu_mul_rows(gu, masked_m, masked=True, keep=True)
    ap = gg.fp8_pack_scales(gg.GG_FP8_ACT_MASKED, a8s, masked_m, max_m, i, e)
    y = gg.fp8_masked_forward(a8, ap, w2, w2p, masked_m)
    da = gg.masked_dgrad(dy, w2b.transpose(1, 2).contiguous(), masked_m)
    dw2 = gg.fp8_masked_wgrad(a8, ap, dy, masked_m)
    dgu = torch.full((e, max_m, 2 * i), 7.0, dtype=BF, device=dev)
    gg.fp8_silu_mul_grad(da, gu8, gu8s, masked_m, masked=True, out=dgu)
    torch.cuda.synchronize()
    rows = live.cpu().reshape(-1).numpy()
    f = oracle.fp8_masked_forward(a8.cpu().numpy(), f32_scales(a8s), w2.cpu().numpy(), f32_scales(w2s),
                                  masked_m.cpu().numpy())
    check_fp8(host(y).reshape(-1, n)[rows], f.value[rows], f.sabs[rows], i, "masked down")
    av = torch.zeros(e, max_m, i, dtype=torch.float64)
    av[live.cpu()] = ref.value(a8[live], a8s[live])
    f = oracle.masked_wgrad(synth.bf16_bits(av.to(BF)), host(dy), masked_m.cpu().numpy())
    L = np.repeat(np.maximum(masked_m.cpu().numpy(), 1), i)[:, None]
    check(host(dw2).reshape(-1, n), f.value, f.sabs, L, "masked dW2")
    want, slack = ref.silu_mul_grad(ref.f64(da[live]), ref.value(gu8[live], gu8s[live]))
    ref.close(dgu[live], want, want.abs() * 2.0 ** -8 + slack, "masked d gate/up")
    assert bool((dgu[~live] == 7.0).all())
