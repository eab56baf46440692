"""GPU tests of the weight gradient from e4m3 activations (gg_fp8_wgrad,
gg_fp8_masked_wgrad): against the fp64 oracle on the values the codes stand
for, and bit for bit against the bf16 wgrad of those values (bf16 holds them
exactly, and the two run the same matrix instructions in the same order)."""
import numpy as np
import pytest
import torch

import oracle
import layer_ref as ref
from moe_grouped_gemm_ragged_amd import binding as gg
from moe_grouped_gemm_ragged_amd import synth
from gpu_util import device, host, say
from parity import check

pytestmark = pytest.mark.gpu
BF, U8 = torch.bfloat16, torch.uint8


def operands(sizes, k, n, seed, spare=0, max_m=None, spread=1.0):
    """e4m3 rows, packed scales, the rows' values as bf16 and dY; NaN wherever
    no expert owns a row.  sizes: rows of each expert (masked: active rows)."""
    dev = device()
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    e = len(sizes)
    total = e * max_m if max_m else int(sum(sizes)) + spare
    x = torch.randn(total, k, generator=g, device=dev) * torch.exp(
        spread * torch.randn(total, k // 128, generator=g, device=dev)).repeat_interleave(128, dim=1)
    codes, scales = (t.cuda() for t in ref.quantise(x.to(BF).cpu()))
    values = ref.value(codes, scales)
    xb = values.to(BF).cuda()
    assert torch.equal(xb.cpu().double(), values), "the values are not exact in bf16"
    dy = torch.randn(total, n, generator=g, device=dev).to(BF)
    row = torch.arange(total, device=dev)
    if max_m:
        groups = torch.tensor(sizes, dtype=torch.int32, device=dev)
        live = row % max_m < groups[row // max_m]
    else:
        groups = torch.tensor(np.cumsum(sizes), dtype=torch.int32, device=dev)
        live = row < groups[-1]
    codes[~live], dy[~live], xb[~live], scales[~live] = 0x7F, float("nan"), float("nan"), 255
    layout = gg.GG_FP8_ACT_MASKED if max_m else gg.GG_FP8_ACT_RAGGED
    packed = gg.fp8_pack_scales(layout, scales.contiguous(), groups, max_m or total, k, e)
    if max_m:
        codes, dy, xb = (t.reshape(e, max_m, -1) for t in (codes, dy, xb))
    return codes, packed, dy, groups, xb


def run(masked, codes, packed, dy, groups, **kw):
    return (gg.fp8_masked_wgrad if masked else gg.fp8_wgrad)(codes, packed, dy, groups, **kw)


def bf16(masked, xb, dy, groups, **kw):
    return (gg.masked_wgrad if masked else gg.wgrad)(xb, dy, groups, **kw)


CASES = [([1], 128, 8, 0, None), ([300, 0, 17, 256, 1, 33], 256, 264, 5, None), ([31, 32, 33, 95, 97, 129], 384, 136, 0, None),
         ([0, 0, 0], 128, 16, 9, None), ([2500, 5], 640, 512, 3, None), ([64, 128, 160, 192], 256, 256, 0, None),
         ([0, 8, 64, 41], 256, 136, 0, 64), ([600, 257, 1, 0], 128, 520, 0, 600)]


@pytest.mark.parametrize("sizes,k,n,spare,max_m", CASES)
@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_fp8_wgrad(sizes, k, n, spare, max_m, dtype):
    codes, packed, dy, groups, xb = operands(sizes, k, n, len(sizes) * k + n, spare, max_m)
    masked = max_m is not None
    say("fp8_wgrad", sizes, k, n, max_m, dtype)
    dw = run(masked, codes, packed, dy, groups, out_dtype=dtype)
    again = run(masked, codes, packed, dy, groups, out_dtype=dtype)
    want = bf16(masked, xb, dy, groups, out_dtype=dtype)
    torch.cuda.synchronize()
    assert torch.equal(dw.view(U8), again.view(U8)), "two calls differ"
    assert torch.equal(dw.view(U8), want.view(U8)), "not the bf16 wgrad of the same values"
    rows = np.asarray(sizes)
    if masked:
        r = oracle.masked_wgrad(synth.bf16_bits(xb), synth.bf16_bits(dy), groups.cpu().numpy())
    else:
        r = oracle.wgrad(synth.bf16_bits(xb), synth.bf16_bits(dy), groups.cpu().numpy())
    L = np.repeat(np.maximum(rows, 1), k)[:, None]
    check(host(dw).reshape(-1, n), r.value, r.sabs, L, f"fp8_wgrad {sizes} {k} {n}")
    for e, count in enumerate(sizes):
        if not count:
            assert bool((dw[e].view(U8) == 0).all()), "an empty expert's dW is not +0"


def test_fp8_wgrad_long_experts_of_every_epilogue():
    """Experts of 2048 rows and more (several tiles a workgroup), more than 512
    experts, and accumulation; every epilogue goes through LDS."""
    for sizes, k, n in (([4100, 2049, 3000], 4096, 2048), ([40] * 520, 256, 256)):
        codes, packed, dy, groups, xb = operands(sizes, k, n, k)
        say("fp8_wgrad", len(sizes), k, n)
        assert torch.equal(run(False, codes, packed, dy, groups), bf16(False, xb, dy, groups))
        for dtype in (torch.float32, BF):
            start = torch.randn(len(sizes), k, n, device="cuda").to(dtype)
            a = run(False, codes, packed, dy, groups, out=start.clone(), alpha=0.5, beta=1.0)
            b = bf16(False, xb, dy, groups, out=start.clone(), alpha=0.5, beta=1.0)
            torch.cuda.synchronize()
            assert torch.equal(a, b), dtype


@pytest.mark.parametrize("experts", [1, 4, 31])
def test_fp8_wgrad_bad_offsets(experts):
    """Offsets that fall, are negative or pass the rows are clamped as the
    packed scales' and the GEMMs' are."""
    codes, packed, dy, groups, xb = operands([37] * experts, 256, 136, experts)
    rng = np.random.default_rng(experts)
    offs = torch.from_numpy(rng.integers(-50, 60 * experts, size=experts).astype(np.int32)).cuda()
    _, scales = ref.quantise(xb.cpu())
    # the codes' own scales, packed again for these offsets: blocks of values are unchanged
    packed = gg.fp8_pack_scales(gg.GG_FP8_ACT_RAGGED, scales.cuda(), offs, xb.shape[0], 256, experts)
    codes2, _ = ref.quantise(xb.cpu())
    say("fp8_wgrad with bad offsets", experts)
    dw = gg.fp8_wgrad(codes2.cuda(), packed, dy, offs)
    want = gg.wgrad(xb, dy, offs)
    torch.cuda.synchronize()
    assert torch.equal(dw, want)


def test_fp8_wgrad_scales_of_all_sizes():
    """Scales far apart within a stage, from about 2^-60 to 2^75."""
    codes, packed, dy, groups, xb = operands([200, 77], 256, 64, 3, spread=12.0)
    say("fp8_wgrad with scales far apart")
    assert torch.equal(run(False, codes, packed, dy, groups), bf16(False, xb, dy, groups))


def test_fp8_wgrad_in_a_graph():
    codes, packed, dy, groups, xb = operands([300, 0, 77, 1000], 384, 264, 5)
    out = torch.zeros(4, 384, 264, device="cuda")
    gg.fp8_wgrad(codes, packed, dy, groups, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    say("fp8_wgrad in a graph")
    with torch.cuda.graph(graph):
        gg.fp8_wgrad(codes, packed, dy, groups, out=out)
    for trial in range(3):
        dy.copy_(torch.randn_like(dy.float()).to(BF))
        want = gg.fp8_wgrad(codes, packed, dy, groups)
        out.fill_(5)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), trial


def test_fp8_wgrad_without_rows():
    """No rows at all (and so no memory behind x, its scales and dY): dW is 0,
    or what beta leaves of it."""
    dev = device()
    groups = torch.zeros(5, dtype=torch.int32, device=dev)
    say("fp8_wgrad without rows")
    for masked in (False, True):
        lead = (5, 0) if masked else (0,)
        x, dy = torch.empty(*lead, 384, dtype=U8, device=dev), torch.empty(*lead, 72, dtype=BF, device=dev)
        scales = torch.empty(gg.fp8_scale_bytes(gg.GG_FP8_ACT_MASKED if masked else gg.GG_FP8_ACT_RAGGED, 0, 384, 5),
                             dtype=U8, device=dev)
        for dtype in (torch.float32, BF):
            out = torch.full((5, 384, 72), 3.0, dtype=dtype, device=dev)
            run(masked, x, scales, dy, groups, out=out)
            assert bool((out == 0).all())
            out.fill_(3.0)
            run(masked, x, scales, dy, groups, out=out, beta=0.5)
            assert bool((out == 1.5).all())


@pytest.mark.parametrize("sizes,k,n,max_m", [([300, 0, 70], 384, 200, None), ([600, 0, 257], 256, 512, 640)])
@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_fp8_wgrad_output_off_the_cache_lines(sizes, k, n, max_m, dtype):
    """An output that begins 16 bytes into a line, overwritten and
    accumulated into; what lies before and behind it stays."""
    codes, packed, dy, groups, xb = operands(sizes, k, n, n, 0, max_m)
    masked, e = max_m is not None, len(sizes)
    pad = 16 // (torch.finfo(dtype).bits // 8)
    whole = torch.randn(e * k * n + 2 * pad, device="cuda").to(dtype)
    before = whole.clone()
    out = whole[pad:-pad].view(e, k, n)
    assert out.data_ptr() % 128 == 16 and out.is_contiguous()
    say("fp8_wgrad off the lines", sizes, k, n, dtype)
    run(masked, codes, packed, dy, groups, out=out, alpha=0.5, beta=1.0)
    want = bf16(masked, xb, dy, groups, out=before[pad:-pad].view(e, k, n).clone(), alpha=0.5, beta=1.0)
    assert torch.equal(out, want)
    run(masked, codes, packed, dy, groups, out=out)
    assert torch.equal(out, bf16(masked, xb, dy, groups, out_dtype=dtype))
    assert torch.equal(run(masked, codes, packed, dy, groups, out_dtype=dtype), out), "and on the lines"
    assert torch.equal(whole[:pad], before[:pad]) and torch.equal(whole[-pad:], before[-pad:])
