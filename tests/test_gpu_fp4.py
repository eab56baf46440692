"""4-bit rows on the GPU: quantisation in every layout against 64 bits (codes
and packed scales equal), back to bf16, gather, SiLU-mul, and the grouped
product with its unused rows and columns."""
import pytest
import torch

import fp4_ref as ref
import layer_ref
from moe_grouped_gemm_ragged_amd import binding as gg
from gpu_util import device, say, sentinel_tensor

pytestmark = pytest.mark.gpu
BF, U8, I32 = torch.bfloat16, torch.uint8, torch.int32
RAGGED, MASKED, WEIGHT = gg.GG_FP4_ACT_RAGGED, gg.GG_FP4_ACT_MASKED, gg.GG_FP4_WEIGHT
FILL = 0xA5

# (layout, groups, rows, experts): experts without rows, one row, whole tiles and one more, offsets
# that go down or past the rows, counts below 0 and past the rows
LAYOUTS = [
    (RAGGED, [1, 1, 130, 130 + 256, 700], 700, 5),
    (RAGGED, [5, 3, 400, 200, 9999], 613, 5),
    (RAGGED, [0, 0, 0], 64, 3),
    (RAGGED, [-4, 31, 32], 33, 3),
    (MASKED, [0, 7, 300, 1, -3, 9999], 300, 6),
    (MASKED, [1, 0], 1, 2),
    (MASKED, [256, 129, 128], 256, 3),
    (WEIGHT, None, 264, 3),
    (WEIGHT, None, 1, 2),
]


def rows_of(layout, rows, experts, width):
    return (rows, width) if layout == RAGGED else (experts, rows, width)


def groups_of(groups, dev):
    return None if groups is None else torch.tensor(groups, dtype=I32, device=dev)


def spread(g, *shape):
    """Normal values whose blocks of 32 are of very different sizes."""
    b = torch.randn(*shape[:-1], shape[-1] // 32, 32, generator=g)
    return (b * torch.exp2(torch.randint(-20, 20, b.shape[:-1], generator=g).float())[..., None]).reshape(shape)


@pytest.mark.parametrize("layout,groups,rows,experts", LAYOUTS)
@pytest.mark.parametrize("k", [32, 160, 256, 416])
def test_quantize(layout, groups, rows, experts, k):
    dev, g = device(), torch.Generator().manual_seed(k + rows)
    x = spread(g, *rows_of(layout, rows, experts, k)).to(BF)
    who = ref.owned(layout, groups, rows, experts)
    x.reshape(-1, k)[who < 0] = float("nan")
    codes = torch.full((*x.shape[:-1], k // 2), FILL, dtype=U8, device=dev)
    scales = torch.full((gg.fp4_scale_bytes(layout, rows, k, experts),), FILL, dtype=U8, device=dev)
    say("fp4 quantize", layout, groups, rows, k)
    gg.fp4_quantize(layout, x.to(dev), groups_of(groups, dev), out=codes, out_scales=scales)
    torch.cuda.synchronize()
    c, b = ref.quantise(x.float())
    want = ref.pack(c).reshape(-1, k // 2)
    want[who < 0] = FILL
    assert torch.equal(codes.cpu().reshape(-1, k // 2), want)
    want = ref.packed_scales(b, layout, groups, rows, experts, FILL)
    assert torch.equal(scales.cpu(), want)


def test_quantize_special_blocks():
    """Zeros of both signs, ties at every border, the largest and smallest
    values, infinities and NaN: their block alone is NaN."""
    dev = device()
    inf, nan = float("inf"), float("nan")
    ties = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, -6.0]
    near = [v * f for v in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0) for f in (1 - 2.0 ** -8, 1 + 2.0 ** -7)]
    blocks = [[0.0] * 32, [-0.0] * 32, ties + [0.0] * 16, near + [6.0] + [-0.0] * 17]
    for s in (2.0 ** -126, 2.0 ** -100, 2.0 ** 40, 2.0 ** 125):
        blocks += [[v * s for v in ties] + [0.0] * 16, [v * s for v in near] + [6.0 * s] + [0.0] * 17]
    blocks += [[2.0 ** -133] + [0.0] * 31, [2.0 ** -127, -(2.0 ** -128)] * 16, [3.3895e38, -3.3895e38] * 16,
               [6.0] * 31 + [6.03125], [1.0] * 31 + [inf], [-inf] + [2.0] * 31, [0.0] * 15 + [nan] + [3.0] * 16,
               [inf, nan] * 16, [1.0] * 32]
    for place in (0, 31):
        b = [0.5] * 32
        b[place] = nan
        blocks.append(b)
    while len(blocks) % 4:
        blocks.append([1.0] * 32)
    x = torch.tensor(blocks, dtype=torch.float64).to(BF).reshape(-1, 128)
    say("fp4 special blocks", tuple(x.shape))
    codes, scales = gg.fp4_quantize(WEIGHT, x[None].to(dev))
    back = gg.fp4_dequantize(WEIGHT, codes, scales)
    torch.cuda.synchronize()
    c, b = ref.quantise(x.float())
    bad = [(i, blocks[i][:4]) for i in range(len(blocks))
           if not torch.equal(ref.pack(c).reshape(-1, 16)[i], codes.cpu().reshape(-1, 16)[i])]
    assert not bad, bad
    assert torch.equal(scales.cpu(), ref.packed_scales(b, WEIGHT, None, x.shape[0], 1, 0))
    want = ref.value(ref.pack(c), b).to(BF)
    assert torch.equal(torch.isnan(back.cpu()[0]), torch.isnan(want))
    assert torch.equal(back.cpu()[0].nan_to_num(7.0), want.nan_to_num(7.0))


@pytest.mark.parametrize("layout,groups,rows,experts", LAYOUTS)
def test_dequantize(layout, groups, rows, experts):
    dev, g, k = device(), torch.Generator().manual_seed(rows), 288
    shape = rows_of(layout, rows, experts, k)
    codes = torch.randint(0, 256, (*shape[:-1], k // 2), generator=g, dtype=U8)
    raw = torch.randint(90, 160, (*shape[:-1], k // 32), generator=g, dtype=U8)
    d = groups_of(groups, dev)
    say("fp4 pack and back", layout, groups, rows)
    scales = torch.full((gg.fp4_scale_bytes(layout, rows, k, experts),), FILL, dtype=U8, device=dev)
    gg.fp4_pack_scales(layout, raw.to(dev), d, out=scales)
    out = sentinel_tensor(shape, BF, dev)
    before = out.clone()
    gg.fp4_dequantize(layout, codes.to(dev), scales, d, out=out)
    torch.cuda.synchronize()
    assert torch.equal(scales.cpu(), ref.packed_scales(raw, layout, groups, rows, experts, FILL))
    who = ref.owned(layout, groups, rows, experts)
    want = ref.value(codes, raw).to(BF).reshape(-1, k)
    want[who < 0] = before.cpu().reshape(-1, k)[who < 0]
    assert torch.equal(out.cpu().reshape(-1, k), want)


def test_dequantize_every_code_and_scale():
    """Each of the 256 scale bytes with each code: exact in bf16 (2^-128 and
    up), infinite past its range, NaN for 255."""
    dev = device()
    raw = torch.arange(256, dtype=torch.int32).to(U8)[:, None].clone()
    codes = ref.pack(torch.arange(16, dtype=torch.int32).to(U8).repeat(256, 2))
    say("fp4 every code and scale")
    scales = gg.fp4_pack_scales(WEIGHT, raw[None].to(dev))
    out = gg.fp4_dequantize(WEIGHT, codes[None].to(dev), scales).cpu()[0]
    want = ref.value(codes, raw).to(BF)
    assert torch.equal(torch.isnan(out), torch.isnan(want))
    assert torch.equal(out.nan_to_num(7.0, float("inf"), float("-inf")), want.nan_to_num(7.0, float("inf"), float("-inf")))


def test_pack_scales_with_wide_rows():
    dev, g = device(), torch.Generator().manual_seed(3)
    rows, k, ld = 200, 96, 7
    raw = torch.randint(0, 256, (2, rows, ld), generator=g, dtype=U8)
    d = raw.to(dev)
    out = torch.full((gg.fp4_scale_bytes(WEIGHT, rows, k, 2),), FILL, dtype=U8, device=dev)
    say("fp4 pack, ld 7")
    rc = gg.call_raw("gg_fp4_pack_scales", WEIGHT, d.data_ptr(), ld, None, rows, k, 2, out.data_ptr(),
                     torch.cuda.current_stream().cuda_stream)
    assert rc == 0, gg.last_error()
    assert torch.equal(out.cpu(), ref.packed_scales(raw[..., :3], WEIGHT, None, rows, 2, FILL))


@pytest.mark.parametrize("tokens,topk,e,k,align", [(33, 8, 16, 160, 8), (1, 2, 4, 32, 1), (300, 3, 5, 416, 16)])
def test_gather_rows(tokens, topk, e, k, align):
    dev, g = device(), torch.Generator().manual_seed(tokens)
    x = spread(g, tokens, k).to(BF)
    ids = torch.rand(tokens, e, generator=g).topk(min(topk, e), dim=1).indices.to(I32)
    ids[torch.rand(ids.shape, generator=g) < 0.1] = -1
    say("fp4 gather", tokens, topk, e, k)
    offs, row_slot, _ = gg.route(ids.contiguous().to(dev), e, align, True)
    used = int(offs[-1])
    cap = row_slot.shape[0] + 3
    row_slot = torch.cat([row_slot, torch.full((3,), 1 << 30, dtype=I32, device=dev)])
    row_slot[used:] = 1 << 30
    row_slot[used - 1] = tokens * ids.shape[1]        # a slot of no token counts as padding
    codes = torch.full((cap, k // 2), FILL, dtype=U8, device=dev)
    scales = torch.full((gg.fp4_scale_bytes(RAGGED, cap, k, e),), FILL, dtype=U8, device=dev)
    gg.fp4_gather_rows(x.to(dev), row_slot, ids.shape[1], offs, out=codes, out_scales=scales)
    torch.cuda.synchronize()
    slot = row_slot.cpu()[:used].long()
    there = (slot >= 0) & (slot < tokens * ids.shape[1])
    src = torch.where(there[:, None], x[(slot // ids.shape[1]).clamp(0, tokens - 1)].float(), 0.0)
    c, b = ref.quantise(src)
    want = torch.full((cap, k // 2), FILL, dtype=U8)
    want[:used] = ref.pack(c)
    assert torch.equal(codes.cpu(), want)
    all_b = torch.zeros(cap, k // 32, dtype=U8)
    all_b[:used] = b
    assert bool((b[~there] == 127).all())
    assert torch.equal(scales.cpu(), ref.packed_scales(all_b, RAGGED, offs.cpu().tolist(), cap, e, FILL))


def scales_of(packed, layout, groups, rows, experts, blocks):
    """Scale bytes [all rows, blocks] back out of the packed layout."""
    total = rows if layout == RAGGED else rows * experts
    at = ref.packed_scales(torch.zeros(total, blocks, dtype=U8), layout, groups, rows, experts, 0)
    index = torch.arange(at.numel()).reshape(-1, -(-blocks // 4), 1024)
    out = torch.zeros(total, blocks, dtype=U8)
    for t, (first, count) in ref.tiles(layout, groups, rows, experts).items():
        r = torch.arange(count)
        for b in range(blocks):
            q = b % 4
            place = 512 * (r // 128) + 16 * (r % 32) + 8 * (q % 2) + 4 * (q // 2) + (r // 32) % 4
            out[first:first + count, b] = packed.cpu()[index[t, b // 4, place]]
    return out


@pytest.mark.parametrize("layout,groups,rows,experts", [c for c in LAYOUTS if c[0] != WEIGHT])
@pytest.mark.parametrize("i", [32, 160, 256])
def test_silu_mul_rows(layout, groups, rows, experts, i):
    dev, g = device(), torch.Generator().manual_seed(rows + i)
    h = (torch.randn(*rows_of(layout, rows, experts, 2 * i), generator=g) * 2).to(BF)
    who = ref.owned(layout, groups, rows, experts)
    h.reshape(-1, 2 * i)[who < 0] = float("nan")
    codes = torch.full((*h.shape[:-1], i // 2), FILL, dtype=U8, device=dev)
    say("fp4 silu", layout, groups, rows, i)
    _, scales = gg.fp4_silu_mul_rows(h.to(dev), groups_of(groups, dev), masked=layout == MASKED, out=codes)
    torch.cuda.synchronize()
    c = codes.cpu().reshape(-1, i // 2)
    assert bool((c[who < 0] == FILL).all())
    live = who >= 0
    if not bool(live.any()):
        return
    a, slack = layer_ref.silu_mul(h.double().reshape(-1, 2 * i)[live])
    b = scales_of(scales, layout, groups, rows, experts, i // 32)[live]
    ref.close4(c[live], b, a, slack, "silu")


def operands(g, layout, groups, rows, experts, k, n, dev, lo=110, hi=135):
    """Random codes with scales, packed; everything of rows nobody owns set to NaN."""
    def make(*shape):
        return (torch.randint(0, 256, (*shape, k // 2), generator=g, dtype=U8),
                torch.randint(lo, hi, (*shape, k // 32), generator=g, dtype=U8))
    x, xs = make(*rows_of(layout, rows, experts, 1)[:-1])
    w, ws = make(experts, n)
    who = ref.owned(layout, groups, rows, experts)
    d = groups_of(groups, dev)
    packed = torch.full((gg.fp4_scale_bytes(layout, rows, k, experts),), 255, dtype=U8, device=dev)
    gg.fp4_pack_scales(layout, xs.to(dev), d, out=packed)
    return x, xs, w, ws, who, d, packed, gg.fp4_pack_scales(WEIGHT, ws.to(dev))


@pytest.mark.parametrize("layout,groups,rows,experts", [c for c in LAYOUTS if c[0] != WEIGHT])
@pytest.mark.parametrize("k,n,dtype", [(32, 8, torch.float32), (96, 264, BF), (128, 72, BF), (160, 256, torch.float32),
                                       (256, 520, BF), (544, 136, BF)])
def test_product(layout, groups, rows, experts, k, n, dtype):
    dev, g = device(), torch.Generator().manual_seed(k * n + rows)
    x, xs, w, ws, who, d, xp, wp = operands(g, layout, groups, rows, experts, k, n, dev)
    out = sentinel_tensor(rows_of(layout, rows, experts, n), dtype, dev)
    before = out.clone()
    say("fp4 product", layout, groups, rows, k, n, dtype)
    f = gg.fp4_forward if layout == RAGGED else gg.fp4_masked_forward
    f(x.to(dev), xp, w.to(dev), wp, d, out=out)
    torch.cuda.synchronize()
    got = out.reshape(-1, n)
    assert torch.equal(got.cpu()[who < 0].view(torch.int16 if dtype == BF else I32),
                       before.reshape(-1, n).cpu()[who < 0].view(torch.int16 if dtype == BF else I32))
    ref.check_product(got, ref.value(x, xs).reshape(-1, k), ref.value(w, ws), who, "product")


@pytest.mark.parametrize("k,n", [(768, 264), (1056, 512)])
def test_product_of_one_scale_is_exact(k, n):
    """With one scale for all, every partial sum is a multiple of 1/4 below
    36 k <= 2^16, which fp32 holds: the result is equal, not close."""
    dev, g = device(), torch.Generator().manual_seed(k)
    groups, rows, e = [100, 100, 500, 756], 760, 4
    x, xs, w, ws, who, d, _, _ = operands(g, RAGGED, groups, rows, e, k, n, dev)
    xs.fill_(127)
    ws.fill_(127)
    say("fp4 exact product", k, n)
    xp, wp = gg.fp4_pack_scales(RAGGED, xs.to(dev), d), gg.fp4_pack_scales(WEIGHT, ws.to(dev))
    out = gg.fp4_forward(x.to(dev), xp, w.to(dev), wp, d, out_dtype=torch.float32).cpu()
    xv, wv = ref.value(x, xs), ref.value(w, ws)
    for r in range(e):
        assert torch.equal(out[who == r].double(), xv[who == r] @ wv[r].t())


def test_product_with_nan_scales():
    """A scale of 255 makes its row (x) or column (w) NaN, and no other."""
    dev, g = device(), torch.Generator().manual_seed(5)
    groups, rows, e, k, n = [40, 300], 300, 2, 288, 264
    x, xs, w, ws, who, d, _, _ = operands(g, RAGGED, groups, rows, e, k, n, dev)
    xs[7, 3] = xs[290, 8] = 255
    ws[1, 5, 0] = ws[0, 263, 8] = 255
    say("fp4 NaN scales")
    xp, wp = gg.fp4_pack_scales(RAGGED, xs.to(dev), d), gg.fp4_pack_scales(WEIGHT, ws.to(dev))
    out = gg.fp4_forward(x.to(dev), xp, w.to(dev), wp, d)
    ref.check_product(out, ref.value(x, xs), ref.value(w, ws), who, "NaN scales")
    nan = torch.isnan(out.cpu())
    want = torch.zeros(rows, n, dtype=torch.bool)
    want[7] = want[290] = True
    want[40:, 5] = want[:40, 263] = True
    assert torch.equal(nan, want)


def test_stream_and_graph():
    """Another stream, and a captured chain replayed with new inputs."""
    dev, g = device(), torch.Generator().manual_seed(11)
    groups, rows, e, k, n = [30, 30, 290], 300, 3, 256, 264
    _, _, w, ws, who, d, _, wp = operands(g, RAGGED, groups, rows, e, k, n, dev)
    w = w.to(dev)
    xs = [spread(g, rows, k).to(BF).to(dev) for _ in range(3)]

    def chain(x, codes, scales, out):
        gg.fp4_quantize(RAGGED, x, d, out=codes, out_scales=scales)
        return gg.fp4_forward(codes, scales, w, wp, d, out=out)

    def buffers():
        return (torch.zeros(rows, k // 2, dtype=U8, device=dev),
                torch.zeros(gg.fp4_scale_bytes(RAGGED, rows, k, e), dtype=U8, device=dev),
                torch.zeros(rows, n, dtype=BF, device=dev))
    say("fp4 eager, stream, graph")
    want = [chain(x, *buffers()).clone() for x in xs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = chain(xs[0], *buffers())
    side.synchronize()
    assert torch.equal(got.view(torch.int16), want[0].view(torch.int16))
    x, b = xs[0].clone(), buffers()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain(x, *b)
    for i in (0, 1, 2, 1):
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(b[2].view(torch.int16), want[i].view(torch.int16))
