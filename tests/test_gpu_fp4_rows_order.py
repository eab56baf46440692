"""4-bit rows: the gather in the order by XCD that full grids take, and SiLU-mul
rows whose gates and products leave the ordinary range."""
import pytest
import torch

import fp4_ref as ref
import layer_ref
from moe_grouped_gemm_ragged_amd import binding as gg
from gpu_util import device, say
from test_gpu_fp4 import FILL, RAGGED, MASKED, scales_of, spread

pytestmark = pytest.mark.gpu
BF, U8, I32 = torch.bfloat16, torch.uint8, torch.int32

# tokens, topk, experts, k, alignment: grids of whole eights, below a full one, and above (units go round)
GATHERS = [(40, 4, 7, 416, 1), (300, 3, 6, 160, 1), (700, 2, 26, 512, 16), (33, 8, 128, 2080, 1), (2000, 8, 64, 2048, 8),
           (4000, 6, 128, 1056, 1)]


@pytest.mark.parametrize("tokens,topk,e,k,align", GATHERS)
def test_gather_by_xcd(tokens, topk, e, k, align):
    dev, g = device(), torch.Generator().manual_seed(tokens)
    x = spread(g, tokens, k).to(BF)
    ids = torch.rand(tokens, e, generator=g).topk(min(topk, e), dim=1).indices.to(I32)
    ids[torch.rand(ids.shape, generator=g) < 0.05] = -1
    ids[ids == e // 2] = -1                              # an expert without rows
    say("fp4 gather by XCD", tokens, topk, e, k)
    offs, row_slot, _ = gg.route(ids.contiguous().to(dev), e, align, True)
    used = int(offs[-1])
    # (so many rows more that the grid is a multiple of 8)
    units = lambda cap: 2 * (-(-cap // 256) + e) * -(-k // 256)
    cap = row_slot.shape[0]
    most = 6 * torch.cuda.get_device_properties(dev).multi_processor_count
    while min(units(cap), most) % 8:
        cap += 256
    row_slot = torch.cat([row_slot[:used], torch.full((cap - used,), 1 << 30, dtype=I32, device=dev)])
    codes = torch.full((cap, k // 2), FILL, dtype=U8, device=dev)
    scales = torch.full((gg.fp4_scale_bytes(RAGGED, cap, k, e),), FILL, dtype=U8, device=dev)
    gg.fp4_gather_rows(x.to(dev), row_slot, ids.shape[1], offs, out=codes, out_scales=scales)
    torch.cuda.synchronize()
    slot = row_slot.cpu()[:used].long()
    there = slot >= 0
    token = (slot // ids.shape[1]).clamp(min=0)
    c, b = ref.quantise(x.float())
    want = torch.full((cap, k // 2), FILL, dtype=U8)
    want[:used] = torch.where(there[:, None], ref.pack(c)[token], 0)
    assert torch.equal(codes.cpu(), want)
    all_b = torch.zeros(cap, k // 32, dtype=U8)
    all_b[:used] = torch.where(there[:, None], b[token], 127)
    assert torch.equal(scales.cpu(), ref.packed_scales(all_b, RAGGED, offs.cpu().tolist(), cap, e, FILL))


INF, NAN = float("inf"), float("nan")
SPECIAL = [  # gate, up
    (INF, 1.0), (INF, -1.0), (INF, 0.0), (-INF, 1.0), (NAN, 1.0), (1.0, NAN), (1.0, INF), (0.0, -INF), (-1.0, INF),
    (1e30, 1e30), (-1e30, 1e30), (20.0, 1e38), (3e38, 1.0), (3.3e38, -1.0), (1.0, 3.3e38), (-3e38, -3e38), (-200.0, 3e38),
    (-104.0, 3e38), (-88.5, 3e38), (-88.0, 3e38), (-87.0, 3e38), (-86.0, -3e38), (-60.0, 1e38), (-60.0, 1.0), (-20.0, 1.0),
    (1e-38, 1.0), (1e-30, 1e-8), (1e-20, 1e-20), (-0.0, 5.0), (0.0, 0.0), (40.0, 1e-38), (-1e-38, 3e38)]


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("rest", [0.0, 1.0, 1e-25])
def test_silu_mul_rows_out_of_range(masked, rest):
    """A block with a product that fp32 does not hold, or a NaN, is NaN (scale
    255, codes 0), and no other block; a very negative gate gives its small
    product, or 0 where the sigmoid is below fp32's range."""
    dev, g = device(), torch.Generator().manual_seed(3)
    i, rows = 128, len(SPECIAL)
    h = (torch.randn(rows, 2 * i, generator=g) * rest).to(BF)
    place = [(37 * r) % i for r in range(rows)]
    for r, (gate, up) in enumerate(SPECIAL):
        h[r, place[r]], h[r, i + place[r]] = gate, up
    say("fp4 silu out of range", masked, rest)
    groups = torch.tensor([rows], dtype=I32, device=dev)
    codes, scales = gg.fp4_silu_mul_rows(h[None].to(dev) if masked else h.to(dev), groups, masked=masked)
    codes = codes.cpu().reshape(rows, i // 2)
    b = scales_of(scales, MASKED if masked else RAGGED, [rows], rows, 1, i // 32)
    a, slack = layer_ref.silu_mul(h.double())
    lost = ~torch.isfinite(a) | (a.abs() > 3.5e38)        # (none of them lies next to fp32's largest value)
    assert bool(((a.abs() < 3.39e38) | lost).all()) and 8 < int(lost.sum()) < 16
    bad = lost.reshape(rows, -1, 32).any(-1)
    assert torch.equal(b == 255, bad)
    assert bool((ref.unpack(codes).reshape(rows, -1, 32)[bad] == 0).all())
    fine = ~bad[..., None].expand(rows, i // 32, 32).reshape(rows, i)
    # the blocks that are not NaN, one a row
    pick = fine.reshape(-1, 32)[:, 0]
    ref.close4(codes.reshape(-1, 16)[pick], b.reshape(-1, 1)[pick], a.reshape(-1, 32)[pick], slack.reshape(-1, 32)[pick], "silu")
