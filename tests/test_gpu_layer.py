"""GPU tests of the layer steps around the grouped GEMM against plain fp64
forms (tests/layer_ref.py): the norm and its gradient, e4m3 rows gathered
with packed scales, the combine gradient, SiLU-mul rows and their gradient.
Sizes from one row up, widths off every power of two, rows nobody owns filled
with NaN on the way in and a sentinel on the way out."""
import numpy as np
import pytest
import torch

import oracle
import layer_ref as ref
from moe_grouped_gemm_ragged_amd import binding as gg
from gpu_util import device, say, sentinel_tensor

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
U8 = torch.uint8


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(BF)


def unchanged(t, mask, before):
    """Elements of t outside mask hold what they held."""
    return torch.equal(t.view(torch.int16 if t.dtype == BF else U8)[~mask],
                       before.view(torch.int16 if t.dtype == BF else U8)[~mask])


# ---------------------------------------------------------------------------
# norm
# ---------------------------------------------------------------------------

NORM_SHAPES = [(1, 8), (1, 2048), (3, 128), (5, 136), (7, 512), (2, 520), (33, 1000), (130, 1024), (4, 4104), (9, 7168),
               (3, 16384), (2, 16512), (2, 32768), (3, 32896), (1, 131080)]


@pytest.mark.parametrize("rows,n", NORM_SHAPES)
@pytest.mark.parametrize("res", [False, True])
def test_rmsnorm(rows, n, res):
    device()
    g = gen(rows * 7 + n)
    x, gamma = randn(g, rows, n, std=1.5), randn(g, n, std=0.5) + 1
    x[0] *= 300                                         # rows of very different sizes
    r = randn(g, rows, n, std=2.0) if res else None
    say("rmsnorm", rows, n, res)
    y, h = gg.rmsnorm(x, gamma, residual=r, eps=1e-5)
    torch.cuda.synchronize()
    want, hw = ref.rmsnorm(x, r, gamma, 1e-5)
    ref.close(y, want, want.abs() * 2.0 ** -8 + ref.rmsnorm_slack(want, n), "y")
    if res:
        ref.close(h, hw, hw.abs() * (2.0 ** -8 + 2.0 ** -24), "h")
    else:
        assert h is None
    if n % 128 == 0:
        say("fp8_rmsnorm", rows, n, res)
        codes, scales, h8, y2 = gg.fp8_rmsnorm(x, gamma, residual=r, eps=1e-5, with_bf16=True)
        torch.cuda.synchronize()
        ref.close8(codes, scales, want, ref.rmsnorm_slack(want, n), "y8")
        assert torch.equal(y, y2) and (not res or torch.equal(h, h8))


def test_rmsnorm_in_place_and_zero_rows():
    device()
    g = gen(1)
    x, r, gamma = randn(g, 70, 768), randn(g, 70, 768), randn(g, 768)
    x[3] = 0
    r[3] = 0
    y, h = gg.rmsnorm(x, gamma, residual=r)
    say("rmsnorm in place")
    r2 = r.clone()
    y2, h2 = gg.rmsnorm(x, gamma, residual=r2, h_out=r2)
    codes, scales, _ = gg.fp8_rmsnorm(x, gamma, residual=r)
    torch.cuda.synchronize()
    assert h2.data_ptr() == r2.data_ptr() and torch.equal(h, h2) and torch.equal(y, y2)
    assert bool((y[3] == 0).all()) and bool((codes[3] & 0x7F == 0).all()) and bool((scales[3] == 127).all())
    empty = x[:0]
    y, h = gg.rmsnorm(empty, gamma, residual=empty)
    assert y.shape == (0, 768) and h.shape == (0, 768)


@pytest.mark.parametrize("rows,n", NORM_SHAPES + [(1025, 264), (2049, 640)])
@pytest.mark.parametrize("res", [False, True])
def test_rmsnorm_grad(rows, n, res):
    device()
    g = gen(rows * 3 + n)
    dy, h, gamma = randn(g, rows, n, std=0.3), randn(g, rows, n, std=1.5), randn(g, n, std=0.5) + 1
    dh = randn(g, rows, n, std=0.3) if res else None
    say("rmsnorm_grad", rows, n, res)
    dx, dgamma = gg.rmsnorm_grad(dy, h, gamma, dh=dh, eps=1e-5)
    again = gg.rmsnorm_grad(dy, h, gamma, dh=dh, eps=1e-5)
    torch.cuda.synchronize()
    wx, slack, wg, slack_g = ref.rmsnorm_grad(dy, h, gamma, dh, 1e-5)
    ref.close(dx, wx, wx.abs() * 2.0 ** -8 + slack, "dx")
    ref.close(dgamma, wg, slack_g, "dgamma")
    assert torch.equal(dx, again[0]) and torch.equal(dgamma, again[1]), "two calls differ"


def test_rmsnorm_rows_that_are_not_finite():
    """An infinity or a NaN changes its own row only (of the gradient: and
    dgamma), and comes out as the formula has it: rho is 0 or NaN."""
    device()
    g = gen(17)
    for rows, n in ((11, 128), (6, 1024), (4, 33024)):
        x, gamma, dy = randn(g, rows, n), randn(g, n), randn(g, rows, n)
        good = [t.clone() for t in gg.fp8_rmsnorm(x, gamma, with_bf16=True) if t is not None]
        dx_good, _ = gg.rmsnorm_grad(dy, x, gamma)
        x[1, 5], x[2, n - 1] = float("inf"), float("nan")
        say("rmsnorm of an infinity and a NaN", rows, n)
        codes, scales, _, y = gg.fp8_rmsnorm(x, gamma, with_bf16=True)
        dx, dgamma = gg.rmsnorm_grad(dy, x, gamma)
        torch.cuda.synchronize()
        rest = [i for i in range(rows) if i not in (1, 2)]
        for a, b in zip((codes, scales, y), good):
            assert torch.equal(a[rest].view(U8), b[rest].view(U8))
        assert torch.equal(dx[rest], dx_good[rest])
        assert bool(torch.isnan(y[2]).all()) and bool(((codes[2] & 0x7F) == 0x7F).all())
        at = torch.arange(n, device="cuda") == 5
        assert torch.equal(torch.isnan(y[1]), at) and bool((y[1][~at] == 0).all())
        assert torch.equal((codes[1] & 0x7F) == 0x7F, at) and bool((scales[1:3] == 127).all())
        assert bool(torch.isnan(dx[2]).all()) and bool(torch.isnan(dgamma).all())


def test_rmsnorm_grad_no_rows_in_place_and_differences():
    device()
    g = gen(5)
    gamma = randn(g, 64)
    none = torch.empty((0, 64), dtype=BF, device="cuda")
    say("rmsnorm_grad without rows")
    dx, dgamma = gg.rmsnorm_grad(none, none, gamma)
    assert dx.shape == (0, 64) and bool((dgamma == 0).all())
    dy, h, dh = randn(g, 40, 64), randn(g, 40, 64), randn(g, 40, 64)
    dx, dgamma = gg.rmsnorm_grad(dy, h, gamma, dh=dh)
    dh2 = dh.clone()
    assert torch.equal(gg.rmsnorm_grad(dy, h, gamma, dh=dh2, out=dh2)[0], dx)
    # against central differences of the fp64 norm: f = <dy, norm(h)> + <dh, h>
    hd, gd, step = ref.f64(h), ref.f64(gamma), 1e-5

    def f(hh, gm):
        y = hh / torch.sqrt(hh.square().mean(-1, keepdim=True) + 1e-6) * gm
        return (ref.f64(dy) * y).sum() + (ref.f64(dh) * hh).sum()

    for t, c in ((0, 0), (7, 33), (39, 63)):
        e = torch.zeros_like(hd)
        e[t, c] = step
        diff = (f(hd + e, gd) - f(hd - e, gd)) / (2 * step)
        # half a bf16 step, and 1e-6 for the difference quotient's own error
        assert abs(float(dx[t, c]) - float(diff)) <= 2.0 ** -8 * abs(float(diff)) + 1e-5
        e = torch.zeros_like(gd)
        e[c] = step
        diff = (f(hd, gd + e) - f(hd, gd - e)) / (2 * step)
        assert abs(float(dgamma[c]) - float(diff)) <= 1e-5 * (1 + abs(float(diff)))


# ---------------------------------------------------------------------------
# routed rows
# ---------------------------------------------------------------------------

def routing(seed, tokens, topk, e, align, pad_empty=True, dropped=0.0):
    rng = np.random.default_rng(seed)
    ids = rng.integers(0, e, size=(tokens, topk)).astype(np.int32)
    if e > 2:
        ids[ids == 1] = 0                                # expert 1 is empty, expert 0 twice as long
    if dropped:
        ids = np.where(rng.random(ids.shape) < dropped, -1, ids).astype(np.int32)
    ids_d = torch.from_numpy(ids).cuda()
    return gg.route(ids_d, e, align, pad_empty)


ROUTED = [(1, 1, 1, 4, 1, False, 0.0), (2, 1, 8, 128, 16, True, 0.0), (3, 37, 3, 7, 1, False, 0.1),
          (4, 700, 4, 9, 8, True, 0.02), (5, 2000, 2, 3, 16, False, 0.0), (6, 300, 9, 2048, 1, False, 0.3),
          (7, 64, 17, 40, 8, True, 0.0), (8, 0, 4, 16, 8, True, 0.0), (9, 5, 2, 4, 8, True, 1.0)]


@pytest.mark.parametrize("seed,tokens,topk,e,align,pad,drop", ROUTED)
@pytest.mark.parametrize("k", [128, 384, 2048])
def test_fp8_gather_rows_bit_exact(seed, tokens, topk, e, align, pad, drop, k):
    dev = device()
    g = gen(seed)
    offs, row_slot, _ = routing(seed, tokens, topk, e, align, pad, drop)
    cap, used = row_slot.shape[0], int(offs[-1])
    src = torch.randint(0, 256, (tokens, k), generator=g, device=dev, dtype=U8)
    scales = torch.randint(1, 255, (tokens, k // 128), generator=g, device=dev, dtype=U8)
    out = torch.full((cap, k), 0xA5, dtype=U8, device=dev)
    packed = torch.full((gg.fp8_scale_bytes(gg.GG_FP8_ACT_RAGGED, cap, k, e),), 0xA5, dtype=U8, device=dev)
    say("fp8_gather_rows", seed, tokens, topk, e, k)
    gg.fp8_gather_rows(src, scales, row_slot, topk, offs, out=out, out_scales=packed)
    torch.cuda.synchronize()
    slots = row_slot[:used].cpu().numpy()
    assert np.array_equal(out[:used].cpu().numpy(), oracle.gather_rows(src.cpu().numpy(), slots, topk))
    assert bool((out[used:] == 0xA5).all()), "rows past the last offset were written"
    rows = torch.full((used, k // 128), 127, dtype=U8)
    at = np.flatnonzero(slots >= 0)
    rows[at] = scales.cpu()[slots[at] // topk]
    assert torch.equal(packed.cpu(), ref.packed_scales(rows, offs.tolist(), cap, fill=0xA5))


@pytest.mark.parametrize("tokens,topk,e,k,align,pad,drop", [
    (4100, 2, 3, 2176, 8, True, 0.0), (9000, 3, 40, 1024, 1, False, 0.05), (20000, 2, 300, 512, 4, True, 0.0),
    (1300, 6, 2048, 7168, 1, False, 0.0), (1100, 4, 16, 8320, 16, True, 0.02), (70000, 2, 5, 128, 8, True, 0.0)])
def test_fp8_gather_rows_of_many_tokens(tokens, topk, e, k, align, pad, drop):
    """More than 8 MB of tokens, which are copied window by window."""
    dev = device()
    assert tokens * k > 8 << 20
    g = gen(tokens)
    offs, row_slot, _ = routing(tokens, tokens, topk, e, align, pad, drop)
    cap, used = row_slot.shape[0], int(offs[-1])
    src = torch.randint(0, 256, (tokens, k), generator=g, device=dev, dtype=U8)
    scales = torch.randint(1, 255, (tokens, k // 128), generator=g, device=dev, dtype=U8)
    out = torch.full((cap, k), 0xA5, dtype=U8, device=dev)
    say("fp8_gather_rows of many tokens", tokens, topk, e, k)
    _, packed = gg.fp8_gather_rows(src, scales, row_slot, topk, offs, out=out)
    slot = row_slot[:used].long()
    want = torch.where((slot >= 0)[:, None], src[slot.clamp(min=0) // topk], torch.zeros(1, dtype=U8, device=dev))
    assert torch.equal(out[:used], want)
    assert bool((out[used:] == 0xA5).all()), "rows past the last offset were written"
    raw = torch.where((slot >= 0)[:, None], scales[slot.clamp(min=0) // topk],
                      torch.full((1, 1), 127, dtype=U8, device=dev))
    same = gg.fp8_pack_scales(gg.GG_FP8_ACT_RAGGED, raw.contiguous(), offs, used, k, e)
    tiles = int(((torch.diff(offs.long(), prepend=offs.new_zeros(1).long()) + 255) // 256).sum())
    n = tiles * (k // 128) * 256
    assert torch.equal(packed[:n], same[:n])


def test_fp8_gather_rows_fewer_than_tokens():
    """Room for fewer rows than there are tokens, of a src of 60 MB."""
    dev = device()
    offs, row_slot, _ = routing(5, 8000, 4, 16, 8, True)
    row_slot, k = row_slot[:333].contiguous(), 7552
    src = torch.randint(0, 256, (8000, k), device=dev, dtype=U8)
    scales = torch.randint(1, 255, (8000, k // 128), device=dev, dtype=U8)
    say("fp8_gather_rows with little room")
    out, packed = gg.fp8_gather_rows(src, scales, row_slot, 4, offs)
    slot = row_slot.long()
    assert torch.equal(out, torch.where((slot >= 0)[:, None], src[slot.clamp(min=0) // 4], torch.zeros_like(out)))
    raw = torch.where((slot >= 0)[:, None], scales[slot.clamp(min=0) // 4], torch.full((1, 1), 127, dtype=U8, device=dev))
    same = gg.fp8_pack_scales(gg.GG_FP8_ACT_RAGGED, raw.contiguous(), offs, 333, k, 16)
    ends = [min(int(v), 333) for v in offs]
    n = sum(-(-(b - a) // 256) for a, b in zip([0] + ends, ends)) * (k // 128) * 256
    assert torch.equal(packed[:n], same[:n])


def test_fp8_gather_rows_feeds_the_packed_layout():
    """The scales are those that gg_fp8_pack_scales writes for the gathered rows."""
    dev = device()
    offs, row_slot, _ = routing(11, 500, 4, 12, 16, True)
    k, used = 512, int(offs[-1])
    src = torch.randint(0, 256, (500, k), device=dev, dtype=U8)
    scales = torch.randint(100, 140, (500, k // 128), device=dev, dtype=U8)
    say("fp8_gather_rows against pack_scales")
    rows, packed = gg.fp8_gather_rows(src, scales, row_slot, 4, offs, out_scales=torch.zeros(
        gg.fp8_scale_bytes(gg.GG_FP8_ACT_RAGGED, row_slot.shape[0], k, 12), dtype=U8, device=dev))
    slot = row_slot[:used].long()                         # (what lies behind them is not initialised)
    raw = torch.zeros(row_slot.shape[0], k // 128, dtype=U8, device=dev)
    raw[:used] = torch.where((slot >= 0)[:, None], scales[slot.clamp(min=0) // 4],
                             torch.full((1, 1), 127, dtype=U8, device=dev))
    want = gg.fp8_pack_scales(gg.GG_FP8_ACT_RAGGED, raw, offs, row_slot.shape[0], k, 12,
                              out=torch.zeros_like(packed))
    assert torch.equal(packed, want)


def test_fp8_gather_rows_bad_slots_and_offsets():
    """Slots past the tokens are padding rows; offsets that fall or pass the
    capacity are clamped as the GEMMs clamp them."""
    dev = device()
    k, cap = 256, 600
    src = torch.randint(0, 256, (10, k), device=dev, dtype=U8)
    scales = torch.randint(1, 255, (10, k // 128), device=dev, dtype=U8)
    row_slot = torch.randint(-3, 40, (cap,), device=dev, dtype=torch.int32)
    offs = torch.tensor([-5, 300, 120, 5000], dtype=torch.int32, device=dev)
    say("fp8_gather_rows with bad slots and offsets")
    rows, packed = gg.fp8_gather_rows(src, scales, row_slot, 2, offs, out_scales=torch.full(
        (gg.fp8_scale_bytes(gg.GG_FP8_ACT_RAGGED, cap, k, 4),), 7, dtype=U8, device=dev))
    slot = row_slot.cpu().long()
    ok = (slot >= 0) & (slot < 20)
    want = torch.where(ok[:, None], src.cpu()[slot.clamp(0, 19) // 2], torch.zeros(1, k, dtype=U8))
    raw = torch.where(ok[:, None], scales.cpu()[slot.clamp(0, 19) // 2], torch.full((1, k // 128), 127, dtype=U8))
    assert torch.equal(rows.cpu(), want)
    assert torch.equal(packed.cpu(), ref.packed_scales(raw, [0, 300, 300, 600], cap, fill=7))


@pytest.mark.parametrize("seed,tokens,topk,e,align,pad,drop", ROUTED)
@pytest.mark.parametrize("n", [8, 520, 2048, 4104])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_combine_rows_grad(seed, tokens, topk, e, align, pad, drop, n, dtype):
    dev = device()
    g = gen(seed + n)
    offs, row_slot, slot_row = routing(seed, tokens, topk, e, align, pad, drop)
    cap, used = row_slot.shape[0], int(offs[-1])
    dout = torch.randn(tokens, n, generator=g, device=dev).to(BF if dtype == "bf16" else torch.float32)
    y = randn(g, cap, n)
    y[:used][row_slot[:used] < 0] = float("nan")          # padding rows are not read
    y[used:] = float("nan")
    w = torch.rand(tokens, topk, generator=g, device=dev) if seed % 2 else None
    dy = sentinel_tensor((cap, n), BF, dev)
    before = dy.clone()
    say("combine_rows_grad", seed, tokens, topk, e, n, dtype)
    _, dw = gg.combine_rows_grad(dout, y, slot_row, row_slot, offs, topk, weights=w, out=dy)
    only, none = gg.combine_rows_grad(dout, None, slot_row, row_slot, offs, topk, weights=w, out=before.clone(),
                                      with_weights=False)
    torch.cuda.synchronize()
    assert none is None and torch.equal(only.view(torch.int16), dy.view(torch.int16))
    live = torch.zeros(cap, dtype=torch.bool, device=dev)
    live[:used] = True
    assert unchanged(dy, live, before)
    d, yy = ref.f64(dout), ref.f64(y)
    ww = torch.ones(tokens, topk, dtype=torch.float64) if w is None else ref.f64(w)
    want = torch.zeros(used, n, dtype=torch.float64)
    slots = row_slot[:used].cpu().long()
    at = (slots >= 0).nonzero()[:, 0]
    want[at] = ww.reshape(-1)[slots[at]][:, None] * d[slots[at] // topk]
    # one product rounded to fp32, then half a bf16 step
    ref.close(dy[:used], want, want.abs() * (2.0 ** -8 + 2.0 ** -23), "dy")
    row = slot_row.cpu().long().reshape(tokens, topk)
    terms = torch.where((row >= 0)[..., None], torch.nan_to_num(yy)[row.clamp(min=0)] * d[:, None, :],
                        torch.zeros(1, dtype=torch.float64)) if tokens else torch.zeros(0, topk, n, dtype=torch.float64)
    ref.close(dw, terms.sum(-1), terms.abs().sum(-1) * (n + 2) * ref.U32, "dweights")


def test_combine_rows_and_its_gradient_agree():
    """<dout, combine(y, w)> as a function of y and w: its derivative along any
    direction is what the gradient says (the combine is linear in each)."""
    dev = device()
    tokens, topk, e, n = 300, 4, 16, 264
    g = gen(77)
    offs, row_slot, slot_row = routing(77, tokens, topk, e, 8, True, 0.05)
    y, dout = randn(g, row_slot.shape[0], n), randn(g, tokens, n)
    w = torch.rand(tokens, topk, generator=g, device=dev)
    say("combine_rows_grad against combine_rows")
    out = gg.combine_rows(y, slot_row, topk, w, out_dtype=torch.float32)
    dy, dw = gg.combine_rows_grad(dout, y, slot_row, row_slot, offs, topk, weights=w)
    used = int(offs[-1])
    f = (ref.f64(out) * ref.f64(dout)).sum()
    kept = (row_slot[:used] >= 0).cpu()
    by_w = (ref.f64(dw) * ref.f64(w)).sum()
    products = ref.f64(dy)[:used][kept] * ref.f64(y)[:used][kept]
    assert abs(float(f - by_w)) <= float((ref.f64(out) * ref.f64(dout)).abs().sum()) * 2 * n * ref.U32 + 1e-9
    # dy is rounded to bf16: half a step of each product
    assert abs(float(f - products.sum())) <= float(products.abs().sum()) * 2.0 ** -8


# ---------------------------------------------------------------------------
# SiLU-mul rows
# ---------------------------------------------------------------------------

def grouped(kind, seed):
    """(groups, leading shape, which rows an expert owns)"""
    rng = np.random.default_rng(seed)
    if kind == "ragged":
        sizes = [0, 130, 1, 0, 77, 300]
        ends = np.cumsum(sizes).astype(np.int32)
        m = int(ends[-1]) + 37
        live = torch.arange(m) < int(ends[-1])
        return torch.from_numpy(ends).cuda(), (m,), live.cuda()
    if kind == "one":
        return torch.tensor([1], dtype=torch.int32, device="cuda"), (1,), torch.ones(1, dtype=torch.bool, device="cuda")
    if kind == "bad":                                    # offsets that fall, are negative and pass the rows
        groups = torch.tensor([-4, 90, 20, 1000], dtype=torch.int32, device="cuda")
        return groups, (333,), torch.ones(333, dtype=torch.bool, device="cuda")
    counts = np.array([0, 8, 64, -3, 41, 900], dtype=np.int32)
    live = torch.arange(64)[None, :] < torch.from_numpy(np.clip(counts, 0, 64))[:, None]
    return torch.from_numpy(counts).cuda(), (6, 64), live.cuda()


KINDS = ["ragged", "one", "bad", "masked"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("width", [8, 200, 128, 768, 2176])
def test_silu_mul_rows(kind, width):
    dev = device()
    groups, lead, live = grouped(kind, width)
    masked = kind == "masked"
    g = gen(width)
    h = randn(g, *lead, 2 * width, std=3.0)
    h[~live] = float("nan")
    a = sentinel_tensor((*lead, width), BF, dev)
    before = a.clone()
    say("silu_mul_rows", kind, width)
    gg.silu_mul_rows(h, groups, masked=masked, out=a)
    torch.cuda.synchronize()
    want, slack = ref.silu_mul(ref.f64(h[live]))
    ref.close(a[live], want, want.abs() * 2.0 ** -8 + slack, "a")
    assert unchanged(a, live, before), "rows nobody owns were written"
    if width % 128:
        return
    a8 = torch.full((*lead, width), 0xA5, dtype=U8, device=dev)
    a8s = torch.full((*lead, width // 128), 0xA5, dtype=U8, device=dev)
    h8 = torch.full((*lead, 2 * width), 0xA5, dtype=U8, device=dev)
    h8s = torch.full((*lead, 2 * width // 128), 0xA5, dtype=U8, device=dev)
    say("fp8_silu_mul_rows", kind, width)
    gg.fp8_silu_mul_rows(h, groups, masked=masked, keep=True, out=a8, out_scales=a8s, kept=h8, kept_scales=h8s)
    a2, k8, k8s = gg.silu_mul_rows(h, groups, masked=masked, keep=True)
    torch.cuda.synchronize()
    ref.close8(a8[live], a8s[live], want, slack, "a8")
    codes, scales = ref.quantise(h[live].cpu())
    assert torch.equal(h8[live].cpu(), codes) and torch.equal(h8s[live].cpu(), scales), "kept rows"
    for t in (a8, a8s, h8, h8s):
        assert bool((t[~live] == 0xA5).all()), "rows nobody owns were written"
    assert torch.equal(a2[live], a[live]) and torch.equal(k8[live], h8[live]) and torch.equal(k8s[live], h8s[live])


def test_kept_rows_at_the_borders():
    """Blocks whose largest value lies at, just below and just above 448 times
    a power of two, tiny and huge ones, blocks of zeros, infinities and NaN,
    and ties between two codes."""
    dev = device()
    width = 128
    h = torch.zeros(12, 2 * width)
    g = torch.Generator().manual_seed(3)
    base = torch.randn(2 * width, generator=g)
    base = (base / base.abs().max())
    tops = [448.0, 450.0, 446.0, 448 * 2.0 ** -20, 450 * 2.0 ** 30, 1e-38, 9e-41, 3e38, 0.0]
    for i, top in enumerate(tops):
        h[i] = base * 0.9 * top
        h[i, 5] = top
        h[i, width + 9] = -top
    h[9] = base * 100
    h[9, 0], h[9, 70], h[9, 200] = float("inf"), float("nan"), -float("inf")
    h[10] = torch.arange(2 * width) / 16.0                # every tie of the first binades
    h[11] = -(torch.arange(2 * width) + 0.5) / 4.0
    h = h.to(BF)
    groups = torch.tensor([12], dtype=torch.int32, device=dev)
    say("kept rows at the borders")
    _, codes, scales = gg.silu_mul_rows(h.cuda(), groups, keep=True)
    torch.cuda.synchronize()
    want, ws = ref.quantise(h)
    assert torch.equal(scales.cpu(), ws), (scales.cpu() - ws).nonzero()
    nan = (want & 0x7F) == 0x7F
    got = codes.cpu()
    assert torch.equal((got & 0x7F) == 0x7F, nan)
    assert torch.equal(got[~nan], want[~nan]), [(int(i), int(j), h[i, j].item(), int(got[i, j]), int(want[i, j]))
                                                 for i, j in (got != want).nonzero()[:8].tolist()]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("width,kept", [(8, False), (200, False), (128, False), (768, False), (2176, False),
                                        (128, True), (768, True), (2176, True)])
def test_silu_mul_grad(kind, width, kept):
    dev = device()
    groups, lead, live = grouped(kind, width)
    masked = kind == "masked"
    g = gen(width + 1)
    h = randn(g, *lead, 2 * width, std=3.0)
    da = randn(g, *lead, width, std=0.5)
    if kept:
        codes, scales = ref.quantise(h.cpu())
        hv = ref.value(codes, scales)[live.cpu()]
        codes[~live.cpu()] = 0x7F
        codes, scales = codes.cuda(), scales.cuda()
    else:
        hv = ref.f64(h)[live.cpu()]
        h[~live] = float("nan")
    da[~live] = float("nan")
    dh, act = sentinel_tensor((*lead, 2 * width), BF, dev), sentinel_tensor((*lead, width), BF, dev)
    b0, b1 = dh.clone(), act.clone()
    say("silu_mul_grad", kind, width, kept)
    if kept:
        gg.fp8_silu_mul_grad(da, codes, scales, groups, masked=masked, out=dh, act=act)
        alone = gg.fp8_silu_mul_grad(da, codes, scales, groups, masked=masked)
    else:
        gg.silu_mul_grad(da, h, groups, masked=masked, out=dh, act=act)
        alone = gg.silu_mul_grad(da, h, groups, masked=masked)
    torch.cuda.synchronize()
    want, slack = ref.silu_mul_grad(ref.f64(da[live]), hv)
    ref.close(dh[live], want, want.abs() * 2.0 ** -8 + slack, "dh")
    wa, sa = ref.silu_mul(hv)
    ref.close(act[live], wa, wa.abs() * 2.0 ** -8 + sa, "act")
    assert unchanged(dh, live, b0) and unchanged(act, live, b1), "rows nobody owns were written"
    assert torch.equal(alone[live], dh[live])


def test_silu_mul_grad_against_differences():
    device()
    g = gen(9)
    h, da = randn(g, 5, 32, std=2.0), randn(g, 5, 16)
    groups = torch.tensor([5], dtype=torch.int32, device="cuda")
    say("silu_mul_grad against differences")
    dh = gg.silu_mul_grad(da, h, groups)
    hd, dd, step = ref.f64(h), ref.f64(da), 1e-5
    for t, c in ((0, 0), (2, 15), (3, 16), (4, 31)):
        e = torch.zeros_like(hd)
        e[t, c] = step
        diff = float(((ref.silu_mul(hd + e)[0] - ref.silu_mul(hd - e)[0]) * dd).sum() / (2 * step))
        assert abs(float(dh[t, c]) - diff) <= 2.0 ** -8 * abs(diff) + 1e-5


def test_silu_extremes():
    """Gates far out on both sides give the limits, not NaN."""
    device()
    gate = torch.tensor([-3e38, -200.0, -100.0, -90.0, -30.0, 0.0, 90.0, 3e38])
    h = torch.cat([gate, torch.full((8,), 0.5)]).to(BF).reshape(1, 16).cuda()
    da = torch.ones(1, 8, dtype=BF, device="cuda")
    groups = torch.tensor([1], dtype=torch.int32, device="cuda")
    say("silu extremes")
    a = gg.silu_mul_rows(h, groups)
    dh, act = gg.silu_mul_grad(da, h, groups, with_act=True)
    hv = ref.f64(h)
    wa, sa = ref.silu_mul(hv)
    ref.close(a, wa, wa.abs() * 2.0 ** -8 + sa, "a")
    ref.close(act, wa, wa.abs() * 2.0 ** -8 + sa, "act")
    assert bool(torch.isfinite(dh).all())


# ---------------------------------------------------------------------------
# streams and graphs
# ---------------------------------------------------------------------------

def test_layer_steps_in_a_graph():
    """Every step captured once and replayed on new inputs, with eager work
    between the replays, gives the eager result each time."""
    dev = device()
    g = gen(21)
    tokens, topk, e, k, width = 200, 4, 8, 256, 128
    offs, row_slot, slot_row = routing(21, tokens, topk, e, 8, True, 0.02)
    cap = row_slot.shape[0]
    x, r, gamma = randn(g, tokens, k), randn(g, tokens, k), randn(g, k)
    hh, da, y, dout = randn(g, cap, 2 * width), randn(g, cap, width), randn(g, cap, k), randn(g, tokens, k)
    w = torch.rand(tokens, topk, generator=g, device=dev)
    ws = torch.empty(gg.rmsnorm_grad_workspace_bytes(tokens, k), dtype=U8, device=dev)
    zero = {"rows8": torch.zeros(cap, k, dtype=U8, device=dev),
            "packed": torch.zeros(gg.fp8_scale_bytes(gg.GG_FP8_ACT_RAGGED, cap, k, e), dtype=U8, device=dev),
            "dy": torch.zeros(cap, k, dtype=BF, device=dev), "a": torch.zeros(cap, width, dtype=BF, device=dev),
            "h8": torch.zeros(cap, 2 * width, dtype=U8, device=dev),
            "h8s": torch.zeros(cap, 2 * width // 128, dtype=U8, device=dev),
            "dh": torch.zeros(cap, 2 * width, dtype=BF, device=dev)}

    def steps():
        y8, s8, h = gg.fp8_rmsnorm(x, gamma, residual=r)
        rows8, packed = gg.fp8_gather_rows(y8, s8, row_slot, topk, offs, out=zero["rows8"], out_scales=zero["packed"])
        a, h8, h8s = gg.silu_mul_rows(hh, offs, keep=True, out=zero["a"], kept=zero["h8"], kept_scales=zero["h8s"])
        dh = gg.fp8_silu_mul_grad(da, h8, h8s, offs, out=zero["dh"])
        dy, dw = gg.combine_rows_grad(dout, y, slot_row, row_slot, offs, topk, weights=w, out=zero["dy"])
        dx, dgamma = gg.rmsnorm_grad(x, h, gamma, dh=r, workspace=ws)
        return y8, s8, h, rows8, packed, a, h8, h8s, dh, dy, dw, dx, dgamma

    say("layer steps in a graph")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        steps()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = steps()
    for trial in range(4):
        for t in (x, r, hh, da, y, dout):
            t.copy_(randn(g, *t.shape))
        torch.cuda.synchronize()
        eager = [t.clone() for t in steps()]
        for t in held:
            t.fill_(3)
        for name in ("rows8", "packed", "dy", "a", "h8", "h8s", "dh"):
            zero[name].zero_()
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(held, eager)):
            assert torch.equal(a.view(U8), b.view(U8)), (trial, i)


def test_two_streams_at_once():
    device()
    g = gen(31)
    x = [randn(g, 3000, 1024) for _ in range(2)]
    gamma = randn(g, 1024)
    dy = randn(g, 3000, 1024)
    want = [gg.rmsnorm_grad(dy, t, gamma) for t in x]
    torch.cuda.synchronize()
    say("rmsnorm_grad on two streams")
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    for i, s in enumerate(streams):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got[i] = gg.rmsnorm_grad(dy, x[i], gamma)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
