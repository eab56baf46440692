"""The expert layer for a few tokens against its formula in 64 bits: token
counts around the 16 of a matrix instruction, odd widths, dropped and repeated
slots, experts that everybody or nobody chose, values that are not finite, the
workspace's end, streams and graphs."""
import pytest
import torch

import fp4_ref
from layer_ref import HALF, U32, close
from moe_grouped_gemm_ragged_amd import binding as gg
from gpu_util import device, say

pytestmark = pytest.mark.gpu
BF, U8, I32 = torch.bfloat16, torch.uint8, torch.int32


class Layer:
    """Weights on the GPU, their 64-bit values, and the library's call."""

    def __init__(self, four, experts, hidden, inter, seed):
        g = torch.Generator().manual_seed(seed)
        self.four, self.experts, self.hidden, self.inter = four, experts, hidden, inter
        self.w13, self.v13, self.s13 = self._make(g, 2 * inter, hidden)
        self.w2, self.v2, self.s2 = self._make(g, hidden, inter)

    def _make(self, g, n, k):
        w = (torch.randn(self.experts, n, k, generator=g) * k ** -0.5).to(BF)
        if not self.four:
            return w.cuda(), w.double(), None
        codes, raw = fp4_ref.quantise(w.float())
        codes = fp4_ref.pack(codes)
        return codes.cuda(), fp4_ref.value(codes, raw), gg.fp4_pack_scales(gg.GG_FP4_WEIGHT, raw.cuda())

    def __call__(self, x, ids, weights=None, **kw):
        weights = None if weights is None else weights.cuda()
        if self.four:
            return gg.fp4_moe_few_tokens(x.cuda(), ids.cuda(), self.w13, self.s13, self.w2, self.s2, weights, **kw)
        return gg.moe_few_tokens(x.cuda(), ids.cuda(), self.w13, self.w2, weights, **kw)

    def check(self, got, x, ids, weights, what):
        """Bound: the two dot products of a (2 L 2^-24 of their terms' sizes, as the GEMMs' tests
        have it), through silu's slope (below 1.1), the activation's arithmetic and its rounding
        to bf16; then the down product over all slots, and the output's rounding."""
        tokens, topk = ids.shape
        ref = torch.zeros(tokens, self.hidden, dtype=torch.float64)
        slack, size = ref.clone(), ref.clone()
        xd = x.double()
        for e in sorted(set(ids.reshape(-1).tolist())):
            if not 0 <= e < self.experts:
                continue
            wt = ((ids == e) * (1.0 if weights is None else weights.double())).sum(-1)
            rows = (ids == e).any(-1)
            xe, we = xd[rows], wt[rows, None]
            h, hs = xe @ self.v13[e].t(), xe.abs() @ self.v13[e].abs().t()
            off = 2 * self.hidden * U32 * hs
            gate, up = h.split(self.inter, 1)
            og, ou = off.split(self.inter, 1)
            act = torch.nn.functional.silu(gate)
            a = we * act * up
            oa = we.abs() * (1.1 * og * (up.abs() + ou) + act.abs() * ou) + (2 * gate.abs() + 16 + topk) * U32 * a.abs()
            oa = oa + HALF[BF] * (a.abs() + oa)
            ref[rows] += a @ self.v2[e].t()
            slack[rows] += oa @ self.v2[e].abs().t()
            size[rows] += (a.abs() + oa) @ self.v2[e].abs().t()
        slack = slack + 2 * (self.inter + 16) * topk * U32 * size
        close(got, ref, slack + HALF[got.dtype] * (ref.abs() + slack), what)


def inputs(seed, tokens, topk, experts, hidden, drop=0.0, repeat=False):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(tokens, hidden, generator=g).to(BF)
    if repeat:
        ids = torch.randint(0, experts, (tokens, topk), generator=g)
    else:
        ids = torch.rand(tokens, experts, generator=g).topk(topk, dim=1).indices
    ids = ids.to(I32)
    if drop:
        lost = torch.rand(ids.shape, generator=g)
        ids[lost < drop] = -1
        ids[lost > 1 - drop] = experts
    return x, ids.contiguous(), torch.rand(tokens, topk, generator=g)


SIZES = [  # tokens, topk, experts, hidden, inter (multiples of 32; bf16 takes 8 off each)
    (1, 1, 1, 32, 32), (1, 8, 16, 512, 96), (2, 2, 3, 160, 32), (15, 3, 8, 288, 160), (16, 4, 5, 96, 64),
    (17, 2, 40, 256, 128), (33, 8, 12, 544, 288), (64, 8, 20, 128, 32), (64, 1, 2, 1056, 544), (64, 8, 8, 416, 96), (16, 8, 8, 1024, 64)]


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("tokens,topk,experts,hidden,inter", SIZES)
@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_layer(four, tokens, topk, experts, hidden, inter, dtype):
    device()
    if not four:
        hidden, inter = hidden - 8, inter - 8
    layer = Layer(four, experts, hidden, inter, tokens)
    x, ids, weights = inputs(tokens + hidden, tokens, topk, experts, hidden, drop=0.1 if tokens > 8 else 0.0)
    say("few tokens", four, tokens, topk, experts, hidden, inter, dtype)
    got = layer(x, ids, weights, out_dtype=dtype)
    torch.cuda.synchronize()
    layer.check(got, x, ids, weights, "layer")


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("tokens,topk,hidden", [(1, 2, 4096), (6, 3, 4128), (40, 2, 4128), (64, 4, 4224)])
def test_wide(four, tokens, topk, hidden):
    """Rows enough for two strips a workgroup in the down product of 4 bits; a
    last span that ends after 32 rows."""
    device()
    layer = Layer(four, 5, hidden, 160, 7)
    x, ids, weights = inputs(tokens, tokens, topk, 5, hidden, drop=0.1 if tokens > 8 else 0.0)
    say("few tokens: wide", four, tokens, topk, hidden)
    layer.check(layer(x, ids, weights), x, ids, weights, "wide")


@pytest.mark.parametrize("four", [False, True])
def test_slots(four):
    """No weights; every token one expert; an expert named twice; all dropped."""
    device()
    layer = Layer(four, 9, 160, 96, 3)
    x, ids, weights = inputs(1, 40, 4, 9, 160, repeat=True)
    say("few tokens: repeated slots", four)
    layer.check(layer(x, ids, weights), x, ids, weights, "repeated")
    layer.check(layer(x, ids), x, ids, None, "without weights")
    same = torch.full_like(ids, 8)
    say("few tokens: one expert", four)
    layer.check(layer(x, same, weights), x, same, weights, "one expert")
    ids[:5] = -1
    ids[5:9] = 9
    ids[9:12] = 1 << 30
    ids[12] = -(1 << 31)
    say("few tokens: dropped", four)
    got = layer(x, ids, weights)
    layer.check(got, x, ids, weights, "dropped")
    assert bool((got[:13] == 0).all())
    got = layer(x, torch.full_like(ids, -1), weights)
    assert bool((got == 0).all())


@pytest.mark.parametrize("four", [False, True])
def test_most_experts_and_slots(four):
    """2048 experts, 512 slots of 64 tokens; slots of few tokens."""
    device()
    layer = Layer(four, 2048, 32, 32, 4)
    for tokens, topk in ((64, 8), (1, 512), (3, 170), (31, 9)):
        x, ids, weights = inputs(tokens, tokens, topk, 2048, 32)
        ids[0, 0] = 2047
        say("few tokens: 2048 experts", four, tokens, topk)
        layer.check(layer(x, ids, weights, out_dtype=torch.float32), x, ids, weights, "2048 experts")


@pytest.mark.parametrize("four", [False, True])
def test_not_finite(four):
    """A token's NaN stays in its row; an expert's reaches its own tokens only."""
    device()
    layer = Layer(four, 6, 96, 64, 5)
    x, ids, weights = inputs(2, 20, 2, 6, 96)
    clean = layer(x, ids, weights)
    x[3, 7] = float("nan")
    x[19, 95] = float("inf")
    say("few tokens: NaN in x", four)
    got = layer(x, ids, weights)
    rows = torch.ones(20, dtype=torch.bool)
    rows[[3, 19]] = False
    assert torch.equal(got[rows.cuda()], clean[rows.cuda()])
    assert bool(torch.isnan(got[3]).all()) and bool((~torch.isfinite(got[19])).all())
    x, ids, weights = inputs(2, 20, 2, 6, 96)
    if four:
        raw = torch.full((6, 96, 2), 120, dtype=U8)
        raw[2] = 255
        layer.s2 = gg.fp4_pack_scales(gg.GG_FP4_WEIGHT, raw.cuda())
        raw[2] = 120
        clean = gg.fp4_moe_few_tokens(x.cuda(), ids.cuda(), layer.w13, layer.s13, layer.w2,
                                      gg.fp4_pack_scales(gg.GG_FP4_WEIGHT, raw.cuda()), weights.cuda())
    else:
        layer.w2[2] = float("inf")
    say("few tokens: an expert's weights not finite", four)
    got = layer(x, ids, weights)
    has = (ids == 2).any(-1).cuda()
    assert bool(has.any()) and bool((~has).any())
    assert torch.equal(got[~has], clean[~has])
    assert bool((~torch.isfinite(got[has])).all())


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("tokens", [5, 37])
def test_workspace_stream_graph(four, tokens):
    """The workspace's contents do not matter and its end is respected; another
    stream; a captured call replayed on new inputs and ids; the same call twice
    gives the same bits."""
    dev = device()
    layer = Layer(four, 11, 288, 96, 6)
    sets = [inputs(s, tokens, 3, 11, 288, drop=0.1) for s in range(3)]
    need = gg.moe_few_tokens_workspace_bytes(tokens, 3, 96, 11)
    ws = torch.full((need + 64,), 0xFF, dtype=U8, device=dev)
    say("few tokens: workspace", four, tokens)
    want = [layer(*s).clone() for s in sets]
    got = layer(*sets[0], workspace=ws)
    assert torch.equal(got, want[0]) and bool((ws[need:] == 0xFF).all())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = layer(*sets[1], workspace=ws)
    side.synchronize()
    assert torch.equal(got, want[1])
    say("few tokens: graph", four, tokens)
    x, ids, weights = (t.cuda() for t in sets[0])
    out = torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        layer(x, ids, weights, out=out, workspace=ws)
    for i in (0, 1, 2, 2, 0):
        for t, s in zip((x, ids, weights), sets[i]):
            t.copy_(s)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i])
        assert torch.equal(layer(*sets[1]), want[1])


@pytest.mark.parametrize("four", [False, True])
def test_two_at_once(four):
    """Two captured calls with a workspace each, replayed at the same time on two
    streams; with one workspace, one after the other; out in x's place."""
    dev = device()
    layer = Layer(four, 24, 1056, 288, 8)
    sets = [tuple(t.cuda() for t in inputs(40 + s, tokens, 4, 24, 1056)) for s, tokens in enumerate((7, 50))]
    want = [layer(*s).clone() for s in sets]
    say("few tokens: two at once", four)
    shared = torch.empty(gg.moe_few_tokens_workspace_bytes(50, 4, 288, 24), dtype=U8, device=dev)
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()

    def capture(spaces):
        graphs, outs = [], []
        for s, ws in zip(sets, spaces):
            outs.append(torch.empty_like(s[0]))
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1]):
                layer(*s, out=outs[-1], workspace=ws)
        return graphs, outs
    own = [torch.empty_like(shared) for _ in sets]
    graphs, outs = capture(own)
    for _ in range(10):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for g, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
    graphs, outs = capture([shared, shared])
    for _ in range(5):
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
    for (x, ids, weights), w in zip(sets, want):
        x = x.clone()
        assert layer(x, ids, weights, out=x) is x
        assert torch.equal(x, w)
