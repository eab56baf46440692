"""Workloads of the 4-bit operators and of the expert layer for a few tokens:
what each computes in plain torch, and the library's calls for the same.

* ``rows``    bf16 rows to 4 bits (e2m1 codes, one power-of-two scale per 32
              values, the scales in the packed layout that the product reads)
              and back to bf16
* ``gemm``    the grouped product of 4-bit rows with 4-bit weights
* ``gateup``  tokens sorted by expert into 4-bit rows, and the gate/up product
* ``down``    SiLU(gate) * up of grouped rows into 4-bit rows, and the down product
* ``layer``   the whole expert layer (gate/up, SiLU-mul, down, weighted sum) for
              a few tokens, with bf16 or with 4-bit weights

``listed()`` gives the fixed cases and ``draw(rng)`` more of the same ranges;
``prepare`` makes a case's inputs, ``run`` computes it once (in plain torch,
or through the library where ``own`` is true), ``exact`` is the definition in
64 bits, ``work`` the bytes and operations a case cannot do without.
"""
import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def listed():
    return [
        # a prompt's activations to 4 bits and back: what a product in 4 bits sees of them
        dict(name="rows4_prompt", op="rows", layout="ragged", rows=65536, k=2048, experts=128, spare=512),
        # one layer's weights as they are loaded
        dict(name="rows4_weights", op="rows", layout="weight", rows=1536, k=2048, experts=64, spare=0),
        # long experts of a wide layer: the matrix cores
        dict(name="gemm4_long", op="gemm", masked=False, rows=65536, k=6144, n=4096, experts=32, spare=0),
        # the down projection of a rollout on the masked layout
        dict(name="gemm4_masked", op="gemm", masked=True, rows=256, k=768, n=2048, experts=64, spare=0),
        # a prompt's gate/up projection from its tokens
        dict(name="gateup4_prompt", op="gateup", tokens=8192, topk=8, experts=128, k=2048, n=1536, align=16, drop=0.0),
        # the same for a decoding batch of odd size, some slots dropped: nearly all tiles almost empty
        dict(name="gateup4_decode", op="gateup", tokens=33, topk=8, experts=128, k=2048, n=1536, align=1, drop=0.02),
        # a prompt's down projection from its gate/up rows
        dict(name="down4_prompt", op="down", masked=False, rows=65536, k=768, n=2048, experts=128, spare=65),
        # a decoding step on the masked layout, a few rows of an expert
        dict(name="down4_masked", op="down", masked=True, rows=8, k=2048, n=7168, experts=64, spare=0),
        # one token of a decoding step, bf16 weights: nothing but eight experts' weights
        dict(name="layer_token", op="layer", four=False, tokens=1, topk=8, experts=128, hidden=2048, inter=768, drop=0.0),
        # an odd batch that reaches most experts
        dict(name="layer_batch", op="layer", four=False, tokens=23, topk=8, experts=128, hidden=2048, inter=768,
             drop=0.03),
        # one token, weights in 4 bits
        dict(name="layer4_token", op="layer", four=True, tokens=1, topk=8, experts=128, hidden=2048, inter=768, drop=0.0),
        # a few tokens of a wide layer, weights in 4 bits
        dict(name="layer4_wide", op="layer", four=True, tokens=4, topk=8, experts=64, hidden=7168, inter=2048, drop=0.0),
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of step between lo and hi, spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(hi // step * step, max(step, int(v) // step * step))


def draw(rng):
    op = rng.choice(["rows", "gemm", "gateup", "down", "layer"])
    if op == "rows":
        layout = rng.choice(["ragged", "masked", "weight"])
        k, experts = _log(rng, 64, 7168, 32), _log(rng, 4, 128)
        most = 65536 * 2048 // k
        rows = _log(rng, 1, most) if layout == "ragged" else _log(rng, 1, max(1, most // experts))
        return dict(op=op, layout=layout, rows=rows, k=k, experts=experts,
                    spare=rng.choice([0, 65]) if layout == "ragged" else 0)
    if op in ("gemm", "down"):
        masked, experts = rng.random() < 0.4, _log(rng, 4, 128)
        k, n = _log(rng, 64, 2048, 32), _log(rng, 64, 2048, 8)
        rows = _log(rng, 1, 256) if masked else _log(rng, 16, 32768)
        return dict(op=op, masked=masked, rows=rows, k=k, n=n, experts=experts, spare=0 if masked else rng.choice([0, 65]))
    if op == "gateup":
        return dict(op=op, tokens=_log(rng, 1, 4096), topk=rng.choice([1, 2, 4, 5, 6, 8]), experts=_log(rng, 8, 128),
                    k=_log(rng, 64, 2048, 32), n=_log(rng, 64, 1536, 8), align=rng.choice([1, 8, 16]),
                    drop=rng.choice([0.0, 0.02]))
    four = rng.random() < 0.5
    step = 32 if four else 8
    return dict(op=op, four=four, tokens=_log(rng, 1, 64), topk=rng.choice([1, 2, 4, 5, 6, 8]),
                experts=_log(rng, 8, 128), hidden=_log(rng, 128, 2048, step), inter=_log(rng, 64, 1024, step),
                drop=rng.choice([0.0, 0.05]))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _randn(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(torch.bfloat16)


def _sizes(c, g, masked):
    """Rows of each expert: a ragged split of c["rows"] over skewed
    probabilities with empty experts, or counts up to c["rows"] (masked)."""
    e = c["experts"]
    if masked:
        counts = torch.randint(0, c["rows"] + 1, (e,), generator=g, device="cuda")
        counts[int(torch.randint(0, e, (1,), generator=g, device="cuda"))] = c["rows"]
        counts[0] = 0
        return counts
    p = torch.randn(e, generator=g, device="cuda").exp()
    p[::max(2, e // 2)] = 0.0
    of = torch.multinomial(p, c["rows"], replacement=True, generator=g)
    return torch.bincount(of, minlength=e)


def _grouped(c, g, masked):
    """The grouped layout: groups as the library takes them, for every row its
    expert, its place in it and whether an expert owns it, and all rows."""
    counts = _sizes(c, g, masked)
    if masked:
        groups, start = counts.to(torch.int32), torch.arange(c["experts"], device="cuda") * c["rows"]
        total = c["experts"] * c["rows"]
    else:
        groups = torch.cumsum(counts, 0).to(torch.int32)
        start, total = groups.long() - counts, c["rows"] + c["spare"]
    row = torch.arange(total, device="cuda")
    # empty experts share their first row with the next one: the last of them owns it
    expert = torch.searchsorted(start, row, right=True) - 1
    place = row - start[expert]
    return dict(groups=groups, start=start, counts=counts, expert=expert, place=place, ok=place < counts[expert],
                total=total, longest=max(1, int(counts.max())))


def _routing(c, g):
    """Top-k experts of every token, and the layout that sorting them gives:
    padded end offsets, each row's slot (-1: padding)."""
    t, k, e, a = c["tokens"], c["topk"], c["experts"], c["align"]
    skew = torch.randn(e, generator=g, device="cuda") * 0.8
    noise = -torch.log(-torch.log(torch.rand(t, e, generator=g, device="cuda").clamp(1e-9, 1 - 1e-7)))
    ids = (skew + noise).topk(k, dim=1).indices.reshape(-1)
    if c["drop"]:
        ids = torch.where(torch.rand(t * k, generator=g, device="cuda") < c["drop"], e, ids)
    counts = torch.bincount(ids, minlength=e + 1)
    padded = (counts[:e] + a - 1) // a * a
    ends = torch.cumsum(padded, 0)
    first = torch.cumsum(counts, 0) - counts
    order = torch.sort(ids, stable=True).indices
    kept = order[:t * k - int(counts[e])]
    of = ids[kept]
    row = ends[of] - padded[of] + torch.arange(kept.numel(), device="cuda") - first[of]
    total = t * k + e * a
    row_slot = torch.full((total,), -1, dtype=torch.int32, device="cuda")
    row_slot[row] = kept.to(torch.int32)
    start = ends - padded
    at = torch.arange(total, device="cuda")
    expert = torch.searchsorted(start, at, right=True) - 1
    place = at - start[expert]
    return dict(groups=ends.to(torch.int32), start=start, counts=padded, expert=expert, place=place,
                ok=place < padded[expert], total=total, longest=max(1, int(padded.max())), row_slot=row_slot)


def _scale_size(rows, k, experts, ragged):
    tiles = -(-rows // 256) + experts if ragged else -(-rows // 256) * experts
    return tiles * -(-k // 128) * 1024


def _packed_place(tile, r, k, stages):
    """Where the packed layout keeps the scale of tile row r and each block of
    32 values: 1024 bytes per tile of 256 rows and 128 values."""
    b = torch.arange(k // 32, device="cuda")
    at = (tile * stages * 1024 + 512 * (r // 128) + 16 * (r % 32) + (r // 32) % 4)[:, None]
    return at + (b // 4) * 1024 + 8 * (b % 2) + 4 * ((b % 4) // 2)


def _weights4(g, experts, n, k):
    """e2m1 codes [E, n, k / 2] (small magnitudes more often, as weights have
    them), a scale byte for every 32 values, and those bytes packed."""
    def byte():
        return torch.randint(0, 256, (experts, n, k // 2), generator=g, device="cuda", dtype=torch.uint8)
    a, b = byte(), byte()
    low, high = torch.minimum(a & 7, b & 7), torch.minimum(a & 0x70, b & 0x70)
    codes = low.bitwise_or_(high).bitwise_or_(a.bitwise_and_(0x88))
    raw = torch.randint(118, 122, (experts, n, k // 32), generator=g, device="cuda", dtype=torch.uint8)
    row = torch.arange(experts * n, device="cuda")
    e, r = row // n, row % n
    stages = -(-k // 128)
    packed = torch.zeros(_scale_size(n, k, experts, False), dtype=torch.uint8, device="cuda")
    at = _packed_place(e * -(-n // 256) + r // 256, r % 256, k, stages)
    packed[at.reshape(-1)] = raw.reshape(-1)
    return codes, raw, packed


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = c["op"]
    s = {"case": c}
    if op == "rows":
        k, e = c["k"], c["experts"]
        if c["layout"] == "weight":
            lead, ragged = (e, c["rows"]), False
            ok = torch.ones(e * c["rows"], dtype=torch.bool, device="cuda")
            s["groups"] = None
        else:
            ragged = c["layout"] == "ragged"
            d = _grouped(c, g, not ragged)
            lead, ok = (d["total"],) if ragged else (e, c["rows"]), d["ok"]
            s["groups"] = d["groups"]
        x = _randn(g, ok.numel(), k, std=0.02 if c["layout"] == "weight" else 1.0)
        x[~ok] = float("nan")                       # rows nobody owns hold anything
        s.update(ok=ok, x=x.reshape(*lead, k), codes=torch.zeros(*lead, k // 2, dtype=torch.uint8, device="cuda"),
                 packed=torch.zeros(_scale_size(lead[0] if ragged else c["rows"], k, e, ragged), dtype=torch.uint8,
                                    device="cuda"),
                 out=torch.zeros(*lead, k, dtype=torch.bfloat16, device="cuda"))
        return s
    if op == "layer":
        t, h, i, e = c["tokens"], c["hidden"], c["inter"], c["experts"]
        ids = torch.rand(t, e, generator=g, device="cuda").topk(min(c["topk"], e), dim=1).indices.to(torch.int32)
        if c["drop"]:
            ids = torch.where(torch.rand(ids.shape, generator=g, device="cuda") < c["drop"], -1, ids)
        w = torch.rand(ids.shape, generator=g, device="cuda")
        s.update(x=_randn(g, t, h), ids=ids.contiguous(), weights=w / w.sum(-1, keepdim=True))
        if c["four"]:
            s["w13"], s["w13_raw"], s["w13_scales"] = _weights4(g, e, 2 * i, h)
            s["w2"], s["w2_raw"], s["w2_scales"] = _weights4(g, e, h, i)
        else:
            s["w13"], s["w2"] = _randn(g, e, 2 * i, h, std=h ** -0.5), _randn(g, e, h, i, std=i ** -0.5)
        return s
    k, n, e = c["k"], c["n"], c["experts"]
    s["w"], s["w_raw"], s["w_scales"] = _weights4(g, e, n, k)
    if op == "gateup":
        s.update(_routing(c, g), x=_randn(g, c["tokens"], k))
        s["codes"] = torch.zeros(s["total"], k // 2, dtype=torch.uint8, device="cuda")
        s["packed"] = torch.zeros(_scale_size(s["total"], k, e, True), dtype=torch.uint8, device="cuda")
        s["out"] = torch.zeros(s["total"], n, dtype=torch.bfloat16, device="cuda")
        return s
    masked = c["masked"]
    s.update(_grouped(c, g, masked))
    lead = (e, c["rows"]) if masked else (s["total"],)
    s["out"] = torch.zeros(*lead, n, dtype=torch.bfloat16, device="cuda")
    per, stages = -(-c["rows"] // 256), -(-k // 128)
    if op == "down":
        h = _randn(g, s["total"], 2 * k, std=1.2)
        h[~s["ok"]] = float("nan")
        s["h"] = h.reshape(*lead, 2 * k)
        s["codes"] = torch.zeros(*lead, k // 2, dtype=torch.uint8, device="cuda")
        s["packed"] = torch.zeros(_scale_size(lead[1] if masked else s["total"], k, e, not masked), dtype=torch.uint8,
                                  device="cuda")
        return s
    codes, raw = _weights4(g, 1, s["total"], k)[:2]
    codes, raw = codes[0], raw[0] + 8
    n256 = (s["counts"] + 255) // 256
    tile = s["expert"] * per if masked else (torch.cumsum(n256, 0) - n256)[s["expert"]]
    at, ok = _packed_place(tile + s["place"] // 256, s["place"] % 256, k, stages), s["ok"]
    packed = torch.zeros(_scale_size(c["rows"] if masked else s["total"], k, e, not masked), dtype=torch.uint8,
                         device="cuda")
    packed[at[ok].reshape(-1)] = raw[ok].reshape(-1)
    codes[~ok] = 0xFF
    s.update(x=codes.reshape(*lead, k // 2), x_raw=raw, x_scales=packed)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return _own(op, state)
    return {"rows": _rows, "gemm": _gemm, "gateup": _gateup, "down": _down, "layer": _layer}[op](state)


def _own(op, s):
    from moe_grouped_gemm_ragged_amd import binding as gg
    c = s["case"]
    if op == "rows":
        layout = {"ragged": gg.GG_FP4_ACT_RAGGED, "masked": gg.GG_FP4_ACT_MASKED, "weight": gg.GG_FP4_WEIGHT}[c["layout"]]
        codes, scales = gg.fp4_quantize(layout, s["x"], s["groups"], out=s["codes"], out_scales=s["packed"])
        return gg.fp4_dequantize(layout, codes, scales, s["groups"], out=s["out"])
    if op == "layer":
        if c["four"]:
            return gg.fp4_moe_few_tokens(s["x"], s["ids"], s["w13"], s["w13_scales"], s["w2"], s["w2_scales"],
                                         weights=s["weights"])
        return gg.moe_few_tokens(s["x"], s["ids"], s["w13"], s["w2"], weights=s["weights"])
    if op == "gateup":
        x, scales = gg.fp4_gather_rows(s["x"], s["row_slot"], c["topk"], s["groups"], out=s["codes"],
                                       out_scales=s["packed"])
        return gg.fp4_forward(x, scales, s["w"], s["w_scales"], s["groups"], out=s["out"])
    if op == "down":
        x, scales = gg.fp4_silu_mul_rows(s["h"], s["groups"], masked=c["masked"], out=s["codes"], out_scales=s["packed"])
    else:
        x, scales = s["x"], s["x_scales"]
    product = gg.fp4_masked_forward if c["masked"] else gg.fp4_forward
    return product(x, scales, s["w"], s["w_scales"], s["groups"], out=s["out"])


def _pow2(e):
    return ((e + 127) << 23).view(torch.float32)


def _to4(v):
    """What the 4-bit rows of v [rows, k] stand for, in v's type: blocks of 32
    with the smallest power of two s with amax / s <= 6 (1 for a block of
    zeros), every value to the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 times s,
    ties to the even code."""
    b = v.reshape(v.shape[0], -1, 32)
    amax = b.abs().amax(-1)
    frac, e = torch.frexp(amax.float())             # 6 = 0.75 * 2^3
    e = torch.where(amax == 0, 0, e - 3 + (frac > 0.75).to(e.dtype)).clamp(-126, 127).to(torch.int32)
    s = _pow2(e).to(v.dtype)[..., None]
    m = b / s
    step = torch.where(m.abs() < 2, 0.5, torch.where(m.abs() < 4, 1.0, 2.0)).to(v.dtype)
    return (torch.round(m / step) * step * s).reshape(v.shape)


def _from4(codes, raw):
    """fp32 values of e2m1 codes [..., k / 2] with scale bytes [..., k / 32]."""
    table = torch.tensor(E2M1, device="cuda")
    nibbles = torch.stack([codes & 15, codes >> 4], dim=-1)
    v = torch.index_select(table, 0, nibbles.reshape(-1).int())
    return (v.reshape(*raw.shape, 32) * _pow2(raw.int() - 127)[..., None]).reshape(*codes.shape[:-1], -1)


def _product(s, x, w):
    """Every row of x [total, k] with its expert's w [E, n, k]: the experts'
    rows side by side, padded with zeros to the longest."""
    place = torch.arange(s["longest"], device="cuda")
    inside = place < s["counts"][:, None]
    at = torch.where(inside, s["start"][:, None] + place, 0)
    y = torch.matmul(torch.where(inside[..., None], x[at], 0.0), w.transpose(1, 2).contiguous())
    ok = s["ok"]
    back = torch.where(ok, s["expert"] * s["longest"] + s["place"], 0)
    y = torch.where(ok[:, None], y.reshape(-1, y.shape[-1])[back], 0.0)
    return y.to(torch.bfloat16).reshape(s["out"].shape)


def _rows(s):
    x = s["x"].reshape(s["ok"].numel(), -1).float()
    return _to4(torch.where(s["ok"][:, None], x, 0.0)).to(torch.bfloat16).reshape(s["x"].shape)


def _gemm(s):
    x = _from4(s["x"].reshape(s["total"], -1), s["x_raw"])
    return _product(s, x, _from4(s["w"], s["w_raw"]))


def _gateup(s):
    slot = s["row_slot"].long()
    x = s["x"].float()[slot.clamp(min=0) // s["case"]["topk"]]
    return _product(s, _to4(torch.where((slot >= 0)[:, None], x, 0.0)), _from4(s["w"], s["w_raw"]))


def _down(s):
    # in 64 bits up to the rounding to 4, whose borders a value may lie next to
    k = s["case"]["k"]
    h = torch.where(s["ok"][:, None], s["h"].reshape(s["total"], 2 * k).double(), 0.0)
    gate, up = h[:, :k], h[:, k:]
    return _product(s, _to4(gate / (1.0 + torch.exp(-gate)) * up).float(), _from4(s["w"], s["w_raw"]))


def _layer(s):
    c, i = s["case"], s["case"]["inter"]
    x, ids = s["x"].float(), s["ids"].long()
    there = (ids >= 0) & (ids < c["experts"])
    wt, ids = torch.where(there, s["weights"], 0.0), torch.where(there, ids, 0)
    few = ids.numel() <= c["experts"]               # the slots' experts, or all of them

    def weights(name):
        w = s[name][ids.reshape(-1)] if few else s[name]
        if not c["four"]:
            return w.float()
        return _from4(w, s[name + "_raw"][ids.reshape(-1)] if few else s[name + "_raw"])

    if few:
        rows = x.repeat_interleave(ids.shape[1], 0)[..., None]
        h = torch.matmul(weights("w13"), rows)[..., 0]
        a = h[:, :i] / (1.0 + torch.exp(-h[:, :i])) * h[:, i:]
        y = torch.matmul(weights("w2"), a[..., None])[..., 0].reshape(*ids.shape, -1)
        return (y * wt[..., None]).sum(1).to(torch.bfloat16)
    share = torch.zeros(c["experts"], c["tokens"], device="cuda")
    share.index_put_((ids, torch.arange(c["tokens"], device="cuda")[:, None].expand_as(ids)), wt, accumulate=True)
    h = torch.matmul(x[None].expand(c["experts"], -1, -1), weights("w13").transpose(1, 2).contiguous())
    a = h[..., :i] / (1.0 + torch.exp(-h[..., :i])) * h[..., i:] * share[..., None]
    return torch.matmul(a, weights("w2").transpose(1, 2).contiguous()).sum(0).to(torch.bfloat16)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    c, op = s["case"], s["case"]["op"]
    if op == "layer":
        return _exact_layer(s)
    if op == "rows":
        x = s["x"].reshape(s["ok"].numel(), c["k"]).masked_fill(~s["ok"][:, None], 0.0)
        out = torch.empty(x.shape, dtype=torch.float64, device="cuda")
        for at in range(0, x.shape[0], 16384):
            out[at:at + 16384] = _nearest4(x[at:at + 16384].double())
        return out.reshape(s["x"].shape)
    out = torch.zeros(s["total"], c["n"], dtype=torch.float64, device="cuda")
    for e, (first, count) in enumerate(zip(s["start"].tolist(), s["counts"].tolist())):
        if not count:
            continue
        rows = slice(first, first + count)
        if op == "gemm":
            x = _value4(s["x"].reshape(s["total"], -1)[rows], s["x_raw"][rows])
        elif op == "gateup":
            slot = s["row_slot"][rows]
            x = s["x"].double()[torch.div(slot.clamp(min=0), c["topk"], rounding_mode="floor").long()]
            x = _nearest4(x.masked_fill((slot < 0)[:, None], 0.0))
        else:
            gate, up = s["h"].reshape(s["total"], -1)[rows].double().split(c["k"], dim=1)
            x = _nearest4(torch.nn.functional.silu(gate) * up)
        out[rows] = x @ _value4(s["w"][e], s["w_raw"][e]).t()
    return out.reshape(s["out"].shape)


def _exact_layer(s):
    c, i = s["case"], s["case"]["inter"]
    out = torch.zeros(c["tokens"], c["hidden"], dtype=torch.float64, device="cuda")
    x = s["x"].double()
    for e in sorted(set(s["ids"].reshape(-1).tolist())):
        if not 0 <= e < c["experts"]:
            continue
        if c["four"]:
            w13, w2 = _value4(s["w13"][e], s["w13_raw"][e]), _value4(s["w2"][e], s["w2_raw"][e])
        else:
            w13, w2 = s["w13"][e].double(), s["w2"][e].double()
        share = (s["weights"].double() * (s["ids"] == e)).sum(-1)
        gate, up = (x @ w13.t()).split(i, dim=1)
        out += share[:, None] * ((torch.nn.functional.silu(gate) * up) @ w2.t())
    return out


def _value4(codes, raw):
    """64-bit values of e2m1 codes (sign, two exponent bits, one mantissa bit;
    the low half of a byte first) with scale bytes."""
    nibble = torch.empty(*codes.shape[:-1], 2 * codes.shape[-1], dtype=torch.int32, device="cuda")
    nibble[..., 0::2], nibble[..., 1::2] = codes & 15, codes >> 4
    e, m = (nibble >> 1) & 3, (nibble & 1).double()
    v = torch.where(e == 0, m / 2, (1 + m / 2) * torch.exp2((e - 1).double()))
    v = torch.where(nibble >= 8, -v, v)
    return v * torch.exp2(raw.double() - 127).repeat_interleave(32, dim=-1)


def _nearest4(v):
    """Blocks of 32 to the nearest e2m1 value times the block's scale, found by
    the borders between neighbours; a value on a border goes to the even code."""
    b = v.reshape(v.shape[0], -1, 32)
    amax = b.abs().amax(-1, keepdim=True)
    s = torch.where(amax > 0, torch.exp2(torch.ceil(torch.log2(amax / 6)).clamp(min=-126)), 1.0)
    m = b.abs() / s
    q = torch.zeros_like(m)
    for border, to, even in ((0.25, 0.5, False), (0.75, 1.0, True), (1.25, 1.5, False), (1.75, 2.0, True),
                             (2.5, 3.0, False), (3.5, 4.0, True), (5.0, 6.0, False)):
        q = torch.where((m >= border) if even else (m > border), to, q)
    return (torch.where(b < 0, -q, q) * s).reshape(v.shape)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    """Bytes and operations of one pass, each input read once and each output
    written once (the expected number of rows or experts where they are drawn)."""
    c, op = case, case["op"]
    if op == "layer":
        t, h, i, e = c["tokens"], c["hidden"], c["inter"], c["experts"]
        slots = t * min(c["topk"], e) * (1 - c["drop"])
        reached = e * (1 - (1 - slots / t / e) ** t)
        per = 17 / 32 if c["four"] else 2
        return {"bytes": reached * 3 * h * i * per + 4 * t * h, "flops": 6 * slots * h * i}
    if op == "rows":
        rows = c["rows"] * c["experts"] if c["layout"] == "weight" else c["rows"]
        if c["layout"] == "masked":
            rows = c["rows"] * c["experts"] // 2
        return {"bytes": rows * c["k"] * (2 + 2 * 17 / 32 + 2), "flops": 4 * rows * c["k"]}
    k, n, e = c["k"], c["n"], c["experts"]
    if op == "gateup":
        rows = c["tokens"] * c["topk"]
        reached = min(e, rows)
        b = c["tokens"] * k * 2 + rows * 2 * n + reached * n * k * 17 / 32
        return {"bytes": b, "flops": 2 * rows * k * n}
    rows = e * c["rows"] // 2 if c["masked"] else c["rows"]
    x = rows * k * (17 / 32 if op == "gemm" else 4)
    return {"bytes": x + min(e, rows) * n * k * 17 / 32 + rows * n * 2, "flops": 2 * rows * k * n}
