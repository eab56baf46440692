"""Host-side checks of the 4-bit entry points (no GPU needed): bad arguments
get their status before anything is enqueued, and the binding refuses tensors
that do not fit."""
import pytest
import torch

from moe_grouped_gemm_ragged_amd import binding as gg

A = 0x10000       # fake, 16-byte aligned: rejected before any use
BIG = (1 << 31) - (1 << 16)
POINTERS = {"x", "src", "offs", "codes", "scales", "dst", "out", "rs", "h", "xs", "w", "ws", "y"}

PACK = dict(layout=0, src=A, ld=8, offs=A, rows=4, k=256, e=4, dst=A, s=None)
QUANT = dict(layout=0, x=A, offs=A, rows=4, k=256, e=4, codes=A, scales=A, s=None)
GATHER = dict(src=A, tokens=4, k=256, rs=A, topk=2, offs=A, e=4, cap=40, codes=A, scales=A, s=None)
SILU = dict(h=A, offs=A, codes=A, scales=A, m=4, n=256, e=4, s=None)
BACK = dict(layout=0, codes=A, scales=A, offs=A, rows=4, k=256, e=4, out=A, s=None)
FWD = dict(x=A, xs=A, w=A, ws=A, offs=A, y=A, dt=0, m=4, k=256, n=64, e=4, s=None)


@pytest.fixture(scope="module")
def lib():
    return gg.load()


def run(name, defaults, case):
    v = dict(defaults, **case)
    return gg.call_raw(name, *[(x or None) if k in POINTERS else x for k, x in v.items()])


SIZES = [(dict(k=0), 2), (dict(k=16), 2), (dict(k=48), 2), (dict(k=(1 << 20) + 32), 2), (dict(e=0), 5), (dict(e=2049), 5)]
ROWS = [(dict(rows=-1), 2), (dict(rows=BIG), 2), (dict(layout=1, rows=1 << 24, e=256), 2),
        (dict(layout=2, rows=1 << 24, e=256), 2), (dict(layout=3), 2), (dict(layout=-1), 2), (dict(offs=0), 1),
        (dict(offs=A + 2), 3)]


@pytest.mark.parametrize("name,defaults,case,status", [
    *[("gg_fp4_pack_scales", PACK, c, s) for c, s in SIZES + ROWS + [
        (dict(src=0), 1), (dict(dst=0), 1), (dict(ld=7), 2), (dict(dst=A + 8), 3), (dict(ld=1 << 61), 2)]],
    *[("gg_fp4_quantize", QUANT, c, s) for c, s in SIZES + ROWS + [
        (dict(x=0), 1), (dict(codes=0), 1), (dict(scales=0), 1), (dict(x=A + 8), 3), (dict(codes=A + 4), 3),
        (dict(scales=A + 8), 3)]],
    *[("gg_fp4_dequantize", BACK, c, s) for c, s in SIZES + ROWS + [
        (dict(codes=0), 1), (dict(out=0), 1), (dict(scales=0), 1), (dict(out=A + 8), 3), (dict(codes=A + 4), 3)]],
    *[("gg_fp4_gather_rows", GATHER, c, s) for c, s in SIZES + [
        (dict(src=0), 1), (dict(rs=0), 1), (dict(offs=0), 1), (dict(codes=0), 1), (dict(scales=0), 1),
        (dict(tokens=-1), 2), (dict(topk=0), 2), (dict(cap=-1), 2), (dict(cap=BIG), 2), (dict(tokens=1 << 30), 2),
        (dict(tokens=1 << 40), 2), (dict(src=A + 8), 3), (dict(rs=A + 2), 3), (dict(codes=A + 8), 3)]],
    *[(n, SILU, c, s) for n in ("gg_fp4_silu_mul_rows", "gg_fp4_masked_silu_mul_rows") for c, s in [
        (dict(h=0), 1), (dict(offs=0), 1), (dict(codes=0), 1), (dict(scales=0), 1), (dict(m=-1), 2), (dict(n=0), 2),
        (dict(n=32), 2), (dict(n=96), 2), (dict(n=(1 << 20) + 64), 2), (dict(m=BIG), 2), (dict(h=A + 8), 3),
        (dict(e=0), 5), (dict(e=2049), 5)]],
    ("gg_fp4_masked_silu_mul_rows", SILU, dict(m=1 << 24, e=256), 2),
    *[(n, FWD, c, s) for n in ("gg_fp4_forward", "gg_fp4_masked_forward") for c, s in [
        (dict(x=0), 1), (dict(xs=0), 1), (dict(w=0), 1), (dict(ws=0), 1), (dict(offs=0), 1), (dict(y=0), 1),
        (dict(k=16), 2), (dict(k=48), 2), (dict(n=0), 2), (dict(n=12), 2), (dict(m=-1), 2), (dict(m=BIG), 2),
        (dict(k=1 << 16, n=1 << 15), 2), (dict(x=A + 8), 3), (dict(xs=A + 8), 3), (dict(w=A + 8), 3),
        (dict(ws=A + 8), 3), (dict(y=A + 8), 3), (dict(offs=A + 2), 3), (dict(dt=2), 4), (dict(e=0), 5),
        (dict(e=2049), 5)]],
    ("gg_fp4_masked_forward", FWD, dict(m=1 << 24, e=256), 2),
])
def test_checks_arguments(lib, name, defaults, case, status):
    assert run(name, defaults, case) == status, (case, gg.last_error())
    assert gg.last_error() != ""


@pytest.mark.parametrize("name,defaults,case", [
    ("gg_fp4_pack_scales", PACK, dict(rows=0, src=0, dst=0)),
    ("gg_fp4_quantize", QUANT, dict(rows=0, x=0, codes=0, scales=0)),
    ("gg_fp4_dequantize", BACK, dict(rows=0, out=0, codes=0, scales=0)),
    ("gg_fp4_gather_rows", GATHER, dict(cap=0, tokens=0, src=0, rs=0, codes=0, scales=0)),
    ("gg_fp4_silu_mul_rows", SILU, dict(m=0, h=0, codes=0, scales=0)),
    ("gg_fp4_forward", FWD, dict(m=0, x=0, xs=0, y=0)),
])
def test_no_rows_need_no_memory(lib, name, defaults, case):
    # (past the argument checks such a call needs no kernel, only the device's properties where there is a device)
    assert run(name, defaults, case) in (0, 6), gg.last_error()


@pytest.mark.parametrize("layout,rows,k,e,expect", [
    (0, 0, 32, 1, 1024), (0, 1, 32, 4, 5 * 1024), (0, 257, 160, 3, 5 * 2048), (1, 256, 128, 3, 3 * 1024),
    (1, 257, 128, 3, 6 * 1024), (2, 264, 2048, 8, 16 * 16 * 1024), (2, 0, 32, 8, 0),
])
def test_scale_bytes(lib, layout, rows, k, e, expect):
    assert gg.fp4_scale_bytes(layout, rows, k, e) == expect


@pytest.mark.parametrize("args", [(3, 1, 32, 1), (-1, 1, 32, 1), (0, -1, 32, 1), (0, BIG, 32, 1), (0, 1, 0, 1),
                                  (0, 1, 48, 1), (0, 1, (1 << 20) + 32, 1), (0, 1, 32, 0), (0, 1, 32, 2049)])
def test_scale_bytes_rejects(lib, args):
    assert lib.gg_fp4_scale_bytes(*args) == -1
    with pytest.raises(ValueError):
        gg.fp4_scale_bytes(*args)


def bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def u8(*shape):
    return torch.zeros(*shape, dtype=torch.uint8)


OFFS = torch.zeros(3, dtype=torch.int32)


@pytest.mark.parametrize("call", [
    lambda: gg.fp4_quantize(0, bf(4, 48), OFFS),
    lambda: gg.fp4_quantize(0, bf(3, 4, 64), OFFS),
    lambda: gg.fp4_quantize(1, bf(2, 4, 64), OFFS),
    lambda: gg.fp4_quantize(2, bf(3, 4, 64), OFFS),
    lambda: gg.fp4_quantize(7, bf(3, 4, 64)),
    lambda: gg.fp4_quantize(2, torch.zeros(3, 4, 64)),
    lambda: gg.fp4_quantize(0, bf(4, 128)[:, ::2], OFFS),
    lambda: gg.fp4_quantize(2, bf(3, 4, 64), out=u8(3, 4, 64)),
    lambda: gg.fp4_quantize(2, bf(3, 4, 64), out_scales=u8(3 * 1024 - 1)),
    lambda: gg.fp4_quantize(2, bf(3, 4, 64)),                               # not on a GPU
    lambda: gg.fp4_dequantize(2, u8(3, 4, 24), u8(1 << 16)),
    lambda: gg.fp4_dequantize(2, u8(3, 4, 32), None),
    lambda: gg.fp4_dequantize(2, u8(3, 4, 32), u8(3 * 1024 - 1)),
    lambda: gg.fp4_dequantize(2, u8(3, 4, 32), u8(1 << 16), out=bf(3, 4, 32)),
    lambda: gg.fp4_pack_scales(0, u8(3, 4, 2), OFFS),
    lambda: gg.fp4_pack_scales(2, torch.zeros(3, 4, 2)),
    lambda: gg.fp4_gather_rows(bf(4, 48), torch.zeros(9, dtype=torch.int32), 2, OFFS),
    lambda: gg.fp4_gather_rows(bf(4, 64), torch.zeros(9), 2, OFFS),
    lambda: gg.fp4_silu_mul_rows(bf(4, 96), OFFS),
    lambda: gg.fp4_silu_mul_rows(bf(4, 64), OFFS, masked=True),
    lambda: gg.fp4_forward(u8(4, 32), u8(1 << 16), u8(3, 8, 16), u8(1 << 16), OFFS),
    lambda: gg.fp4_forward(u8(4, 24), u8(1 << 16), u8(3, 8, 24), u8(1 << 16), OFFS),
    lambda: gg.fp4_forward(u8(4, 32), u8(7), u8(3, 8, 32), u8(1 << 16), OFFS),
    lambda: gg.fp4_forward(u8(4, 32), u8(1 << 16), u8(3, 8, 32), u8(7), OFFS),
    lambda: gg.fp4_forward(u8(4, 32), None, u8(3, 8, 32), u8(1 << 16), OFFS),
    lambda: gg.fp4_forward(u8(4, 32), u8(1 << 16), u8(2, 8, 32), u8(1 << 16), OFFS),
    lambda: gg.fp4_forward(u8(4, 32), u8(1 << 16), u8(3, 8, 32), u8(1 << 16), OFFS, out=bf(4, 9)),
    lambda: gg.fp4_forward(u8(4, 32), u8(1 << 16), u8(3, 8, 32), u8(1 << 16), OFFS, out_dtype=torch.float16),
    lambda: gg.fp4_masked_forward(u8(4, 32), u8(1 << 16), u8(3, 8, 32), u8(1 << 16), OFFS),
])
def test_binding_refuses(call):
    with pytest.raises((TypeError, ValueError)):
        call()
