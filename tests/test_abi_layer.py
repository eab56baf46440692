"""Host-side checks of the layer steps' entry points (no GPU needed): bad
arguments get their status before anything is enqueued, calls with nothing to
do need no memory, and the binding refuses tensors that do not fit."""
import pytest
import torch

from moe_grouped_gemm_ragged_amd import binding as gg

A = 0x10000       # fake, 16-byte aligned: rejected before any use


@pytest.fixture(scope="module")
def lib():
    return gg.load()


def run(name, defaults, case):
    v = dict(defaults, **case)
    return gg.call_raw(name, *[(x or None) if k in POINTERS else x for k, x in v.items()])


POINTERS = {"x", "res", "gamma", "h", "y", "y8", "s8", "dy", "dh", "dx", "dg", "ws", "src", "ss", "rs", "offs", "dst",
            "ds", "dout", "sr", "w", "dw", "xs", "a", "a8", "as8", "h8", "hs8", "da", "act"}

NORM = dict(x=A, res=0, gamma=A, h=0, y=A, y8=0, s8=0, rows=4, n=64, eps=1e-6, s=None)
NORM_GRAD = dict(dy=A, h=A, gamma=A, dh=0, dx=A, dg=A, ws=A, rows=4, n=64, eps=1e-6, s=None)
GATHER = dict(src=A, ss=A, tokens=4, k=256, rs=A, topk=2, offs=A, e=4, cap=40, dst=A, ds=A, s=None)
COMBINE = dict(dout=A, dt=0, y=A, n=64, sr=A, rs=A, offs=A, e=4, w=A, topk=2, tokens=4, cap=40, dy=A, dw=A, s=None)
SILU = dict(h=A, offs=A, a=A, a8=0, as8=0, h8=0, hs8=0, m=4, n=256, e=4, s=None)
SILU_GRAD = dict(da=A, h=A, hs8=0, offs=A, dh=A, act=0, m=4, n=256, e=4, s=None)
BIG = (1 << 31) - (1 << 16)


@pytest.mark.parametrize("case,status", [
    (dict(x=0), 1), (dict(gamma=0), 1), (dict(y=0), 1), (dict(y8=A, n=128), 1),
    (dict(rows=-1), 2), (dict(rows=BIG), 2), (dict(n=0), 2), (dict(n=12), 2), (dict(n=(1 << 20) + 8), 2),
    (dict(y8=A, s8=A, n=64), 2), (dict(eps=-1.0), 2), (dict(eps=float("nan")), 2), (dict(eps=float("inf")), 2),
    (dict(x=A + 8), 3), (dict(res=A + 2), 3), (dict(gamma=A + 4), 3), (dict(h=A + 8), 3), (dict(y=A + 8), 3),
    (dict(y8=A + 8, s8=A, n=128), 3),
])
def test_rmsnorm_checks_arguments(lib, case, status):
    assert run("gg_rmsnorm", NORM, case) == status, (case, gg.last_error())
    assert gg.last_error() != ""


@pytest.mark.parametrize("case,status", [
    (dict(dy=0), 1), (dict(h=0), 1), (dict(gamma=0), 1), (dict(dx=0), 1), (dict(dg=0), 1), (dict(ws=0), 1),
    (dict(rows=-1), 2), (dict(n=20), 2), (dict(eps=-1e-9), 2), (dict(rows=BIG), 2),
    (dict(dy=A + 8), 3), (dict(dh=A + 8), 3), (dict(ws=A + 4), 3), (dict(dg=A + 2), 3),
])
def test_rmsnorm_grad_checks_arguments(lib, case, status):
    assert run("gg_rmsnorm_grad", NORM_GRAD, case) == status, (case, gg.last_error())


def test_rmsnorm_grad_workspace(lib):
    # a whole number of fp32 rows, one at least, no more than there are rows of h
    for rows in (0, 1, 3, 1000, 1 << 20):
        for n in (8, 64, 7168, 1 << 20):
            size = gg.rmsnorm_grad_workspace_bytes(rows, n)
            assert size % (4 * n) == 0 and 1 <= size // (4 * n) <= max(1, rows)
    for rows, n in ((-1, 64), (4, 12), (4, 0), (BIG, 64)):
        assert lib.gg_rmsnorm_grad_workspace_bytes(rows, n) == -1


@pytest.mark.parametrize("case,status", [
    (dict(src=0), 1), (dict(ss=0), 1), (dict(rs=0), 1), (dict(offs=0), 1), (dict(dst=0), 1), (dict(ds=0), 1),
    (dict(tokens=-1), 2), (dict(k=64), 2), (dict(k=192), 2), (dict(topk=0), 2), (dict(cap=-1), 2), (dict(cap=BIG), 2),
    (dict(tokens=1 << 30), 2), (dict(tokens=1 << 40), 2), (dict(src=A + 8), 3), (dict(ds=A + 4), 3), (dict(rs=A + 2), 3),
    (dict(e=0), 5), (dict(e=2049), 5),
])
def test_fp8_gather_checks_arguments(lib, case, status):
    assert run("gg_fp8_gather_rows", GATHER, case) == status, (case, gg.last_error())


@pytest.mark.parametrize("case,status", [
    (dict(dout=0), 1), (dict(y=0), 1), (dict(sr=0), 1), (dict(rs=0), 1), (dict(offs=0), 1), (dict(dy=0), 1),
    (dict(n=12), 2), (dict(n=0), 2), (dict(topk=0), 2), (dict(tokens=-1), 2), (dict(cap=-1), 2), (dict(cap=BIG), 2),
    (dict(tokens=1 << 30), 2), (dict(tokens=1 << 40), 2),
    (dict(dout=A + 8), 3), (dict(y=A + 8), 3), (dict(dy=A + 8), 3), (dict(w=A + 2), 3), (dict(dw=A + 2), 3),
    (dict(dt=2), 4), (dict(e=0), 5),
])
def test_combine_grad_checks_arguments(lib, case, status):
    assert run("gg_combine_rows_grad", COMBINE, case) == status, (case, gg.last_error())


@pytest.mark.parametrize("name", ["gg_silu_mul_rows", "gg_masked_silu_mul_rows"])
@pytest.mark.parametrize("case,status", [
    (dict(h=0), 1), (dict(offs=0), 1), (dict(a=0), 1), (dict(a8=A), 1), (dict(h8=A), 1),
    (dict(m=-1), 2), (dict(n=0), 2), (dict(n=24), 2), (dict(h8=A, hs8=A, n=128), 2), (dict(a8=A, as8=A, n=128), 2),
    (dict(m=BIG), 2), (dict(h=A + 8), 3), (dict(a=A + 8), 3), (dict(h8=A + 8, hs8=A), 3), (dict(e=0), 5),
])
def test_silu_rows_check_arguments(lib, name, case, status):
    assert run(name, SILU, case) == status, (name, case, gg.last_error())


@pytest.mark.parametrize("name", ["gg_silu_mul_grad", "gg_masked_silu_mul_grad"])
@pytest.mark.parametrize("case,status", [
    (dict(da=0), 1), (dict(h=0), 1), (dict(offs=0), 1), (dict(dh=0), 1),
    (dict(m=-1), 2), (dict(n=24), 2), (dict(hs8=A, n=128), 2), (dict(da=A + 8), 3), (dict(act=A + 8), 3), (dict(e=0), 5),
])
def test_silu_grad_checks_arguments(lib, name, case, status):
    assert run(name, SILU_GRAD, case) == status, (name, case, gg.last_error())


@pytest.mark.parametrize("name,defaults", [("gg_masked_silu_mul_rows", SILU), ("gg_masked_silu_mul_grad", SILU_GRAD)])
def test_masked_row_limit(lib, name, defaults):
    assert run(name, defaults, dict(m=1 << 24, e=256)) == 2 and "max_m" in gg.last_error()


@pytest.mark.parametrize("name,defaults,case", [
    ("gg_rmsnorm", NORM, dict(rows=0, x=0, y=0)),
    ("gg_silu_mul_grad", SILU_GRAD, dict(m=0, da=0, h=0, dh=0)),
    ("gg_silu_mul_rows", SILU, dict(m=0, h=0, a=0)),
])
def test_no_rows_need_no_memory(lib, name, defaults, case):
    # an empty tensor's pointer may be NULL; such a call gets past the pointer checks (and
    # then needs no kernel, only the device's properties where there is a device)
    assert run(name, defaults, case) != 1, gg.last_error()


@pytest.mark.parametrize("name", ["gg_fp8_wgrad", "gg_fp8_masked_wgrad"])
def test_fp8_wgrad_without_rows_needs_no_operands(lib, name):
    assert run(name, WGRAD, dict(m=0, x=0, xs=0, dy=0)) != 1, gg.last_error()
    assert run(name, WGRAD, dict(m=0, offs=0)) == 1 and run(name, WGRAD, dict(m=0, dw=0)) == 1


def bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def u8(*shape):
    return torch.zeros(*shape, dtype=torch.uint8)


I = torch.zeros(4, dtype=torch.int32)


@pytest.mark.parametrize("error,call", [
    (TypeError, lambda: gg.rmsnorm(torch.zeros(4, 8), bf(8))),
    (ValueError, lambda: gg.rmsnorm(bf(4, 8), bf(16))),
    (ValueError, lambda: gg.rmsnorm(bf(4, 8), bf(8), residual=bf(3, 8))),
    (ValueError, lambda: gg.rmsnorm(bf(8, 4).t(), bf(8))),
    (ValueError, lambda: gg.rmsnorm(bf(4, 8), bf(8), h_out=bf(4, 8))),
    (ValueError, lambda: gg.fp8_rmsnorm(bf(4, 64), bf(64))),
    (ValueError, lambda: gg.fp8_rmsnorm(bf(4, 128), bf(128), out_scales=u8(4, 2))),
    (ValueError, lambda: gg.rmsnorm_grad(bf(4, 8), bf(4, 16), bf(8))),
    (TypeError, lambda: gg.rmsnorm_grad(bf(4, 8), bf(4, 8), bf(8), dgamma=bf(8))),
    (ValueError, lambda: gg.rmsnorm_grad(bf(4, 8), bf(4, 8), bf(8), workspace=u8(8))),
    (ValueError, lambda: gg.fp8_gather_rows(u8(4, 64), u8(4, 1), I, 2, I)),
    (ValueError, lambda: gg.fp8_gather_rows(u8(4, 256), u8(4, 1), I, 2, I)),
    (TypeError, lambda: gg.fp8_gather_rows(u8(4, 256), u8(4, 2), I.long(), 2, I)),
    (TypeError, lambda: gg.combine_rows_grad(bf(2, 8).half(), bf(4, 8), I, I, I, 2)),
    (ValueError, lambda: gg.combine_rows_grad(bf(3, 8), bf(4, 8), I, I, I, 2)),
    (ValueError, lambda: gg.combine_rows_grad(bf(2, 8), None, I, I, I, 2)),
    (ValueError, lambda: gg.combine_rows_grad(bf(2, 8), bf(5, 8), I, I, I, 2)),
    (ValueError, lambda: gg.silu_mul_rows(bf(4, 24), I)),
    (ValueError, lambda: gg.silu_mul_rows(bf(4, 128), I, keep=True)),
    (ValueError, lambda: gg.silu_mul_rows(bf(3, 4, 16), I, masked=True)),
    (ValueError, lambda: gg.fp8_silu_mul_rows(bf(4, 128), I)),
    (ValueError, lambda: gg.silu_mul_grad(bf(4, 8), bf(4, 8), I)),
    (TypeError, lambda: gg.fp8_silu_mul_grad(bf(4, 128), bf(4, 256), u8(4, 2), I)),
    (ValueError, lambda: gg.fp8_silu_mul_grad(bf(4, 128), u8(4, 256), u8(4, 1), I)),
    # fitting tensors, but not on a GPU
    (ValueError, lambda: gg.rmsnorm(bf(4, 8), bf(8))),
    (ValueError, lambda: gg.silu_mul_grad(bf(4, 8), bf(4, 16), I)),
])
def test_binding_refuses(error, call):
    with pytest.raises(error):
        call()


WGRAD = dict(x=A, xs=A, dy=A, offs=A, dw=A, dt=1, m=64, k=256, n=64, e=4, alpha=1.0, beta=0.0, s=None)


@pytest.mark.parametrize("name", ["gg_fp8_wgrad", "gg_fp8_masked_wgrad"])
@pytest.mark.parametrize("case,status", [
    (dict(x=0), 1), (dict(xs=0), 1), (dict(dy=0), 1), (dict(offs=0), 1), (dict(dw=0), 1),
    (dict(k=64), 2), (dict(k=200), 2), (dict(n=20), 2), (dict(m=-1), 2), (dict(m=BIG), 2),
    (dict(x=A + 8), 3), (dict(xs=A + 8), 3), (dict(dw=A + 4), 3), (dict(dt=2), 4), (dict(e=0), 5), (dict(e=2049), 5),
])
def test_fp8_wgrad_checks_arguments(lib, name, case, status):
    assert run(name, WGRAD, case) == status, (name, case, gg.last_error())


@pytest.mark.parametrize("error,call", [
    (TypeError, lambda: gg.fp8_wgrad(bf(4, 128), u8(4096), bf(4, 8), I)),
    (ValueError, lambda: gg.fp8_wgrad(u8(4, 64), u8(4096), bf(4, 8), I)),
    (ValueError, lambda: gg.fp8_wgrad(u8(4, 128), u8(8), bf(4, 8), I)),
    (ValueError, lambda: gg.fp8_wgrad(u8(4, 128), u8(4096), bf(5, 8), I)),
    (ValueError, lambda: gg.fp8_wgrad(u8(4, 128), u8(4096), bf(4, 8), I, beta=1.0)),
    (ValueError, lambda: gg.fp8_wgrad(u8(4, 128), u8(4096), bf(4, 8), I, out=torch.zeros(4, 8, 128))),
    (TypeError, lambda: gg.fp8_wgrad(u8(4, 128), u8(4096), bf(4, 8), I, out=torch.zeros(4, 128, 8).half())),
    (ValueError, lambda: gg.fp8_masked_wgrad(u8(3, 4, 128), u8(4096), bf(3, 4, 8), I)),
])
def test_fp8_wgrad_binding_refuses(error, call):
    with pytest.raises(error):
        call()


@pytest.mark.parametrize("f", [gg.silu_mul_rows, gg.fp8_silu_mul_rows])
@pytest.mark.parametrize("shape", [(256,), (4, 4, 256), (4, 4, 4, 256)])
@pytest.mark.parametrize("masked", [False, True])
def test_silu_rows_binding_refuses_other_ranks(f, shape, masked):
    if masked and len(shape) == 3:
        shape = (3, *shape[1:])                # (a rank that is taken, with experts that do not match)
    with pytest.raises(ValueError):
        f(bf(*shape), I, masked=masked)
