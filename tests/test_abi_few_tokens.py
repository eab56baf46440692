"""Host-side checks of the expert layer for a few tokens (no GPU needed)."""
import pytest
import torch

from moe_grouped_gemm_ragged_amd import binding as gg

A = 0x10000
POINTERS = {"x", "ids", "wt", "w13", "s13", "w2", "s2", "out", "ws"}
BF = dict(x=A, ids=A, wt=A, w13=A, w2=A, out=A, dt=0, ws=A, tokens=4, topk=2, hidden=64, inter=32, e=8, s=None)
FOUR = dict(x=A, ids=A, wt=A, w13=A, s13=A, w2=A, s2=A, out=A, dt=0, ws=A, tokens=4, topk=2, hidden=64, inter=32, e=8,
            s=None)


@pytest.fixture(scope="module")
def lib():
    return gg.load()


def run(name, defaults, case):
    v = dict(defaults, **case)
    return gg.call_raw(name, *[(x or None) if k in POINTERS else x for k, x in v.items()])


BOTH = [(dict(x=0), 1), (dict(ids=0), 1), (dict(w13=0), 1), (dict(w2=0), 1), (dict(out=0), 1), (dict(ws=0), 1),
        (dict(tokens=-1), 2), (dict(topk=0), 2), (dict(hidden=0), 2), (dict(inter=0), 2), (dict(hidden=4), 2),
        (dict(hidden=(1 << 20) + 32), 2), (dict(inter=1 << 20), 2), (dict(hidden=1 << 16, inter=1 << 13), 2),
        (dict(x=A + 8), 3), (dict(w13=A + 8), 3), (dict(w2=A + 8), 3), (dict(out=A + 8), 3), (dict(ws=A + 8), 3),
        (dict(ids=A + 2), 3), (dict(wt=A + 2), 3), (dict(dt=2), 4), (dict(dt=-1), 4), (dict(e=0), 5), (dict(e=2049), 5),
        (dict(tokens=65), 5), (dict(tokens=64, topk=9), 5), (dict(tokens=1, topk=513), 5), (dict(tokens=1 << 62), 5)]


@pytest.mark.parametrize("name,defaults,case,status", [
    *[("gg_moe_few_tokens", BF, c, s) for c, s in BOTH + [(dict(hidden=12), 2), (dict(inter=12), 2)]],
    *[("gg_fp4_moe_few_tokens", FOUR, c, s) for c, s in BOTH + [
        (dict(s13=0), 1), (dict(s2=0), 1), (dict(s13=A + 8), 3), (dict(s2=A + 4), 3), (dict(hidden=72), 2),
        (dict(inter=40), 2)]],
])
def test_checks_arguments(lib, name, defaults, case, status):
    assert run(name, defaults, case) == status, (case, gg.last_error())
    assert gg.last_error() != ""


@pytest.mark.parametrize("name,defaults", [("gg_moe_few_tokens", BF), ("gg_fp4_moe_few_tokens", FOUR)])
def test_no_tokens_need_nothing(lib, name, defaults):
    assert run(name, defaults, dict(tokens=0, x=0, ids=0, wt=0, out=0, ws=0)) == 0, gg.last_error()


def test_workspace(lib):
    for tokens, topk, inter, e in ((0, 1, 8, 1), (1, 8, 768, 128), (64, 8, 2048, 256), (3, 170, 40, 2048)):
        need = gg.moe_few_tokens_workspace_bytes(tokens, topk, inter, e)
        assert need == 16 + 16 * min(tokens * topk, e) + tokens * topk * inter * 4
    for args in ((-1, 1, 8, 1), (65, 1, 8, 1), (1, 0, 8, 1), (64, 9, 8, 1), (1, 1, 12, 1), (1, 1, 0, 1), (1, 1, 8, 0),
                 (1, 1, 8, 2049)):
        assert lib.gg_moe_few_tokens_workspace_bytes(*args) == -1


def test_limits_match():
    text = open(gg.header_path()).read()
    assert f"#define GG_FEW_TOKENS_MAX {gg.FEW_TOKENS_MAX}\n" in text
    assert f"#define GG_FEW_SLOTS_MAX {gg.FEW_SLOTS_MAX}\n" in text


def bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def u8(*shape):
    return torch.zeros(*shape, dtype=torch.uint8)


IDS = torch.zeros(4, 2, dtype=torch.int32)


@pytest.mark.parametrize("call", [
    lambda: gg.moe_few_tokens(bf(4, 64), IDS, bf(3, 64, 64), bf(3, 64, 32)),              # not on a GPU
    lambda: gg.moe_few_tokens(bf(5, 64), IDS, bf(3, 64, 64), bf(3, 64, 32)),
    lambda: gg.moe_few_tokens(bf(4, 64), IDS.reshape(-1), bf(3, 64, 64), bf(3, 64, 32)),
    lambda: gg.moe_few_tokens(bf(4, 64), IDS.long(), bf(3, 64, 64), bf(3, 64, 32)),
    lambda: gg.moe_few_tokens(bf(4, 64), IDS, bf(3, 63, 64), bf(3, 64, 31)),
    lambda: gg.moe_few_tokens(bf(4, 64), IDS, bf(3, 64, 64), bf(2, 64, 32)),
    lambda: gg.moe_few_tokens(bf(4, 64), IDS, bf(3, 64, 64), bf(3, 64, 64)),
    lambda: gg.moe_few_tokens(bf(4, 64), IDS, bf(3, 64, 72), bf(3, 64, 32)),
    lambda: gg.moe_few_tokens(bf(4, 64), IDS, u8(3, 64, 64), bf(3, 64, 32)),
    lambda: gg.moe_few_tokens(bf(4, 64), IDS, bf(3, 64, 64), bf(3, 64, 32), weights=torch.zeros(2, 4)),
    lambda: gg.moe_few_tokens(bf(4, 64), IDS, bf(3, 64, 64), bf(3, 64, 32), workspace=u8(31)),
    lambda: gg.moe_few_tokens(bf(4, 64), IDS, bf(3, 64, 64), bf(3, 64, 32), out=bf(4, 32)),
    lambda: gg.moe_few_tokens(bf(4, 64), IDS, bf(3, 64, 64), bf(3, 64, 32), out_dtype=torch.float16),
    lambda: gg.moe_few_tokens(bf(65, 64), torch.zeros(65, 2, dtype=torch.int32), bf(3, 64, 64), bf(3, 64, 32)),
    lambda: gg.fp4_moe_few_tokens(bf(4, 64), IDS, u8(3, 64, 32), None, u8(3, 64, 16), u8(1 << 16)),
    lambda: gg.fp4_moe_few_tokens(bf(4, 64), IDS, u8(3, 64, 32), u8(9), u8(3, 64, 16), u8(1 << 16)),
    lambda: gg.fp4_moe_few_tokens(bf(4, 64), IDS, u8(3, 64, 32), u8(1 << 16), u8(3, 64, 16), u8(9)),
    lambda: gg.fp4_moe_few_tokens(bf(4, 80), IDS, u8(3, 64, 40), u8(1 << 16), u8(3, 80, 16), u8(1 << 16)),
    lambda: gg.fp4_moe_few_tokens(bf(4, 64), IDS, bf(3, 64, 32), u8(1 << 16), u8(3, 64, 16), u8(1 << 16)),
])
def test_binding_refuses(call):
    with pytest.raises((TypeError, ValueError)):
        call()
