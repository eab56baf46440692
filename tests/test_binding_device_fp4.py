"""The 4-bit calls and the few-token layer launch with their tensors' device
current and on that device's stream (host only: tensors without memory on a second
GPU, and a library that records instead of launching), and refuse tensors of
several devices."""
import contextlib

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from moe_grouped_gemm_ragged_amd import binding as gg

DEV = torch.device("cuda", 1)
BF, U8, I32, F32 = torch.bfloat16, torch.uint8, torch.int32, torch.float32
RAGGED, MASKED, WEIGHT = gg.GG_FP4_ACT_RAGGED, gg.GG_FP4_ACT_MASKED, gg.GG_FP4_WEIGHT
E, M, K, N, T = 3, 16, 256, 128, 4


def t(*shape, dtype=BF, device=DEV):
    return torch.empty(*shape, dtype=dtype, device=device)


def packed(layout, rows, k):
    return t(gg.fp4_scale_bytes(layout, rows, k, E), dtype=U8)


CALLS = {
    "fp4_pack_scales": lambda o: gg.fp4_pack_scales(RAGGED, t(M, K // 32, dtype=U8), o),
    "fp4_quantize": lambda o: gg.fp4_quantize(RAGGED, t(M, K), o),
    "fp4_quantize weights": lambda o: gg.fp4_quantize(WEIGHT, t(E, N, K)),
    "fp4_dequantize": lambda o: gg.fp4_dequantize(MASKED, t(E, M, K // 2, dtype=U8), packed(MASKED, M, K), o),
    "fp4_gather_rows": lambda o: gg.fp4_gather_rows(t(T, K), t(M, dtype=I32), 2, o),
    "fp4_silu_mul_rows": lambda o: gg.fp4_silu_mul_rows(t(M, K), o),
    "fp4_silu_mul_rows masked": lambda o: gg.fp4_silu_mul_rows(t(E, M, K), o, masked=True),
    "fp4_forward": lambda o: gg.fp4_forward(t(M, K // 2, dtype=U8), packed(RAGGED, M, K), t(E, N, K // 2, dtype=U8),
                                            packed(WEIGHT, N, K), o),
    "fp4_masked_forward": lambda o: gg.fp4_masked_forward(t(E, M, K // 2, dtype=U8), packed(MASKED, M, K),
                                                          t(E, N, K // 2, dtype=U8), packed(WEIGHT, N, K), o),
    "moe_few_tokens": lambda o: gg.moe_few_tokens(t(T, K), t(T, 2, dtype=I32), t(E, 2 * N, K), t(E, K, N),
                                                  t(T, 2, dtype=F32)),
    "fp4_moe_few_tokens": lambda o: gg.fp4_moe_few_tokens(t(T, K), t(T, 2, dtype=I32), t(E, 2 * N, K // 2, dtype=U8),
                                                          packed(WEIGHT, 2 * N, K), t(E, K, N // 2, dtype=U8),
                                                          packed(WEIGHT, K, N)),
}


@pytest.fixture
def recorded(monkeypatch):
    lib, current, seen = gg.load(), [0], []

    class Library:
        def __getattr__(self, f):
            if f.endswith("_bytes") or f == "gg_last_error":
                return getattr(lib, f)
            return lambda *args: seen.append((f, current[0], args[-1])) or 0

    @contextlib.contextmanager
    def device(d):
        before, current[0] = current[0], torch.device(d).index
        yield
        current[0] = before

    def stream(d=None):
        return type("Stream", (), {"cuda_stream": 1000 + torch.device("cuda", d if isinstance(d, int) else d.index).index})

    monkeypatch.setattr(gg, "_lib", Library())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_stream", stream)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 1000 + i, raising=False)
    monkeypatch.setattr(torch.Tensor, "data_ptr", lambda self: 4096)
    return current, seen


@pytest.mark.parametrize("name", CALLS)
def test_launches_on_the_tensors_device(name, recorded):
    current, seen = recorded
    with FakeTensorMode():
        CALLS[name](t(E, dtype=I32))
    assert seen and all(d == 1 and s == 1001 for _, d, s in seen), seen
    assert current[0] == 0


def test_refuses_several_devices(recorded):
    _, seen = recorded
    other = torch.device("cuda", 0)
    with FakeTensorMode():
        o = t(E, dtype=I32)
        for call in (
                lambda: gg.fp4_quantize(RAGGED, t(M, K, device=other), o),
                lambda: gg.fp4_gather_rows(t(T, K), t(M, dtype=I32, device=other), 2, o),
                lambda: gg.fp4_forward(t(M, K // 2, dtype=U8), packed(RAGGED, M, K),
                                       t(E, N, K // 2, dtype=U8, device=other), packed(WEIGHT, N, K), o),
                lambda: gg.moe_few_tokens(t(T, K), t(T, 2, dtype=I32), t(E, 2 * N, K), t(E, K, N, device=other)),
                lambda: gg.moe_few_tokens(t(T, K), t(T, 2, dtype=I32), t(E, 2 * N, K), t(E, K, N),
                                          t(T, 2, dtype=F32, device=other)),
                lambda: gg.moe_few_tokens(t(T, K), t(T, 2, dtype=I32), t(E, 2 * N, K), t(E, K, N),
                                          workspace=t(1 << 16, dtype=U8, device=other))):
            with pytest.raises((ValueError, RuntimeError)):
                call()
    assert not seen
