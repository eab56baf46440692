"""Every call of the binding launches with its tensors' device current and on
that device's stream (host only: tensors without memory on a second GPU, and a
library that records instead of launching)."""
import contextlib

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from moe_grouped_gemm_ragged_amd import binding as gg

DEV = torch.device("cuda", 1)
BF, U8, I32, F32 = torch.bfloat16, torch.uint8, torch.int32, torch.float32
E, M, K, N = 3, 16, 256, 128


def t(*shape, dtype=BF):
    return torch.empty(*shape, dtype=dtype, device=DEV)


def packed(layout, rows, k, experts=E):
    return t(gg.fp8_scale_bytes(layout, rows, k, experts), dtype=U8)


CALLS = {
    "forward": lambda o: gg.forward(t(M, K), t(E, K, N), o),
    "forward scaled": lambda o: gg.forward(t(M, K), t(E, K, N), o, out=t(M, N), beta=1.0),
    "dgrad": lambda o: gg.dgrad(t(M, N), t(E, K, N), o),
    "wgrad": lambda o: gg.wgrad(t(M, K), t(M, N), o),
    "masked_forward": lambda o: gg.masked_forward(t(E, M, K), t(E, K, N), o),
    "masked_dgrad": lambda o: gg.masked_dgrad(t(E, M, N), t(E, K, N), o),
    "masked_wgrad": lambda o: gg.masked_wgrad(t(E, M, K), t(E, M, N), o),
    "forward_nk": lambda o: gg.forward_nk(t(M, K), t(E, N, K), o),
    "forward_bias": lambda o: gg.forward_bias(t(M, K), t(E, K, N), o, t(E, N)),
    "bias_grad": lambda o: gg.bias_grad(t(M, N), o),
    "bias_scale_grad": lambda o: gg.bias_scale_grad(t(M, N), o, t(E, N)),
    "offsets_from_splits": lambda o: gg.offsets_from_splits(t(E, dtype=torch.int64), 8),
    "route": lambda o: gg.route(t(5, 2, dtype=I32), E, 8),
    "gather_rows": lambda o: gg.gather_rows(t(5, K), t(M, dtype=I32), 2, o),
    "combine_rows": lambda o: gg.combine_rows(t(M, N), t(10, dtype=I32), 2, t(5, 2, dtype=F32)),
    "fp8_pack_scales": lambda o: gg.fp8_pack_scales(gg.GG_FP8_ACT_RAGGED, t(M, K // 128, dtype=F32), o, M, K, E),
    "fp8_forward": lambda o: gg.fp8_forward(t(M, K, dtype=U8), packed(0, M, K), t(E, N, K, dtype=U8),
                                            packed(2, N, K), o),
    "fp8_masked_forward": lambda o: gg.fp8_masked_forward(t(E, M, K, dtype=U8), packed(1, M, K),
                                                          t(E, N, K, dtype=U8), packed(2, N, K), o),
    "rmsnorm": lambda o: gg.rmsnorm(t(M, K), t(K), residual=t(M, K)),
    "fp8_rmsnorm": lambda o: gg.fp8_rmsnorm(t(M, K), t(K)),
    "rmsnorm_grad": lambda o: gg.rmsnorm_grad(t(M, K), t(M, K), t(K)),
    "fp8_gather_rows": lambda o: gg.fp8_gather_rows(t(5, K, dtype=U8), t(5, K // 128, dtype=U8), t(M, dtype=I32), 2, o),
    "combine_rows_grad": lambda o: gg.combine_rows_grad(t(5, N), t(M, N), t(10, dtype=I32), t(M, dtype=I32), o, 2),
    "silu_mul_rows": lambda o: gg.silu_mul_rows(t(M, K), o, keep=True),
    "silu_mul_grad": lambda o: gg.silu_mul_grad(t(M, N), t(M, 2 * N), o),
    "fp8_wgrad": lambda o: gg.fp8_wgrad(t(M, K, dtype=U8), packed(0, M, K), t(M, N), o),
    "fp8_masked_wgrad": lambda o: gg.fp8_masked_wgrad(t(E, M, K, dtype=U8), packed(1, M, K), t(E, M, N), o),
}


@pytest.mark.parametrize("name", CALLS)
def test_launches_on_the_tensors_device(name, monkeypatch):
    lib, current, seen = gg.load(), [0], []

    class Library:
        def __getattr__(self, f):
            if f.endswith("_bytes") or f.endswith("_bound") or f == "gg_last_error":
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
    with FakeTensorMode():
        CALLS[name](t(E, dtype=I32))
    assert seen and all(d == 1 and s == 1001 for _, d, s in seen), seen
    assert current[0] == 0
