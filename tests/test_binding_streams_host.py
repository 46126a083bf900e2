"""Where the binding takes the memory of a call that is given a stream of its own.

The caching allocator may hand out a block of the current stream's pool that was freed there while kernels queued on that stream
still use it; only work on that stream comes after them.  So what a call writes on another stream has to come from that
stream's pool, and what it returns is kept until both streams are done with it.  Streams, allocator and library are stand-ins
here: nothing runs on a GPU."""
import contextlib

import pytest
import torch

import nvfp4_block_scaled_16_b200 as nv
from nvfp4_block_scaled_16_b200 import binding

M, N, K, R, A, E = 4, 128, 64, 16, 3, 2


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


class Library:
    """Entry points that succeed without doing anything; sizes are 4096 bytes."""

    def __getattr__(self, name):
        return lambda *args: 4096 if name.endswith(("_workspace", "_bytes")) else 0


@pytest.fixture
def machine(monkeypatch):
    """(allocations, uses): the stream current at each allocation, and the (address, stream) pairs of record_stream."""
    current, allocations, uses = [Stream(0)], [], []

    @contextlib.contextmanager
    def switch(stream):
        current.append(stream)
        yield
        current.pop()

    def noting(make):
        def allocate(*args, **kwargs):
            t = make(*args, **kwargs)
            allocations.append((t.data_ptr(), current[-1].cuda_stream))
            return t
        return allocate

    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current[-1])
    monkeypatch.setattr(torch.cuda, "stream", switch)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: Stream(handle))
    monkeypatch.setattr(torch.cuda, "device", lambda device: contextlib.nullcontext())
    monkeypatch.setattr(torch, "empty", noting(torch.empty))
    monkeypatch.setattr(torch.Tensor, "new_empty", noting(torch.Tensor.new_empty))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: uses.append((t.data_ptr(), s.cuda_stream)))
    monkeypatch.setattr(binding, "load_library", Library)
    monkeypatch.setattr(binding, "_ptr", lambda t: None if t is None else t.data_ptr())
    monkeypatch.setattr(binding, "_index_of", lambda name, t: 0)
    monkeypatch.setattr(binding, "_operand", lambda name, t, *rest: t.data_ptr())
    monkeypatch.setattr(binding, "_call", lambda fn, index, args, stream: 0)
    binding._workspace_bytes.cache_clear()
    yield allocations, uses
    binding._workspace_bytes.cache_clear()


def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


one, per_expert = torch.zeros(1), torch.zeros(E)
a, b, x, mask = u8(M, K // 2), u8(N, K // 2), bf16(M, K), torch.zeros(E, dtype=torch.int32)
ids = torch.zeros((M, 2), dtype=torch.int32)
CALLS = {
    "nvfp4_global_scale": (x, None, None, one),
    "nvfp4_global_scale_batched": (bf16(E, M, K),),
    "nvfp4_quantize": (x, one),
    "nvfp4_global_scale_quantize": (x, one),
    "nvfp4_quantize_masked_batched": (bf16(E, M, K), per_expert),
    "nvfp4_silu_mul_quantize_batched": (bf16(E, M, 2 * K), per_expert),
    "nvfp4_gemm": (a, b, u8(512), u8(512), one),
    "nvfp4_gemm_bf16a": (x, b, u8(512), one),
    "nvfp4_gemm_bf16a_static": (x, b, u8(512), one, one),
    "nvfp4_grouped_gemm_masked": (u8(E, M, K // 2), u8(E, N, K // 2), u8(E, 512), u8(E, 512), mask, per_expert),
    "nvfp4_gemm_lowrank_bias": (a, b, u8(512), u8(512), one, bf16(M, R), bf16(N, R)),
    "nvfp4_gemm_silu_mul_quantize": (a, b, b, u8(512), u8(512), u8(512), one, one, one),
    "nvfp4_grouped_gemm_silu_mul_quantize_masked": (u8(E, M, K // 2), u8(E, N, K // 2), u8(E, N, K // 2), u8(E, 512), u8(E, 512),
                                                    u8(E, 512), mask, per_expert, per_expert, per_expert),
    "nvfp4_silu_and_mul": (bf16(M, 2 * K),),
    "nvfp4_quantize_smooth": (x, bf16(K), one),
    "nvfp4_lora_down": (x, bf16(R, K)),
    "nvfp4_quantize_smooth_lora_down": (x, bf16(K), one, bf16(R, K)),
    "nvfp4_lora_down_batched": (x, bf16(A, R, K), torch.zeros(M, dtype=torch.int32)),
    "nvfp4_gemm_lora_batched": (a, b, u8(512), u8(512), one, bf16(M, R), bf16(A, N, R), torch.zeros(M, dtype=torch.int32)),
    "nvfp4_moe_route": (torch.zeros((M, E)), 2),
    "nvfp4_moe_few_tokens": (x, ids, torch.zeros((M, 2)), u8(E, N, K // 2), u8(E, N, K // 2), u8(E, K, N // 2), u8(E, 512),
                             u8(E, 512), u8(E, 512), per_expert, per_expert, per_expert),
}


def tensors(result):
    return [t for t in (result if isinstance(result, tuple) else (result,)) if t is not None]


@pytest.mark.parametrize("name", sorted(CALLS))
def test_memory_of_a_call_on_another_stream_comes_from_that_stream(machine, name):
    allocations, uses = machine
    out = tensors(getattr(nv, name)(*CALLS[name], stream=Stream(7)))
    assert out and allocations and all(stream == 7 for _, stream in allocations)
    made = {address for address, _ in allocations}
    for t in out:                                # the caller goes on with them on the current stream
        assert t.data_ptr() in made and (t.data_ptr(), 0) in uses


@pytest.mark.parametrize("name", sorted(CALLS))
@pytest.mark.parametrize("stream", [None, Stream(0)])
def test_memory_of_a_call_on_the_current_stream(machine, name, stream):
    allocations, uses = machine
    out = tensors(getattr(nv, name)(*CALLS[name], stream=stream))
    assert out and allocations and all(at == 0 for _, at in allocations) and not uses


def test_outputs_and_workspace_of_the_caller_are_used_as_they_are(machine):
    allocations, uses = machine
    out, ws = bf16(M, K), u8(8192)
    got = nv.nvfp4_moe_few_tokens(*CALLS["nvfp4_moe_few_tokens"], out=out, workspace=ws, stream=Stream(7))
    assert got is out and not allocations and not uses
