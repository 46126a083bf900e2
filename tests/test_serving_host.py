"""Argument checks of the serving-step entry points (router, few-token expert layer, batched adapters): sizes, null and
misaligned pointers, workspaces, and the binding's types, shapes and devices.  No kernel is launched."""
import ctypes

import pytest
import torch

import nvfp4_block_scaled_16_b200 as nv

INVALID = 1
P = ctypes.c_void_p
A16, A1 = P(1 << 20), P((1 << 20) + 1)
BIG = 1 << 50


@pytest.fixture(scope="module")
def lib():
    from nvfp4_block_scaled_16_b200 import build
    build.build()
    return nv.load_library()


@pytest.mark.parametrize("t,E,topk,weighting", [(-1, 8, 2, 0), (4, 0, 1, 0), (4, 1025, 2, 0), (4, 8, 0, 0), (4, 8, 9, 0),
                                               (4, 64, 33, 0), (4, 8, 2, 3), (4, 8, 2, -1)])
def test_route_refuses_sizes(lib, t, E, topk, weighting):
    assert lib.nvfp4_moe_route(A16, 0, t, E, topk, weighting, A16, A16, None) == INVALID


def test_route_refuses_pointers_and_accepts_no_tokens(lib):
    assert lib.nvfp4_moe_route(None, 0, 4, 8, 2, 0, A16, A16, None) == INVALID
    assert lib.nvfp4_moe_route(A16, 0, 4, 8, 2, 0, None, A16, None) == INVALID
    assert lib.nvfp4_moe_route(A16, 0, 4, 8, 2, 0, A16, None, None) == INVALID
    assert lib.nvfp4_moe_route(A1, 0, 4, 8, 2, 0, A16, A16, None) == INVALID
    assert lib.nvfp4_moe_route(A1, 1, 4, 8, 2, 0, A16, A16, None) == INVALID
    assert lib.nvfp4_moe_route(None, 0, 0, 8, 2, 0, None, None, None) == 0


MOE = dict(t=4, topk=2, E=8, n=128, k=256)


def moe_call(lib, pointers=None, nbytes=BIG, **sizes):
    s = {**MOE, **sizes}
    return lib.nvfp4_moe_few_tokens(*(pointers or [A16] * 14), nbytes, s["t"], s["topk"], s["E"], s["n"], s["k"], None)


@pytest.mark.parametrize("sizes", [dict(t=65), dict(t=-1), dict(topk=0), dict(topk=17), dict(E=0), dict(E=1025), dict(n=96),
                                   dict(n=0), dict(k=0), dict(k=224), dict(k=-64), dict(n=1 << 18), dict(k=1 << 18)])
def test_moe_refuses_sizes(lib, sizes):
    assert moe_call(lib, **sizes) == INVALID
    s = {**MOE, **sizes}
    assert nv.nvfp4_moe_few_tokens_workspace(s["t"], s["topk"], s["E"], s["n"], s["k"]) == -1


def test_moe_refuses_pointers_and_short_workspaces(lib):
    for i in range(14):
        p = [A16] * 14
        p[i] = None
        assert moe_call(lib, p) == INVALID, i
        p[i] = A1
        assert moe_call(lib, p) == INVALID, i
    need = nv.nvfp4_moe_few_tokens_workspace(4, 2, 8, 128, 256)
    assert need > 0 and moe_call(lib, nbytes=need - 1) == INVALID
    assert moe_call(lib, [None] * 14, 0, t=0) == 0          # no tokens: nothing is read


def test_moe_workspace_grows_with_its_arguments(lib):
    base = nv.nvfp4_moe_few_tokens_workspace(8, 2, 16, 512, 512)
    assert nv.nvfp4_moe_few_tokens_workspace(64, 2, 16, 512, 512) > base
    assert nv.nvfp4_moe_few_tokens_workspace(8, 2, 16, 4096, 512) > base
    assert nv.nvfp4_moe_few_tokens_workspace(8, 2, 16, 512, 4096) > base


@pytest.mark.parametrize("m,k,r,adapters", [(-1, 128, 16, 2), (4, 96, 16, 2), (4, 0, 16, 2), (4, 128, 0, 2), (4, 128, 12, 2),
                                            (4, 128, 264, 2), (4, 128, 16, 0), (4, 128, 16, 65537)])
def test_lora_refuses_sizes(lib, m, k, r, adapters):
    assert lib.nvfp4_lora_down_batched(A16, m, k, A16, r, adapters, A16, A16, None) == INVALID
    assert nv.nvfp4_gemm_lora_batched_workspace(m, 128, k, r, adapters) == -1
    assert lib.nvfp4_gemm_lora_batched(*[A16] * 7, r, adapters, A16, None, A16, A16, BIG, m, 128, k, None) == INVALID


def test_lora_down_refuses_pointers(lib):
    good = [A16, 4, 128, A16, 16, 2, A16, A16, None]
    for i in (0, 3, 6, 7):
        for bad in (None, A1):
            args = list(good)
            args[i] = bad
            assert lib.nvfp4_lora_down_batched(*args) == INVALID, (i, bad)
    assert lib.nvfp4_lora_down_batched(None, 0, 128, None, 16, 2, None, None, None) == 0


def test_gemm_lora_refuses_pointers_widths_and_short_workspaces(lib):
    need = nv.nvfp4_gemm_lora_batched_workspace(400, 128, 256, 16, 2)
    good = [A16] * 7 + [16, 2, A16, None, A16, A16, need, 400, 128, 256, None]
    assert need > 0
    assert nv.nvfp4_gemm_lora_batched_workspace(4, 128, 256, 16, 2) == 0      # few rows need none
    few = [A16] * 7 + [16, 2, A16, None, A16, None, 0, 4, 128, 256, None]
    for i in (0, 1, 2, 3, 4, 5, 6, 9, 11):
        args = list(few)
        args[i] = None
        assert lib.nvfp4_gemm_lora_batched(*args) == INVALID, i
    for i in (0, 1, 2, 3, 4, 5, 6, 9, 11, 12):
        for bad in (None, A1):
            args = list(good)
            args[i] = bad
            assert lib.nvfp4_gemm_lora_batched(*args) == INVALID, (i, bad)
    for i, bad in ((10, A1), (13, need - 1), (15, 100), (16, 96)):          # bias, workspace bytes, n, k
        args = list(good)
        args[i] = bad
        assert lib.nvfp4_gemm_lora_batched(*args) == INVALID, (i, bad)
    assert lib.nvfp4_gemm_lora_batched(*[None] * 7, 16, 2, None, None, None, None, 0, 0, 128, 256, None) == 0
    assert lib.nvfp4_gemm_lora_batched(*[None] * 7, 16, 2, None, None, None, None, 0, 4, 0, 256, None) == 0


def test_binding_refuses_host_tensors_and_other_objects(lib):
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        nv.nvfp4_moe_route(torch.zeros((4, 8)), 2)
    with pytest.raises(TypeError):
        nv.nvfp4_moe_route([[1.0]], 1)
    with pytest.raises(ValueError, match="CUDA"):
        nv.nvfp4_moe_few_tokens(x, *[None] * 11)
    with pytest.raises(ValueError, match="CUDA"):
        nv.nvfp4_lora_down_batched(x, None, None)
    with pytest.raises(ValueError, match="CUDA"):
        nv.nvfp4_gemm_lora_batched(x, *[None] * 7)
