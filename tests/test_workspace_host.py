"""A workspace whose elements share memory, or leave some out between them, is refused: its size in bytes says
nothing of the memory behind its address."""
import ctypes

import pytest
import torch

import token_level_sparse_hs2_b200 as hs2

CPU = -1


@pytest.fixture(scope="module")
def calls():
    from token_level_sparse_hs2_b200 import build
    build.build()
    return hs2._calls()


WORKSPACES = [torch.zeros(1, dtype=torch.uint8).expand(1 << 20), torch.zeros(1 << 20, dtype=torch.uint8)[::2]]


@pytest.mark.parametrize("ws", WORKSPACES)
def test_gemm(calls, ws):
    with pytest.raises(ValueError, match="workspace must be one piece of memory"):
        calls.gemm_fp8(torch.zeros((4, 256), dtype=torch.uint8), hs2.fp8_scales(4, 256, device="cpu"), torch.zeros((300, 256), dtype=torch.uint8),
                       hs2.fp8_scales(300, 256, 128, device="cpu"), torch.zeros((4, 300)), ws, CPU, 0)


@pytest.mark.parametrize("ws", WORKSPACES)
def test_prefix(calls, ws):
    k = torch.zeros((1008, 128), dtype=torch.bfloat16)
    c = hs2.KvCache(k, k, [200, 500], [100, 300], 1, 32)
    with pytest.raises(ValueError, match="workspace must be one piece of memory"):
        calls.prefix_attn(ctypes.addressof(c.view), k, k, 5, 100, torch.zeros((2, 1, 32, 128), dtype=torch.bfloat16), 0.1,
                          torch.zeros((2, 1, 32, 128)), torch.zeros((2, 1, 32)), ws, CPU, 0)
