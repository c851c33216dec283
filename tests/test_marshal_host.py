"""Refusals of the module that turns torch tensors into calls of the operators around the block. The
device given is that of CPU tensors, so that each call gets as far as the fault it is made with; every
call here is refused before anything runs."""
import ctypes

import pytest
import torch

import token_level_sparse_hs2_b200 as hs2

CPU = -1   # device index of a CPU tensor


@pytest.fixture(scope="module")
def calls():
    from token_level_sparse_hs2_b200 import build
    build.build()
    return hs2._calls()


def refused(f, args, kind, words):
    with pytest.raises(kind, match=words):
        f(*args.values())


def norm_args():
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    return dict(x=x, weight=torch.ones(256), eps=1e-6, residual=x.clone(), residual_out=x.clone(), out=torch.zeros((4, 256)),
                codes=torch.zeros((4, 256), dtype=torch.uint8), scales=hs2.fp8_scales(4, 256, device="cpu"), device=CPU, stream=0)


B, F, D = torch.bfloat16, torch.float32, torch.float64


@pytest.mark.parametrize("name,value,kind,words", [
    ("x", None, TypeError, "x must be a tensor"), ("x", torch.zeros((4, 256)), TypeError, "x: dtype Float"),
    ("x", torch.zeros(256, dtype=B), ValueError, "x must be 2-D"), ("x", torch.zeros((256, 4), dtype=B).t(), ValueError, "x must have contiguous rows"),
    ("weight", torch.zeros(255), ValueError, r"weight must be \[256\]"), ("weight", torch.zeros(512)[::2], ValueError, "weight must be contiguous"),
    ("weight", torch.zeros(256, dtype=D), TypeError, "weight: dtype Double"), ("eps", "small", TypeError, "real number"),
    ("residual", None, ValueError, "both or neither"), ("residual_out", None, ValueError, "both or neither"),
    ("residual_out", torch.zeros((4, 256)), TypeError, "residual_out: dtype Float"),
    ("residual_out", torch.zeros((4, 512), dtype=B)[:, :256], ValueError, "one row stride"),
    ("out", torch.zeros((3, 256)), ValueError, r"out must be \[4, 256\], not \[3, 256\]"), ("out", torch.zeros((4, 256), dtype=D), TypeError, "out: dtype"),
    ("codes", None, ValueError, "codes and scales"), ("scales", None, ValueError, "codes and scales"),
    ("codes", torch.zeros((4, 256), dtype=torch.int8), TypeError, "codes: dtype"),
    ("scales", torch.zeros((4, 2)), ValueError, r"scales must be \[2, 4\]"), ("device", 0, ValueError, "x is on cpu, the current device is cuda:0"),
    ("device", None, TypeError, "integer"), ("stream", 1.5, TypeError, "int"),
])
def test_norm(calls, name, value, kind, words):
    refused(calls.rms_norm, {**norm_args(), name: value}, kind, words)


def test_number_of_arguments(calls):
    for f in (calls.rms_norm, calls.fp8_quantize, calls.gemm_fp8, calls.prefix_attn):
        with pytest.raises(TypeError, match="arguments expected, not 1"):
            f(0)


@pytest.mark.parametrize("name,value,kind,words", [
    ("x", torch.zeros((200, 256)), TypeError, "x: dtype"), ("codes", torch.zeros((200, 255), dtype=torch.uint8), ValueError, "codes must be"),
    ("scales", torch.zeros((2, 200)), ValueError, r"scales must be \[2, 2\]"), ("block_rows", 1, ValueError, r"scales must be \[2, 200\]"),
    ("block_rows", 2 ** 31, ValueError, "block_rows out of range"), ("block_rows", 2 ** 63, OverflowError, "int"), ("block_rows", "1", TypeError, "int"),
    ("device", 0, ValueError, "current device"),
])
def test_quantize(calls, name, value, kind, words):
    args = dict(x=torch.zeros((200, 256), dtype=B), codes=torch.zeros((200, 256), dtype=torch.uint8),
                scales=hs2.fp8_scales(200, 256, 128, device="cpu"), block_rows=128, device=CPU, stream=0)
    refused(calls.fp8_quantize, {**args, name: value}, kind, words)


@pytest.mark.parametrize("name,value,kind,words", [
    ("a", torch.zeros((4, 256)), TypeError, "a: dtype"), ("a", torch.zeros((4, 128), dtype=torch.uint8), ValueError, "same number of columns"),
    ("w", torch.zeros((256, 300), dtype=torch.uint8).t(), ValueError, "w must have contiguous rows"),
    ("w", torch.zeros(256, dtype=torch.uint8), ValueError, "w must be 2-D"), ("a_scale", torch.zeros((2, 5)), ValueError, r"a_scale must be \[2, 4\]"),
    ("w_scale", torch.zeros((2, 4)), ValueError, r"w_scale must be \[2, 3\]"), ("w_scale", torch.zeros((2, 3), dtype=D), TypeError, "w_scale: dtype"),
    ("out", torch.zeros((4, 299)), ValueError, r"out must be \[4, 300\]"), ("out", torch.zeros((300, 4)).t(), ValueError, "contiguous rows"),
    ("out", torch.zeros((4, 300), dtype=torch.float16), TypeError, "out: dtype Half"), ("workspace", None, TypeError, "workspace must be a tensor"),
])
def test_gemm(calls, name, value, kind, words):
    args = dict(a=torch.zeros((4, 256), dtype=torch.uint8), a_scale=hs2.fp8_scales(4, 256, device="cpu"),
                w=torch.zeros((300, 256), dtype=torch.uint8), w_scale=hs2.fp8_scales(300, 256, 128, device="cpu"),
                out=torch.zeros((4, 300)), workspace=torch.zeros(256, dtype=torch.uint8), device=CPU, stream=0)
    refused(calls.gemm_fp8, {**args, name: value}, kind, words)


@pytest.mark.parametrize("name,value,kind,words", [
    ("q", torch.zeros((2, 1, 32, 128)), TypeError, "q: dtype"), ("q", torch.zeros((1, 1, 32, 128), dtype=B), ValueError, r"q must be \[2, 1, 32, 128\]"),
    ("q", torch.zeros((2, 1, 128, 32), dtype=B).transpose(2, 3), ValueError, "q must be contiguous"),
    ("out", torch.zeros((2, 1, 16, 128)), ValueError, "out must be"), ("out", torch.zeros((2, 1, 32, 128), dtype=D), TypeError, "out: dtype"),
    ("lse", torch.zeros((2, 32)), ValueError, "lse must be"), ("lse", torch.zeros((2, 1, 32), dtype=D), TypeError, "lse: dtype"),
    ("prefix_len", 2 ** 31, ValueError, "prefix_len out of range"), ("prefix_len", 1.0, TypeError, "int"), ("workspace", 0, TypeError, "workspace must be"),
    ("device", 0, ValueError, "k is on cpu"),
])
def test_prefix(calls, name, value, kind, words):
    k = torch.zeros((1008, 128), dtype=B)
    c = hs2.KvCache(k, k, [200, 500], [100, 300], 1, 32)
    args = dict(view=ctypes.addressof(c.view), k=k, v=k, prefix_start=5, prefix_len=100, q=torch.zeros((2, 1, 32, 128), dtype=B),
                scale=0.1, out=torch.zeros((2, 1, 32, 128)), lse=torch.zeros((2, 1, 32)), workspace=torch.zeros(4096, dtype=torch.uint8),
                device=CPU, stream=0)
    refused(calls.prefix_attn, {**args, name: value}, kind, words)
