"""KvCache refuses tensors that the kernels would read past their end or with another type: the calls that
take a cache look at nothing but its addresses."""
import pytest
import torch

import token_level_sparse_hs2_b200 as hs2

ROWS = 64


def parts(**change):
    k = torch.zeros((ROWS, 128), dtype=torch.uint8)
    return {**dict(k=k, v=k.clone(), kv_start=[0], kv_len=[9], n_q=1, n_heads=16, k_scale=torch.ones(ROWS), v_scale=torch.ones(ROWS)), **change}


@pytest.mark.parametrize("name", ["k_scale", "v_scale"])
@pytest.mark.parametrize("value,kind", [
    (torch.ones(ROWS - 1), ValueError), (torch.ones(2 * ROWS)[::2], ValueError), (torch.ones((1, ROWS)).expand(2, ROWS), ValueError),
    (torch.ones(ROWS, dtype=torch.float64), TypeError), (torch.ones(2 * ROWS, dtype=torch.bfloat16), TypeError),
    (torch.ones(ROWS, device="meta"), ValueError),
])
def test_scales(name, value, kind):
    with pytest.raises(kind, match=name):
        hs2.KvCache(**parts(**{name: value}))


@pytest.mark.parametrize("k,v,kind", [
    (torch.bfloat16, torch.uint8, TypeError), (torch.uint8, torch.bfloat16, TypeError), (torch.bfloat16, torch.float8_e4m3fn, TypeError),
    (torch.bfloat16, torch.float32, TypeError), (torch.uint8, torch.int8, TypeError),
])
def test_one_type_of_keys_and_values(k, v, kind):
    with pytest.raises(kind, match="v"):
        hs2.KvCache(**parts(k=torch.zeros((ROWS, 128), dtype=k), v=torch.zeros((ROWS, 128), dtype=v)))


def test_one_device():
    with pytest.raises(ValueError, match="v is on"):
        hs2.KvCache(**parts(v=torch.zeros((ROWS, 128), dtype=torch.uint8, device="meta")))


def test_what_is_taken():
    hs2.KvCache(**parts())
    hs2.KvCache(**parts(k=torch.zeros((ROWS, 128), dtype=torch.float8_e4m3fn)))       # codes either way
    hs2.KvCache(**parts(k_scale=torch.ones((ROWS, 1)), v_scale=torch.ones(ROWS + 7)))
    bf16 = torch.zeros((ROWS, 128), dtype=torch.bfloat16)
    hs2.KvCache(**parts(k=bf16, v=bf16, k_scale=None, v_scale=None))
    hs2.KvCache(**parts(k_scale=None, v_scale=None))                                   # refused by every call
