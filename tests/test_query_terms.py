"""The two e4m3 terms in which the attention of a shared prefix holds a query row for an e4m3 cache: after a
power of two that puts the row's largest element in [128, 256), every bf16 element of 1/4 or more (2^-9 of the
largest and more) is their sum exactly; a smaller one to within 2^-10, 2^-17 of the largest. On the CPU, over every
bf16 value below 256."""
import torch


def test_the_querys_two_terms():
    x = torch.arange(1, 0x4380, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).float()      # up to 256
    x = x[(x >= 2.0 ** -30) & (x < 256)]
    hi = x.to(torch.float8_e4m3fn).float()
    lo = (x - hi).to(torch.float8_e4m3fn).float()
    off = (x - hi - lo).abs()
    assert (off[x >= 0.25] == 0).all() and off.max() == 2.0 ** -10 and (off[(x >= 0.125) & (x < 0.25)] > 0).any()
