"""Infinities and NaN in what hs2_fp8_quantize and hs2_rms_norm turn into codes: a NaN has the code NaN and leaves its
block's scale to the other elements (1 where none is left); an infinity makes the scale infinite, its own code
NaN and the block's other codes 0, so that no value of the block is finite. Other blocks are as without it."""
import pytest
import torch

import token_level_sparse_hs2_b200 as hs2
from tests import operator_refs as R
from tests.test_gpu_norm import check_codes

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from token_level_sparse_hs2_b200 import build
    build.build()


def quantized(x, block_rows):
    rows, cols = x.shape
    codes, scales = torch.empty((rows, cols), dtype=torch.float8_e4m3fn, device="cuda"), hs2.fp8_scales(rows, cols, block_rows)
    hs2.fp8_quantize(x.cuda(), codes, scales, block_rows)
    return codes.float().cpu(), scales.cpu()


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,cols", [(5, 400), (200, 272), (129, 2064)])
def test_quantizer(rows, cols, block_rows):
    g = torch.Generator().manual_seed(rows)
    x = torch.randn((rows, cols), generator=g).bfloat16()
    codes0, scales0 = quantized(x, block_rows)
    i, last = rows - 1, (cols - 1) // 128
    bad = x.clone()
    bad[1, 5], bad[i, cols - 1] = NAN, -INF
    bad[3, 128:256] = NAN                      # a whole block of a row
    codes, scales = quantized(bad, block_rows)
    # NaN: the others' scale and codes
    without = x.clone()
    without[1, 5] = 0
    without[3, 128:256] = 0
    if block_rows == 128:
        without[i, cols - 1] = 0               # (the infinity's block is looked at below)
    want, want_scales = R.quantize(without, block_rows)
    keep = torch.ones((rows, cols), dtype=torch.bool)
    keep[1, 5], keep[3, 128:256] = False, False
    r0 = i // block_rows * block_rows
    keep[r0:, last * 128:] = False
    assert torch.isnan(codes[1, 5]) and torch.isnan(codes[3, 128:256]).all()
    assert torch.equal(codes[keep].double(), want[keep])
    same = torch.ones(scales.shape, dtype=torch.bool)
    same[last, i // block_rows] = False
    assert torch.equal(scales[same], want_scales[same])
    if block_rows == 1:
        assert scales[1, 3] == 1               # nothing left
    # infinity: the block's scale, and no finite value
    assert scales[last, i // block_rows] == INF
    block = codes[r0:, last * 128:]
    assert torch.isnan(codes[i, cols - 1])
    others = ~torch.isnan(block)
    assert (block[others] == 0).all() and others.sum() == block.numel() - torch.isnan(bad[r0:, last * 128:]).sum() - 1
    # the rows and columns without any are as they were
    if block_rows == 1:
        assert torch.equal(codes[[0, 2]], codes0[[0, 2]]) and torch.equal(scales[:, [0, 2]], scales0[:, [0, 2]])


def test_norm_codes():
    g = torch.Generator().manual_seed(2)
    x, w = torch.randn((6, 400), generator=g).bfloat16(), torch.ones(400)
    bad, h = x.clone(), torch.zeros((6, 400))
    bad[1, 3], bad[2, 200] = INF, NAN
    h[4, 7] = -INF                             # in the residual
    codes, scales = torch.empty((6, 400), dtype=torch.float8_e4m3fn, device="cuda"), hs2.fp8_scales(6, 400)
    out, res = torch.empty((6, 400), device="cuda"), h.cuda()
    hs2.rms_norm(bad.cuda(), w.cuda(), 1e-6, residual=res, residual_out=res, out=out, codes=codes, scales=scales)
    c, s = codes.float().cpu(), scales.cpu()
    # an infinite mean square: 1 / sqrt is 0, the infinite element's own y NaN, the others' 0
    for row, col in ((1, 3), (4, 7)):
        assert torch.isnan(c[row, col]) and torch.isnan(c[row]).sum() == 1 and c[row].nan_to_num().abs().sum() == 0
        assert (s[:, row] == 1).all() and torch.isinf(res[row, col])
    assert torch.isnan(c[2]).all() and (s[:, 2] == 1).all() and torch.isnan(out[2]).all()
    good = [0, 3, 5]
    y = R.rms_norm(x, w, 1e-6)[1]
    check_codes(y[good], codes[good], scales[:, good])


def test_a_product_with_them_is_non_finite_in_their_rows_alone():
    g = torch.Generator().manual_seed(3)
    x, wt = torch.randn((9, 256), generator=g).bfloat16(), torch.randn((300, 256), generator=g).bfloat16()
    w, sw = torch.empty((300, 256), dtype=torch.float8_e4m3fn, device="cuda"), hs2.fp8_scales(300, 256, 128)
    hs2.fp8_quantize(wt.cuda(), w, sw, 128)
    outs = []
    for bad in (False, True):
        if bad:
            x[2, 7], x[5, 200] = INF, NAN
        a, sa, out = torch.empty((9, 256), dtype=torch.float8_e4m3fn, device="cuda"), hs2.fp8_scales(9, 256), torch.empty((9, 300), device="cuda")
        hs2.fp8_quantize(x.cuda(), a, sa)
        hs2.gemm_fp8(a, sa, w, sw, out, torch.empty(256, dtype=torch.uint8, device="cuda"))
        outs.append(out.cpu())
    rows = [0, 1, 3, 4, 6, 7, 8]
    assert torch.equal(outs[0][rows], outs[1][rows])
    assert torch.isnan(outs[1][[2, 5]]).all()
