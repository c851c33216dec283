"""GPU parity of hs2_rms_norm and hs2_fp8_quantize, through the binding, against plain float64.

Tolerances, all relative to the exact value. The float32 sum of squares is a chain of at most
8 chunks x 8 fused multiply-adds per thread, 5 shuffle additions and 16 words of other warps: its
error is at most 85 half steps of float32 (2^-24 each), halved by the root; the addition, the
division by d, the added eps, the root and two products add six: y is within 49 x 2^-24, plus the
output's own half step (bf16 2^-8). The residual is one addition: half a step of its type (and of
float32). A scale is within y's error and one more division; a code is within half an e4m3 step of
the exact quotient by the scale that was written, widened by y's error and the quotient's."""
import numpy as np
import pytest
import torch

import token_level_sparse_hs2_b200 as hs2
from tests import operator_refs as R

pytestmark = pytest.mark.gpu
Y_TOL = 49 * 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from token_level_sparse_hs2_b200 import build
    build.build()


def strided(rows, cols, pad, dtype, fill=None):
    """A [rows, cols] view of a buffer with `pad` more columns, and the buffer."""
    buf = torch.empty((rows, cols + pad), dtype=dtype, device="cuda")
    if fill is not None:
        buf.fill_(fill)
    return buf[:, :cols], buf


def inputs(rows, d, seed, res=None, wdtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, d), generator=g).bfloat16()
    r = None if res is None else (3 * torch.randn((rows, d), generator=g)).to(res)
    w = (1 + 0.3 * torch.randn(d, generator=g)).to(wdtype)
    return x, r, w


def check_codes(y, codes, scales, tol=Y_TOL):
    values = codes.float().cpu().double()
    for j, (c0, c1) in enumerate(R.column_blocks(y.shape[1])):
        part, s = y[:, c0:c1], scales[j].cpu().double()
        amax = part.abs().amax(1)
        want = torch.where(amax > 0, amax / 448, torch.ones_like(amax))
        assert ((s - want).abs() <= (tol + 2.0 ** -23) * want).all()
        q = part / s[:, None]
        off = (values[:, c0:c1] - q.clamp(-448, 448)).abs()
        assert (off <= R.e4m3_half_step(q) * (1 + 2.0 ** -20) + q.abs() * (tol + 2.0 ** -22)).all()


SHAPES = [(1, 8), (3, 64), (1, 4096), (8, 4096), (37, 136), (129, 1000), (5, 4104), (2, 16384), (1, 32768),
          (700, 32), (2000, 256), (300, 2832)]


@pytest.mark.parametrize("rows,d", SHAPES)
@pytest.mark.parametrize("res", [None, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_norm(rows, d, res, out):
    wd = torch.float32 if out == torch.bfloat16 and res is None else torch.bfloat16
    x, r, w = inputs(rows, d, rows + d, res, wd)
    xs, _ = strided(rows, d, 8, torch.bfloat16)
    xs.copy_(x)
    y, ybuf = strided(rows, d, 16, out, fill=7.0)
    ro = rbuf = rd = None
    if res is not None:
        rd, _ = strided(rows, d, 24, res)
        rd.copy_(r)
        ro, rbuf = strided(rows, d, 24, res, fill=5.0)
    hs2.rms_norm(xs, w.cuda(), 1e-5, rd, ro, y)
    h, want = R.rms_norm(x, w, 1e-5, r)
    assert ((y.cpu().double() - want).abs() <= (Y_TOL + HALF[out]) * want.abs() + 1e-40).all()
    assert (ybuf[:, d:] == 7).all()                      # nothing behind a row is written
    if res is not None:
        assert ((ro.cpu().double() - h).abs() <= (HALF[res] + 2.0 ** -24) * h.abs()).all()
        assert (rbuf[:, d:] == 5).all()


@pytest.mark.parametrize("rows,d", [(1, 16), (3, 64), (8, 4096), (37, 144), (129, 1008), (5, 4112), (2, 16384),
                                    (1, 32768), (700, 32), (2000, 256), (300, 2832)])
@pytest.mark.parametrize("res", [None, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("both", [False, True])
def test_norm_codes(rows, d, res, both):
    x, r, w = inputs(rows, d, 3 * rows + d, res)
    codes, cbuf = strided(rows, d, 16, torch.uint8, fill=0x55)
    sbuf = torch.full((-(-d // 128), -(-rows // 4) * 4 + 4), -3.0, device="cuda")
    scales = sbuf[:, :rows]
    y = torch.empty((rows, d), device="cuda") if both else None
    rd = None if r is None else r.cuda()
    ro = None if r is None else rd                       # in place
    hs2.rms_norm(x.cuda(), w.cuda(), 1e-6, rd, ro, y, codes, scales)
    h, want = R.rms_norm(x, w, 1e-6, r)
    check_codes(want, codes.view(torch.float8_e4m3fn), scales)
    assert (cbuf[:, d:] == 0x55).all() and (sbuf[:, rows:] == -3).all()
    if both:
        assert ((y.cpu().double() - want).abs() <= Y_TOL * want.abs() + 1e-40).all()
    if r is not None:
        assert ((ro.cpu().double() - h).abs() <= (HALF[res] + 2.0 ** -24) * h.abs()).all()


def test_norm_zero_rows_and_zero_blocks():
    x = torch.zeros((5, 400), dtype=torch.bfloat16)
    x[1, :128] = 1                                       # blocks 1..3 of row 1 are zero
    x[2] = torch.finfo(torch.bfloat16).tiny              # far below eps
    codes = torch.empty((5, 400), dtype=torch.float8_e4m3fn, device="cuda")
    scales = hs2.fp8_scales(5, 400)
    w = torch.ones(400, dtype=torch.bfloat16)
    hs2.rms_norm(x.cuda(), w.cuda(), 1e-6, codes=codes, scales=scales)
    check_codes(R.rms_norm(x, w, 1e-6)[1], codes, scales)
    s = scales.cpu()
    assert (s[:, 0] == 1).all() and (s[1:, 1] == 1).all() and s[0, 1] != 1
    assert (codes.float()[0] == 0).all()
    hs2.rms_norm(x[:0].cuda(), w.cuda(), 1e-6, codes=codes[:0], scales=hs2.fp8_scales(0, 400)[:, :0])   # no row


def test_norm_non_finite_rows_stay_their_own():
    x = torch.ones((4, 256), dtype=torch.bfloat16)
    x[1, 3], x[2, 200] = float("inf"), float("nan")
    y = torch.empty((4, 256), device="cuda")
    w = torch.ones(256)
    hs2.rms_norm(x.cuda(), w.cuda(), 0.0, out=y)
    y = y.cpu()
    assert (y[0] == 1).all() and (y[3] == 1).all()
    assert (y[1, :3] == 0).all() and torch.isnan(y[1, 3]) and torch.isnan(y[2]).all()


def test_norm_outputs_near_the_smallest_float32():
    """y of a few 2^-149 (a weight of 2^-148): out within one step, and blocks whose max|y| / 448 rounds to
    zero have the scale 1 and codes 0."""
    g = torch.Generator().manual_seed(11)
    x = torch.randn((6, 272), generator=g).bfloat16()
    w = torch.full((272,), 2.0 ** -148)
    y, out = R.rms_norm(x, w, 1e-6)[1], torch.empty((6, 272), device="cuda")
    codes, scales = torch.empty((6, 272), dtype=torch.float8_e4m3fn, device="cuda"), hs2.fp8_scales(6, 272)
    hs2.rms_norm(x.cuda(), w.cuda(), 1e-6, out=out, codes=codes, scales=scales)
    assert ((out.cpu().double() - y).abs() <= 2.0 ** -149).all()
    assert (scales == 1).all() and (codes.float() == 0).all()


def test_norm_in_place_on_x():
    x, _, w = inputs(33, 512, 1)
    want = R.rms_norm(x, w, 1e-6)[1]
    xd = x.cuda()
    hs2.rms_norm(xd, w.cuda(), 1e-6, out=xd)
    assert ((xd.cpu().double() - want).abs() <= (Y_TOL + 2.0 ** -8) * want.abs()).all()


def test_norm_on_another_stream_and_in_a_graph():
    x, r, w = inputs(16, 4096, 2, torch.bfloat16)
    xd, rd, wd = x.cuda(), r.cuda(), w.cuda()
    ro = torch.empty_like(rd)
    codes = torch.empty((16, 4096), dtype=torch.float8_e4m3fn, device="cuda")
    scales = hs2.fp8_scales(16, 4096)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    hs2.rms_norm(xd, wd, 1e-6, rd, ro, codes=codes, scales=scales, stream=s)
    s.synchronize()
    want = codes.float().clone(), scales.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        hs2.rms_norm(xd, wd, 1e-6, rd, ro, codes=codes, scales=scales)
    x2, r2, _ = inputs(16, 4096, 3, torch.bfloat16)
    for xi, ri in ((x2, r2), (x, r)):
        xd.copy_(xi)
        rd.copy_(ri)
        g.replay()
        check_codes(R.rms_norm(xi, w, 1e-6, ri)[1], codes, scales)
    assert torch.equal(codes.float(), want[0]) and torch.equal(scales, want[1])


@pytest.mark.parametrize("rows,cols", [(1, 16), (1, 128), (3, 4096), (127, 144), (128, 128), (130, 2064), (1000, 272), (70, 1024),
                                       (33, 2000), (65, 640), (200, 1152), (67, 512), (9, 16384)])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_matches_the_definition_bit_for_bit(rows, cols, block_rows):
    g = torch.Generator().manual_seed(rows * cols)
    x = (torch.randn((rows, cols), generator=g) * torch.exp(3 * torch.randn((rows, 1), generator=g))).bfloat16()
    x[rows // 2, :cols // 2] = 0
    if rows > 2:
        x[2] = 0
    xs, _ = strided(rows, cols, 8, torch.bfloat16)
    xs.copy_(x)
    codes, cbuf = strided(rows, cols, 16, torch.uint8, fill=0x55)
    nr = -(-rows // block_rows)
    sbuf = torch.full((-(-cols // 128), -(-nr // 4) * 4 + 4), -3.0, device="cuda")
    hs2.fp8_quantize(xs, codes, sbuf[:, :nr], block_rows)
    values, scales = R.quantize(x, block_rows)
    assert torch.equal(sbuf[:, :nr].cpu(), scales)
    assert torch.equal(codes.view(torch.float8_e4m3fn).float().cpu().double(), values)
    assert (cbuf[:, cols:] == 0x55).all() and (sbuf[:, nr:] == -3).all()


def test_quantize_of_wide_offsets():
    """More than 2^31 elements between the first and the last row's start."""
    rows, cols, stride = 70000, 128, 32768
    buf = torch.zeros((rows - 1) * stride + cols, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((rows, cols), (stride, 1))
    x[-1], x[65536] = 3.0, -2.0
    codes = torch.empty((rows, cols), dtype=torch.float8_e4m3fn, device="cuda")
    scales = hs2.fp8_scales(rows, cols)
    hs2.fp8_quantize(x, codes, scales)
    v = codes.float()
    assert (v[-1] == 448).all() and (v[65536] == -448).all() and v.abs().sum() == 2 * 448 * cols
    y = torch.empty((rows, cols), device="cuda")
    hs2.rms_norm(x, torch.ones(cols, device="cuda"), 1e-6, out=y)
    assert (y[-1] - 1).abs().max() < 1e-6 and (y[65536] + 1).abs().max() < 1e-6 and (y != 0).sum() == 2 * cols


@pytest.mark.parametrize("rows,d", [(1300, 3584), (1200, 4880), (1190, 8192), (1185, 4112), (400, 8192), (310, 5120), (300, 12288), (150, 9000)])
@pytest.mark.parametrize("res", [None, torch.bfloat16, torch.float32])
def test_norm_of_many_wide_rows(rows, d, res):
    """CTAs that go from row to row, two and four chunks of 8 columns per thread."""
    x, r, w = inputs(rows, d, rows - d + 9000, res)
    h, y = R.rms_norm(x, w, 1e-6, r)
    out = torch.empty((rows, d), dtype=torch.float32, device="cuda")
    codes, scales = (torch.empty((rows, d), dtype=torch.float8_e4m3fn, device="cuda"), hs2.fp8_scales(rows, d)) if d % 16 == 0 else (None, None)
    rd = None if r is None else r.cuda()
    hs2.rms_norm(x.cuda(), w.cuda(), 1e-6, residual=rd, residual_out=rd, out=out, codes=codes, scales=scales)
    # as in test_norm
    assert ((out.cpu().double() - y).abs() <= (Y_TOL + HALF[torch.float32]) * y.abs() + 1e-40).all()
    if rd is not None:
        assert ((rd.cpu().double() - h).abs() <= (HALF[res] + 2.0 ** -24) * h.abs()).all()
    if codes is not None:
        check_codes(y, codes, scales)
