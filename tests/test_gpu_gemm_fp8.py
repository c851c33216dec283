"""GPU parity of hs2_gemm_fp8, through the binding, against plain float64.

Tolerance per element, with mag = sum of |scaled terms|: a block's product adds at most 128 exact
products into a float32 sum, each addition within 2^-23 of the magnitude so far (truncation
allowed): 128 x 2^-23 mag; the product of the two scales, the product with it and the addition to
the running sum of kb blocks (and up to 8 joined ranges) add (kb + 10) x 2^-24 mag; then the
output's half step (bf16 2^-8, float32 2^-24) of the value."""
import pytest
import torch

import token_level_sparse_hs2_b200 as hs2
from tests import operator_refs as R

pytestmark = pytest.mark.gpu
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from token_level_sparse_hs2_b200 import build
    build.build()


def codes_of(rows, cols, g, pad=0):
    """Random finite e4m3 codes on the device, in a buffer with `pad` more columns of NaN codes."""
    c = torch.randint(0, 256, (rows, cols + pad), generator=g, dtype=torch.int32).to(torch.uint8)
    c[(c & 0x7f) == 0x7f] = 0x40
    c[:, cols:] = 0x7f
    return c.cuda()[:, :cols].view(torch.float8_e4m3fn)


def scales_of(blocks, rows, g, spread=1.0):
    s = hs2.fp8_scales(rows, blocks * 128)
    s.copy_(torch.exp(spread * torch.randn((blocks, rows), generator=g)))
    return s


def workspace():
    return torch.full((256,), 0x33, dtype=torch.uint8, device="cuda")


def check(out, a, sa, w, sw):
    ref, mag = R.gemm(a.float().cpu(), sa.cpu(), w.float().cpu(), sw.cpu())
    kb = sa.shape[0]
    tol = mag * (128 * 2.0 ** -23 + (kb + 10) * 2.0 ** -24) + HALF[out.dtype] * ref.abs() + 1e-38
    off = (out.cpu().double() - ref).abs()
    bad = ~(off <= tol)
    assert not bad.any(), (bad.nonzero()[:5].tolist(), int(bad.sum()), float((off / tol).max()))


SHAPES = [(1, 1, 16), (1, 256, 4096), (2, 129, 128), (7, 128, 144), (8, 1000, 4112), (31, 4096, 512), (32, 130, 272),
          (33, 640, 2048), (64, 64, 1024), (65, 257, 4096), (127, 384, 1040), (128, 128, 128), (129, 8, 640), (200, 1000, 2064),
          (300, 520, 16384), (1024, 256, 272), (777, 1000, 2064), (2500, 1280, 400), (1, 4096, 65536),
          (9473, 100, 2064), (5000, 333, 272), (1300, 2000, 1040), (20000, 256, 16), (2049, 2305, 4112)]


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_product(m, n, k, dtype):
    g = torch.Generator().manual_seed(m * 7919 + n * 31 + k)
    pad = 16 if (m + n) % 2 else 0
    a, w = codes_of(m, k, g, pad), codes_of(n, k, g, 32 - pad)
    kb = -(-k // 128)
    sa, sw = scales_of(kb, m, g), scales_of(kb, -(-n // 128), g)
    buf = torch.full((m + 1, n + 3 + pad), 9.0, dtype=dtype, device="cuda")
    out, ws = buf[:m, :n], workspace()
    hs2.gemm_fp8(a, sa, w, sw, out, ws)
    hs2.read_device_status(ws)
    check(out, a, sa, w, sw)
    assert (buf[m:] == 9).all() and (buf[:, n:] == 9).all()     # nothing behind the result is written
    again = torch.empty((m, n), dtype=dtype, device="cuda")
    hs2.gemm_fp8(a, sa, w, sw, again, ws)
    assert torch.equal(again, out)                              # the order of the sums is fixed


def test_aligned_wide_stores_and_row_strides():
    """Output rows that allow wide stores (n not a multiple of a piece) and ones that do not."""
    g = torch.Generator().manual_seed(11)
    for m, n in ((300, 1000), (260, 999), (40, 1004), (1500, 333), (4900, 1001), (5000, 1000)):
        a, w = codes_of(m, 512, g), codes_of(n, 512, g)
        sa, sw = scales_of(4, m, g), scales_of(4, -(-n // 128), g)
        first = None
        for ldo, off in ((1008, 0), (1008, 8), (1011, 0), (1009, 1)):
            for dtype in (torch.bfloat16, torch.float32):
                buf = torch.full((m * ldo + 16,), -5.0, dtype=dtype, device="cuda")
                out = buf[off:off + m * ldo].view(m, ldo)[:, :n]
                hs2.gemm_fp8(a, sa, w, sw, out, workspace())
                if first is None:
                    first = {}
                if dtype not in first:
                    first[dtype] = out.clone()
                    check(out, a, sa, w, sw)
                assert torch.equal(out, first[dtype])
                assert (buf == -5).sum() >= buf.numel() - m * n


def test_zero_and_non_finite_values_stay_in_their_rows_and_columns():
    g = torch.Generator().manual_seed(5)
    for m in (8, 200):
        a, w = codes_of(m, 256, g), codes_of(300, 256, g)
        sa, sw = scales_of(2, m, g), scales_of(2, 3, g)
        out0 = torch.empty((m, 300), device="cuda")
        hs2.gemm_fp8(a, sa, w, sw, out0, workspace())
        a2, w2 = a.view(torch.uint8).clone(), w.view(torch.uint8).clone()
        a2[3, 7], w2[290, 100] = 0x7f, 0xff                     # NaN codes
        sa2 = hs2.fp8_scales(m, 256)
        sa2.copy_(sa)
        sa2[0, 5], sa2[1, 6] = float("inf"), 0.0
        out = torch.empty_like(out0)
        hs2.gemm_fp8(a2, sa2, w2, sw, out, workspace())
        assert torch.isnan(out[3]).all() and torch.isnan(out[:, 290]).all() and not torch.isfinite(out[5]).any()
        keep = torch.ones((m, 300), dtype=torch.bool, device="cuda")
        keep[[3, 5, 6]] = False
        keep[:, 290] = False
        assert torch.equal(out[keep], out0[keep])


def test_quantised_operands_give_the_product():
    """bf16 activations and weights, quantised by the library: within e4m3's own rounding of the
    exact product (each factor within 2^-4 of itself or 2^-10 of its block's scale)."""
    g = torch.Generator().manual_seed(3)
    m, n, k = 130, 400, 1040
    x, wt = torch.randn((m, k), generator=g).bfloat16(), torch.randn((n, k), generator=g).bfloat16()
    a, sa = torch.empty((m, k), dtype=torch.float8_e4m3fn, device="cuda"), hs2.fp8_scales(m, k)
    w, sw = torch.empty((n, k), dtype=torch.float8_e4m3fn, device="cuda"), hs2.fp8_scales(n, k, 128)
    hs2.fp8_quantize(x.cuda(), a, sa)
    hs2.fp8_quantize(wt.cuda(), w, sw, 128)
    out = torch.empty((m, n), device="cuda")
    hs2.gemm_fp8(a, sa, w, sw, out, workspace())
    check(out, a, sa, w, sw)
    ref, mag = x.double() @ wt.double().t(), x.double().abs() @ wt.double().abs().t()
    assert ((out.cpu().double() - ref).abs() <= (2 * 2.0 ** -4 + 2.0 ** -8 + 2.0 ** -6) * mag).all()


def test_streams_graphs_and_two_calls_at_once():
    g = torch.Generator().manual_seed(8)
    for m in (8, 1000):
        a, w = codes_of(m, 4096, g), codes_of(2048, 4096, g)
        sa, sw = scales_of(32, m, g, 0.2), scales_of(32, 16, g, 0.2)
        want = torch.empty((m, 2048), dtype=torch.bfloat16, device="cuda")
        hs2.gemm_fp8(a, sa, w, sw, want, workspace())
        torch.cuda.synchronize()
        outs, streams = [torch.zeros_like(want) for _ in range(2)], [torch.cuda.Stream() for _ in range(2)]
        wss = [workspace() for _ in range(2)]
        torch.cuda.synchronize()
        for _ in range(5):
            for o, s, ws in zip(outs, streams, wss):
                hs2.gemm_fp8(a, sa, w, sw, o, ws, stream=s)
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o in outs)
        graph, out, ws = torch.cuda.CUDAGraph(), torch.zeros_like(want), workspace()
        with torch.cuda.graph(graph):
            hs2.gemm_fp8(a, sa, w, sw, out, ws)
        for _ in range(2):
            out.zero_()
            graph.replay()
            assert torch.equal(out, want)
        hs2.read_device_status(ws)


def test_wide_offsets():
    """Rows of the result more than 2^31 elements apart."""
    g = torch.Generator().manual_seed(2)
    m, n, ldo = 600, 128, 2 ** 22
    a, w = codes_of(m, 128, g), codes_of(n, 128, g)
    sa, sw = scales_of(1, m, g), scales_of(1, 1, g)
    small = torch.empty((m, n), dtype=torch.bfloat16, device="cuda")
    hs2.gemm_fp8(a, sa, w, sw, small, workspace())
    buf = torch.zeros(((m - 1) * ldo + n,), dtype=torch.bfloat16, device="cuda")
    out = buf.as_strided((m, n), (ldo, 1))
    hs2.gemm_fp8(a, sa, w, sw, out, workspace())
    assert torch.equal(out, small)
