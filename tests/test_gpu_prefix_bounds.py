"""hs2_prefix_attn within bounds that count each rounding of the kernel once.

The scores of most cases here are sums of products of small whole numbers (times powers of two), so the
tensor cores' sums are exact and what is left is arithmetic that can be bounded. With z = score / ln 2 and the
largest |z| of a row Z, T keys and n = T / 128 + 2 tiles:

  weight    the factor c log2 e has two roundings and the K scale's product one (e4m3), z - m one more:
            |error of z| <= 3 x 2^-24 Z + 2^-24 (2 Z + 8); the exponential is within 2^-22 of itself. So
            a weight is within dw = ln 2 (5 Z + 8) 2^-24 + 2^-22 of its value.
  lse       dw, 34 + 2 n + 60 additions of a sum of positive terms and of the joined ranges (2^-24 each),
            2 n rescalings at most (2^-22 + 2^-24 each), then logarithms, exponentials and products by
            constants of a few steps: 2^-20 + 2^-21 |lse|.
  output    each weight (times its V scale, one product) rounded to bf16 once, 2^-8; dw for the weight and dw for
            the sum; T additions of the tensor cores within 2^-23 of the magnitude so far (truncation
            allowed); the sum's additions as above; the ranges' weights, within the lse's error, twice; all
            of a = sum of weight x |v|; then the output's half step (bf16 2^-8, float32 2^-24).

The e4m3 cache's query is held as two e4m3 terms after a power of two that puts the row's largest element in
[128, 256). An element of at least 2^-9 of the largest is at least 1/4 then: its bf16 steps, 2^-9 or more, are
within reach of the second term, and the sum is exact. Of a smaller one the last bits below 2^-9 are lost:
at most 2^-10 of the scaled unit, 2^-17 of the row's largest element."""
import math

import pytest
import torch

import token_level_sparse_hs2_b200 as hs2  # noqa: F401
from tests.test_gpu_prefix import HALF, Case

pytestmark = pytest.mark.gpu
C = 128 ** -0.5


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from token_level_sparse_hs2_b200 import build
    build.build()


def whole_numbers(c, fp8, seed):
    """q = i / 32 with |i| <= 100, keys of whole numbers up to 8 (quarters of them; codes times scales)."""
    g = torch.Generator().manual_seed(seed)
    c.q = (torch.randint(-100, 101, c.q.shape, generator=g) / 32).bfloat16()
    k = torch.randint(-8, 9, c.k64.shape, generator=g).double()
    used = torch.zeros(len(k), dtype=torch.bool)
    used[c.start:c.start + c.prefix] = True
    for f, t in zip(c.first, c.lens):
        used[f:f + t] = True
    if fp8:
        ks = 0.25 * torch.exp(0.5 * torch.randn(len(k), generator=g))
        c.k64 = k * ks.double()[:, None]
        codes, ks = k.float().to(torch.float8_e4m3fn).view(torch.uint8), ks.clone()
        codes[~used], ks[~used] = 0x7f, float("nan")
        c.k, c.ks = codes.view(torch.float8_e4m3fn).cuda(), ks.cuda()
    else:
        c.k64 = k / 4
        kb = c.k64.bfloat16()
        kb[~used] = float("nan")
        c.k = kb.cuda()


def check(c, got, lse, score_error=None):
    """score_error(q, k): a bound of what the scores' sums lose, [H, T] of q [H, 128] and k [T, 128]."""
    for b, (f, t) in enumerate(zip(c.first, c.lens)):
        for i in range(c.n_q):
            rows = torch.cat([torch.arange(c.start, c.start + c.prefix), torch.arange(f, f + t - c.n_q + i + 1)])
            q, k, v = c.q[b, i].double(), c.k64[rows], c.v64[rows]
            x = q @ k.t() * C
            T, z = len(rows), (x.abs().amax(1) / math.log(2))
            tiles = T / 128 + 2
            dw = math.log(2) * (5 * z + 8) * 2.0 ** -24 + 2.0 ** -22
            if score_error is not None:
                dw = dw + score_error(q, k).amax(1)
            want = torch.logsumexp(x, 1)
            tol = dw + (94 + 2 * tiles) * 2.0 ** -24 + 2 * tiles * (2.0 ** -22 + 2.0 ** -24) + 2.0 ** -20 + 2.0 ** -21 * want.abs()
            off = (lse[b, i].cpu().double() - want).abs()
            assert (off <= tol).all(), ("lse", b, i, float((off / tol).max()))
            p = torch.exp(x - want[:, None])
            ref, mag = p @ v, p @ v.abs()
            rel = 2.0 ** -8 + 2 * dw + T * 2.0 ** -23 + (94 + 2 * tiles) * 2.0 ** -24 + 2 * tol
            tol = rel[:, None] * mag + HALF[got.dtype] * ref.abs()
            off = (got[b, i].cpu().double() - ref).abs()
            assert (off <= tol).all(), ("out", b, i, float((off / tol).max()))


SHAPES = [([1], 1, 16, 1), ([300, 1, 77], 1, 32, 128), ([64] * 4, 1, 32, 129), ([1, 2, 3, 4, 5, 6, 7, 8, 9], 1, 32, 3000), ([17] * 9, 1, 16, 777),
          ([1100, 3], 1, 32, 500), ([700, 10], 1, 16, 0), ([5, 9], 5, 16, 130), ([33, 40], 33, 32, 515), ([129], 129, 16, 1000)]


@pytest.mark.parametrize("lens,n_q,heads,prefix", SHAPES)
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_exact_scores(lens, n_q, heads, prefix, fp8, dtype):
    c = Case(lens, n_q, heads, prefix, fp8, seed=prefix + n_q)
    whole_numbers(c, fp8, seed=len(lens) + prefix)
    check(c, *c.run(dtype))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("q0", [8.0, 32.0, -32.0])
def test_growing_and_falling_scores(fp8, q0):
    """Scores that grow from key to key: the maximum moves with every tile (8: 4 octaves per 64 keys) or
    every half of one (32), and the output is rescaled each time; or fall, and it never moves again."""
    c = Case([50, 60, 70], 1, 32, 2000, fp8, seed=1)
    c.q[:] = 0
    c.q[..., 0] = q0
    grow = torch.arange(c.prefix).bfloat16() / 16
    at = slice(c.start, c.start + c.prefix)
    c.k64[at, 0] = grow.double()
    if fp8:                              # growth by the K scales: codes 1
        k = c.k.view(torch.uint8)
        k[at, 0] = torch.ones(1).to(torch.float8_e4m3fn).view(torch.uint8).item()
        c.ks[at] = grow.float().cuda()
    else:
        c.k[at, 0] = grow.cuda()
    # (other dimensions meet zeros of q)
    check(c, *c.run())


def lost_bits(q, k):
    """What the two e4m3 terms of q lose of each score, and the sums' additions: 2 x 128 products."""
    top = q.abs().amax(1, keepdim=True)
    lost = torch.where(q.abs() < 2.0 ** -9 * top, 2.0 ** -17 * top.expand_as(q), torch.zeros_like(q))
    return C * (lost @ k.abs().t() + 256 * 2.0 ** -23 * (q.abs() @ k.abs().t()))


@pytest.mark.parametrize("lens,n_q,prefix", [([40, 50], 1, 700), ([9] * 17, 1, 1300), ([30, 20], 9, 260)])
@pytest.mark.parametrize("octaves", [8, 10, 12, 20])
def test_channels_far_above_the_others(lens, n_q, prefix, octaves):
    """A few channels of every query row 2^8 to 2^20 times the others, in an e4m3 cache."""
    c = Case(lens, n_q, 32, prefix, True, seed=octaves)
    g = torch.Generator().manual_seed(octaves)
    big = torch.rand(c.q.shape, generator=g) < 3 / 128
    big[..., 7] = True
    q = torch.randn(c.q.shape, generator=g) * torch.where(big, 2.0 ** octaves, 1.0)
    c.q = (q * (4.0 / q.abs().amax(-1, keepdim=True))).bfloat16()
    check(c, *c.run(), score_error=lost_bits)
    # rows without the large channels
    c.q = (q.masked_fill(big, 0) * 2.0).bfloat16()
    check(c, *c.run(), score_error=lost_bits)
