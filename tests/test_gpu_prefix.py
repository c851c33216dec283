"""GPU parity of hs2_prefix_attn, through the binding, against plain float64 attention over each
sequence's prefix and own rows.

Tolerance of the output, per element, with a = sum of weight x |v|: each weight is rounded to
bf16 for its product with V, within 2^-8 of itself (the exponential and the float32 arguments
add less than 2^-12: the arguments are below 64 in magnitude, in float32 after the products'
128 additions), so (2^-8 + 2^-11) a, doubled for the own rows' pass, whose e4m3 form rounds the
probabilities scaled by the V scales once more, plus the output's half step (bf16 2^-8, float32
2^-24). The log-sum-exp sums positive float32 exponentials: 1e-4 + 1e-5 |lse|, the bound that the
block's own passes are held to (their exponentials are a polynomial within 7.5e-5)."""
import numpy as np
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


class Case:
    """A cache with a prefix and sequences; every row that is neither holds NaN."""

    def __init__(self, lens, n_q, heads, prefix, fp8=False, seed=0, start=None, gap=3, q_scale=1.0, spread=0.0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.n_q, self.heads, self.prefix = list(lens), n_q, heads, prefix
        self.start = 5 if start is None else start
        at, self.first = self.start + prefix + gap, []
        for t in self.lens:
            self.first.append(at)
            at += t + gap
        rows = at + 130
        used = torch.zeros(rows, dtype=torch.bool)
        used[self.start:self.start + prefix] = True
        for f, t in zip(self.first, self.lens):
            used[f:f + t] = True
        k, v = (torch.randn((rows, 128), generator=g).bfloat16() for _ in range(2))
        self.ks = self.vs = None
        if fp8:
            if spread:                                   # rows of very different scales
                k = (k.float() * torch.exp(spread * torch.randn((rows, 1), generator=g))).bfloat16()
                v = (v.float() * torch.exp(spread * torch.randn((rows, 1), generator=g))).bfloat16()
            (k, ks), (v, vs) = R.quantize(k), R.quantize(v)
            self.k64, self.v64 = k * ks[0].double()[:, None], v * vs[0].double()[:, None]
            k, v = (t.float().to(torch.float8_e4m3fn).view(torch.uint8) for t in (k, v))
            self.ks, self.vs = ks[0].clone(), vs[0].clone()
            k[~used], v[~used] = 0x7f, 0x7f
            self.ks[~used], self.vs[~used] = float("nan"), float("inf")
            self.ks, self.vs = self.ks.cuda(), self.vs.cuda()
            k, v = k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn)
        else:
            self.k64, self.v64 = k.double(), v.double()
            k[~used], v[~used] = float("nan"), float("inf")
        self.k, self.v = k.cuda(), v.cuda()
        self.q = (q_scale * torch.randn((len(self.lens), n_q, heads, 128), generator=g)).bfloat16()

    def cache(self):
        return hs2.KvCache(self.k, self.v, self.first, self.lens, self.n_q, self.heads, self.ks, self.vs)

    def run(self, out_dtype=torch.float32, ws_fill=0xff, stream=None, scale=None, lse=True):
        cache = self.cache()
        ws = torch.full((hs2.prefix_attn_workspace_size(cache, self.prefix),), ws_fill, dtype=torch.uint8, device="cuda")
        out = torch.full(self.q.shape, float("nan"), dtype=out_dtype, device="cuda")
        l = torch.full(self.q.shape[:3], float("nan"), device="cuda") if lse else None
        q = self.q.cuda()
        torch.cuda.synchronize()
        hs2.prefix_attn(cache, self.start, self.prefix, q, out, l, ws, scale=scale, stream=stream)
        hs2.read_device_status(ws, stream)
        return out, l

    def reference(self, scale=None):
        scale = 128 ** -0.5 if scale is None else scale
        out = torch.empty(self.q.shape, dtype=torch.float64)
        mag, lse = torch.empty_like(out), torch.empty(self.q.shape[:3], dtype=torch.float64)
        for b, (f, t) in enumerate(zip(self.first, self.lens)):
            rows = torch.cat([torch.arange(self.start, self.start + self.prefix), torch.arange(f, f + t)])
            k, v = self.k64[rows], self.v64[rows]
            x = torch.einsum("qhd,td->qht", self.q[b].double(), k) * scale
            last = self.prefix + t - self.n_q + torch.arange(self.n_q)
            x.masked_fill_((torch.arange(len(rows)) > last[:, None])[:, None], -torch.inf)
            lse[b] = torch.logsumexp(x, -1)
            p = torch.exp(x - lse[b][..., None])
            out[b], mag[b] = p @ v, p @ v.abs()
        return out, mag, lse

    def check(self, got, lse, scale=None):
        out, mag, want = self.reference(scale)
        tol = 2 * (2.0 ** -8 + 2.0 ** -11) * mag + HALF[got.dtype] * out.abs()
        off = (got.cpu().double() - out).abs()
        assert (off <= tol).all(), float((off / tol).nan_to_num(1e9).max())
        if lse is not None:
            assert ((lse.cpu().double() - want).abs() <= 1e-4 + 1e-5 * want.abs()).all()


DECODE = [([1], 1, 16, 1), ([1, 5], 1, 16, 127), ([300, 1, 77], 1, 32, 128), ([64] * 4, 1, 32, 129), ([3] * 5, 1, 32, 1000),
          ([1, 2, 3, 4, 5, 6, 7, 8, 9], 1, 32, 5000), ([17] * 33, 1, 16, 777), ([200] * 8, 1, 32, 4096), ([2] * 128, 1, 32, 300),
          ([1000, 10], 1, 16, 20011), ([1100] * 9, 1, 32, 500), ([2000, 3, 1500, 700] * 5, 1, 16, 77), ([3000] * 8, 1, 32, 6000)]
CHUNKS = [([2], 2, 16, 1), ([5, 9], 5, 16, 130), ([33, 40, 33], 33, 32, 515), ([129, 300], 129, 32, 1000), ([17], 17, 32, 9001),
          ([700], 513, 16, 250), ([1500, 900, 1200], 3, 32, 3000), ([2000, 1000], 70, 16, 140)]


@pytest.mark.parametrize("lens,n_q,heads,prefix", DECODE + CHUNKS)
@pytest.mark.parametrize("fp8", [False, True])
def test_prefix(lens, n_q, heads, prefix, fp8):
    c = Case(lens, n_q, heads, prefix, fp8, seed=prefix + n_q)
    c.check(*c.run())
    c.check(*c.run(torch.bfloat16, ws_fill=0))


@pytest.mark.parametrize("fp8", [False, True])
def test_no_prefix_is_plain_attention(fp8):
    for lens, n_q in (([40, 1, 900], 1), ([40, 50], 7)):
        c = Case(lens, n_q, 32, 0, fp8, seed=4)
        c.check(*c.run())
        c.check(*c.run(torch.bfloat16, lse=False))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("start,gap", [(0, 0), (1, 0), (64, 1), (4099, 2)])
def test_prefix_anywhere_and_rows_beside_it_unused(fp8, start, gap):
    c = Case([20, 31], 1, 32, 333, fp8, seed=7, start=start, gap=gap)
    c.check(*c.run())


@pytest.mark.parametrize("fp8", [False, True])
def test_sharp_and_flat_scores(fp8):
    c = Case([50, 60, 70], 1, 32, 3000, fp8, seed=1, q_scale=4.0)
    c.check(*c.run())                                   # scores of many units: the maximum moves
    c.check(*c.run(scale=1e-6), scale=1e-6)             # all but uniform weights
    c = Case([50, 60, 70], 1, 32, 3000, fp8, seed=1, q_scale=0.0)
    c.check(*c.run())
    c.q[:] = 0
    c.q[..., 0] = 8
    c.k64[c.start:c.start + c.prefix, 0] = torch.arange(c.prefix).bfloat16().double() / 16
    if not fp8:                                         # growing scores: every tile moves the maximum
        c.k[c.start:c.start + c.prefix, 0] = (torch.arange(c.prefix).bfloat16() / 16).cuda()
        c.check(*c.run())


def test_rows_of_very_different_scales():
    c = Case([50, 60], 1, 32, 2500, True, seed=2, spread=1.5, q_scale=0.3)
    c.check(*c.run())


def test_the_mass_may_lie_in_either_part():
    for where in ("prefix", "own"):
        c = Case([40, 40], 1, 16, 1000, seed=3)
        u = c.q[0, 0, 0].double()
        c.q[:] = c.q[0, 0, 0]
        row = c.start + 17 if where == "prefix" else c.first[0] + 30
        c.k64[row] = (u / u.norm() * 128).bfloat16().double()
        c.k[row] = c.k64[row].bfloat16().cuda()
        c.check(*c.run())


@pytest.mark.parametrize("fp8", [False, True])
def test_one_sequences_nan_stays_its_own(fp8):
    c = Case([40, 50, 60], 1, 32, 700, fp8, seed=6)
    want, lse = c.run()
    if fp8:
        c.k.view(torch.uint8)[c.first[1] + 3] = 0x7f
        c.v.view(torch.uint8)[c.first[1] + 4] = 0x7f
    else:
        c.k[c.first[1] + 3] = float("nan")
        c.v[c.first[1] + 4] = float("inf")
    out, lse2 = c.run()
    for b in (0, 2):
        assert torch.equal(out[b], want[b]) and torch.equal(lse2[b], lse[b])
    assert not torch.isfinite(out[1]).any()


@pytest.mark.parametrize("fp8", [False, True])
def test_query_rows_of_any_magnitude(fp8):
    c = Case([40, 50], 1, 32, 700, fp8, seed=13)
    c.q *= torch.exp2(torch.linspace(-100, 5, 32)).bfloat16()[:, None]     # heads from 2^-100 to 2^5
    c.q[1, 0, 3] = 0
    c.q[1, 0, 4, 1:] = 0                                                   # one element alone
    c.check(*c.run())
    want, lse = c.run()
    c.q[0, 0, 7, 5], c.q[0, 0, 8, 9] = float("inf"), float("nan")
    out, lse2 = c.run()
    keep = torch.ones(32, dtype=torch.bool)
    keep[7:9] = False
    assert torch.equal(out[0, 0][keep], want[0, 0][keep]) and torch.equal(out[1], want[1]) and torch.equal(lse2[1], lse[1])
    assert torch.isnan(out[0, 0, 7:9]).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_streams_graphs_repeats(fp8):
    a, b = Case([30] * 9, 1, 32, 6000, fp8, seed=8), Case([200] * 3, 40, 32, 1500, fp8, seed=9)
    want = [c.run() for c in (a, b)]
    s = torch.cuda.Stream()
    for c, w in zip((a, b), want):
        got = c.run(stream=s)
        assert torch.equal(got[0], w[0]) and torch.equal(got[1], w[1])
    state = []
    for c in (a, b):
        cache = c.cache()
        state.append((c, cache, c.q.cuda(), torch.empty(c.q.shape, device="cuda"), torch.empty(c.q.shape[:3], device="cuda"),
                      torch.empty(hs2.prefix_attn_workspace_size(cache, c.prefix), dtype=torch.uint8, device="cuda")))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for c, cache, q, out, lse, ws in state:
            hs2.prefix_attn(cache, c.start, c.prefix, q, out, lse, ws)
    for _ in range(2):
        for st in state:
            st[3].zero_()
        g.replay()
        for st, w in zip(state, want):
            assert torch.equal(st[3], w[0]) and torch.equal(st[4], w[1])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        for (c, cache, q, out, lse, ws), st in zip(state, streams):   # at once, each with its workspace
            hs2.prefix_attn(cache, c.start, c.prefix, q, out, lse, ws, stream=st)
    torch.cuda.synchronize()
    for st, w in zip(state, want):
        assert torch.equal(st[3], w[0])


def test_many_pairs_and_long_prefix():
    """More row blocks than SMs, and a prefix long enough for many ranges: sampled rows."""
    for lens, n_q, heads, prefix, fp8 in (([1300], 1200, 32, 700, False), ([600] * 2, 600, 32, 900, True), ([9, 9], 1, 32, 150001, False)):
        c = Case(lens, n_q, heads, prefix, fp8, seed=12)
        out, lse = c.run()
        sample = sorted({0, min(1, n_q - 1), n_q // 2, n_q - 1})
        full = c.q
        ref = torch.empty((len(lens), len(sample), heads, 128), dtype=torch.float64)
        for b, (f, t) in enumerate(zip(c.first, c.lens)):
            for j, i in enumerate(sample):
                rows = torch.cat([torch.arange(c.start, c.start + prefix), torch.arange(f, f + t - n_q + i + 1)])
                x = torch.einsum("hd,td->ht", full[b, i].double(), c.k64[rows]) / 128 ** 0.5
                w = torch.softmax(x, -1)
                ref[b, j] = w @ c.v64[rows]
                tol = 2 * (2.0 ** -8 + 2.0 ** -11) * (w @ c.v64[rows].abs()) + 2.0 ** -24 * ref[b, j].abs()
                assert ((out[b, i].cpu().double() - ref[b, j]).abs() <= tol).all()
                want = torch.logsumexp(x, -1)
                assert ((lse[b, i].cpu().double() - want).abs() <= 1e-4 + 1e-5 * want.abs()).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_overlapping_rows(fp8):
    """Two sequences with the same own rows, and one whose own rows are the prefix's last."""
    c = Case([90, 90, 300], 1, 32, 1000, fp8, seed=21)
    c.first[1] = c.first[0]
    c.first[2] = c.start + c.prefix - 300
    c.check(*c.run())


@pytest.mark.parametrize("fp8", [False, True])
def test_a_later_tokens_key_does_not_reach_earlier_queries(fp8):
    c = Case([140, 9], 6, 16, 400, fp8, seed=22)
    want, lse = c.run()
    row = c.first[0] + 140 - 2                       # the token of query 4
    if fp8:
        c.k.view(torch.uint8)[row] = 0x7f
    else:
        c.k[row] = float("nan")
    out, lse2 = c.run()
    assert torch.equal(out[0, :4], want[0, :4]) and torch.equal(lse2[0, :4], lse[0, :4])
    assert torch.equal(out[1], want[1]) and not torch.isfinite(out[0, 4:]).any()


@pytest.mark.parametrize("fp8", [False, True])
def test_rows_behind_32_bit_offsets(fp8):
    """Prefix and own rows whose elements lie more than 2^31 (bf16) or 2^32 bytes into the cache."""
    c = Case([50, 300], 1, 32, 1500, fp8, seed=23)
    want, lse = c.run()
    at = (1 << 31) // 128 + 77 if not fp8 else (1 << 32) // 128 + 77
    for name in ("k", "v", "ks", "vs"):
        small = getattr(c, name)
        if small is not None:
            big = torch.empty((at + small.shape[0],) + small.shape[1:], dtype=small.dtype, device="cuda")
            big[at:] = small
            setattr(c, name, big)
    c.start += at
    c.first = [f + at for f in c.first]
    out, lse2 = c.run()
    assert torch.equal(out, want) and torch.equal(lse2, lse)


@pytest.mark.parametrize("lens,n_q,prefix,splits", [([150, 100, 90, 500], 80, 700, range(2, 8)), ([60, 50, 45], 40, 3000, range(8, 16)),
                                                    ([30, 40], 21, 5000, range(16, 32)), ([200, 90], 19, 9001, range(16, 32))])
def test_many_rows_by_number_of_parts(lens, n_q, prefix, splits):
    c = Case(lens, n_q, 32, prefix, seed=31)
    rows = len(lens) * n_q * 32
    parts = (hs2.prefix_attn_workspace_size(c.cache(), prefix) - 256) // (rows * 129 * 4)
    assert rows > 8 * 148 and parts in splits
    c.check(*c.run())
    c.check(c.run(torch.bfloat16, lse=False)[0], None)
