"""The operators around the block in one run, as a decode step uses them: residual stream and norm to
e4m3, the queries of the full layer and two sparse layers and the new token's K and V as e4m3
products, the cache append, attention behind a shared prefix, the importance scores of prefix and own
rows, the selection over both, a sparse layer, and the output projection of the quantised result.

Every step is checked against float64 on the step's own inputs as the GPU produced them, with the
tolerances of the operator's own tests (operator_refs, test_gpu_prefix), so that no error of an earlier step
widens a later one's bound."""
import numpy as np
import pytest
import torch

import token_level_sparse_hs2_b200 as hs2
from tests import operator_refs as R
from tests.test_gpu_gemm_fp8 import check as check_product
from tests.test_gpu_norm import check_codes

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from token_level_sparse_hs2_b200 import build
    build.build()


def quantised_weight(n, k, g):
    w = (torch.randn((n, k), generator=g) / k ** 0.5).bfloat16().cuda()
    codes, scales = torch.empty((n, k), dtype=torch.float8_e4m3fn, device="cuda"), hs2.fp8_scales(n, k, 128)
    hs2.fp8_quantize(w, codes, scales, 128)
    return codes, scales


class Step:
    """A batch behind a shared prefix and everything one decode step of it writes."""

    def __init__(self, fp8, B=5, H=32, d=512, prefix=3000, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.B, self.H, self.d, self.prefix, self.fp8 = B, H, d, prefix, fp8
        self.lens = [int(x) for x in torch.randint(1, 400, (B,), generator=g)]
        self.start, at = [], prefix + 9
        for t in self.lens:
            self.start.append(at)
            at += t + 3
        k, v = (torch.randn((at, 128), generator=g).bfloat16() for _ in range(2))
        self.ks = self.vs = None
        if fp8:
            (k, ks), (v, vs) = R.quantize(k), R.quantize(v)
            k, v = k.float().to(torch.float8_e4m3fn), v.float().to(torch.float8_e4m3fn)
            self.ks, self.vs = ks[0].cuda(), vs[0].cuda()
        self.k, self.v = k.cuda(), v.cuda()
        self.x, self.res = torch.randn((B, d), generator=g).bfloat16().cuda(), torch.randn((B, d), generator=g).cuda()
        self.wn = (1 + 0.1 * torch.randn(d, generator=g)).bfloat16().cuda()
        self.wq, self.wkv, self.wo = quantised_weight(3 * H * 128, d, g), quantised_weight(256, d, g), quantised_weight(d, H * 128, g)
        dev = dict(device="cuda")
        self.h, self.codes, self.cs = torch.empty((B, d), **dev), torch.empty((B, d), dtype=torch.float8_e4m3fn, **dev), hs2.fp8_scales(B, d)
        self.q = torch.empty((3, B, H * 128), dtype=torch.bfloat16, **dev)
        self.new_kv = torch.empty((2, B, 128), dtype=torch.bfloat16, **dev)
        self.out, self.lse = torch.empty((B, 1, H, 128), dtype=torch.bfloat16, **dev), torch.empty((B, 1, H), **dev)
        self.width = prefix + max(self.lens)
        self.scores = torch.zeros((B, (self.width + 3) // 4 * 4), **dev)
        self.idx, self.count = torch.zeros((B, 1152), dtype=torch.int32, **dev), torch.zeros(B, dtype=torch.int32, **dev)
        self.sparse = torch.empty((B, 1, H, 128), dtype=torch.bfloat16, **dev)
        self.oc, self.os = torch.empty((B, H * 128), dtype=torch.float8_e4m3fn, **dev), hs2.fp8_scales(B, H * 128)
        self.y = torch.empty((B, d), **dev)
        self.own = hs2.KvCache(self.k, self.v, self.start, self.lens, 1, H, self.ks, self.vs)
        self.pre = hs2.KvCache(self.k, self.v, [0] * B, [prefix] * B, 1, H, self.ks, self.vs)
        # positions 0 .. prefix + len of a sequence, and the cache as one long sequence for the sparse layer
        fake = torch.zeros((self.width + 1, 128), dtype=torch.bfloat16, **dev)
        self.logical = hs2.KvCache(fake, fake, [0] * B, [prefix + t for t in self.lens], 1, H)
        self.rows = hs2.KvCache(self.k, self.v, [0] * B, [self.k.shape[0]] * B, 1, H, self.ks, self.vs)
        n = max(hs2.workspace_size(c) for c in (self.own, self.pre, self.logical, self.rows))
        self.ws = torch.empty(max(n, hs2.prefix_attn_workspace_size(self.own, prefix)), dtype=torch.uint8, **dev)
        self.first = torch.tensor(self.start, dtype=torch.int32, **dev)[:, None]

    def run(self):
        hs2.rms_norm(self.x, self.wn, 1e-6, self.res, self.h, codes=self.codes, scales=self.cs)
        rows = self.H * 128
        for i in range(3):
            hs2.gemm_fp8(self.codes, self.cs, self.wq[0][i * rows:(i + 1) * rows], self.wq[1][:, i * self.H:(i + 1) * self.H],
                         self.q[i], self.ws)
        for i in range(2):
            hs2.gemm_fp8(self.codes, self.cs, self.wkv[0][i * 128:(i + 1) * 128], self.aligned_scales(i), self.new_kv[i], self.ws)
        hs2.kv_append(self.own, self.new_kv[0], self.new_kv[1])
        q = [t.view(self.B, 1, self.H, 128) for t in self.q]
        hs2.prefix_attn(self.own, 0, self.prefix, q[0], self.out, self.lse, self.ws)
        hs2.score_pass(self.pre, q[0], self.lse, self.scores, self.ws)
        hs2.score_pass(self.own, q[0], self.lse, self.scores[:, self.prefix:], self.ws)
        hs2.topk_select(self.logical, self.scores, self.idx, self.count, self.ws)
        at = torch.where(self.idx < self.prefix, self.idx, self.idx - self.prefix + self.first)   # cache rows
        hs2.sparse_gather_attn(self.rows, q[1], at, self.count, self.sparse, self.ws)
        hs2.fp8_quantize(self.sparse.view(self.B, -1), self.oc, self.os)
        hs2.gemm_fp8(self.oc, self.os, self.wo[0], self.wo[1], self.y, self.ws)

    def aligned_scales(self, i):
        # the scales of 128 of the 256 features: one column, on 16 bytes of its own
        if not hasattr(self, "kv_scales"):
            self.kv_scales = []
            for j in range(2):
                s = hs2.fp8_scales(128, self.d, 128)
                s.copy_(self.wkv[1][:, j:j + 1])
                self.kv_scales.append(s)
        return self.kv_scales[i]

    def check(self):
        h, y = R.rms_norm(self.x.cpu(), self.wn.cpu(), 1e-6, self.res.cpu())
        assert ((self.h.cpu().double() - h).abs() <= 2.0 ** -23 * h.abs()).all()
        check_codes(y, self.codes, self.cs)
        rows = self.H * 128
        for i in range(3):
            check_product(self.q[i], self.codes, self.cs, self.wq[0][i * rows:(i + 1) * rows], self.wq[1][:, i * self.H:(i + 1) * self.H])
        for i in range(2):
            check_product(self.new_kv[i], self.codes, self.cs, self.wkv[0][i * 128:(i + 1) * 128], self.kv_scales[i])
        k, v = self.k.float().cpu().double(), self.v.float().cpu().double()
        last = [f + t - 1 for f, t in zip(self.start, self.lens)]
        for cache, new, scale in ((k, self.new_kv[0], self.ks), (v, self.new_kv[1], self.vs)):
            if self.fp8:
                values, s = R.quantize(new.cpu())
                assert torch.equal(cache[last], values) and torch.equal(scale.cpu()[last], s[0])
                cache *= scale.cpu().double()[:, None]
            else:
                assert torch.equal(cache[last], new.cpu().double())
        q = self.q.view(3, self.B, self.H, 128).cpu().double()
        for b in range(self.B):
            at = torch.cat([torch.arange(self.prefix), torch.arange(self.start[b], self.start[b] + self.lens[b])])
            x = q[0, b] @ k[at].t() / 128 ** 0.5
            lse = torch.logsumexp(x, -1)
            p = torch.exp(x - lse[:, None])
            ref, mag = p @ v[at], p @ v[at].abs()
            got = self.out[b, 0].cpu().double()
            assert ((got - ref).abs() <= 2 * (2.0 ** -8 + 2.0 ** -11) * mag + 2.0 ** -8 * ref.abs()).all()
            got_lse = self.lse[b, 0].cpu().double()
            assert ((got_lse - lse).abs() <= 1e-4 + 1e-5 * lse.abs()).all()
            s = torch.exp(x - got_lse[:, None]).sum(0)
            n = len(at)
            assert ((self.scores[b, :n].cpu().double() - s).abs() <= 1e-3 * s + 1e-9 * self.H / n).all()
            # the selection is the best 1,024 of the scores as they are, and the last 128 positions
            score, nc = self.scores[b, :n].cpu().numpy(), max(0, n - 128)
            best = np.sort(np.lexsort((np.arange(nc), -score[:nc]))[:1024])
            want = np.concatenate([best, np.arange(nc, n)])
            c = int(self.count[b])
            assert np.array_equal(self.idx[b, :c].cpu().numpy(), want)
            sel = at[torch.from_numpy(want)]
            p = torch.softmax(q[1, b] @ k[sel].t() / 128 ** 0.5, -1)
            ref, mag = p @ v[sel], p @ v[sel].abs()
            assert ((self.sparse[b, 0].cpu().double() - ref).abs() <= 2 * (2.0 ** -8 + 2.0 ** -11) * mag + 2.0 ** -8 * ref.abs()).all()
        values, s = R.quantize(self.sparse.view(self.B, -1).cpu())
        assert torch.equal(self.oc.float().cpu().double(), values) and torch.equal(self.os.cpu(), s)
        check_product(self.y, self.oc, self.os, self.wo[0], self.wo[1])


@pytest.mark.parametrize("fp8", [False, True])
def test_a_decode_step(fp8):
    step = Step(fp8)
    step.run()
    step.check()


def test_a_decode_step_in_a_graph():
    step = Step(True, B=3, prefix=1500, seed=4)
    step.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step.run()
    for _ in range(2):
        step.x.normal_()
        step.res.normal_()
        g.replay()
        torch.cuda.synchronize()
        step.check()
