"""The steps of a decode call behind a shared prefix, as the README gives them (attention, scores of both
parts, selection over them, a sparse layer), against the block's own calls on a cache in which every sequence
holds its own copy of the prefix.

Tolerances: outputs of either path are within 2^-8 a + 2^-11 a + half a step of the exact ones (a = sum of
weight x |v|: test_gpu_prefix_bounds, and the block's passes hold theirs to at least that); the two lse within 1e-4 +
1e-5 |lse| each, which the scores' exponentials turn into as much of each score, and their own passes 1e-4 more.
The selection is exact on the scores as they are; the sparse layer reads the same rows, so it is equal bit for bit."""
import numpy as np
import pytest
import torch

import token_level_sparse_hs2_b200 as hs2
from tests import operator_refs as R

pytestmark = pytest.mark.gpu
H = 32


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from token_level_sparse_hs2_b200 import build
    build.build()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("prefix_start,prefix_len,own_len", [(0, 2999, [1, 300, 77, 5]), (13, 40, [1500, 3]), (1, 6001, [129] * 9)])
def test_the_documented_steps(prefix_start, prefix_len, own_len, fp8):
    g = torch.Generator().manual_seed(prefix_len)
    B = len(own_len)
    own_start, at = [], prefix_start + prefix_len + 3
    for t in own_len:
        own_start.append(at)
        at += t + 1
    k, v = (torch.randn((at, 128), generator=g).bfloat16() for _ in range(2))
    ks = vs = None
    if fp8:
        (k, ks), (v, vs) = R.quantize(k), R.quantize(v)
        k, v, ks, vs = k.float().to(torch.float8_e4m3fn), v.float().to(torch.float8_e4m3fn), ks[0].cuda(), vs[0].cuda()
    k, v = k.cuda(), v.cuda()
    scale = (ks, vs) if fp8 else ()
    q, q_sparse = (torch.randn((B, 1, H, 128), generator=g).bfloat16().cuda() for _ in range(2))
    new = dict(device="cuda")

    # the steps
    own = hs2.KvCache(k, v, own_start, own_len, 1, H, *scale)
    pre = hs2.KvCache(k, v, [prefix_start] * B, [prefix_len] * B, 1, H, *scale)
    both = hs2.KvCache(k, v, [0] * B, [prefix_len + t for t in own_len], 1, H, *scale)
    rows = hs2.KvCache(k, v, [0] * B, [k.shape[0]] * B, 1, H, *scale)
    ws = torch.empty(max(hs2.prefix_attn_workspace_size(own, prefix_len), *(hs2.workspace_size(c) for c in (own, pre, both, rows))),
                     dtype=torch.uint8, **new)
    out, lse = torch.empty((B, 1, H, 128), **new), torch.empty((B, 1, H), **new)
    scores = torch.empty((B, prefix_len + max(own_len)), **new)
    idx, count = torch.empty((B, hs2.TOPK + hs2.WINDOW), dtype=torch.int32, **new), torch.empty(B, dtype=torch.int32, **new)
    sparse = torch.empty((B, 1, H, 128), **new)
    first = torch.tensor(own_start, dtype=torch.int32, **new)[:, None]
    hs2.prefix_attn(own, prefix_start, prefix_len, q, out, lse, ws)
    hs2.score_pass(pre, q, lse, scores, ws)
    hs2.score_pass(own, q, lse, scores[:, prefix_len:], ws)
    hs2.topk_select(both, scores, idx, count, ws)
    at = torch.where(idx < prefix_len, prefix_start + idx, first + (idx - prefix_len))
    hs2.sparse_gather_attn(rows, q_sparse, at, count, sparse, ws)
    hs2.read_device_status(ws)

    # every sequence with a copy of the prefix
    order = torch.cat([torch.cat([torch.arange(prefix_start, prefix_start + prefix_len), torch.arange(s, s + t)]) for s, t in zip(own_start, own_len)]).cuda()
    lens = [prefix_len + t for t in own_len]
    starts = [sum(lens[:b]) for b in range(B)]
    flat = lambda t: t.view(torch.uint8)[order].view(t.dtype) if fp8 and t.dim() == 2 else t[order]  # noqa: E731
    alone = hs2.KvCache(flat(k), flat(v), starts, lens, 1, H, *(s[order].contiguous() for s in scale))
    ws2 = torch.empty(hs2.workspace_size(alone), dtype=torch.uint8, **new)
    out2, lse2, scores2, sparse2 = torch.empty_like(out), torch.empty_like(lse), torch.empty_like(scores), torch.empty_like(sparse)
    hs2.full_attn_scores(alone, q, out2, lse2, scores2, ws2)
    hs2.sparse_gather_attn(alone, q_sparse, idx, count, sparse2, ws2)
    hs2.read_device_status(ws2)

    assert ((lse - lse2).abs() <= 2 * (1e-4 + 1e-5 * lse.abs())).all()
    assert torch.equal(sparse, sparse2)
    vf = v.float() * (vs[:, None] if fp8 else 1)
    kf = k.float() * (ks[:, None] if fp8 else 1)
    for b, n in enumerate(lens):
        r = order[starts[b]:starts[b] + n]
        p = torch.softmax(q[b, 0].double() @ kf[r].double().t() / 128 ** 0.5, -1)
        mag = p @ vf[r].double().abs()
        assert ((out[b, 0] - out2[b, 0]).abs() <= 2 * (2.0 ** -8 + 2.0 ** -11) * mag + 2.0 ** -23 * out[b, 0].abs()).all()
        s, s2 = scores[b, :n].double(), scores2[b, :n].double()
        tol = 2 * (1e-4 + 1e-5 * float(lse[b].abs().max())) + 2e-4
        assert ((s - s2).abs() <= tol * s2).all()
        score, nc = scores[b, :n].cpu().numpy(), max(0, n - hs2.WINDOW)
        best = np.sort(np.lexsort((np.arange(nc), -score[:nc]))[:hs2.TOPK])
        want = np.concatenate([best, np.arange(nc, n)])
        assert int(count[b]) == len(want) and np.array_equal(idx[b, :len(want)].cpu().numpy(), want)
