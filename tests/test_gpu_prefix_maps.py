"""hs2_prefix_attn where the host makes only some of the kernel's tensor maps (no map of the query for an
e4m3 cache, none of a prefix that has no rows): calls of every kind in turn on one workspace, also captured
and replayed, equal the same calls alone."""
import pytest
import torch

import token_level_sparse_hs2_b200 as hs2
from tests.test_gpu_prefix import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from token_level_sparse_hs2_b200 import build
    build.build()


def test_calls_with_and_without_a_prefix_in_turn():
    cases = [Case([40, 1, 900], 1, 32, prefix, fp8, seed=prefix + fp8) for prefix in (0, 700) for fp8 in (False, True)]
    cases += [Case([50, 60], 7, 16, 0, fp8, seed=3) for fp8 in (False, True)]
    alone = []
    for c in cases:
        got = c.run()
        c.check(*got)
        alone.append(got)
    caches, qs = [c.cache() for c in cases], [c.q.cuda() for c in cases]
    ws = torch.empty(max(hs2.prefix_attn_workspace_size(k, c.prefix) for k, c in zip(caches, cases)), dtype=torch.uint8, device="cuda")
    outs = [(torch.zeros_like(o), torch.zeros_like(l)) for o, l in alone]

    def run():
        for c, cache, q, (out, lse) in zip(cases, caches, qs, outs):
            hs2.prefix_attn(cache, c.start, c.prefix, q, out, lse, ws)

    def equal():
        hs2.read_device_status(ws)
        for got, want in zip(outs, alone):
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
            got[0].zero_()

    run()
    run()
    equal()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(2):
        graph.replay()
        equal()
