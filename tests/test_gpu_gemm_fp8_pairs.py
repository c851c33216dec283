"""Products by CTA pairs in a row, each started while the one before it ends: what the leader of a pair
signals to the other CTA's shared memory has to have arrived before that CTA leaves, since the next kernel's
barriers may lie there. Results are equal to those of calls that stand alone, bit for bit, and the status
word stays clear."""
import pytest
import torch

import token_level_sparse_hs2_b200 as hs2
from tests.test_gpu_gemm_fp8 import check, codes_of, scales_of, workspace

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from token_level_sparse_hs2_b200 import build
    build.build()


# one block along k (all stages but one unused), fewer blocks than stages, as many, one more; one tile per pair and several
@pytest.mark.parametrize("m,n,k", [(20000, 256, 16), (9473, 256, 272), (5000, 512, 640), (2500, 1280, 768), (4900, 1001, 896),
                                   (2049, 2305, 2064)])
def test_calls_in_a_row_equal_calls_alone(m, n, k):
    g = torch.Generator().manual_seed(m + n + k)
    kb = -(-k // 128)
    ops = [(codes_of(m, k, g), scales_of(kb, m, g), codes_of(n, k, g), scales_of(kb, -(-n // 128), g)) for _ in range(3)]
    alone, outs, ws = [], [torch.empty((m, n), dtype=torch.bfloat16, device="cuda") for _ in range(3)], workspace()
    for op in ops:
        out = torch.empty((m, n), dtype=torch.bfloat16, device="cuda")
        hs2.gemm_fp8(*op, out, ws)
        hs2.read_device_status(ws)
        alone.append(out)
    check(alone[0][:300], ops[0][0][:300], ops[0][1][:, :300], *ops[0][2:])
    status = [workspace() for _ in range(30)]
    x = torch.randn((64, 4096), device="cuda").bfloat16()
    y, w = torch.empty_like(x), torch.ones(4096, device="cuda")
    torch.cuda.synchronize()
    for i in range(30):              # each leaves memory to the next: products of other inputs, and norms in between
        hs2.gemm_fp8(*ops[i % 3], outs[i % 3], status[i])
        if i % 4 == 3:
            hs2.rms_norm(x, w, out=y)
    for s in status:
        hs2.read_device_status(s)
    for out, want in zip(outs, alone):
        assert torch.equal(out, want)
