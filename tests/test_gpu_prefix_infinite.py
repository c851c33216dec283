"""hs2_prefix_attn for rows whose every score is -inf, by the formula: the log-sum-exp of nothing but exp(-inf)
is -inf, and the output's weights exp(-inf - lse) are NaN, however many ranges the tiles are split into."""
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


@pytest.mark.parametrize("prefix,own,one_range", [(0, 1, True), (0, 100, True), (1, 2, False), (100, 3, False), (5000, 3, False)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_whose_every_score_is_minus_infinity(prefix, own, one_range, dtype):
    c = Case([own] if one_range else [own, 4], 1, 16, prefix, seed=prefix)
    # the workspace holds partial results of two ranges or more, or the status word alone
    assert (hs2.prefix_attn_workspace_size(c.cache(), prefix) == 256) == one_range
    c.q[:, 0, :, 0] = 1.0
    c.q[0, 0, 5] = 0                           # one element alone, a small one
    c.q[0, 0, 5, 0] = 2.0 ** -100
    used = list(range(c.start, c.start + prefix)) + list(range(c.first[0], c.first[0] + own))
    c.k[used, 0] = float("-inf")               # every row that sequence 0 sees
    c.k64[used, 0] = float("-inf")
    out, lse = c.run(dtype)
    ref, _, want = c.reference()
    assert torch.isnan(ref[0]).all() and (want[0] == -torch.inf).all()
    assert torch.isnan(out[0]).all(), out[0].isnan().sum()
    assert (lse[0] == -torch.inf).all()
    assert torch.isfinite(lse[1:]).all() and torch.isfinite(out[1:]).all()       # its own rows are finite
