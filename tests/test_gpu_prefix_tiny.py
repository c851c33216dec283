"""hs2_prefix_attn with queries and softmax scales so small that their product is below float32: every weight
is the same, positions that a row does not see keep none, whatever the cache's type."""
import pytest
import torch

from tests.test_gpu_prefix import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from token_level_sparse_hs2_b200 import build
    build.build()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("scale", [1e-8, 1e-15, 1e-30, 1e-44])
@pytest.mark.parametrize("lens,n_q,prefix", [([40, 3], 1, 100), ([9], 5, 0)])
def test_uniform_weights(lens, n_q, prefix, scale, fp8):
    c = Case(lens, n_q, 16, prefix, fp8, seed=17)
    c.q *= 2.0 ** -125
    c.check(*c.run(scale=scale), scale=scale)
