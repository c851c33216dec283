"""The weights' scales of hs2_gemm_fp8 as a slice of a larger array (one projection of a fused one): they are
read element by element, so any start and row stride serve."""
import pytest
import torch

import token_level_sparse_hs2_b200 as hs2
from tests.test_operators_host import A, GEMM, L, refused  # noqa: F401


@pytest.mark.parametrize("change", [dict(sw=A + 4), dict(sw=A + 12), dict(swld=3), dict(swld=7, sw=A + 8)])
def test_any_start_and_stride_is_taken(L, change):  # noqa: F811
    # as far as the next argument's check
    refused(L, L.hs2_gemm_fp8, list({**GEMM, **change, "ws": None}.values()), 1, b"workspace")


@pytest.mark.parametrize("change,word", [(dict(sw=A + 2), b"w_scale"), (dict(swld=2), b"scale_ld"), (dict(sa=A + 4), b"aligned"),
                                         (dict(sald=5), b"scale_ld")])
def test_what_stays_refused(L, change, word):  # noqa: F811
    refused(L, L.hs2_gemm_fp8, list({**GEMM, **change}.values()), 1, word)


@pytest.mark.gpu
@pytest.mark.parametrize("m", [1, 40, 100, 5000])          # tiles of 32, 64 and 128 tokens and of CTA pairs
@pytest.mark.parametrize("n,k", [(256, 1040), (100, 128), (500, 2048)])
def test_products_with_a_slice_of_the_scales(m, n, k):
    from tests.test_gpu_gemm_fp8 import check, codes_of, scales_of, workspace
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from token_level_sparse_hs2_b200 import build
    build.build()
    g = torch.Generator().manual_seed(m + n + k)
    kb, nb = -(-k // 128), -(-n // 128)
    a, sa, w = codes_of(m, k, g), scales_of(kb, m, g), codes_of(n, k, g)
    fused = torch.full((kb, nb + 6), float("nan"), device="cuda")
    for first in (1, 2, 3):
        sw = fused[:, first:first + nb]
        sw.copy_(torch.exp(torch.randn((kb, nb), generator=g)))
        out, whole = (torch.empty((m, n), device="cuda") for _ in range(2))
        hs2.gemm_fp8(a, sa, w, sw, out, workspace())
        own = hs2.fp8_scales(n, k, 128)
        own.copy_(sw)
        hs2.gemm_fp8(a, sa, w, own, whole, workspace())
        assert torch.equal(out, whole)
        fused.fill_(float("nan"))
        if first == 1:
            check(out[:200], a[:200], sa[:, :200], w, own)
