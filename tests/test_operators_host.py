"""Refusals of the operators around the block, on the CPU: every bad argument is an error before
any launch, with a message, and nothing is written."""
import ctypes

import pytest
import torch

import token_level_sparse_hs2_b200 as hs2

BF16, F32 = hs2.OUT_BF16, hs2.OUT_F32
P = ctypes.c_void_p
A = 4096                       # an aligned address that nothing reads: the checks come first


@pytest.fixture(scope="module")
def L():
    from token_level_sparse_hs2_b200 import build
    build.build()
    return hs2.lib()


def refused(L, fn, args, status, word=b""):
    got = fn(*args)
    assert got == status, (got, L.hs2_last_error())
    assert word in L.hs2_last_error(), L.hs2_last_error()


NORM = dict(rows=4, d=256, x=A, xs=256, res=A, ro=A, rt=BF16, rs=256, w=A, wt=BF16, eps=1e-6, out=A, ot=BF16,
            os=256, codes=A, cs=256, scales=A, ld=4, stream=None)


@pytest.mark.parametrize("change,status,word", [
    (dict(rows=-1), 1, b"rows"), (dict(rows=2 ** 31), 1, b"rows"),
    (dict(d=0), 2, b"d 0"), (dict(d=12), 2, b"d 12"), (dict(d=32776), 2, b"d 32776"),
    (dict(d=248, xs=256), 2, b"codes"),
    (dict(x=None), 1, b"x"), (dict(w=None), 1, b"weight"), (dict(x=A + 8), 1, b"x"),
    (dict(w=A + 2), 1, b"weight"), (dict(xs=248), 1, b"x"), (dict(xs=260), 1, b"x"), (dict(wt=2), 1, b"weight_dtype"),
    (dict(res=None), 1, b"both"), (dict(ro=None), 1, b"both"), (dict(rt=5), 1, b"residual_dtype"),
    (dict(rs=128), 1, b"residual"), (dict(ro=A + 4), 1, b"residual_out"),
    (dict(eps=-1.0), 1, b"eps"), (dict(eps=float("nan")), 1, b"eps"), (dict(eps=float("inf")), 1, b"eps"),
    (dict(out=None, codes=None, scales=None), 1, b"both NULL"), (dict(ot=3), 1, b"out_dtype"),
    (dict(os=255), 1, b"out"), (dict(out=A + 8), 1, b"out"),
    (dict(codes=None), 1, b"codes"), (dict(scales=None), 1, b"scales"), (dict(cs=264), 1, b"codes_stride"),
    (dict(cs=240), 1, b"codes_stride"), (dict(ld=3), 1, b"scale_ld"), (dict(ld=6), 1, b"scale_ld"),
    (dict(scales=A + 4), 1, b"aligned"), (dict(codes=A + 8), 1, b"aligned"),
])
def test_norm_refusals(L, change, status, word):
    refused(L, L.hs2_rms_norm, list({**NORM, **change}.values()), status, word)


def test_no_rows_is_no_work(L):
    assert L.hs2_rms_norm(*{**NORM, "rows": 0, "x": None, "res": None, "ro": None, "out": None, "codes": None,
                            "scales": None}.values()) == 0
    assert L.hs2_fp8_quantize(0, 128, None, 128, 1, None, 128, None, 4, None) == 0


QUANT = dict(rows=4, cols=256, x=A, xs=256, br=1, codes=A, cs=256, scales=A, ld=4, stream=None)


@pytest.mark.parametrize("change,status,word", [
    (dict(rows=-1), 1, b"rows"), (dict(cols=8), 2, b"cols"), (dict(cols=264, xs=264), 2, b"cols"), (dict(cols=65552), 2, b"cols"),
    (dict(br=2), 2, b"block_rows"), (dict(br=0), 2, b"block_rows"), (dict(x=None), 1, b"x"), (dict(xs=248), 1, b"x"),
    (dict(codes=None), 1, b"codes"), (dict(scales=None), 1, b"scales"), (dict(cs=250), 1, b"codes_stride"),
    (dict(ld=0), 1, b"scale_ld"), (dict(ld=2, br=128), 1, b"scale_ld"),
])
def test_quantize_refusals(L, change, status, word):
    refused(L, L.hs2_fp8_quantize, list({**QUANT, **change}.values()), status, word)


def test_binding_refuses_wrong_tensors(L):
    x, w = torch.zeros((4, 256), dtype=torch.bfloat16), torch.ones(256)
    y, c = torch.zeros((4, 256)), torch.zeros((4, 256), dtype=torch.uint8)
    s = hs2.fp8_scales(4, 256, device="cpu")
    for bad in (dict(x=x.float()), dict(x=x.t()), dict(x=x[0]), dict(out=y[:3]), dict(out=y.half()), dict(residual=x),
                dict(codes=c), dict(scales=s), dict(codes=c, scales=s[:1]), dict(codes=c, scales=s.double()),
                dict(weight=w[:128]), dict(residual=x, residual_out=y)):
        args = dict(x=x, weight=w, out=y)
        args.update(bad)
        with pytest.raises((TypeError, ValueError)):
            hs2.rms_norm(**args)
    for args in ((x.float(), c, s), (x, c[:, :128], s), (x, c, s[:, :2]), (x, c.float(), s)):
        with pytest.raises((TypeError, ValueError)):
            hs2.fp8_quantize(*args)


def test_scale_arrays_have_the_layout_the_library_reads():
    for rows, cols, br, want in ((1, 16, 1, (1, 1, 4)), (5, 4096, 1, (32, 5, 8)), (129, 300, 128, (3, 2, 4))):
        s = hs2.fp8_scales(rows, cols, br, device="cpu")
        assert tuple(s.shape) == want[:2] and s.stride(0) == want[2] and s.stride(1) == 1


def ws_ptr():
    buf = torch.zeros(1024, dtype=torch.uint8)
    return buf, buf.data_ptr() + (-buf.data_ptr()) % 256


GEMM = dict(m=4, n=300, k=256, a=A, lda=256, sa=A, sald=4, w=A, ldw=256, sw=A, swld=4, out=A, ot=BF16, ldo=300, ws=A,
            wsb=256, stream=None)


@pytest.mark.parametrize("change,status,word", [
    (dict(m=-1), 1, b"m"), (dict(m=2 ** 31), 1, b"m"), (dict(n=0), 2, b"n 0"), (dict(n=2 ** 24 + 1), 2, b"n "),
    (dict(k=0), 2, b"k 0"), (dict(k=264, lda=272, ldw=272), 2, b"k 264"), (dict(k=65552, lda=65552, ldw=65552), 2, b"k"),
    (dict(a=None), 1, b"codes"), (dict(a=A + 8), 1, b"aligned"), (dict(lda=248), 1, b"codes_stride"),
    (dict(lda=264), 1, b"codes_stride"), (dict(sa=None), 1, b"scales"), (dict(sald=3), 1, b"scale_ld"), (dict(sald=6), 1, b"scale_ld"),
    (dict(w=None), 1, b"w"), (dict(w=A + 1), 1, b"aligned"), (dict(ldw=128), 1, b"codes_stride"), (dict(sw=None), 1, b"w_scale"),
    (dict(swld=2), 1, b"scale_ld"), (dict(out=None), 1, b"out"), (dict(out=A + 1), 1, b"out"), (dict(ot=F32, out=A + 2), 1, b"out"),
    (dict(ot=2), 1, b"out_dtype"), (dict(ldo=299), 1, b"ldo"), (dict(ws=None), 1, b"workspace"), (dict(ws=A + 64), 1, b"workspace"),
    (dict(wsb=255), 3, b"workspace"),
])
def test_gemm_refusals(L, change, status, word):
    refused(L, L.hs2_gemm_fp8, list({**GEMM, **change}.values()), status, word)


def test_gemm_without_rows_is_no_work(L):
    assert L.hs2_gemm_fp8(*{**GEMM, "m": 0, "a": None, "sa": None, "out": None, "ws": None, "wsb": 0}.values()) == 0


def test_gemm_binding_refuses_wrong_tensors(L):
    a, w = torch.zeros((4, 256), dtype=torch.uint8), torch.zeros((300, 256), dtype=torch.uint8)
    good = dict(a=a, a_scale=hs2.fp8_scales(4, 256, device="cpu"), w=w, w_scale=hs2.fp8_scales(300, 256, 128, device="cpu"),
                out=torch.zeros((4, 300)), workspace=torch.zeros(256, dtype=torch.uint8))
    for bad in (dict(a=a.float()), dict(a=a[:, :128]), dict(w=w.t()), dict(a_scale=good["w_scale"]), dict(w_scale=good["a_scale"][:1]),
                dict(out=torch.zeros((4, 299))), dict(out=torch.zeros((4, 300), dtype=torch.float16)), dict(out=torch.zeros((300, 4)).t())):
        with pytest.raises((TypeError, ValueError)):
            hs2.gemm_fp8(**{**good, **bad})


def prefix_call(L, c, start=5, length=100, q=A, scale=0.1, out=A, ot=F32, lse=A, ws=A, wsb=1 << 40):
    return L.hs2_prefix_attn(c.ref(), start, length, q, ctypes.c_float(scale), out, ot, lse, ws, wsb, None)


@pytest.mark.parametrize("change,status,word", [
    (dict(start=-1), 1, b"prefix rows"), (dict(start=909), 1, b"prefix rows"), (dict(length=-1), 1, b"prefix_len"),
    (dict(length=1009), 1, b"prefix_len"), (dict(q=None), 1, b"q / out"), (dict(out=None), 1, b"q / out"), (dict(q=A + 8), 1, b"aligned"),
    (dict(out=A + 4), 1, b"aligned"), (dict(scale=0.0), 1, b"softmax_scale"), (dict(scale=float("inf")), 1, b"softmax_scale"),
    (dict(ot=7), 1, b"out_dtype"), (dict(ws=None), 1, b"workspace"), (dict(ws=A + 16), 1, b"workspace"), (dict(wsb=4096), 3, b"required"),
])
def test_prefix_refusals(L, change, status, word):
    k = torch.zeros((1008, 128), dtype=torch.bfloat16)
    c = hs2.KvCache(k, k, [200, 500], [100, 300], 1, 32)
    got = prefix_call(L, c, **change)
    assert got == status and word in L.hs2_last_error(), (got, L.hs2_last_error())


def test_prefix_workspace_covers_the_plan(L):
    k = torch.zeros((200000, 128), dtype=torch.bfloat16)
    sizes = [hs2.prefix_attn_workspace_size(hs2.KvCache(k, k, [150000], [100], 1, 32), p) for p in (0, 1000, 100000)]
    # the status word; then O and log-sum-exp of 32 rows for each range of at least two
    assert sizes[0] >= 256 and sizes[1] >= 256 + 2 * 32 * 129 * 4 and sizes[1] < sizes[2]
    bad = hs2.KvCache(k, k, [150000], [100], 1, 32)
    bad.view.n_heads = 8
    with pytest.raises(hs2.HS2Error):
        hs2.prefix_attn_workspace_size(bad, 10)
    with pytest.raises(hs2.HS2Error):
        hs2.prefix_attn_workspace_size(hs2.KvCache(k, k, [150000], [100], 1, 32), 200001)


def test_prefix_binding_refuses_wrong_tensors(L):
    k = torch.zeros((1008, 128), dtype=torch.bfloat16)
    c = hs2.KvCache(k, k, [200, 500], [100, 300], 1, 32)
    q, lse = torch.zeros((2, 1, 32, 128), dtype=torch.bfloat16), torch.zeros((2, 1, 32))
    ws = torch.zeros(4096, dtype=torch.uint8)
    for bad in (dict(q=q.float()), dict(q=q[:1]), dict(q=q.transpose(0, 1)), dict(out=q[:, :, :16]), dict(out=q.half()),
                dict(lse=lse.double()), dict(lse=lse[0])):
        args = dict(q=q, out=q.clone(), lse=lse)
        args.update(bad)
        with pytest.raises((TypeError, ValueError)):
            hs2.prefix_attn(c, 5, 100, args["q"], args["out"], args["lse"], ws)
