"""CPU pins of the block-scaled layer's 64-bit definitions and of the C ABI's refusals (no launch is reached)."""
import ctypes

import numpy as np
import pytest
import torch

import linear8_ref as R


def test_decode_is_the_format():
    b = np.arange(256, dtype=np.uint8)
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(R.decode_e4m3(b), want, equal_nan=True)


def test_rounding_is_the_format():
    x = torch.cat([torch.linspace(-448, 448, 40001), torch.randn(20000) * 1e-2, torch.randn(20000) * 30]).clamp(-448, 448)
    assert np.array_equal(R.round_e4m3(x.double().numpy()), x.to(torch.float8_e4m3fn).double().numpy())


@pytest.mark.parametrize("amax,byte", [
    (448.0, 127), (np.nextafter(448.0, 1000), 128), (224.0, 126), (1.75, 119), (1.7500001, 120), (1.0, 119),
    (0.0, 127), (2.0 ** -149, 0), (3.38e38, 247), (np.inf, 255), (np.nan, 255)])
def test_scale_of_a_block(amax, byte):
    x = np.zeros((1, 130))
    x[0, 77] = -amax
    codes, s = R.quantize(x, 1)
    assert s.tolist() == [[byte, 127]]
    assert np.isnan(codes[0, :128]).all() == (byte == 255)


def _lib():
    from token_mixing_feature_b200 import rankmixer as rm
    return rm, rm._lib


P = 1 << 20   # a 16-byte aligned address that nothing touches: every call below ends at its checks


def _norm(rm, **kw):
    d = dict(X=P, Y=P, ld_x=64, ld_y=64, rows=4, D=64, dtype=rm.RM_BF16, eps=1e-5)
    return rm.rm_rmsnorm_args(**{**d, **kw})


@pytest.mark.parametrize("kw,status", [
    (dict(X=None), "INVALID_ARG"), (dict(X=P + 8), "INVALID_ARG"), (dict(Y=None), "INVALID_ARG"),
    (dict(dtype=2), "INVALID_ARG"), (dict(rows=-1), "INVALID_ARG"), (dict(D=0), "INVALID_ARG"),
    (dict(D=72, ld_x=72, ld_y=72), "UNSUPPORTED"), (dict(D=16400, ld_x=16400, ld_y=16400), "UNSUPPORTED"),
    (dict(ld_x=48), "INVALID_ARG"), (dict(ld_x=65), "INVALID_ARG"), (dict(Yq=P, ld_yq=64), "INVALID_ARG"),
    (dict(Yq=P, Ys=P, ld_yq=72, ld_ys=1), "INVALID_ARG"), (dict(Yq=P, Ys=P, ld_yq=64, ld_ys=0), "INVALID_ARG"),
    (dict(R=P, ld_r=8), "INVALID_ARG"), (dict(Sum=P + 2, ld_sum=64), "INVALID_ARG"), (dict(gamma=P + 4), "INVALID_ARG"),
    (dict(eps=-1.0), "INVALID_ARG"), (dict(eps=float("nan")), "INVALID_ARG"), (dict(rows=1 << 31), "UNSUPPORTED"),
    (dict(rows=0), "OK")])
def test_norm_refuses(kw, status):
    rm, lib = _lib()
    assert lib.rm_rmsnorm_forward(ctypes.byref(_norm(rm, **kw)), None) == getattr(rm, "RM_" + (
        "OK" if status == "OK" else "ERR_" + status))
    assert lib.rm_rmsnorm_forward(None, None) == rm.RM_ERR_INVALID_ARG


@pytest.mark.parametrize("kw,status", [
    (dict(dY=None), "INVALID_ARG"), (dict(S=P + 8), "INVALID_ARG"), (dict(dX=None), "INVALID_ARG"),
    (dict(rstd=None), "INVALID_ARG"), (dict(dgamma=P, workspace=None), "INVALID_ARG"),
    (dict(dgamma=P, workspace=P, workspace_bytes=64), "INVALID_ARG"), (dict(ld_dx=56), "INVALID_ARG"),
    (dict(dSum=P, ld_dsum=24), "INVALID_ARG"), (dict(D=24, ld_dy=24, ld_s=24, ld_dx=24), "UNSUPPORTED"),
    (dict(rows=0), "OK")])
def test_norm_grad_refuses(kw, status):
    rm, lib = _lib()
    d = dict(dY=P, S=P, rstd=P, dX=P, ld_dy=64, ld_s=64, ld_dx=64, rows=4, D=64, dtype=rm.RM_F32)
    a = rm.rm_rmsnorm_grad_args(**{**d, **kw})
    assert lib.rm_rmsnorm_backward(ctypes.byref(a), None) == getattr(rm, "RM_" + ("OK" if status == "OK" else "ERR_" + status))


def test_norm_grad_workspace():
    rm, _ = _lib()
    assert rm.rm_rmsnorm_backward_workspace_bytes(0, 64) == 0
    assert rm.rm_rmsnorm_backward_workspace_bytes(5, 72) == 0
    for rows in (1, 7, 4096, 1 << 20):
        for D in (16, 1536, 16384):
            n = rm.rm_rmsnorm_backward_workspace_bytes(rows, D)
            assert 4 * D <= n <= 4 * D * min(rows, 1024)


@pytest.mark.parametrize("kw,status", [
    (dict(src=None), "INVALID_ARG"), (dict(dst=None), "INVALID_ARG"), (dict(scale=None), "INVALID_ARG"),
    (dict(block_rows=64), "INVALID_ARG"), (dict(cols=40), "UNSUPPORTED"), (dict(src_ld=60), "INVALID_ARG"),
    (dict(dst_ld=40), "INVALID_ARG"), (dict(G=2, dst_gstride=0), "INVALID_ARG"), (dict(G=2, scale_gstride=0), "INVALID_ARG"),
    (dict(dst_t=P, scale_t=P, dst_t_ld=9, scale_t_ld=1), "INVALID_ARG"), (dict(dst_t=P), "INVALID_ARG"),
    (dict(dst_t=P, scale_t=P, dst_t_ld=16, scale_t_ld=0), "INVALID_ARG"), (dict(dtype=2), "INVALID_ARG"),
    (dict(G=1 << 20, rows=1 << 20, cols=1 << 10, src_ld=1 << 10, dst_ld=1 << 10, scale_ld=8), "UNSUPPORTED"),
    (dict(rows=0), "OK"), (dict(G=0), "OK")])
def test_quantize_refuses(kw, status):
    rm, lib = _lib()
    d = dict(src=P, src_gstride=640, src_ld=64, dst=P, dst_gstride=640, dst_ld=64, scale=P, scale_gstride=10, scale_ld=1,
             G=1, rows=10, cols=64, block_rows=1, dtype=rm.RM_BF16)
    a = rm.rm_quant_block_args(**{**d, **kw})
    assert lib.rm_quantize_fp8_block(ctypes.byref(a), None) == getattr(rm, "RM_" + ("OK" if status == "OK" else "ERR_" + status))


@pytest.mark.parametrize("kw,status", [
    (dict(A=None), "INVALID_ARG"), (dict(W=P + 8), "INVALID_ARG"), (dict(a_scale=None), "INVALID_ARG"),
    (dict(w_scale=None), "INVALID_ARG"), (dict(out=None), "INVALID_ARG"), (dict(N=40), "UNSUPPORTED"),
    (dict(K=0), "INVALID_ARG"), (dict(N=0), "INVALID_ARG"), (dict(M=-1), "INVALID_ARG"), (dict(a_ld=200), "INVALID_ARG"),
    (dict(a_ld=201), "INVALID_ARG"), (dict(w_ld=199), "INVALID_ARG"), (dict(as_ld=1), "INVALID_ARG"),
    (dict(w_block_rows=1, ws_ld=1), "INVALID_ARG"), (dict(w_block_rows=32), "INVALID_ARG"), (dict(act=4), "INVALID_ARG"),
    (dict(act=-1), "INVALID_ARG"), (dict(o_ld=60), "INVALID_ARG"), (dict(o_ld=66), "INVALID_ARG"),
    (dict(G=2, o_gstride=0), "INVALID_ARG"), (dict(out_dtype=2), "INVALID_ARG"), (dict(out_dtype=3), "INVALID_ARG"),
    (dict(out_dtype=2, out_scale=P, os_ld=1, o_ld=64, resid=P, r_ld=64), "INVALID_ARG"), (dict(bias=P + 4), "INVALID_ARG"),
    (dict(resid=P, r_ld=8), "INVALID_ARG"), (dict(device_status=P + 2), "INVALID_ARG"), (dict(M=0), "OK"), (dict(G=0), "OK")])
def test_matmul_refuses(kw, status):
    rm, lib = _lib()
    d = dict(A=P, a_ld=208, a_scale=P, as_ld=2, W=P, w_ld=208, w_scale=P, ws_ld=2, out=P, o_ld=64, G=1, M=8, N=64, K=200,
             a_gstride=2080, w_gstride=20800, as_gstride=32, ws_gstride=2, o_gstride=640, w_block_rows=128,
             act=rm.RM_ACT_NONE, out_dtype=rm.RM_BF16)
    a = rm.rm_matmul_fp8_args(**{**d, **kw})
    assert lib.rm_matmul_fp8_block(ctypes.byref(a), None) == getattr(rm, "RM_" + ("OK" if status == "OK" else "ERR_" + status))


def test_which_kernel():
    """The ends of the product's launch rule: few rows at any size, large products on the CTA pairs."""
    from linear8_route import few_rows
    rm, _ = _lib()
    assert few_rows(rm, 1, 1, 16, 16, "bf16") and few_rows(rm, 32, 32, 6144, 1536, "e4m3", "tanh")
    assert few_rows(rm, 1, 64, 1024, 16384, "bf16")
    for out in ("bf16", "f32", "e4m3"):
        assert not few_rows(rm, 32, 512, 6144, 1536, out) and not few_rows(rm, 1, 8192, 8192, 8192, out, "erf")
    # up to two 64 x 128 tiles an SM: where the epilogue is long and K is not
    for K in (256, 2048):
        for out, act in (("f32", None), ("bf16", "tanh"), ("bf16", "erf"), ("e4m3", "tanh"), ("e4m3", "relu")):
            assert few_rows(rm, 8, 256, 1024, K, out, act) and not few_rows(rm, 5, 320, 1600, K, out, act)
        for out, act in (("e4m3", None), ("bf16", None), ("bf16", "relu")):
            assert not few_rows(rm, 8, 256, 1024, K, out, act)
    assert not few_rows(rm, 8, 256, 1024, 4096, "f32")


def test_quantize_refuses_widths_next_to_2_to_31():
    """Tiles are counted in ints: the last 255 widths are refused like the last 255 heights."""
    rm, lib = _lib()
    for rows, cols in ((1, 0x7ffffff0), (0x7ffffff0, 16)):
        a = rm.rm_quant_block_args(src=P, src_gstride=1 << 33, src_ld=cols, dst=P, dst_gstride=1 << 33, dst_ld=cols, scale=P,
                                   scale_gstride=1 << 30, scale_ld=1 << 24, G=1, rows=rows, cols=cols, block_rows=1,
                                   dtype=rm.RM_BF16)
        assert lib.rm_quantize_fp8_block(ctypes.byref(a), None) == rm.RM_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw", [dict(scale_t=P, scale_t_ld=1), dict(dst=None, dst_t=P, dst_t_ld=16, scale_t=P, scale_t_ld=1)])
def test_quantize_refuses_scales_alone(kw):
    rm, lib = _lib()
    d = dict(src=P, src_gstride=640, src_ld=64, dst=P, dst_gstride=640, dst_ld=64, scale=P, scale_gstride=10, scale_ld=1,
             G=1, rows=10, cols=64, block_rows=1, dtype=rm.RM_BF16)
    a = rm.rm_quant_block_args(**{**d, **kw})
    assert lib.rm_quantize_fp8_block(ctypes.byref(a), None) == rm.RM_ERR_INVALID_ARG
