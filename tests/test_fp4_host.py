"""Host checks of the microscaled entry points: what they refuse, before any
device is touched (no GPU needed), and the sizes they state."""
import ctypes

import pytest
import torch

INVALID, UNSUPPORTED = 1, 2
P, I = ctypes.c_void_p, ctypes.c_int64
A16 = P(0x10000)          # aligned fakes, never dereferenced: validation fails first
OFF8, OFF2, OFF1 = P(0x10008), P(0x10002), P(0x10001)


@pytest.fixture(scope="module")
def lib():
    from quantized_gemm_token_b200 import build
    import quantized_gemm_token_b200 as dq
    build.build()
    return dq._load()


def _quant(lib, fn, M=4, K=64, ld=64, fmt=1, x=A16, q=A16, ldq=32, sf=A16, s=A16):
    return getattr(lib, fn)(x, M, K, ld, fmt, q, ldq, sf, s, None)


@pytest.mark.parametrize("fn", ["dq_quantize_rows_fp4", "dq_quantize_weight_fp4"])
@pytest.mark.parametrize("bad,status", [
    (dict(fmt=2), INVALID), (dict(fmt=-1), INVALID), (dict(M=-1), INVALID), (dict(K=0), INVALID), (dict(ld=63), INVALID),
    (dict(ldq=31), INVALID), (dict(x=None), INVALID), (dict(q=None), INVALID), (dict(sf=None), INVALID),
    (dict(s=None), INVALID), (dict(K=48, ldq=24), UNSUPPORTED), (dict(K=16, ldq=8), UNSUPPORTED),
    (dict(M=(1 << 30) + 1), UNSUPPORTED), (dict(sf=OFF8), UNSUPPORTED), (dict(s=OFF2), UNSUPPORTED),
    (dict(x=OFF1), UNSUPPORTED)])
def test_quantize_refusals(lib, fn, bad, status):
    assert _quant(lib, fn, **bad) == status


def test_mx_needs_no_row_scales(lib):
    # accepted as far as the device check: not an argument error
    assert _quant(lib, "dq_quantize_rows_fp4", fmt=0, s=None) != INVALID


def _linear(lib, A=A16, sfa=A16, sr=A16, M=4, K=64, W=A16, sfw=A16, sc=A16, N=16, fmt=1, b=None, out=A16, dt=0):
    return lib.dq_fp4_linear(A, sfa, sr, M, K, W, sfw, sc, N, fmt, b, out, dt, None)


@pytest.mark.parametrize("bad,status", [
    (dict(fmt=7), INVALID), (dict(M=-1), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(dt=1), INVALID),
    (dict(dt=9), INVALID), (dict(A=None), INVALID), (dict(sfa=None), INVALID), (dict(W=None), INVALID),
    (dict(sfw=None), INVALID), (dict(out=None), INVALID), (dict(K=80), UNSUPPORTED), (dict(N=12), UNSUPPORTED),
    (dict(N=(1 << 30) + 8), UNSUPPORTED), (dict(A=OFF8), UNSUPPORTED), (dict(sfa=OFF8), UNSUPPORTED),
    (dict(W=OFF8), UNSUPPORTED), (dict(sfw=OFF8), UNSUPPORTED), (dict(out=OFF8), UNSUPPORTED),
    (dict(sc=OFF8), UNSUPPORTED), (dict(sr=OFF2), UNSUPPORTED), (dict(b=OFF8), UNSUPPORTED)])
def test_linear_refusals(lib, bad, status):
    assert _linear(lib, **bad) == status


@pytest.mark.parametrize("args,status", [
    ((A16, A16, None, 4, 64, 5, A16), INVALID), ((A16, A16, None, -1, 64, 1, A16), INVALID),
    ((None, A16, None, 4, 64, 1, A16), INVALID), ((A16, None, None, 4, 64, 1, A16), INVALID),
    ((A16, A16, None, 4, 64, 1, None), INVALID), ((A16, A16, None, 4, 40, 1, A16), UNSUPPORTED),
    ((OFF8, A16, None, 4, 64, 1, A16), UNSUPPORTED), ((A16, A16, OFF2, 4, 64, 1, A16), UNSUPPORTED),
    ((A16, A16, None, 4, 64, 1, OFF8), UNSUPPORTED)])
def test_dequantize_refusals(lib, args, status):
    assert lib.dq_fp4_dequantize(*args, None) == status


@pytest.mark.parametrize("args,status", [
    ((A16, 4, 64, 3, A16), INVALID), ((A16, -1, 64, 1, A16), INVALID), ((None, 4, 64, 1, A16), INVALID),
    ((A16, 4, 64, 1, None), INVALID), ((A16, 4, 72, 1, A16), UNSUPPORTED), ((A16, 4, 64, 1, OFF8), UNSUPPORTED)])
def test_tile_scales_refusals(lib, args, status):
    assert lib.dq_fp4_tile_scales(*args, None) == status


@pytest.mark.parametrize("args,status", [
    ((A16, -1, 64, 64, A16, A16), INVALID), ((A16, 4, 0, 64, A16, A16), INVALID), ((A16, 4, 64, 63, A16, A16), INVALID),
    ((None, 4, 64, 64, A16, A16), INVALID), ((A16, 4, 64, 64, None, A16), INVALID), ((A16, 4, 64, 64, A16, None), INVALID),
    ((A16, 4, 40, 40, A16, A16), UNSUPPORTED), ((OFF1, 4, 64, 64, A16, A16), UNSUPPORTED),
    ((A16, 4, 64, 64, OFF8, A16), UNSUPPORTED), ((A16, 4, 64, 64, A16, OFF8), UNSUPPORTED)])
def test_act8_pack_refusals(lib, args, status):
    assert lib.dq_act8_pack(*args, None) == status


@pytest.mark.parametrize("args,status", [
    ((A16, A16, -1, 64, A16), INVALID), ((None, A16, 4, 64, A16), INVALID), ((A16, A16, 4, 64, None), INVALID),
    ((A16, A16, 4, 24, A16), UNSUPPORTED), ((A16, A16, 4, 64, OFF8), UNSUPPORTED)])
def test_act8_unpack_refusals(lib, args, status):
    assert lib.dq_act8_unpack(*args, None) == status


def _grad(lib, dy=A16, M=4, N=16, ld=16, codes=A16, scales=A16, K=32, dw=A16, dt=0, acc=0, db=None):
    return lib.dq_act8_weight_grad(dy, M, N, ld, codes, scales, K, dw, dt, acc, db, None)


@pytest.mark.parametrize("bad,status", [
    (dict(M=-1), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(ld=15), INVALID), (dict(dt=1), INVALID),
    (dict(dw=None), INVALID), (dict(dy=None), INVALID), (dict(codes=None), INVALID), (dict(scales=None), INVALID),
    (dict(acc=1), INVALID), (dict(K=24), UNSUPPORTED), (dict(N=12), UNSUPPORTED), (dict(ld=20), UNSUPPORTED),
    (dict(dy=OFF8), UNSUPPORTED), (dict(codes=OFF8), UNSUPPORTED), (dict(scales=OFF8), UNSUPPORTED),
    (dict(dw=OFF8), UNSUPPORTED), (dict(db=OFF8), UNSUPPORTED), (dict(M=(1 << 30) + 1), UNSUPPORTED)])
def test_weight_grad_refusals(lib, bad, status):
    assert _grad(lib, **bad) == status


def test_sizes(lib):
    assert lib.dq_fp4_scales_size(1, 64, 1) == 512 and lib.dq_fp4_scales_size(129, 96, 1) == 2 * 2 * 512
    assert lib.dq_fp4_scales_size(128, 128, 0) == 512 and lib.dq_fp4_scales_size(128, 160, 0) == 1024
    assert lib.dq_fp4_scales_size(0, 64, 1) == 0 and lib.dq_fp4_scales_size(4, 40, 1) == 0
    assert lib.dq_fp4_scales_size(4, 64, 2) == 0 and lib.dq_fp4_scales_size(-1, 64, 1) == 0
    assert lib.dq_act8_codes_size(33, 16) == 64 * 16 and lib.dq_act8_scales_size(33, 16) == 32
    assert lib.dq_act8_codes_size(0, 16) == 0 and lib.dq_act8_codes_size(-1, 16) == 0


def test_host_tensors_are_refused(lib):
    import quantized_gemm_token_b200 as dq
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    u8 = torch.zeros((4, 32), dtype=torch.uint8)
    sf = torch.zeros((1, 1, 512), dtype=torch.uint8)
    calls = [lambda: dq.dq_quantize_rows_fp4(x), lambda: dq.dq_quantize_weight_fp4(x.float()),
             lambda: dq.dq_fp4_dequantize(u8, sf), lambda: dq.dq_fp4_linear(u8, sf, None, u8, sf, None),
             lambda: dq.dq_fp4_tile_scales(u8), lambda: dq.dq_act8_pack(x), lambda: dq.Act8.save(x),
             lambda: dq.dq_act8_unpack(torch.zeros((2, 16, 16), dtype=torch.int8), u8[:1, :16], 4),
             lambda: dq.dq_act8_weight_grad(x, torch.zeros((2, 16, 16), dtype=torch.int8), u8[:1, :16])]
    for c in calls:
        with pytest.raises(TypeError):
            c()
    with pytest.raises(ValueError):
        dq.dq_quantize_rows_fp4(x, fmt="int4")


def test_plain_forms_agree():
    """The 64-bit forms the GPU tests use, against hand-worked values."""
    import numpy as np
    import mx_ref as ref
    # e2m1 ties go to the even code; 5 is halfway between 4 and 6
    v = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.01, 7.0, 100.0])
    assert ref.nearest(v, ref.E2M1).tolist() == [0, 2, 2, 4, 4, 6, 6, 7, 7, 7]
    # e4m3: 448 the largest, 2^-9 the least, 17 halfway between 16 and 18
    assert ref.E4M3[126] == 448.0 and ref.E4M3[1] == 2.0 ** -9 and ref.E4M3[ref.nearest(np.array([17.0]), ref.E4M3)[0]] == 16.0
    # mx: largest 7 -> scale 2^(2 - 2) = 1, 7 saturates at 6
    x = np.zeros((1, 32))
    x[0, :4] = [7.0, -2.5, 0.3, 1.0]
    c, E, s = ref.quantize_fp4(x, "mx")
    assert E[0, 0] == 127 and c[0, :4].tolist() == [7, 12, 1, 2] and s is None
    # nv: row maximum 2688 = 6 * 448 exactly: s = 1, the block scale 448
    x = np.zeros((1, 32))
    x[0, 0], x[0, 16] = 2688.0, 3.0
    c, E, s = ref.quantize_fp4(x, "nv")
    assert s[0] == 1.0 and ref.E4M3[E[0, 0]] == 448.0 and ref.E4M3[E[0, 1]] == 0.5 and c[0, 0] == 7 and c[0, 16] == 7
    # just above it the row scale doubles
    assert ref.quantize_fp4(x * (1 + 2.0 ** -7), "nv")[2][0] == 2.0
    # 8-bit: largest 1.5 -> scale 1, code 96; 255 / 128 would round to 128 and is kept at 127
    q, E = ref.act8(np.array([[1.5], [-0.25], [0.0]]))
    assert E[0, 0] == 127 and q[:, 0].tolist() == [96, -16, 0]
    assert ref.act8(np.array([[255 / 128]]))[0][0, 0] == 127
