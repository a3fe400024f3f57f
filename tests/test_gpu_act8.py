"""8-bit activation checkpoints against plain 64-bit forms (tests/mx_ref.py)."""
import numpy as np
import pytest
import torch

import mx_ref as ref

pytestmark = pytest.mark.gpu

dq = pytest.importorskip("quantized_gemm_token_b200") if torch.cuda.is_available() else None


@pytest.fixture(autouse=True)
def _sync_and_check():
    yield
    if torch.cuda.is_available():
        assert dq.dq_sync_status() == dq.DQ_OK


def _x(M, K, seed, kind="normal"):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((M, K), generator=g)
    if kind == "outliers":
        x[:, torch.rand(K, generator=g) < 0.03] *= 20
    elif kind == "wide":
        x *= torch.exp2(torch.randint(-126, 120, (M, K), generator=g).float())
    elif kind == "edges":
        x[:, 0] = 0
        x[:, 1] = torch.sign(x[:, 1]) * 2.0 ** -133
        x[:, 2] = 255.0 * 2.0 ** 120                 # the largest finite mantissa: 127.5 steps
        x[:, 3] *= 2.0 ** -130
        x[:, 4] = -0.0
    return x.bfloat16()


def _check(x, codes, scales):
    q, E = ref.act8(x.double().numpy())
    assert np.array_equal(scales.cpu().numpy(), E)
    assert np.array_equal(codes.cpu().numpy(), ref.act8_layout(q))
    return ref.act8_values(q, E)


@pytest.mark.parametrize("kind", ["normal", "outliers", "wide", "edges"])
@pytest.mark.parametrize("M,K", [(1, 16), (15, 32), (31, 48), (32, 512), (33, 528), (100, 1280), (777, 1040), (2080, 16)])
def test_pack_and_unpack_bit_exact(M, K, kind):
    x = _x(M, K, M + K, kind)
    codes, scales = dq.dq_act8_pack(x.cuda())
    v = _check(x, codes, scales)
    out = dq.dq_act8_unpack(codes, scales, M)
    assert tuple(out.shape) == (M, K)
    assert np.array_equal(out.cpu().double().numpy(), v)
    # off by half a step of the block's scale at most
    step = np.repeat(2.0 ** (scales.cpu().numpy().astype(np.float64) - 133), 32, axis=0)[:M]
    assert (np.abs(v - x.double().numpy()) <= step / 2).all()


@pytest.mark.parametrize("M,K", [(75, 272), (3, 16)])
def test_pack_into_codes_aligned_to_16_bytes_only(M, K):
    g = 2 * -(-M // 32)
    x = _x(M, K, 6)
    buf = torch.full((g * K * 16 + 48,), 77, dtype=torch.int8, device="cuda")
    codes = buf[16:16 + g * K * 16].view(g, K, 16)
    assert codes.data_ptr() % 32 == 16
    _, scales = dq.dq_act8_pack(x.cuda(), codes=codes)
    _check(x, codes, scales)
    assert bool((buf[:16] == 77).all()) and bool((buf[16 + g * K * 16:] == 77).all())


@pytest.mark.parametrize("offset,pad", [(0, 8), (0, 1), (1, 0), (2, 2), (4, 4)])
def test_pack_strides_and_offsets(offset, pad):
    M, K = 75, 272
    x = _x(M, K + offset + pad, 3).cuda()[:, offset:offset + K]
    _check(x.cpu(), *dq.dq_act8_pack(x))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_non_finite_blocks_read_back_as_nan(bad):
    x = _x(100, 64, 3)
    x[40, 5] = bad
    x[99, 63] = bad
    codes, scales = dq.dq_act8_pack(x.cuda())
    _check(x, codes, scales)
    nan = torch.isnan(dq.dq_act8_unpack(codes, scales, 100)).cpu()
    want = torch.zeros_like(nan)
    want[32:64, 5] = True
    want[96:, 63] = True
    assert torch.equal(nan, want)


def test_rows_behind_the_last_token_stay():
    x = _x(41, 64, 5).cuda()
    codes, scales = dq.dq_act8_pack(x)
    buf = torch.full((64, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    dq.dq_act8_unpack(codes, scales, 41, out=buf[:41])
    assert bool((buf[41:] == 3.0).all())


def test_no_tokens():
    codes, scales = dq.dq_act8_pack(torch.empty((0, 32), dtype=torch.bfloat16, device="cuda"))
    assert tuple(dq.dq_act8_unpack(codes, scales, 0).shape) == (0, 32)
