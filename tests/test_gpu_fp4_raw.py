"""fp32 output of the 4-bit product (the sum itself): operands with a NaN or an
infinity must not come back as finite numbers.  An nv row carries its NaN in
the row scale alone (codes and block scales are 0), an mx block in the block
scale."""
import pytest
import torch

pytestmark = pytest.mark.gpu

dq = pytest.importorskip("quantized_gemm_token_b200") if torch.cuda.is_available() else None


@pytest.fixture(autouse=True)
def _sync_and_check():
    yield
    if torch.cuda.is_available():
        assert dq.dq_sync_status() == dq.DQ_OK


def _operands(M, N, K, fmt):
    g = torch.Generator().manual_seed(M + N)
    x, w = torch.randn((M, K), generator=g).bfloat16(), torch.randn((N, K), generator=g)
    clean = dq.dq_quantize_rows_fp4(x.cuda(), fmt), dq.dq_quantize_weight_fp4(w.cuda(), fmt)
    bad_rows, bad_cols = sorted({0, M // 2, M - 1}), sorted({1, 37, N - 1})
    for i, (r, v) in enumerate(zip(bad_rows, (float("nan"), float("inf"), -float("inf")))):
        x[r, (31 * i) % K] = v
    for i, (c, v) in enumerate(zip(bad_cols, (float("inf"), float("nan"), -float("inf")))):
        w[c, (17 * i + 5) % K] = v
    return clean, (dq.dq_quantize_rows_fp4(x.cuda(), fmt), dq.dq_quantize_weight_fp4(w.cuda(), fmt)), bad_rows, bad_cols


# few tokens (with and without a split of the features), many tokens (whole and narrow tiles, ragged both ways)
@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("M,N,K", [(1, 72, 64), (17, 136, 4096), (64, 264, 2080), (130, 200, 288), (700, 1096, 544)])
def test_non_finite_operands_are_nan_in_the_raw_sum(M, N, K, fmt):
    (A, W), (Ab, Wb), rows, cols = _operands(M, N, K, fmt)
    want = dq.dq_fp4_linear(*A, *W, fmt=fmt, out_dtype="f32")
    assert not bool(torch.isnan(want).any())
    for a, w, rr, cc in ((Ab, W, rows, []), (A, Wb, [], cols), (Ab, Wb, rows, cols)):
        nan = torch.zeros((M, N), dtype=torch.bool, device="cuda")
        nan[rr] = True
        nan[:, cc] = True
        got = dq.dq_fp4_linear(*a, *w, fmt=fmt, out_dtype="f32")
        assert torch.equal(torch.isnan(got), nan)
        assert torch.equal(got[~nan], want[~nan])
        # the scaled output agrees on what is NaN
        assert torch.equal(torch.isnan(dq.dq_fp4_linear(*a, *w, fmt=fmt)), nan)


@pytest.mark.parametrize("M", [5, 300])
def test_finite_row_scales_leave_the_raw_sum_alone(M):
    (A, W), _, _, _ = _operands(M, 136, 288, "nv")
    with_scales = dq.dq_fp4_linear(*A, *W, out_dtype="f32")
    assert torch.equal(dq.dq_fp4_linear(A[0], A[1], None, W[0], W[1], None, out_dtype="f32"), with_scales)
    assert torch.equal(dq.dq_fp4_linear(A[0], A[1], A[2], W[0], W[1], None, out_dtype="f32"), with_scales)
    assert torch.equal(dq.dq_fp4_linear(A[0], A[1], None, W[0], W[1], W[2], out_dtype="f32"), with_scales)
