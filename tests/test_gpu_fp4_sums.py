"""How much of a sum the tensor core's accumulator loses, at its worst: operands
of one sign and long rows.

Every product is exact.  The accumulator (fp32, 24 bits) takes one MMA's
products, 64 features, per addition and truncates, so an MMA loses less than
one place, 2^-23 of the sum so far.  A row (or its share, where the few-token
kernel splits it over up to 8 CTAs) is one chain of MMAs.  With operands of one
sign the sums so far are known exactly, and the bound is
    2^-23 sum over the MMAs of (the sum so far) + 8 2^-24 sum
(the second term: the shares' additions), about 2^-24 K / 64 of the sum.  A
split only shortens the chain.  Whatever the signs, no sum so far exceeds the
magnitude sum: |error| <= (ceil(K / 64) 2^-23 + 8 2^-24) sum |a w|.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

dq = pytest.importorskip("quantized_gemm_token_b200") if torch.cuda.is_available() else None


@pytest.fixture(autouse=True)
def _sync_and_check():
    yield
    if torch.cuda.is_available():
        assert dq.dq_sync_status() == dq.DQ_OK


def _bound(a, w):
    """(exact sum, bound) of the product of positive operands in 64 bits."""
    so_far = torch.zeros((a.shape[0], w.shape[0]), dtype=torch.float64, device=a.device)
    lost = torch.zeros_like(so_far)
    for k in range(0, a.shape[1], 64):
        so_far += a[:, k:k + 64] @ w[:, k:k + 64].T
        lost += so_far
    return so_far, 2.0 ** -23 * lost + 8 * 2.0 ** -24 * so_far


def _positive(R, K, seed, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.rand((R, K), generator=g, device="cuda") + 0.05).to(dtype)


def _values(q, fmt):
    # codes times block scales have at most six significant bits: exact in bf16
    return dq.dq_fp4_dequantize(q[0], q[1], None, fmt).double()


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("K", [4096, 8192, 8224, 16384, 28672, 65536, 262144])
@pytest.mark.parametrize("M,N", [(16, 136), (64, 128), (300, 264)])
def test_one_signed_rows(M, N, K, fmt):
    A, W = dq.dq_quantize_rows_fp4(_positive(M, K, K, torch.bfloat16), fmt), dq.dq_quantize_weight_fp4(
        _positive(N, K, K + 1, torch.float32), fmt)
    want, tol = _bound(_values(A, fmt), _values(W, fmt))
    got = dq.dq_fp4_linear(*A, *W, fmt=fmt, out_dtype="f32").double()
    err = (got - want).abs()
    assert bool((err <= tol).all()), f"{float((err / tol).max()):.3g} of the bound, {float((err / want).max()):.3g} of the sum"


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("M,K", [(1, 65536), (64, 16416), (33, 28672)])
def test_one_signed_rows_that_are_not_split(M, K, fmt):
    """More channel tiles than SMs: the few-token kernel sums a whole row in one
    CTA.  128 weight rows, repeated."""
    reps = 149
    A = dq.dq_quantize_rows_fp4(_positive(M, K, K, torch.bfloat16), fmt)
    W = dq.dq_quantize_weight_fp4(_positive(128, K, K + 1, torch.float32), fmt)
    want, tol = _bound(_values(A, fmt), _values(W, fmt))
    wide = W[0].repeat(reps, 1), W[1].repeat(reps, 1, 1), None if W[2] is None else W[2].repeat(reps)
    got = dq.dq_fp4_linear(*A, *wide, fmt=fmt, out_dtype="f32").view(M, reps, 128)
    assert torch.equal(got, got[:, :1].expand_as(got))
    err = (got[:, 0].double() - want).abs()
    assert bool((err <= tol).all()), f"{float((err / tol).max()):.3g} of the bound, {float((err / want).max()):.3g} of the sum"


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("M,N,K", [(7, 72, 20000), (40, 19080, 8480), (64, 136, 66080), (300, 200, 16640), (1799, 1288, 8224),
                                   (257, 4104, 24608)])
def test_long_rows_of_both_signs(M, N, K, fmt):
    """Rows of 8224 features and more, ragged every way, with bias and scales."""
    g = torch.Generator(device="cuda").manual_seed(K)
    x = torch.randn((M, K), generator=g, device="cuda").bfloat16()
    w = torch.randn((N, K), generator=g, device="cuda")
    b = torch.randn(N, generator=g, device="cuda").bfloat16()
    A, W = dq.dq_quantize_rows_fp4(x, fmt), dq.dq_quantize_weight_fp4(w, fmt)
    a, v = _values(A, fmt), _values(W, fmt)
    acc, mag = a @ v.T, a.abs() @ v.abs().T
    # zero-mean operands: the sum so far stays below 8 sqrt(k) of a term's size (about 1.6 times the terms' mean
    # magnitude), so the MMAs lose less than 2^-23 8 1.6 (2 / 3) sqrt(K) K / 64 of a mean term, 2^-25.9 sqrt(K) of the
    # magnitude sum
    rel = 2.0 ** -25.9 * K ** 0.5 + 8 * 2.0 ** -24
    got = dq.dq_fp4_linear(*A, *W, fmt=fmt, out_dtype="f32")
    assert bool(((got.double() - acc).abs() <= rel * mag).all())
    f = 1.0 if fmt == "mx" else A[2].double()[:, None] * W[2].double()
    y = acc * f + b.double()
    got = dq.dq_fp4_linear(*A, *W, b, fmt=fmt).double()
    tol = rel * mag * f + 2.0 ** -8 * y.abs() + 3 * 2.0 ** -24 * ((acc * f).abs() + y.abs())
    assert bool(((got - y).abs() <= tol).all())
