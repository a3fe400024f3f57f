"""33 to 64 tokens of the 4-bit product, on both sides of the rule that sends
them to the few-token kernel: rows of more than seven 256-feature stages, or at
least as many channel tiles as SMs; split over a cluster or not, with a 48- or a
64-token tile.  Expected values: 64-bit products of what the stored codes stand
for.  Zero-mean operands: 2^-20 of the magnitude sum, as the other product tests."""
import pytest
import torch

pytestmark = pytest.mark.gpu

dq = pytest.importorskip("quantized_gemm_token_b200") if torch.cuda.is_available() else None


@pytest.fixture(autouse=True)
def _sync_and_check():
    yield
    if torch.cuda.is_available():
        assert dq.dq_sync_status() == dq.DQ_OK


# (N, K): rows around seven stages of 256 features; split 2, 4 or 8 ways; 149 channel tiles (no split) with long and
# with short rows; 148 and 147 tiles (at and below the SM count of a B200)
@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("M", [33, 47, 48, 49, 63, 64])
@pytest.mark.parametrize("N,K", [(136, 1792), (136, 1824), (640, 2080), (4104, 4096), (9480, 2048), (19064, 1824),
                                 (19072, 288), (18944, 800), (18816, 800)])
def test_33_to_64_tokens(M, N, K, fmt):
    g = torch.Generator(device="cuda").manual_seed(M * N + K)
    x = torch.randn((M, K), generator=g, device="cuda").bfloat16()
    w = torch.randn((N, K), generator=g, device="cuda")
    b = torch.randn(N, generator=g, device="cuda").bfloat16()
    A, W = dq.dq_quantize_rows_fp4(x, fmt), dq.dq_quantize_weight_fp4(w, fmt)
    a, v = (dq.dq_fp4_dequantize(t[0], t[1], None, fmt).double() for t in (A, W))
    acc, mag = a @ v.T, a.abs() @ v.abs().T
    buf = torch.full((M + 64, N), 7.0, device="cuda")
    dq.dq_fp4_linear(*A, *W, fmt=fmt, out=buf[:M], out_dtype="f32")
    assert bool(((buf[:M].double() - acc).abs() <= 2.0 ** -20 * mag).all()) and bool((buf[M:] == 7.0).all())
    f = 1.0 if fmt == "mx" else A[2].double()[:, None] * W[2].double()
    y = acc * f + b.double()
    out = torch.full((M + 64, N), 7.0, dtype=torch.bfloat16, device="cuda")
    dq.dq_fp4_linear(*A, *W, b, fmt=fmt, out=out[:M])
    tol = 2.0 ** -20 * mag * f + 2.0 ** -8 * y.abs() + 3 * 2.0 ** -24 * ((acc * f).abs() + y.abs())
    assert bool(((out[:M].double() - y).abs() <= tol).all()) and bool((out[M:] == 7.0).all())
