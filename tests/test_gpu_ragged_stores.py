"""Output blocks past the last column are not stored and must not disturb the
ones still being stored: short tiles follow one another at once, the last tile
of every row block is ragged, and every call runs on cold caches.  The bf16
output of each GEMM is compared bit for bit with the epilogue's definition
applied to the accumulators that the same GEMM returns."""
import pytest
import torch

pytestmark = pytest.mark.gpu

dq = pytest.importorskip("quantized_gemm_token_b200") if torch.cuda.is_available() else None


@pytest.fixture(autouse=True)
def _sync_and_check():
    yield
    if torch.cuda.is_available():
        assert dq.dq_sync_status() == dq.DQ_OK


@pytest.fixture(scope="module")
def flush():
    return torch.empty(1 << 28, dtype=torch.uint8, device="cuda")


def _operands(M, N, K, seed, quantize_rows, quantize_weight):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((M, K), generator=g, device="cuda").bfloat16()
    w = torch.randn((N, K), generator=g, device="cuda")
    return quantize_rows(x), quantize_weight(w)


@pytest.mark.parametrize("M,N,K", [(20000, 4104, 32), (5000, 4136, 32), (5000, 4168, 256), (5000, 4104, 2048),
                                   (5000, 4200, 2048)])
def test_int8_ragged_last_tiles(M, N, K, flush):
    (q, s), (wq, sw) = _operands(M, N, K, N + K, dq.dq_quantize_rows, dq.dq_quantize_weight)
    acc = dq.dq_int8_linear(q, s, wq, sw, out_dtype="s32")
    want = ((acc.float() * s[:, None]) * sw).bfloat16()
    for _ in range(10):
        flush.fill_(1)
        assert torch.equal(dq.dq_int8_linear(q, s, wq, sw), want)


@pytest.mark.parametrize("M,N,K", [(20000, 4104, 32), (5000, 4136, 32), (5000, 4104, 2048)])
def test_fp8_ragged_last_tiles(M, N, K, flush):
    (q, s), (wq, sw) = _operands(M, N, K, N + K, dq.dq_quantize_rows_fp8, dq.dq_quantize_weight_fp8)
    acc = dq.dq_fp8_linear(q, s, wq, sw, out_dtype="f32")
    want = ((acc * s[:, None]) * sw).bfloat16()
    for _ in range(10):
        flush.fill_(1)
        assert torch.equal(dq.dq_fp8_linear(q, s, wq, sw), want)
