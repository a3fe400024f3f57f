"""The weight gradient's output type: a given tensor states it, out_dtype need
not repeat it."""
import pytest
import torch

pytestmark = pytest.mark.gpu

dq = pytest.importorskip("quantized_gemm_token_b200") if torch.cuda.is_available() else None


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_the_given_tensor_states_the_type(dtype):
    g = torch.Generator().manual_seed(0)
    x, dy = torch.randn((40, 64), generator=g).bfloat16().cuda(), torch.randn((40, 24), generator=g).bfloat16().cuda()
    kept = dq.Act8.save(x)
    want = kept.weight_grad(dy, out_dtype=dtype)[0]
    out = torch.empty((24, 64), dtype=dtype, device="cuda")
    assert kept.weight_grad(dy, out=out)[0] is out and torch.equal(out, want)
    out.zero_()
    assert dq.dq_act8_weight_grad(dy, kept.codes, kept.scales, out=out)[0] is out and torch.equal(out, want)
    assert kept.weight_grad(dy)[0].dtype == torch.bfloat16              # nothing given: bf16
    if dtype == torch.float32:
        kept.weight_grad(dy, out=out, accumulate=True)
        assert torch.equal(out, want + want)


def test_types_that_disagree_are_refused():
    x, dy = torch.zeros((40, 64), dtype=torch.bfloat16, device="cuda"), torch.zeros((40, 24), dtype=torch.bfloat16, device="cuda")
    kept = dq.Act8.save(x)
    with pytest.raises(TypeError):
        kept.weight_grad(dy, out=torch.empty((24, 64), device="cuda"), out_dtype="bf16")
    with pytest.raises(ValueError):
        kept.weight_grad(dy, out=torch.empty((24, 64), dtype=torch.float16, device="cuda"))
    with pytest.raises(ValueError):
        kept.weight_grad(dy, out=torch.empty((24, 64), dtype=torch.bfloat16, device="cuda"), accumulate=True)
    with pytest.raises(ValueError):
        kept.weight_grad(dy, accumulate=True)
