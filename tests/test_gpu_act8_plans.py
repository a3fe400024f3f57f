"""The weight gradient's launch plans: whole waves of tiles with the remaining
ones split in a launch of their own, tiles of 256 channels split over two or
four pairs, and gradients added to by a split; and what its sums lose.

dW: a chain of at most 128 MMAs of 16 tokens truncates less than 2^-23 of its
sum so far per MMA; chains (and split parts) are added in fp32.  With zero-mean
operands a chain's sum so far stays below 2^-4 of the whole magnitude sum, which
gives 2^-20 of it.  db: an unsplit tile of 256 channels sums each channel in 16
parts (8 warps x 2 token slots), so the longest chain is M / 16 additions:
(M / 16 + 48) 2^-24 sum |dy|.
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


def _case(M, N, K, seed, positive=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x, dy = torch.randn((M, K), generator=g, device="cuda"), torch.randn((M, N), generator=g, device="cuda") * 0.1
    if positive:
        x, dy = x.abs(), dy.abs()
    dy = dy.bfloat16()
    codes, scales = dq.dq_act8_pack(x.bfloat16())
    return dy, codes, scales, dq.dq_act8_unpack(codes, scales, M).double()


def _check(dw, db, dy, x, base=0.0, dbase=0.0):
    d = dy.double()
    want = d.T @ x + base
    tol = 2.0 ** -20 * (d.abs().T @ x.abs()) + 2.0 ** -24 * want.abs()
    if dw.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * want.abs()
    err = (dw.double() - want).abs()
    assert bool((err <= tol).all()), f"{float((err / tol).max()):.3g} of the bound"
    if db is not None:
        want = d.sum(0) + dbase
        tol = (dy.shape[0] / 16 + 48) * 2.0 ** -24 * d.abs().sum(0) + 2.0 ** -24 * want.abs()
        assert bool(((db.double() - want).abs() <= tol).all())


# On 74 pairs: 100 tiles of 256 x 256 (74 whole, 26 split two ways in a second launch), 115 (whole tiles, two waves,
# ragged edges), 78 (74 whole, 4 split four ways in a second launch), 30 (two ways at once), 12 (four ways at once); 32
# tiles of 128 channels (two ways), 6 (four ways)
PLANS = [(12000, 5120, 1280), (12001, 5864, 1040), (16400, 6648, 752), (8192, 1280, 1536), (8192, 768, 1024),
         (4160, 1000, 784), (2048, 384, 512)]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", PLANS)
def test_plans(M, N, K, out):
    dy, codes, scales, x = _case(M, N, K, M + N)
    dw, db = dq.dq_act8_weight_grad(dy, codes, scales, out_dtype=out, bias_grad=True)
    _check(dw, db, dy, x)
    again, dbn = dq.dq_act8_weight_grad(dy, codes, scales, out_dtype=out, bias_grad=True)
    assert torch.equal(again, dw) and torch.equal(dbn, db)
    _check(dq.dq_act8_weight_grad(dy, codes, scales, out_dtype=out)[0], None, dy, x)


@pytest.mark.parametrize("with_db", [True, False])
@pytest.mark.parametrize("M,N,K", PLANS)
def test_plans_that_add_to_gradients(M, N, K, with_db):
    dy, codes, scales, x = _case(M, N, K, M + K)
    g = torch.Generator(device="cuda").manual_seed(1)
    base, dbase = torch.randn((N, K), generator=g, device="cuda"), torch.randn(N, generator=g, device="cuda")
    # the rows and numbers behind the gradients stay as they are
    dw, db = torch.full((N + 8, K), 7.0, device="cuda"), torch.full((N + 8,), 7.0, device="cuda")
    dw[:N], db[:N] = base, dbase
    dq.dq_act8_weight_grad(dy, codes, scales, out=dw[:N], out_dtype="f32", accumulate=True, bias_grad=db[:N] if with_db else False)
    if with_db:
        _check(dw[:N], db[:N], dy, x, base.double(), dbase.double())
    else:
        _check(dw[:N], None, dy, x, base.double())
        assert torch.equal(db[:N], dbase)
    assert bool((dw[N:] == 7.0).all()) and bool((db[N:] == 7.0).all())


@pytest.mark.parametrize("M,N,K", [(16, 72, 144), (1024, 264, 256), (2048, 512, 512), (8192, 512, 512), (65792, 256, 256)])
def test_one_signed_sums(M, N, K):
    """The worst case of a truncating accumulator: all products positive.  The
    bound follows the exact sums so far, chain by chain (splits only shorten
    chains; joins: the chains and four parts)."""
    dy, codes, scales, x = _case(M, N, K, M, positive=True)
    d = dy.double()
    total = torch.zeros((N, K), dtype=torch.float64, device="cuda")
    chain, lost = torch.zeros_like(total), torch.zeros_like(total)
    n = -(-M // 16)
    for i in range(n):
        if i % 128 == 0:
            chain.zero_()
        part = d[16 * i:16 * i + 16].T @ x[16 * i:16 * i + 16]
        chain += part
        total += part
        lost += chain
    tol = 2.0 ** -23 * lost + 2.0 ** -24 * (-(-n // 128) + 4) * total
    dw, db = dq.dq_act8_weight_grad(dy, codes, scales, out_dtype="f32", bias_grad=True)
    err = (dw.double() - total).abs()
    assert bool((err <= tol).all()), f"{float((err / tol).max()):.3g} of the bound, {float((err / total).max()):.3g} of the sum"
    assert bool(((db.double() - d.sum(0)).abs() <= (M / 16 + 48) * 2.0 ** -24 * d.sum(0)).all())
