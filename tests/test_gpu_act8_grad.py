"""Weight and bias gradients from an 8-bit checkpoint against plain 64-bit sums.

Both factors are exact bf16 numbers, so every product is exact in fp32; the
fp32 sum is the tensor core's: |dW - exact| <= ACC_REL * sum_m |dy x| (as for
the other tensor-core fp32 sums here); a bf16 output adds half a bf16 step.
db is a chain of at most M fp32 additions split over 32 to 256 partial sums:
bounded by (M / 32 + 48) 2^-24 sum_m |dy|.
"""
import numpy as np
import pytest
import torch

import mx_ref as ref

pytestmark = pytest.mark.gpu

dq = pytest.importorskip("quantized_gemm_token_b200") if torch.cuda.is_available() else None

ACC_REL = 2.0 ** -20


@pytest.fixture(autouse=True)
def _sync_and_check():
    yield
    if torch.cuda.is_available():
        assert dq.dq_sync_status() == dq.DQ_OK


def _case(M, N, K, seed, pad=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((M, K), generator=g)
    x[:, torch.rand(K, generator=g) < 0.05] *= 20
    x = x.bfloat16()
    dy = (torch.randn((M, N + pad), generator=g) * 0.1).bfloat16().cuda()[:, :N]
    codes, scales = dq.dq_act8_pack(x.cuda())
    q, E = ref.act8(x.double().numpy())
    return dy, codes, scales, torch.from_numpy(ref.act8_values(q, E)).cuda()


def _check(dw, db, dy, x, base=None, dbase=None):
    d = dy.double()
    want = d.T @ x
    mag = d.abs().T @ x.abs()
    tol = ACC_REL * mag
    if base is not None:
        want = want + base
        tol = tol + 2.0 ** -24 * want.abs()
    if dw.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * want.abs()
    err = (dw.double() - want).abs()
    assert bool((err <= tol).all()), f"worst {float((err / tol.clamp_min(1e-300)).max()):.3g} of the bound"
    if db is not None:
        s = d.sum(0)
        t = (dy.shape[0] / 32 + 48) * 2.0 ** -24 * d.abs().sum(0)
        if dbase is not None:
            s = s + dbase
            t = t + 2.0 ** -24 * s.abs()
        assert bool(((db.double() - s).abs() <= t).all())


SHAPES = [(1, 8, 16), (7, 64, 128), (33, 72, 144), (64, 200, 48), (65, 192, 272), (200, 136, 1296), (1001, 264, 400),
          (640, 1000, 256), (2048, 384, 512), (4100, 64, 64), (257, 2056, 2064)]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_weight_and_bias_gradients(M, N, K, out):
    dy, codes, scales, x = _case(M, N, K, M + N + K)
    dw, db = dq.dq_act8_weight_grad(dy, codes, scales, out_dtype=out, bias_grad=True)
    assert dw.dtype == (torch.bfloat16 if out == "bf16" else torch.float32) and tuple(dw.shape) == (N, K)
    _check(dw, db, dy, x)
    again, none = dq.dq_act8_weight_grad(dy, codes, scales, out_dtype=out)
    assert none is None and torch.equal(again, dw)


@pytest.mark.parametrize("M,N,K", [(33, 72, 144), (300, 1000, 272), (2048, 2056, 2048)])
def test_accumulate(M, N, K):
    dy, codes, scales, x = _case(M, N, K, 5)
    g = torch.Generator().manual_seed(1)
    base, dbase = torch.randn((N, K), generator=g).cuda(), torch.randn((N,), generator=g).cuda()
    dw, db = base.clone(), dbase.clone()
    dq.dq_act8_weight_grad(dy, codes, scales, out=dw, out_dtype="f32", accumulate=True, bias_grad=db)
    _check(dw, db, dy, x, base.double(), dbase.double())


@pytest.mark.parametrize("pad", [8, 64, 72])
def test_strided_output_gradient(pad):
    dy, codes, scales, x = _case(130, 328, 160, pad, pad)
    _check(*dq.dq_act8_weight_grad(dy, codes, scales, out_dtype="f32", bias_grad=True), dy, x)


def test_each_token_alone():
    """A one-hot output gradient reads the checkpoint back, bit for bit."""
    M, N, K = 100, 104, 336
    _, codes, scales, x = _case(M, N, K, 8)
    dy = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    dy[torch.arange(M), torch.arange(M)] = 1
    dw, _ = dq.dq_act8_weight_grad(dy, codes, scales, out_dtype="f32")
    assert torch.equal(dw[:M].double(), x)
    assert bool((dw[M:] == 0).all())


def test_many_tokens_full_grid():
    dy, codes, scales, x = _case(6000, 1536, 2560, 2)
    _check(*dq.dq_act8_weight_grad(dy, codes, scales, out_dtype="f32", bias_grad=True), dy, x)


@pytest.mark.parametrize("out,accumulate", [("bf16", False), ("f32", False), ("f32", True)])
@pytest.mark.parametrize("M,N,K", [(130, 2312, 2064), (2048, 2560, 2048), (1601, 2184, 2320)])
def test_more_tiles_than_one_wave(M, N, K, out, accumulate):
    """81 to 90 tiles of 256 x 256: the ones past the first wave are halved (with
    a half that lies outside the matrix, and ragged ones) or split."""
    dy, codes, scales, x = _case(M, N, K, 4)
    if accumulate:
        base, dbase = torch.ones((N, K), device="cuda"), torch.ones((N,), device="cuda")
        dw, db = dq.dq_act8_weight_grad(dy, codes, scales, out=base.clone(), out_dtype=out, accumulate=True,
                                        bias_grad=dbase.clone())
        _check(dw, db, dy, x, base.double(), dbase.double())
    else:
        dw, db = dq.dq_act8_weight_grad(dy, codes, scales, out_dtype=out, bias_grad=True)
        _check(dw, db, dy, x)
        again, _ = dq.dq_act8_weight_grad(dy, codes, scales, out_dtype=out)
        assert torch.equal(again, dw)


def test_against_differences():
    """dW and db of L = sum (x W^T + b - t)^2 / 2 against central differences of
    L in 64 bits (exact for a quadratic but for rounding); dY is rounded to bf16
    first, which moves dW by at most 2^-8 sum |dy x|."""
    M, N, K = 96, 24, 48
    _, codes, scales, x = _case(M, N, K, 4)
    g = torch.Generator().manual_seed(7)
    w, b = torch.randn((N, K), generator=g).double().cuda(), torch.randn(N, generator=g).double().cuda()
    t = torch.randn((M, N), generator=g).double().cuda()

    def loss(w, b):
        return float(((x @ w.T + b - t) ** 2).sum()) / 2

    r = x @ w.T + b - t
    dw, db = dq.dq_act8_weight_grad(r.bfloat16(), codes, scales, out_dtype="f32", bias_grad=True)
    mag = r.abs().T @ x.abs()
    h = 2.0 ** -10
    for n, k in [(0, 0), (5, 17), (23, 47), (11, 30)]:
        e = torch.zeros_like(w)
        e[n, k] = h
        diff = (loss(w + e, b) - loss(w - e, b)) / (2 * h)
        assert abs(float(dw[n, k]) - diff) <= (2.0 ** -8 + ACC_REL) * float(mag[n, k]) + 1e-6 * abs(diff)
    for n in (0, 9, 23):
        e = torch.zeros_like(b)
        e[n] = h
        diff = (loss(w, b + e) - loss(w, b - e)) / (2 * h)
        assert abs(float(db[n]) - diff) <= 2.0 ** -7 * float(r.abs().sum(0)[n]) + 1e-6 * abs(diff)


def test_non_finite_checkpoint_blocks_reach_their_feature_only():
    M, N, K = 70, 40, 64
    x = torch.randn((M, K), generator=torch.Generator().manual_seed(0)).bfloat16()
    x[69, 9] = float("inf")
    codes, scales = dq.dq_act8_pack(x.cuda())
    dy = torch.ones((M, N), dtype=torch.bfloat16, device="cuda")
    dw, _ = dq.dq_act8_weight_grad(dy, codes, scales)
    nan = torch.isnan(dw)
    assert bool(nan[:, 9].all()) and int(nan.sum()) == N


@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_no_tokens_give_zeros(out):
    codes, scales = dq.dq_act8_pack(torch.empty((0, 32), dtype=torch.bfloat16, device="cuda"))
    dy = torch.empty((0, 16), dtype=torch.bfloat16, device="cuda")
    dw, db = dq.dq_act8_weight_grad(dy, codes, scales, out_dtype=out, bias_grad=True)
    assert bool((dw == 0).all()) and bool((db == 0).all()) and tuple(dw.shape) == (16, 32)


@pytest.mark.parametrize("M,N,K", [(130, 72, 80), (2048, 1032, 1040)])
def test_memory_behind_the_gradients_stays(M, N, K):
    dy, codes, scales, _ = _case(M, N, K, 3)
    for dt, name in ((torch.bfloat16, "bf16"), (torch.float32, "f32")):
        buf = torch.full((N + 40, K), 5.0, dtype=dt, device="cuda")
        dbuf = torch.full((N + 64,), 5.0, device="cuda")
        dq.dq_act8_weight_grad(dy, codes, scales, out=buf[:N], out_dtype=name, bias_grad=dbuf[:N])
        assert bool((buf[N:] == 5.0).all()) and bool((dbuf[N:] == 5.0).all())
