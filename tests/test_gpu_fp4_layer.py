"""The microscaled layer as a user runs it: forward, the input kept in 8 bits,
input, weight and bias gradients; captured and replayed, on other streams, two
calls at once; and what the binding refuses.

Expected values are 64-bit products of the values that the stored codes stand
for (the codes themselves are checked bit for bit elsewhere), with the bounds
of the product tests: ACC_REL of the magnitude sum for the fp32 accumulation,
half a bf16 step (2^-8) for the output, 2^-24 per further fp32 operation."""
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


def _values(x, fmt):
    c, E, s = ref.quantize_fp4(x.double().cpu().numpy(), fmt)
    return torch.from_numpy(ref.values_fp4(c, E, s, fmt)).cuda()


def _close(got, want, mag, bf16):
    tol = ACC_REL * mag + 4 * 2.0 ** -24 * want.abs()
    if bf16:
        tol = tol + 2.0 ** -8 * want.abs()
    assert bool(((got.double() - want).abs() <= tol).all())


def _step(layer, x, dy):
    """One training step's calls."""
    y = layer(x)
    kept = dq.Act8.save(x)
    dw, db = kept.weight_grad(dy, out_dtype="f32", bias_grad=True)
    return y, layer.backward_input(dy), dw, db


def _inputs(M, K, N, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((M, K), generator=g)
    x[:, torch.rand(K, generator=g) < 0.02] *= 20
    return x.bfloat16().cuda(), (torch.randn((M, N), generator=g) * 0.1).bfloat16().cuda()


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("M,K,N", [(1, 64, 32), (40, 288, 160), (333, 512, 416), (2100, 256, 1056)])
def test_training_step(M, K, N, fmt):
    g = torch.Generator().manual_seed(M)
    w = (torch.randn((N, K), generator=g) * 0.02).cuda()
    b = torch.randn(N, generator=g).bfloat16().cuda()
    layer = dq.Fp4Linear.from_float(w, b, fmt, backward=True)
    x, dy = _inputs(M, K, N, M + 1)
    y, dx, dw, db = _step(layer, x, dy)
    xq, wq = _values(x, fmt), _values(w, fmt)
    _close(y, xq @ wq.T + b.double(), xq.abs() @ wq.abs().T + b.double().abs(), True)
    dq_, wt = _values(dy, fmt), _values(w.t().contiguous(), fmt)
    _close(dx, dq_ @ wt.T, dq_.abs() @ wt.abs().T, True)
    q, E = ref.act8(x.double().cpu().numpy())
    x8 = torch.from_numpy(ref.act8_values(q, E)).cuda()
    d = dy.double()
    _close(dw, d.T @ x8, d.abs().T @ x8.abs(), False)
    assert bool(((db.double() - d.sum(0)).abs() <= (M / 8 + 64) * 2.0 ** -24 * d.abs().sum(0)).all())
    assert torch.equal(dq.Act8.save(x).restore().double(), x8)


def test_checkpoint_serves_the_int8_layer():
    """The int8 layer's input kept in 8 bits: with outlier features the
    checkpoint's gradient is nearer to the unquantized one than the gradient
    of the layer's own per-token codes."""
    M, K, N = 512, 512, 256
    x, dy = _inputs(M, K, N, 3)
    layer = dq.Int8DynamicLinear.from_float(torch.randn((N, K), generator=torch.Generator().manual_seed(1)).cuda())
    layer(x)
    dw, _ = dq.Act8.save(x).weight_grad(dy, out_dtype="f32")
    exact = dy.double().T @ x.double()
    q, s = dq.dq_quantize_rows(x)
    own = dy.double().T @ (q.double() * s.double()[:, None])
    assert float((dw.double() - exact).norm()) < 0.3 * float((own - exact).norm())


@pytest.mark.parametrize("M", [1, 16, 300])
def test_captured_step_replays_on_new_inputs(M):
    K, N = 512, 288
    layer = dq.Fp4Linear.from_float(torch.randn((N, K), generator=torch.Generator().manual_seed(1)).cuda(), backward=True)
    x, dy = _inputs(M, K, N, 0)
    _step(layer, x, dy)                        # first calls resolve devices and limits
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = _step(layer, x, dy)
    for seed in (5, 6):
        x2, dy2 = _inputs(M, K, N, seed)
        x.copy_(x2)
        dy.copy_(dy2)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, _step(layer, x2, dy2)):
            assert torch.equal(a, b)


def test_two_graphs_of_one_layer_at_once():
    K, N = 1024, 512
    layer = dq.Fp4Linear.from_float(torch.randn((N, K), generator=torch.Generator().manual_seed(1)).cuda(), backward=True)
    ins = [_inputs(M, K, N, M) for M in (33, 700)]
    want = [tuple(t.clone() for t in _step(layer, *i)) for i in ins]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for i in ins:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(_step(layer, *i))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in ins]
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        for a, b in zip(o, w):
            assert torch.equal(a, b)


def test_calls_on_other_streams_at_once():
    K, N = 768, 320
    layer = dq.Fp4Linear.from_float(torch.randn((N, K), generator=torch.Generator().manual_seed(1)).cuda())
    ins = [_inputs(M, K, N, M) for M in (8, 64, 400, 1500)]
    want = [layer(x).clone() for x, _ in ins]
    grads = [dq.Act8.save(x).weight_grad(dy, out_dtype="f32")[0].clone() for x, dy in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ins]
    for _ in range(10):
        got, dws = [], []
        for (x, dy), s in zip(ins, streams):
            got.append(layer(x, stream=s))
            dws.append(dq.Act8.save(x, stream=s).weight_grad(dy, out_dtype="f32", stream=s)[0])
        torch.cuda.synchronize()
        for a, b in zip(got + dws, want + grads):
            assert torch.equal(a, b)


def test_binding_refusals():
    x = torch.zeros((8, 64), dtype=torch.bfloat16, device="cuda")
    q, sf, s = dq.dq_quantize_rows_fp4(x)
    for bad in (x.float(), x.half()):
        with pytest.raises(TypeError):
            dq.dq_quantize_rows_fp4(bad)
        with pytest.raises(TypeError):
            dq.dq_act8_pack(bad)
    for bad in (x[:, :40], x.t(), x[:, ::2], x[0], x[:1].expand(8, 64)):
        with pytest.raises(ValueError):
            dq.dq_quantize_rows_fp4(bad)
    for bad in (x[:, :40], x.t(), x[:1].expand(8, 64)):
        with pytest.raises(ValueError):
            dq.dq_act8_pack(bad)
    with pytest.raises(ValueError):
        dq.dq_quantize_rows_fp4(x, "mx", s_row=s)            # mx has none
    with pytest.raises(ValueError):
        dq.dq_quantize_rows_fp4(x, sf=sf[:, :, :256])
    with pytest.raises(ValueError):
        dq.dq_fp4_linear(q, sf, s, q[:, :16], sf, s)         # K differs, not contiguous
    with pytest.raises(ValueError):
        dq.dq_fp4_linear(q, sf, s[:4], q, sf, s)
    wide = dq.dq_quantize_rows_fp4(torch.zeros((8, 128), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        dq.dq_fp4_linear(*wide, *wide, fmt="mx")             # scale tiles of the other format
    with pytest.raises(ValueError):
        dq.dq_fp4_linear(q, sf, s, q, sf, s, out_dtype="s32")
    with pytest.raises(ValueError):
        dq.dq_fp4_linear(q, sf, s, q, sf, s, out=torch.empty((8, 16), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(TypeError):
        dq.dq_fp4_linear(q, sf, s, q, sf, s, out=torch.empty((8, 8), device="cuda"))
    with pytest.raises(TypeError):
        dq.dq_fp4_linear(q, sf, s, q, sf, s, bias=torch.zeros(8, device="cuda"))
    seven = dq.dq_quantize_weight_fp4(torch.zeros((12, 64), device="cuda"))
    with pytest.raises(dq.DQError):
        dq.dq_fp4_linear(q, sf, s, *seven)                   # N % 8
    buf = torch.zeros(8 * 8 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(8, 8)
    with pytest.raises(dq.DQError):
        dq.dq_fp4_linear(q, sf, s, q, sf, s, out=buf)        # misaligned
    codes, scales = dq.dq_act8_pack(x)
    dy = torch.zeros((8, 16), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        dq.dq_act8_weight_grad(torch.zeros((40, 16), dtype=torch.bfloat16, device="cuda"), codes, scales)
    with pytest.raises(ValueError):
        dq.dq_act8_weight_grad(dy, codes[:, :32], scales)
    with pytest.raises(ValueError):
        dq.dq_act8_weight_grad(dy, codes, scales, accumulate=True)
    with pytest.raises(ValueError):
        dq.dq_act8_weight_grad(dy, codes, scales, out=torch.zeros((16, 64), dtype=torch.bfloat16, device="cuda"),
                               accumulate=True)
    with pytest.raises(dq.DQError):
        dq.dq_act8_weight_grad(dy[:, :12], codes, scales)    # N % 8
    with pytest.raises(dq.DQError):
        dq.dq_act8_weight_grad(torch.zeros((8, 20), dtype=torch.bfloat16, device="cuda")[:, :16], codes, scales)
    with pytest.raises(ValueError):
        dq.dq_act8_unpack(codes, scales, 40)
    with pytest.raises(ValueError):
        dq.Act8(codes, scales, 8).weight_grad(dy[:4])
    layer = dq.Fp4Linear.from_float(torch.zeros((16, 64), device="cuda"))
    with pytest.raises(ValueError):
        layer.backward_input(dy)
