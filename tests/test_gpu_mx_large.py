"""The microscaled operators where offsets pass 2^31 elements, and where token
blocks outnumber a grid's rows: the last rows against the plain forms."""
import numpy as np
import pytest
import torch

import mx_ref as ref

pytestmark = pytest.mark.gpu

dq = pytest.importorskip("quantized_gemm_token_b200") if torch.cuda.is_available() else None

M, K = 131080, 16416            # 2.15e9 elements


@pytest.fixture(scope="module")
def x():
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=g)
    yield x
    del x
    torch.cuda.empty_cache()


ENDS = [slice(0, 3), slice(M - 40, M)]


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_quantize_dequantize_and_product(x, fmt):
    q, sf, s = dq.dq_quantize_rows_fp4(x, fmt)
    back = dq.dq_fp4_dequantize(q, sf, s, fmt)
    tiles = sf.cpu().numpy()
    for rows in ENDS:
        codes, E, sr = ref.quantize_fp4(x[rows].double().cpu().numpy(), fmt)
        got, want = q[rows].cpu().numpy(), ref.pack4(codes)
        lut = ref.E2M1_ALL
        assert np.array_equal(lut[got & 15], lut[want & 15]) and np.array_equal(lut[got >> 4], lut[want >> 4])
        r = np.arange(rows.start, rows.stop)[:, None]
        b = np.arange(E.shape[1])[None]
        assert np.array_equal(tiles[r // 128, b // 4, 16 * (r % 32) + 4 * (r % 128 // 32) + b % 4], E)
        assert sr is None or np.array_equal(s[rows].cpu().numpy(), sr)
        assert torch.equal(back[rows].double().cpu(), torch.from_numpy(ref.values_fp4(codes, E, sr, fmt)))
    N = 16424                   # 2.15e9 outputs
    w = torch.randn((N, K), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    W = dq.dq_quantize_weight_fp4(w, fmt)
    del w
    y = dq.dq_fp4_linear(q, sf, s, *W, fmt=fmt)
    wv = dq.dq_fp4_dequantize(*W, fmt)[-200:].double()
    for rows in ENDS:
        a = back[rows].double()
        want, mag = a @ wv.T, a.abs() @ wv.abs().T
        tol = (2.0 ** -25.9 * K ** 0.5 + 2.0 ** -21) * mag + (2.0 ** -8 + 2.0 ** -22) * want.abs()
        assert bool(((y[rows, -200:].double() - want).abs() <= tol).all())
    assert dq.dq_sync_status() == dq.DQ_OK


def test_checkpoint_and_gradients(x):
    kept = dq.Act8.save(x)
    back = kept.restore()
    for rows in (slice(0, 32), slice(M - M % 32 - 32, M)):
        q, E = ref.act8(x[rows].double().cpu().numpy())
        assert torch.equal(back[rows].double().cpu(), torch.from_numpy(ref.act8_values(q, E)))
    N = 72
    dy = torch.randn((M, N), generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").bfloat16()
    dw, db = kept.weight_grad(dy, out_dtype="f32", bias_grad=True)
    d = dy.double()
    for cols in (slice(0, 32), slice(K - 48, K)):
        xv = back[:, cols].double()
        # zero-mean operands: 2^-20 of the magnitude sum
        assert bool(((dw[:, cols].double() - d.T @ xv).abs() <= 2.0 ** -20 * (d.abs().T @ xv.abs())).all())
    assert bool(((db.double() - d.sum(0)).abs() <= (M / 16 + 48) * 2.0 ** -24 * d.abs().sum(0)).all())
    assert dq.dq_sync_status() == dq.DQ_OK


@pytest.mark.parametrize("tokens", [65535 * 16 + 5, 65535 * 32 + 40])
def test_more_token_blocks_than_a_grid_has_rows(tokens):
    g = torch.Generator(device="cuda").manual_seed(tokens)
    x = torch.empty((tokens, 16), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    back = dq.Act8.save(x).restore()
    e = torch.nn.functional.pad(x.float(), (0, 0, 0, -tokens % 32)).view(-1, 32, 16)
    scale = torch.exp2(torch.frexp(e.abs().amax(1, keepdim=True)).exponent.float() - 7)
    want = ((e / scale).round().clamp(-127, 127) * scale).view(-1, 16)[:tokens].bfloat16()
    assert torch.equal(back, want)
