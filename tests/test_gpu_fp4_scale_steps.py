"""bf16 values against every mantissa step of the nv block scale: the kernel
decides a code without a division, from a product that is snapped to a grid;
the steps with the most significant bits (15 / 8) are the tightest."""
import numpy as np
import pytest
import torch

import mx_ref as ref

pytestmark = pytest.mark.gpu

dq = pytest.importorskip("quantized_gemm_token_b200") if torch.cuda.is_available() else None


@pytest.mark.parametrize("shift", [-90, 0, 60])
@pytest.mark.parametrize("neighbour", [0.0, 1.0])
def test_every_step_of_the_block_scale(shift, neighbour):
    """Block maxima 6 d with d = 8 .. 15 sixteenths (times 64), so that each block's
    scale has the mantissa d / 8, and below each maximum all bf16 values from 2^-5
    times it (the least border is 1 / 24 of it) up to it, at three places
    of the exponent range; with a neighbour block the row scale is another one."""
    pats = (torch.arange(0x3a00, 0x4480, dtype=torch.int32) << 16).view(torch.float32)      # 2^-11 .. 2^10
    rows, steps = [], []
    for d in range(8, 16):
        top = 6.0 * d / 16 * 64
        v = pats[(pats >= top / 32) & (pats <= top)]
        v = torch.cat([v, torch.zeros(-v.numel() % 15)]).view(-1, 15)
        rows.append(torch.cat([torch.full((v.shape[0], 1), top), v], 1))
        steps += [d] * v.shape[0]
    blk = torch.cat(rows)
    other = torch.full_like(blk, neighbour * 2000.0)
    x = torch.cat([blk, other], 1)
    x[1::2] *= -1
    x = (x.double() * 2.0 ** shift).bfloat16()
    q, sf, s = dq.dq_quantize_rows_fp4(x.cuda())
    codes, E, sr = ref.quantize_fp4(x.double().numpy(), "nv")
    assert np.array_equal(8 + (E[:, 0] & 7), np.array(steps)) and bool((E[:, 0] >= 8).all())     # all eight, as built
    lut, got, want = ref.E2M1_ALL, q.cpu().numpy(), ref.pack4(codes)
    assert np.array_equal(lut[got & 15], lut[want & 15]) and np.array_equal(lut[got >> 4], lut[want >> 4])
    assert np.array_equal(sf.cpu().numpy(), ref.tile_scales(E, "nv")) and np.array_equal(s.cpu().numpy(), sr)
