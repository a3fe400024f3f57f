"""The two sets of plain forms of the microscaled operators, written apart:
perf/operators.py (fp32 tensor expressions, and its 64-bit forms) and
tests/mx_ref.py (numpy).  They have to give the same codes, scales and values
on the same inputs, borders and ends of the range included (CPU)."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import mx_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ops():
    spec = importlib.util.spec_from_file_location("operators_plain_forms", os.path.join(ROOT, "perf", "operators.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _x(M, K, kind):
    g = torch.Generator().manual_seed(M + K)
    x = torch.randn((M, K), generator=g)
    if kind == "outliers":
        x[:, torch.rand(K, generator=g) < 0.03] *= 20
    elif kind == "wide":
        x *= torch.exp2(torch.randint(-60, 60, (M, K), generator=g).float())
    elif kind == "ties":
        x = torch.randint(-28, 29, (M, K), generator=g).float() / 8
    elif kind == "edges":
        x[0] = 0
        x[-1, :K // 2] = 0
        if M > 4:
            x[1] = torch.sign(x[1]) * 2.0 ** -130
            x[2, 0] = 3.38e38
            x[3] *= 2.0 ** -118
            x[4] = -0.0
    return x.bfloat16()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("kind", ["normal", "outliers", "wide", "ties", "edges"])
@pytest.mark.parametrize("M,K", [(1, 32), (5, 96), (33, 160), (130, 288), (8, 4096)])
def test_four_bit_forms_agree(ops, M, K, kind, fmt):
    x = _x(M, K, kind)
    codes, E, s = ref.quantize_fp4(x.double().numpy(), fmt)
    oc, oe, os_ = ops._quantize(x, fmt)
    lut = ref.E2M1_ALL                              # a zero code's sign is free
    assert np.array_equal(lut[oc.numpy()], lut[codes]) and np.array_equal(oe.numpy(), E)
    assert np.array_equal(os_.numpy(), np.ones(M, np.float32) if s is None else s)
    assert np.array_equal(ops._tile(oe, fmt).numpy(), ref.tile_scales(E, fmt))
    assert torch.equal(ops._untile(ops._tile(oe, fmt), M, E.shape[1]), oe)
    p = ops._pack(oc)
    assert torch.equal(torch.stack((p & 15, p >> 4), 2).view(M, K), oc)
    want = torch.from_numpy(ref.values_fp4(codes, E, None, fmt))
    assert torch.equal(ops._values(oc, oe, fmt).double(), want)
    assert torch.equal(ops._exact_fp4(x, fmt), want if s is None else want * torch.from_numpy(s).double()[:, None])


@pytest.mark.parametrize("kind", ["normal", "outliers", "wide", "ties", "edges"])
@pytest.mark.parametrize("M,K", [(1, 16), (31, 48), (32, 16), (70, 272), (257, 128)])
def test_checkpoint_forms_agree(ops, M, K, kind):
    x = _x(M, K, kind)
    q, E = ref.act8(x.double().numpy())
    oq, oe = ops._act8(x)
    assert np.array_equal(oq[:M].numpy(), q) and bool((oq[M:] == 0).all()) and np.array_equal(oe.numpy(), E)
    assert np.array_equal(ops._act8_layout(oq).numpy(), ref.act8_layout(q))
    want = torch.from_numpy(ref.act8_values(q, E))
    assert torch.equal(ops._act8_values(ops._act8_layout(oq), oe, M).double(), want)
    assert torch.equal(ops._exact_act8(x), want)
