"""The microscaled 4-bit layer against plain 64-bit forms (tests/mx_ref.py).

Codes, block scales and row scales are bit-equal by definition.  The product:
every a * w * sfa * sfw is exact in fp32 (2 + 2 bits times 4 + 4 bits of e4m3
scales), the fp32 sum's order and rounding are the tensor core's, so |acc -
exact| is bounded by ACC_REL * sum |a w sfa sfw|, as for the FP8 layer; a bf16
output adds one bf16 rounding (2^-8 relative) after two or three fp32 ones.
"""
import numpy as np
import pytest
import torch

import mx_ref as ref

pytestmark = pytest.mark.gpu

dq = pytest.importorskip("quantized_gemm_token_b200") if torch.cuda.is_available() else None

# sixteen times the fp32 unit roundoff, as the other tensor-core fp32 sums here
ACC_REL = 2.0 ** -20


@pytest.fixture(autouse=True)
def _sync_and_check():
    yield
    if torch.cuda.is_available():
        assert dq.dq_sync_status() == dq.DQ_OK


def _x(M, K, seed, kind="normal", dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((M, K), generator=g)
    if kind == "outliers":
        x[:, torch.rand(K, generator=g) < 0.03] *= 20
    elif kind == "wide":             # magnitudes over the whole range of the format
        x *= torch.exp2(torch.randint(-60, 60, (M, K), generator=g).float())
    elif kind == "ties":             # small integers: many quotients on a border
        x = torch.randint(-28, 29, (M, K), generator=g).float() / 8
    elif kind == "edges":            # zero rows and blocks, subnormals, the largest finite value
        x[0] = 0
        x[-1, : K // 2] = 0
        if M > 2:
            x[1] = torch.sign(x[1]) * 2.0 ** -130
            x[2, 0] = 3.38e38
        if M > 4:
            x[3] *= 2.0 ** -118
            x[4] = -0.0
    return x.to(dtype)


def _check_quantized(x, fmt, q, sf, s):
    codes, E, sr = ref.quantize_fp4(x.double().numpy(), fmt)
    got = q.cpu().numpy()
    want = ref.pack4(codes)
    # a zero code's sign is free: both nibbles stand for 0
    lut = ref.E2M1_ALL
    assert np.array_equal(lut[got & 15], lut[want & 15]) and np.array_equal(lut[got >> 4], lut[want >> 4])
    assert np.array_equal(sf.cpu().numpy(), ref.tile_scales(E, fmt))
    if fmt == "nv":
        assert np.array_equal(s.cpu().numpy(), sr, equal_nan=True)
    else:
        assert s is None
    return codes, E, sr


SHAPES = [(1, 32), (1, 64), (3, 96), (5, 480), (33, 160), (130, 1280), (129, 4096), (40, 8192), (3, 16384), (2, 16416), (2, 28672), (1, 32768), (1, 32800)]


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("kind", ["normal", "outliers", "wide", "ties", "edges"])
@pytest.mark.parametrize("M,K", SHAPES)
def test_quantize_rows_bit_exact(M, K, kind, fmt):
    x = _x(M, K, M * 7 + K, kind)
    q, sf, s = dq.dq_quantize_rows_fp4(x.cuda(), fmt)
    codes, E, sr = _check_quantized(x, fmt, q, sf, s)
    out = dq.dq_fp4_dequantize(q, sf, s, fmt).cpu()
    # exact in bf16, but for the infinity past its range: 3.38e38 is quantized
    # to 6 * 352 * 2^117 = 2112 * 2^117, the largest bf16 is 2040 * 2^117
    want = torch.from_numpy(ref.values_fp4(codes, E, sr, fmt))
    assert torch.equal(out, want.bfloat16())
    assert torch.equal(out.double(), want) or kind == "edges"


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_every_bf16_value_against_every_scale(fmt):
    """All 2^15 non-negative finite bf16 patterns below a block maximum, for
    eight maxima with every mantissa step of the e4m3 scale."""
    pats = torch.arange(0x3a00, 0x4300, dtype=torch.int32)           # 2^-11 .. 2^7
    vals = (pats << 16).view(torch.float32)
    rows = []
    for top in (1.0, 1.0625, 1.1875, 1.3125, 1.5, 1.6875, 1.875, 1.9921875):
        v = vals[vals <= top * 64]
        v = torch.cat([v, torch.zeros(-v.numel() % 15)]).view(-1, 15)
        blk = torch.cat([torch.full((v.shape[0], 1), top * 64), v], 1)
        rows.append(blk)
    x = torch.cat(rows)
    x = torch.cat([x, torch.zeros((-x.shape[0] % 8, 16))]).view(-1, 128).bfloat16()
    x[1::2] *= -1
    q, sf, s = dq.dq_quantize_rows_fp4(x.cuda(), fmt)
    _check_quantized(x, fmt, q, sf, s)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("kind", ["normal", "wide", "ties", "edges"])
@pytest.mark.parametrize("N,K", [(8, 32), (72, 96), (136, 2080)])
def test_quantize_weight_bit_exact(N, K, kind, fmt):
    w = _x(N, K, N + K, kind, torch.float32)
    q, sf, s = dq.dq_quantize_weight_fp4(w.cuda(), fmt)
    _check_quantized(w, fmt, q, sf, s)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("kind", ["normal", "wide", "ties", "edges"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("R,K", [(300, 64), (257, 128), (200, 192), (131, 256), (70, 544), (33, 640), (40, 768),
                                 (19, 2560), (20, 3584), (9, 5120), (7, 6112), (3, 12288), (2, 20480)])
def test_quantize_rows_of_every_split(R, K, dtype, kind, fmt):
    """Rows that share a warp (8 or 16 threads each), and one to eight runs of 16
    features per thread, filled or with idle places."""
    x = _x(R, K, R + K, kind, dtype)
    f = dq.dq_quantize_rows_fp4 if dtype == torch.bfloat16 else dq.dq_quantize_weight_fp4
    _check_quantized(x, fmt, *f(x.cuda(), fmt))


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("kind", ["normal", "outliers", "wide", "edges"])
@pytest.mark.parametrize("N,K", [(130, 1280), (9, 8192), (3, 16384), (2, 16416)])
def test_quantize_long_weight_rows(N, K, kind, fmt):
    w = _x(N, K, N + K, kind, torch.float32)
    _check_quantized(w, fmt, *dq.dq_quantize_weight_fp4(w.cuda(), fmt))


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("offset,pad", [(0, 8), (0, 4), (0, 3), (1, 0), (4, 4)])
def test_quantize_weight_strides_and_offsets(offset, pad, fmt):
    N, K = 37, 416
    w = _x(N, K + pad + offset, 5, "wide", torch.float32).cuda()[:, offset:offset + K]
    _check_quantized(w.cpu(), fmt, *dq.dq_quantize_weight_fp4(w, fmt))


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_fp32_values_beside_a_border(fmt):
    """Every rounding border of a code times every mantissa step of the block
    scale, the fp32 values next to it on either side, and their negatives."""
    rows = []
    borders = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    for d in (8, 9, 10, 11, 12, 13, 14, 15):
        b = borders * (d * 2.0 ** -4)
        near = torch.stack([torch.nextafter(b, torch.zeros(7)), b, torch.nextafter(b, torch.full((7,), 9.0))]).flatten()
        near = torch.cat([near, -near, torch.zeros(3)])
        for part in near.split(15):
            rows.append(torch.cat([torch.tensor([6.0 * d * 2.0 ** -4]), part]))
    w = torch.stack(rows)
    w = torch.cat([w, torch.zeros((-w.shape[0] % 4, 16))]).view(-1, 64)
    _check_quantized(w, fmt, *dq.dq_quantize_weight_fp4(w.cuda(), fmt))


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("offset,pad", [(0, 8), (0, 3), (1, 0), (4, 12)])
def test_quantize_strides_and_offsets(offset, pad, fmt):
    """Column slices of a wider matrix, aligned or not, and a strided q."""
    M, K = 37, 416
    wide = _x(M, K + pad + offset, 5, "outliers").cuda()
    x = wide[:, offset:offset + K]
    qbuf = torch.full((M, K // 2 + 6), 0xEE, dtype=torch.uint8, device="cuda")
    q, sf, s = dq.dq_quantize_rows_fp4(x, fmt, q=qbuf[:, :K // 2])
    _check_quantized(x.cpu(), fmt, q, sf, s)
    assert bool((qbuf[:, K // 2:] == 0xEE).all())


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_non_finite_inputs_become_nan(bad, fmt):
    x = _x(130, 256, 3)
    x[7, 40] = bad
    x[129, 255] = bad
    q, sf, s = dq.dq_quantize_rows_fp4(x.cuda(), fmt)
    _check_quantized(x, fmt, q, sf, s)
    out = dq.dq_fp4_dequantize(q, sf, s, fmt).cpu()
    nan = torch.isnan(out)
    if fmt == "nv":
        want = torch.zeros_like(nan)
        want[7] = want[129] = True
    else:
        want = torch.zeros_like(nan)
        want[7, 32:64] = True
        want[129, 224:] = True
    assert torch.equal(nan, want)
    w = _x(72, 256, 4, dtype=torch.float32)
    wq, sw, sc = dq.dq_quantize_weight_fp4(w.cuda(), fmt)
    for rows in (slice(0, 130), slice(0, 40)):
        xs = x[rows].cuda()
        y = dq.dq_fp4_linear(*dq.dq_quantize_rows_fp4(xs, fmt), wq, sw, sc, fmt=fmt)
        hit = torch.isnan(y).all(1).cpu()
        some = torch.isnan(y).any(1).cpu()
        want = torch.tensor([r in (7, 129) for r in range(xs.shape[0])])
        assert torch.equal(hit, want) and torch.equal(some, want)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("R,K", [(1, 32), (128, 256), (130, 4128), (300, 96)])
def test_tile_scales(R, K, fmt):
    G = K // (32 if fmt == "mx" else 16)
    E = np.random.default_rng(R + K).integers(0, 255, (R, G)).astype(np.uint8)
    got = dq.dq_fp4_tile_scales(torch.from_numpy(E).cuda(), fmt)
    assert np.array_equal(got.cpu().numpy(), ref.tile_scales(E, fmt))


# ---------------------------------------------------------------- product

def _operand(R, K, fmt, seed, kind="normal"):
    x = _x(R, K, seed, kind)
    codes, E, s = ref.quantize_fp4(x.double().numpy(), fmt)
    q = torch.from_numpy(ref.pack4(codes)).cuda()
    sf = torch.from_numpy(ref.tile_scales(E, fmt)).cuda()
    v = ref.values_fp4(codes, E, None, fmt)
    return q, sf, None if s is None else torch.from_numpy(s).cuda(), v


def _check_product(M, N, K, fmt, bias=False, seed=0, kind="normal"):
    qa, sa, sr, a = _operand(M, K, fmt, seed + 1, kind)
    qw, sw, sc, w = _operand(N, K, fmt, seed + 2)
    acc = a @ w.T
    mag = np.abs(a) @ np.abs(w).T
    got = dq.dq_fp4_linear(qa, sa, sr, qw, sw, sc, fmt=fmt, out_dtype="f32").cpu().double().numpy()
    err = np.abs(got - acc)
    assert (err <= ACC_REL * mag).all(), f"fp32 error {np.max(err / np.maximum(mag, 1e-300)):.3g} of the magnitude sum"
    b = (torch.randn(N, generator=torch.Generator().manual_seed(seed)) * 2).bfloat16() if bias else None
    f = np.ones((M, N)) if sr is None else sr.cpu().double().numpy()[:, None] * sc.cpu().double().numpy()
    y = acc * f + (b.double().numpy() if bias else 0.0)
    got = dq.dq_fp4_linear(qa, sa, sr, qw, sw, sc, b.cuda() if bias else None, fmt=fmt).cpu().double().numpy()
    # accumulation, then the fp32 ops (2^-24 each of the intermediate values), then half a bf16 step
    tol = ACC_REL * mag * f + 2.0 ** -8 * np.abs(y) + 3 * 2.0 ** -24 * (np.abs(acc * f) + np.abs(y))
    assert (np.abs(got - y) <= tol).all()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("M,N,K", [(1, 8, 32), (1, 264, 512), (5, 136, 96), (16, 128, 4096), (17, 520, 1056), (48, 72, 288),
                                   (64, 640, 2048), (100, 256, 736), (128, 384, 1280), (129, 136, 544), (200, 64, 64),
                                   (256, 1032, 1024)])
def test_few_tokens(M, N, K, fmt):
    _check_product(M, N, K, fmt, bias=M % 2 == 1, seed=M)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("M,N,K", [(257, 8, 32), (257, 192, 256), (300, 384, 1056), (512, 1160, 544), (700, 136, 2080),
                                   (1024, 2048, 736), (1799, 1280, 1280), (2300, 4104, 288), (2048, 4096, 4096)])
def test_many_tokens(M, N, K, fmt):
    _check_product(M, N, K, fmt, bias=M % 2 == 1, seed=M)


@pytest.mark.parametrize("N", [4104, 4136, 4168, 4200, 8])
@pytest.mark.parametrize("K", [32, 288])
def test_ragged_last_tiles_in_quick_succession(N, K):
    """Blocks of the output past the last column are not stored and must not
    disturb the ones still being stored: with few features the tiles follow one
    another at once, and the first calls run cold."""
    M = 5000
    x, w = _x(M, K, N).cuda(), _x(N, K, N + 1, dtype=torch.float32).cuda()
    A, W = dq.dq_quantize_rows_fp4(x, "mx"), dq.dq_quantize_weight_fp4(w, "mx")
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    want = dq.dq_fp4_linear(*A, *W, fmt="mx", out_dtype="f32").bfloat16()
    for _ in range(5):
        flush.fill_(1)
        assert torch.equal(dq.dq_fp4_linear(*A, *W, fmt="mx"), want)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("M", [3, 300])
def test_one_hot_reads_the_weight_back(M, fmt):
    """A one-hot activation (value 1, block scale 1) makes each output one
    weight value: nothing rounds, so every code and scale position is checked."""
    K, N = 320, 200
    qw, sw, sc, w = _operand(N, K, fmt, 9, "wide" if fmt == "mx" else "outliers")
    for k0 in range(0, K, M):
        hot = np.zeros((M, K), np.uint8)
        rows = np.arange(min(M, K - k0))
        hot[rows, k0 + rows] = 2                                     # e2m1 code of 1.0
        E = np.full((M, K // (32 if fmt == "mx" else 16)), 127 if fmt == "mx" else 56, np.uint8)   # scale 1
        qa = torch.from_numpy(ref.pack4(hot)).cuda()
        sa = torch.from_numpy(ref.tile_scales(E, fmt)).cuda()
        got = dq.dq_fp4_linear(qa, sa, None, qw, sw, None, fmt=fmt, out_dtype="f32").cpu().double().numpy()
        assert np.array_equal(got[rows], w.T[k0 + rows])
        if M < K and k0 > 2 * M:
            break


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("M", [1, 40, 300])
def test_output_canaries_and_repeat(M, fmt):
    """Rows behind the last one stay as they were; a repeated call gives the same bits."""
    N, K = 200, 800
    qa, sa, sr, _ = _operand(M, K, fmt, 1)
    qw, sw, sc, _ = _operand(N, K, fmt, 2)
    buf = torch.full((M + 300, N), 7.0, dtype=torch.bfloat16, device="cuda")
    y = dq.dq_fp4_linear(qa, sa, sr, qw, sw, sc, fmt=fmt, out=buf[:M]).clone()
    assert bool((buf[M:] == 7.0).all())
    for _ in range(3):
        assert torch.equal(dq.dq_fp4_linear(qa, sa, sr, qw, sw, sc, fmt=fmt), y)


def test_no_tokens():
    q, sf, s = dq.dq_quantize_rows_fp4(torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"))
    qw, sw, sc, _ = _operand(16, 64, "nv", 2)
    y = dq.dq_fp4_linear(q, sf, s, qw, sw, sc)
    assert tuple(y.shape) == (0, 16)
    assert tuple(dq.dq_fp4_dequantize(q, sf, s).shape) == (0, 64)
