"""Plain 64-bit numpy forms of the microscaled formats: 4-bit codes with block
scales ("mx": 32 features, ue8m0; "nv": 16 features, e4m3 and a power-of-two
row scale) and the 8-bit activation checkpoint.  Written from the definitions
in include/dq.h; every function works on values (float64) or on the stored
bytes and shares no code with the library."""
import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E2M1_ALL = np.concatenate([E2M1, -E2M1])
# all e4m3 values by code 0..126 (finite, non-negative)
E4M3 = np.array([(c % 8) * 2.0 ** -9 if c < 8 else (8 + c % 8) * 2.0 ** (c // 8 - 10) for c in range(127)])


def floor_log2(a):
    """floor(log2 a) for a > 0 (a large negative number for 0)."""
    return np.where(a > 0, np.frexp(a)[1] - 1, -10000).astype(np.int64)


def nearest(v, table):
    """Index of the nearest entry of an increasing table for v >= 0; ties to
    the even index; saturating."""
    mid = (table[1:] + table[:-1]) / 2            # exact: few significant bits
    lo = np.searchsorted(mid, v, side="left")     # ties stay below
    hi = np.searchsorted(mid, v, side="right")    # ties go above
    return np.where(lo % 2 == 0, lo, hi)


def quantize_fp4(x, fmt):
    """x float64 [R, K] holding bf16 or fp32 values -> (codes uint8 [R, K] 0..15,
    scale bytes [R, K / block], row scales fp32 [R] or None)."""
    x = np.asarray(x, np.float64)
    R, K = x.shape
    b = 32 if fmt == "mx" else 16
    blk = x.reshape(R, K // b, b)
    with np.errstate(invalid="ignore"):
        top = np.abs(blk).max(axis=2)
    if fmt == "mx":
        bad = ~np.isfinite(top)
        E = np.clip(floor_log2(np.where(bad, 1.0, top)) - 2 + 127, 0, 254)
        y = np.where(bad[..., None], 0.0, np.where(np.isfinite(blk), blk, 0.0)) / (2.0 ** (E - 127.0))[..., None]
        E = np.where(bad, 255, E)
        s = None
    else:
        row = top.max(axis=1) if K else np.zeros(R)
        bad = ~np.isfinite(row)
        row = np.where(bad, 0.0, row)
        p = np.full(R, -110, np.int64)
        m, e = np.frexp(row / 2688.0)             # 2^p >= row / 2688
        # row / 2688 is rounded; it is a power of two only where it is exactly one (row has <= 24 bits, 2688 = 21 * 2^7)
        exact = (m == 0.5) & (2688.0 * 2.0 ** (e - 1.0) == row)
        p = np.where(row > 0, np.maximum(np.where(exact, e - 1, e), -110), -110)
        sv = 2.0 ** p.astype(np.float64)
        r = ((top / sv[:, None]).astype(np.float32) / np.float32(6)).astype(np.float64)
        E = nearest(np.where(bad[:, None], 0.0, r), E4M3)
        d = E4M3[E]
        with np.errstate(divide="ignore", invalid="ignore"):
            # exact quotient against the borders: compare x with border * d * s in 64 bits
            y = np.where((d > 0)[..., None] & ~bad[:, None, None],
                         np.where(np.isfinite(blk), blk, 0.0) / sv[:, None, None] / d[..., None], 0.0)
        E = np.where(bad[:, None], 0, E)
        s = np.where(bad, np.nan, sv).astype(np.float32)
    codes = nearest(np.abs(y), E2M1) + 8 * np.signbit(y)
    return codes.reshape(R, K).astype(np.uint8), E.astype(np.uint8), s


def pack4(codes):
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def scale_values(E, fmt):
    if fmt == "mx":
        return np.where(E == 255, np.nan, 2.0 ** (E.astype(np.float64) - 127))
    v = E4M3[np.minimum(E & 127, 126)]
    return np.where((E & 127) == 127, np.nan, np.where(E & 128, -v, v))


def values_fp4(codes, E, s, fmt):
    """float64 values [R, K] (row scale included when given)."""
    R, K = codes.shape
    v = E2M1_ALL[codes].reshape(R, E.shape[1], -1) * scale_values(E, fmt)[..., None]
    v = v.reshape(R, K)
    return v if s is None else v * s.astype(np.float64)[:, None]


def tile_scales(E, fmt):
    R, G = E.shape
    rb, gb = -(-R // 128), -(-G // 4)
    out = np.zeros((rb, gb, 512), np.uint8)
    for r in range(R):
        for g in range(G):
            out[r // 128, g // 4, 16 * (r % 32) + 4 * (r % 128 // 32) + g % 4] = E[r, g]
    return out


def act8(x):
    """x float64 [M, K] (bf16 values) -> (codes int8 [M, K], scale bytes [ceil(M/32), K])."""
    x = np.asarray(x, np.float64)
    M, K = x.shape
    p = np.zeros((-(-M // 32) * 32, K))
    p[:M] = x
    blk = p.reshape(-1, 32, K)
    with np.errstate(invalid="ignore"):
        top = np.abs(blk).max(axis=1)
    bad = ~np.isfinite(top)
    E = np.clip(floor_log2(np.where(bad, 1.0, top)) + 127, 0, 254)
    y = np.where(bad[:, None], 0.0, np.where(np.isfinite(blk), blk, 0.0)) * (2.0 ** (133.0 - E))[:, None]
    q = np.clip(np.rint(y), -127, 127).reshape(-1, K)[:M]
    return q.astype(np.int8), np.where(bad, 255, E).astype(np.uint8)


def act8_values(q, E):
    M, K = q.shape
    s = np.where(E == 255, np.nan, 2.0 ** (E.astype(np.float64) - 133))
    return q.astype(np.float64) * np.repeat(s, 32, axis=0)[:M]


def act8_layout(q):
    """[M, K] -> [2 ceil(M/32), K, 16], zero padded."""
    M, K = q.shape
    p = np.zeros((-(-M // 32) * 32, K), np.int8)
    p[:M] = q
    return np.ascontiguousarray(p.reshape(-1, 16, K).transpose(0, 2, 1))
