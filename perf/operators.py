"""The microscaled operators as a user's program calls them, for timing and
comparison: the 4-bit layer (quantise the activations, multiply by the 4-bit
weight), its quantiser, the 8-bit activation checkpoint and the weight
gradient that reads it.

Formats (all scales are stored values, see include/dq.h):

* 4-bit codes: e2m1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign bit), two to a byte
  along the features, the even feature in the low nibble.
  "mx": blocks of 32 features, scale 2^(E - 127) with E = floor(log2 max|x|) -
  2 + 127 in 0..254.  "nv": blocks of 16 features; per row s, the least power
  of two with max|row| <= 2688 s (at least 2^-110), and per block the e4m3
  value nearest to max|block| / (6 s); a code stands for e2m1 * e4m3 * s.
  Block scales lie in tiles of 128 rows x 4 blocks, 512 bytes each: byte
  16 (r % 32) + 4 (r % 128 / 32) + b % 4 of tile (r / 128, b / 4).
* 8-bit checkpoint: blocks of 32 consecutive tokens of one feature, scale
  2^(E - 127) with E = floor(log2 max|x|) + 127 in 0..254, codes rint(64 x /
  scale) in -127..127; codes [token / 16, feature, token % 16], scales
  [token / 32, feature].

A plain form is written in elementary torch operations in fp32; ``exact``
evaluates the same definitions in fp64 by other means.
"""
import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # decoding one sequence: a single token against the wide few-token weight
        dict(name="linear_1", op="linear", fmt="nv", M=1, K=8192, N=28672, bias=False),
        # a small decoding batch on the same weight
        dict(name="linear_16", op="linear", fmt="mx", M=16, K=8192, N=28672, bias=False),
        # the language-model layer of the default benchmark
        dict(name="linear_2048", op="linear", fmt="nv", M=2048, K=4096, N=4096, bias=False),
        # seven images of 257 patches through the vision layer, an odd token count, with a bias
        dict(name="linear_1799_bias", op="linear", fmt="mx", M=1799, K=1280, N=5120, bias=True),
        # a long prefill
        dict(name="linear_16384", op="linear", fmt="nv", M=16384, K=8192, N=8192, bias=False),
        # the quantiser alone, its codes read back as values: the memory-bound sweep's matrix, and one image
        dict(name="quantize_16384", op="quantize", fmt="nv", M=16384, K=8192, pad=0),
        dict(name="quantize_257", op="quantize", fmt="mx", M=257, K=1280, pad=64),
        # saving and restoring a layer's input: the vision layer's tokens, and a short odd sequence
        dict(name="act8_65792", op="act8", M=65792, K=1280, pad=0),
        dict(name="act8_777", op="act8", M=777, K=4096, pad=128),
        # weight gradients: the language-model layer, the vision layer over a whole batch, a narrow odd layer
        dict(name="wgrad_2048", op="wgrad", M=2048, K=4096, N=4096, out="bf16", bias=False, pad=0),
        dict(name="wgrad_65792_f32", op="wgrad", M=65792, K=1280, N=5120, out="f32", bias=True, pad=0),
        dict(name="wgrad_1001", op="wgrad", M=1001, K=1296, N=264, out="bf16", bias=True, pad=8),
    ]


def _log(rng, lo, hi, step):
    return max(step, int(round(lo * (hi / lo) ** rng.random() / step)) * step)


def draw(rng):
    op = rng.choice(["linear", "linear", "quantize", "act8", "wgrad"])
    fmt = rng.choice(["nv", "mx"])
    pad = rng.choice([0, 0, 8, 72])
    if op == "linear":
        M, K, N = _log(rng, 1, 16384, 1), _log(rng, 64, 8192, 32), _log(rng, 64, 28672, 8)
        N = min(N, max(64, 16384 * 8192 // M // 8 * 8))
        return dict(op=op, fmt=fmt, M=M, K=K, N=N, bias=rng.random() < 0.5)
    M, K = _log(rng, 1, 65536, 1), _log(rng, 64, 8192, 32)
    K = min(K, max(64, 16384 * 8192 // M // 32 * 32))
    if op == "quantize":
        return dict(op=op, fmt=fmt, M=M, K=K, pad=pad)
    if op == "act8":
        return dict(op=op, M=M, K=K - rng.choice([0, 0, 16]), pad=pad)
    M = max(M, 16)
    N = _log(rng, 64, 8192, 8)
    N = min(N, max(64, 65792 * 1280 * 5120 // (M * K) // 8 * 8))
    return dict(op=op, M=M, K=K - rng.choice([0, 0, 16]), N=N, out=rng.choice(["bf16", "f32"]), bias=rng.random() < 0.5,
                pad=pad)


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _activations(g, M, K, pad=0):
    """bf16 [M, K] ~ N(0, 1) with 1 % of the features twenty times larger; with
    `pad`, the left columns of a wider matrix."""
    x = torch.randn((M, K + pad), generator=g, device="cuda")
    big = torch.rand((K + pad,), generator=g, device="cuda") < 0.01
    return (x * torch.where(big, 20.0, 1.0)).bfloat16()[:, :K]


def _weight(g, N, K):
    """A bf16 master weight ~ N(0, 0.02), held in fp32."""
    return (torch.randn((N, K), generator=g, device="cuda") * 0.02).bfloat16().float()


def prepare(case, seed):
    g = _gen(seed)
    op, M, K = case["op"], case["M"], case["K"]
    st = dict(case, x=_activations(g, M, K, case.get("pad", 0)))
    if op == "linear":
        codes, scales, row = _quantize(_weight(g, case["N"], K), case["fmt"])
        st.update(w=_pack(codes), sfw=_tile(scales, case["fmt"]), s_col=row if case["fmt"] == "nv" else None)
        st["b"] = torch.randn((case["N"],), generator=g, device="cuda").mul_(0.1).bfloat16() if case["bias"] else None
    elif op == "wgrad":
        q, e = _act8(st.pop("x"))
        st.update(codes=_act8_layout(q), scales=e)
        dy = torch.randn((M, case["N"] + case["pad"]), generator=g, device="cuda") * 0.05
        st["dy"] = dy.bfloat16()[:, :case["N"]]
    return st


# ---------------------------------------------------------------- plain forms

def _pow2(e):
    """2^e exactly, from its bits (two normal factors reach the subnormals)."""
    e = e.int()
    lo = torch.div(e, 2, rounding_mode="floor")
    return ((lo + 127) << 23).view(torch.float32) * ((e - lo + 127) << 23).view(torch.float32)


def _floor_log2(a):
    """floor(log2 a) of positive fp32 values; far below every format's range for 0."""
    return torch.where(a > 0, torch.frexp(a).exponent.int() - 1, -200)


def _e2m1(y):
    """Signed index of the nearest e2m1 value, ties to the even index."""
    a = y.abs()
    i = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int()
         + (a >= 3.5).int() + (a > 5.0).int())
    return i + 8 * (y < 0).int()


def _quantize(x, fmt):
    """(4-bit codes [M, K], block scale bytes [M, K / block], row scales [M])."""
    x = x.float()
    M, K = x.shape
    blk = x.view(M, K // (32 if fmt == "mx" else 16), -1)
    top = blk.abs().amax(2)
    if fmt == "mx":
        e = (_floor_log2(top) - 2).clamp(-127, 127)
        # in two steps, each a normal power of two
        y = blk * _pow2(-(e // 2))[..., None] * _pow2(-(e - e // 2))[..., None]
        return _e2m1(y).view(M, K).byte(), (e + 127).byte(), torch.ones((M,), device=x.device)
    frac, e = torch.frexp(top.amax(1))
    e = torch.where(frac > 0, e.int() - torch.where(frac <= 0.65625, 12, 11), -110).clamp(-110, 127)
    s = _pow2(e)
    inv = _pow2(-e)
    sf = (top * inv[:, None] / 6.0).to(torch.float8_e4m3fn)
    d = sf.float()[..., None]
    y = torch.where(d > 0, blk * inv[:, None, None] / d, 0.0)
    return _e2m1(y).view(M, K).byte(), sf.view(torch.uint8), s


def _pack(codes):
    return codes[:, 0::2] | (codes[:, 1::2] << 4)


def _tile(scales, fmt):
    """Block scale bytes [R, G] -> tiles of 128 rows x 4 blocks, zero padded."""
    R, G = scales.shape
    rb, gb = -(-R // 128), -(-G // 4)
    p = torch.zeros((rb * 128, gb * 4), dtype=torch.uint8, device=scales.device)
    p[:R, :G] = scales
    return p.view(rb, 4, 32, gb, 4).permute(0, 3, 2, 1, 4).reshape(rb, gb, 512).contiguous()


def _untile(sf, R, G):
    rb, gb, _ = sf.shape
    return sf.view(rb, gb, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rb * 128, gb * 4)[:R, :G]


def _scale_values(b, fmt):
    return _pow2(b.int() - 127) if fmt == "mx" else b.contiguous().view(torch.float8_e4m3fn).float()


def _values(codes, scales, fmt):
    """What the codes stand for, without the row scale: fp32 [R, K]."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    R, K = codes.shape
    d = _scale_values(scales, fmt)
    return (lut[codes.int()].view(R, d.shape[1], -1) * d[..., None]).view(R, K)


def _act8(x):
    """(int8 codes [M, K], scale bytes [ceil(M / 32), K])."""
    x = x.float()
    M, K = x.shape
    p = torch.zeros((-(-M // 32) * 32, K), device=x.device)
    p[:M] = x
    blk = p.view(-1, 32, K)
    e = _floor_log2(blk.abs().amax(1)).clamp(-127, 127)
    up = 6 - e
    y = blk * _pow2(up // 2)[:, None] * _pow2(up - up // 2)[:, None]
    return y.round().clamp(-127, 127).to(torch.int8).view(-1, K), (e + 127).byte()


def _act8_layout(q):
    return q.view(q.shape[0] // 16, 16, q.shape[1]).transpose(1, 2).contiguous()


def _act8_values(codes, scales, M):
    G, K, _ = codes.shape
    q = codes.transpose(1, 2).reshape(G // 2, 32, K).float()
    return (q * _pow2(scales.int() - 133)[:, None]).view(-1, K)[:M]


# ---------------------------------------------------------------- one pass

def run(st):
    op = st["op"]
    if own:
        import quantized_gemm_token_b200 as dq
        if op == "linear":
            q, sf, s = dq.dq_quantize_rows_fp4(st["x"], st["fmt"])
            return dq.dq_fp4_linear(q, sf, s, st["w"], st["sfw"], st["s_col"], st["b"], fmt=st["fmt"])
        if op == "quantize":
            q, sf, s = dq.dq_quantize_rows_fp4(st["x"], st["fmt"])
            return dq.dq_fp4_dequantize(q, sf, s, fmt=st["fmt"])
        if op == "act8":
            codes, scales = dq.dq_act8_pack(st["x"])
            return dq.dq_act8_unpack(codes, scales, st["M"])
        return dq.dq_act8_weight_grad(st["dy"], st["codes"], st["scales"], out_dtype=st["out"], bias_grad=st["bias"])
    if op == "linear":
        fmt, K = st["fmt"], st["K"]
        q, b, s = _quantize(st["x"], fmt)
        w4 = torch.stack((st["w"] & 15, st["w"] >> 4), 2).view(st["N"], K)
        w = _values(w4, _untile(st["sfw"], st["N"], K // (32 if fmt == "mx" else 16)), fmt)
        y = _values(q, b, fmt) @ w.T
        if fmt == "nv":
            y = y * s[:, None] * st["s_col"]
        if st["b"] is not None:
            y = y + st["b"].float()
        return y.bfloat16()
    if op == "quantize":
        q, b, s = _quantize(st["x"], st["fmt"])
        return (_values(q, b, st["fmt"]) * s[:, None]).bfloat16()
    if op == "act8":
        q, e = _act8(st["x"])
        return _act8_values(_act8_layout(q), e, st["M"]).bfloat16()
    x = _act8_values(st["codes"], st["scales"], st["M"])
    dy = st["dy"].float()
    dw = dy.T @ x
    dw = dw.bfloat16() if st["out"] == "bf16" else dw
    return (dw, dy.sum(0)) if st["bias"] else (dw, None)


def work(case):
    op, M, K = case["op"], case["M"], case["K"]
    per = 2.0 if op not in ("linear", "quantize") else 0.5 + (1 / 32 if case["fmt"] == "mx" else 1 / 16)
    if op == "linear":
        N = case["N"]
        return {"bytes": 2 * M * K + per * N * K + 2 * M * N, "flops": 2 * M * N * K}
    if op == "quantize":
        return {"bytes": 2 * M * K + 2 * M * K, "flops": 4 * M * K}
    if op == "act8":
        return {"bytes": 2 * M * K + 2 * M * K, "flops": 4 * M * K}
    N = case["N"]
    return {"bytes": M * K * (1 + 1 / 32) + 2 * M * N + (2 if case["out"] == "bf16" else 4) * N * K, "flops": 2 * M * N * K}


# ---------------------------------------------------------------- in 64 bits

def _exponent(v):
    """floor(log2 v) of positive fp64 values (from the bits: a rounded log2 may
    fall short of a whole number), far below every format's range for 0."""
    return torch.where(v > 0, torch.frexp(v).exponent.double() - 1, -200.0)


def _grid(v, least, digits):
    """v >= 0 to the nearest number of `digits` significant bits, the spacing
    no finer than 2^least; ties to even."""
    step = torch.exp2(torch.clamp(_exponent(v) - (digits - 1), min=least))
    return torch.round(v / step) * step


def _exact_fp4(x, fmt):
    """The values that the 4-bit codes of x stand for, in fp64."""
    x = x.double()
    M, K = x.shape
    if fmt == "mx":
        b = x.reshape(M, K // 32, 32)
        top = b.abs().amax(2, keepdim=True)
        scale = torch.exp2(torch.clamp(_exponent(top) - 2, -127, 127))
    else:
        b = x.reshape(M, K // 16, 16)
        row = x.abs().amax(1)
        r = row / 2688
        s = torch.exp2(torch.clamp(_exponent(r) + (torch.exp2(_exponent(r)) < r), min=-110))
        scale = _grid(b.abs().amax(2, keepdim=True) / (6 * s[:, None, None]), -9, 4) * s[:, None, None]
    v = torch.where(scale > 0, b.abs() / scale, 0.0)
    return (torch.sign(b) * torch.clamp(_grid(v, -1, 2), max=6.0) * scale).reshape(M, K)


def _exact_act8(x):
    x = x.double()
    M, K = x.shape
    p = torch.nn.functional.pad(x, (0, 0, 0, -M % 32)).reshape(-1, 32, K)
    top = p.abs().amax(1, keepdim=True)
    scale = torch.exp2(torch.clamp(_exponent(top), -127, 127) - 6)
    return (torch.clamp(torch.round(p / scale), -127, 127) * scale).reshape(-1, K)[:M]


def exact(case, seed):
    g = _gen(seed)
    op, M, K = case["op"], case["M"], case["K"]
    x = _activations(g, M, K, case.get("pad", 0))
    if op == "linear":
        w = _exact_fp4(_weight(g, case["N"], K), case["fmt"])
        y = _exact_fp4(x, case["fmt"]) @ w.T
        if case["bias"]:
            y = y + torch.randn((case["N"],), generator=g, device="cuda").mul_(0.1).bfloat16().double()
        return y
    if op == "quantize":
        return _exact_fp4(x, case["fmt"])
    if op == "act8":
        return _exact_act8(x)
    xh = _exact_act8(x)
    dy = (torch.randn((M, case["N"] + case["pad"]), generator=g, device="cuda") * 0.05).bfloat16()[:, :case["N"]].double()
    dw = dy.T @ xh
    return (dw, dy.sum(0)) if case["bias"] else (dw, None)
