// fp4_quant.cu -- microscaled 4-bit floating point (e2m1): quantization of
// bf16 rows and fp32 weights, dequantization, and the tiling of block scales.
//
// Formats (OCP Microscaling Formats v1.0 for "mx"; the two-level block-16
// e4m3 form for "nv"):
//   MX  blocks of 32 features, ue8m0 scale byte E = floor(log2 a) - 2 + 127
//       (a the block's largest magnitude, E clamped to 0..254), code =
//       e2m1(x / 2^(E - 127)), nearest, ties to even, saturating at 6.
//   NV  per row s = the least power of two with max|row| <= 2688 s (2688 =
//       6 * 448), at least 2^-110; blocks of 16 features, ue4m3 scale d =
//       e4m3(fp32(a / s / 6)), code = e2m1(x / (d s)) (0 where d = 0).
// The row scale is a power of two so that x / s is exact and a code depends
// on the exact quotient alone, where a general fp32 scale would round x / (d s)
// twice.  It gives up little: the e4m3 block scale takes up a factor below 2,
// but for the row's largest block, which a free scale max|row| / 2688 would give
// the scale 448 exactly (relative error of a row, against a free scale: normal
// values 9.50 % and 9.50 %, with 1 % of features twenty times larger 9.10 % and
// 8.97 %, two features of 1024 a hundred times larger 6.0 % and 5.5 %).
// A block (MX) or row (NV) that holds a NaN or an infinity gets the scale NaN
// (E = 255; s = NaN with block scales and codes 0), so everything computed with
// its scales is NaN.
//
// Both are bound by HBM: one pass over x, 0.53 or 0.56 bytes written for 2
// read.  A row stays in registers between the row maximum and the codes.
// Measured, 16384 x 8192: nv 53.3 us (6.45 TB/s, 1.00 of the measured copy
// rate), mx 49.0 us (6.94 TB/s; the mix reads more than it writes); fp32
// weights, 28672 x 8192: 151 us (7.1 TB/s), nv and mx.
#include <cuda_bf16.h>

#include "internal.h"
#include "mx.h"
#include "sm100.cuh"

namespace dq {
namespace {

// Eight fp32 values -> eight e2m1 codes (value 2i in the low nibble of byte
// i), nearest with ties to even, saturating.
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

__device__ __forceinline__ uint32_t e4m3_byte(float v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(v));
  return r & 0xffu;
}
__device__ __forceinline__ float e4m3_value(uint32_t byte) {
  uint32_t h2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<uint16_t>(byte)));
  float f;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.f32.f16 %0, lo;\n\t}" : "=f"(f) : "r"(h2));
  return f;
}

// 2^e for -149 <= e <= 127, from its bits.
__device__ __forceinline__ float pow2i(int e) {
  return e >= -126 ? __uint_as_float(static_cast<uint32_t>(e + 127) << 23)
                   : __uint_as_float(1u << (e + 149));
}

// Scale byte and the factor that takes x to its code's range, for a block of
// largest magnitude `a` (fp32 bits, any payload for NaN).
__device__ __forceinline__ uint32_t mx_scale(uint32_t abits, float& inv) {
  if (abits >= 0x7f800000u) {
    inv = 0.0f;
    return 255u;
  }
  // floor(log2 a): subnormals (and 0) lie below every clamped scale
  const int e = max(static_cast<int>(abits >> 23) - 2, 0);
  inv = pow2i(127 - e);
  return static_cast<uint32_t>(e);
}

// log2 of the NV row scale for the row's largest magnitude (fp32 bits, finite).
__device__ __forceinline__ int nv_row_exp(uint32_t abits) {
  // a = 1.f * 2^e <= 2688 * 2^p, 2688 = 1.3125 * 2^11
  const int e = static_cast<int>(abits >> 23) - 127;
  const int p = e - ((abits & 0x7fffffu) <= 0x280000u ? 11 : 10);
  return max(p, -110);
}

// Code of one value against the scale d s of its block, |x| / s = ax exact:
// the number of rounding borders (ties to the even code) that ax passes.
// border * d has at most 7 significant bits, so every comparison is exact.
__device__ __forceinline__ uint32_t e2m1_by_borders(float ax, float d, bool neg) {
  uint32_t c = ax > 0.25f * d;
  c += ax >= 0.75f * d;
  c += ax > 1.25f * d;
  c += ax >= 1.75f * d;
  c += ax > 2.5f * d;
  c += ax >= 3.5f * d;
  c += ax > 5.0f * d;
  c = d > 0.0f ? c : 0u;
  return c | (neg ? 8u : 0u);
}

// ---------------------------------------------------------------- rows
// A run of 16 features: 32 bytes of bf16, 64 of fp32, as 32-bit words.
template <bool WIDE, int W>
__device__ __forceinline__ void load_run(uint32_t (&w)[W], const void* p) {
#pragma unroll
  for (int i = 0; i < W; i += 8) {
    const char* a = static_cast<const char*>(p) + 4 * i;
    if (WIDE) {
      asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3]), "=r"(w[i + 4]), "=r"(w[i + 5]),
                     "=r"(w[i + 6]), "=r"(w[i + 7])
                   : "l"(a));
    } else {
      const uint4 u = __ldcs(reinterpret_cast<const uint4*>(a)), v = __ldcs(reinterpret_cast<const uint4*>(a) + 1);
      w[i] = u.x, w[i + 1] = u.y, w[i + 2] = u.z, w[i + 3] = u.w;
      w[i + 4] = v.x, w[i + 5] = v.y, w[i + 6] = v.z, w[i + 7] = v.w;
    }
  }
}

// Register-resident: 2^tpr_log2 (8..256) threads own a row, up to VPT runs of
// 16 features each: an NV block is one run, an MX block two neighbouring lanes'.
//
// For NV and bf16 rows, two roundings are decided without a division, both because
// bf16 has 8 significant bits.  (1) The e4m3 scale of t / 6, t = a / s exact: a rounding
// border B of e4m3 has 5 significant bits and 6 B at most 7, so t / 6 is either
// exactly a border or at least 2^-8 (relative) away from it; t * fp32(1/6) is
// within 2^-23 of t / 6, so rounding it to 12 significant bits restores the
// borders exactly and moves nothing across one.  (2) The code of x / (s d):
// the product with c = 1 / (s d) (approximate reciprocal) is within 2^-22 of
// the quotient X / d, X = x / s; border * d has at most 7 significant bits, so
// X / d is a border or at least 2^-10 away from it (2^-8 relative, the least
// border being 1/4), and rounding to a multiple of 2^-10 (adding and
// subtracting 1.5 * 2^13) again restores ties and crosses nothing.
//
// fp32 rows: the block's scale by a division; the code from the fp32 quotient X / d with
// Markstein's correction (q = X c, c = fp32(1 / d); r = X - q d, exact; q + r c), which is
// RN(X / d (1 + e)), |e| < 2^-45.  A border B is met only if X / d is B: else
// X differs from B d (at most 7 significant bits) by at least its own last
// place, so X / d is 2 / m (m < 1.9 the mantissa of d) half places or more away from B.
template <typename T, bool NV, int VPT, bool WIDE>
__global__ void __launch_bounds__(256) fp4_rows_kernel(const T* __restrict__ x, int64_t M, int64_t K,
                                                       int64_t ldx, uint8_t* __restrict__ q, int64_t ldq,
                                                       uint8_t* __restrict__ sf, int64_t sf_atoms,
                                                       float* __restrict__ s_row, int tpr_log2) {
  constexpr bool F32 = sizeof(T) == 4;
  constexpr int W = F32 ? 16 : 8;
  griddep_launch_dependents();
  griddep_wait();
  const int tpr = 1 << tpr_log2;
  const int t = threadIdx.x & (tpr - 1);
  const int r_local = threadIdx.x >> tpr_log2;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (256 >> tpr_log2) + r_local;
  const int nu = static_cast<int>(K / 16);
  const bool in = row < M;               // rows up to the next multiple of 128 get zero scales
  __shared__ uint32_t warp_max[8];

  uint32_t v[VPT][W];
  const T* xr = x + row * ldx;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int u = t + i * tpr;
#pragma unroll
    for (int j = 0; j < W; ++j) v[i][j] = 0u;
    if (in && u < nu) load_run<WIDE>(v[i], xr + u * 16);
  }
  // magnitudes order like their bits, NaN above infinity above the rest
  uint32_t top[VPT];
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    uint32_t b;
    if constexpr (F32) {
      b = v[i][0] & 0x7fffffffu;
#pragma unroll
      for (int j = 1; j < W; ++j) b = max(b, v[i][j] & 0x7fffffffu);
    } else {
      uint32_t m = v[i][0] & 0x7fff7fffu;
#pragma unroll
      for (int j = 1; j < W; ++j) m = __vmaxu2(m, v[i][j] & 0x7fff7fffu);
      b = max(m & 0xffffu, m >> 16) << 16;
    }
    if (!NV) b = max(b, __shfl_xor_sync(0xffffffffu, b, 1));
    top[i] = b;                          // fp32 bits
    amax = max(amax, b);
  }
  float inv_s = 1.0f;
  bool bad_row = false;
  if constexpr (NV) {
    if (tpr >= 32) amax = __reduce_max_sync(0xffffffffu, amax);
    else
      for (int o = tpr >> 1; o > 0; o >>= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (tpr > 32) {
      const int warp = threadIdx.x >> 5;
      if ((threadIdx.x & 31) == 0) warp_max[warp] = amax;
      __syncthreads();
      const int wpr = tpr >> 5;
      amax = 0;
      for (int w = 0; w < wpr; ++w) amax = max(amax, warp_max[r_local * wpr + w]);
    }
    bad_row = amax >= 0x7f800000u;
    const int p = nv_row_exp(amax);
    inv_s = pow2i(-p);
    if (t == 0 && in) s_row[row] = bad_row ? __uint_as_float(0x7fc00000u) : pow2i(p);
  }
  const int64_t srow_off = (row >> 7) * sf_atoms * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4;
  uint8_t* qr = q + row * ldq;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int u = t + i * tpr;
    uint32_t byte;
    float c = 0.0f, d = 0.0f;
    bool zero;
    if constexpr (NV) {
      const float a = __uint_as_float(top[i]) * inv_s;
      uint32_t r;
      if constexpr (F32) r = __float_as_uint(__fdiv_rn(a, 6.0f));
      else r = (__float_as_uint(a * (1.0f / 6.0f)) + 0x800u) & 0xfffff000u;
      byte = bad_row ? 0u : e4m3_byte(__uint_as_float(r));
      zero = byte == 0;
      d = e4m3_value(byte);
      if constexpr (F32) {
        c = __frcp_rn(d);
      } else {
        float rcp;
        asm("rcp.approx.f32 %0, %1;" : "=f"(rcp) : "f"(d));
        c = zero ? 0.0f : rcp * inv_s;
      }
    } else {
      byte = mx_scale(top[i], c);
      zero = byte == 255u;
    }
    uint32_t codes[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint64_t c2 = pack_f2(c, c), up = pack_f2(12288.0f, 12288.0f), down = pack_f2(-12288.0f, -12288.0f);
      float y[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint64_t p;
        if constexpr (F32) {
          p = pack_f2(__uint_as_float(v[i][8 * h + 2 * j]), __uint_as_float(v[i][8 * h + 2 * j + 1]));
          if constexpr (NV) {
            const uint64_t X = mul_f2(p, pack_f2(inv_s, inv_s)), quot = mul_f2(X, c2);
            p = fma_f2(fma_f2(quot, pack_f2(-d, -d), X), c2, quot);
          } else {
            p = mul_f2(p, c2);
          }
        } else {
          const uint32_t w = v[i][4 * h + j];
          p = pack_f2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
          p = NV ? add_f2(fma_f2(p, c2, up), down) : mul_f2(p, c2);
        }
        unpack_f2(p, y[2 * j], y[2 * j + 1]);
      }
      codes[h] = zero ? 0u : e2m1x8(y);
    }
    // four neighbouring blocks' scale bytes as one word (an MX block's two lanes hold the same byte)
    uint32_t word = u < nu ? byte << (8 * ((NV ? u : u >> 1) & 3)) : 0u;
    word |= __shfl_xor_sync(0xffffffffu, word, NV ? 1 : 2);
    word |= __shfl_xor_sync(0xffffffffu, word, NV ? 2 : 4);
    if (u < nu) {
      if (in) *reinterpret_cast<uint2*>(qr + static_cast<int64_t>(u) * 8) = make_uint2(codes[0], codes[1]);
      if ((u & (NV ? 3 : 7)) == 0)
        *reinterpret_cast<uint32_t*>(sf + srow_off + static_cast<int64_t>(u >> (NV ? 2 : 3)) * 512) = in ? word : 0u;
    }
  }
}

template <typename T>
__device__ __forceinline__ float elem_f32(const T* p);
template <>
__device__ __forceinline__ float elem_f32<uint16_t>(const uint16_t* p) {
  return __uint_as_float(static_cast<uint32_t>(*p) << 16);
}
template <>
__device__ __forceinline__ float elem_f32<float>(const float* p) {
  return *p;
}

// Any stride, alignment or row length: one CTA per row, two
// passes over the row (the second from L2).  A thread takes one group of four
// blocks at a time, so a scale word has one writer.
template <typename T, bool NV>
__global__ void __launch_bounds__(256) fp4_generic_kernel(const T* __restrict__ x, int64_t M, int64_t rows,
                                                          int64_t K, int64_t ldx, uint8_t* __restrict__ q,
                                                          int64_t ldq, uint8_t* __restrict__ sf, int64_t sf_atoms,
                                                          float* __restrict__ s_row) {
  constexpr int B = NV ? 16 : 32;
  __shared__ uint32_t warp_max[8];
  griddep_launch_dependents();
  griddep_wait();
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const bool in = row < M;
    const T* xr = x + row * ldx;
    uint32_t amax = 0;
    if (NV) {
      if (in)
        for (int64_t k = threadIdx.x; k < K; k += 256) amax = max(amax, __float_as_uint(elem_f32(xr + k)) & 0x7fffffffu);
      amax = __reduce_max_sync(0xffffffffu, amax);
      __syncthreads();                   // the previous row's maxima have been read
      if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = amax;
      __syncthreads();
      for (int w = 0; w < 8; ++w) amax = max(amax, warp_max[w]);
    }
    const bool bad_row = amax >= 0x7f800000u;
    const int p = nv_row_exp(amax);
    const float inv_s = NV ? pow2i(-p) : 1.0f;
    if (NV && threadIdx.x == 0 && in) s_row[row] = bad_row ? __uint_as_float(0x7fc00000u) : pow2i(p);
    uint8_t* qr = q + row * ldq;
    for (int64_t g = threadIdx.x; g < sf_atoms; g += 256) {
      uint32_t word = 0;
      for (int b = 0; in && b < 4; ++b) {
        const int64_t k0 = (g * 4 + b) * B;
        if (k0 >= K) break;
        uint32_t top = 0;
        for (int j = 0; j < B; ++j) top = max(top, __float_as_uint(elem_f32(xr + k0 + j)) & 0x7fffffffu);
        uint32_t byte;
        float c = 0.0f, d = 0.0f;
        if (NV) {
          byte = bad_row ? 0u : e4m3_byte(__fdiv_rn(__uint_as_float(top) * inv_s, 6.0f));
          d = e4m3_value(byte);
        } else {
          byte = mx_scale(top, c);
        }
        word |= byte << (8 * b);
        for (int j = 0; j < B; j += 8) {
          uint32_t codes = 0;
          if (NV) {
            for (int u = 0; u < 8; ++u) {
              const float f = elem_f32(xr + k0 + j + u);
              codes |= e2m1_by_borders(fabsf(f) * inv_s, d, __float_as_uint(f) >> 31) << (4 * u);
            }
            if (bad_row) codes = 0;
          } else if (byte != 255u) {
            float y[8];
            for (int u = 0; u < 8; ++u) y[u] = elem_f32(xr + k0 + j + u) * c;
            codes = e2m1x8(y);
          }
          uint8_t* o = qr + (k0 + j) / 2;
          for (int u = 0; u < 4; ++u) o[u] = static_cast<uint8_t>(codes >> (8 * u));
        }
      }
      *reinterpret_cast<uint32_t*>(sf + ((row >> 7) * sf_atoms + g) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4) =
          word;
    }
  }
}

// ---------------------------------------------------------------- dequantize
// A block takes 512 runs of 16 codes, a thread two of them with all their
// loads in flight: w = bf16((e2m1 * d) * s).  The block product is exact: for
// NV in fp16 (six significant bits, 2^-10 .. 2688), two at a time.  HBM
// bound (16384 x 8192, nv: 52.5 us, 1.02 of the copy rate; 61.9 with one run
// per thread).  WIDE: a 32-byte aligned output, one store per run.
// A run's row: rows have per_row runs; inv = floor(2^64 / per_row) + 1, so
// the high half of i * inv is i / per_row for i * per_row < 2^64 (any matrix that
// fits the memory).
constexpr int DEQ_RUNS = 2;
template <bool NV, bool WIDE>
__global__ void __launch_bounds__(256) fp4_dequant_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ sf,
                                                          const float* __restrict__ s_row, int64_t n, uint32_t per_row,
                                                          uint64_t inv, int64_t sf_atoms, uint16_t* __restrict__ out) {
  griddep_launch_dependents();
  griddep_wait();
  for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * (256 * DEQ_RUNS) + threadIdx.x; i0 < n;
       i0 += static_cast<int64_t>(gridDim.x) * (256 * DEQ_RUNS)) {
    uint2 c[DEQ_RUNS];
    uint32_t byte[DEQ_RUNS];
    float s[DEQ_RUNS];
#pragma unroll
    for (int j = 0; j < DEQ_RUNS; ++j) {
      const int64_t i = i0 + 256 * j;
      if (i >= n) continue;
      const int64_t row = static_cast<int64_t>(__umul64hi(static_cast<uint64_t>(i), inv));
      const uint32_t u = static_cast<uint32_t>(i) - static_cast<uint32_t>(row) * per_row;
      c[j] = __ldcs(reinterpret_cast<const uint2*>(q + i * 8));
      const uint32_t blk = NV ? u : u >> 1;
      byte[j] = __ldg(sf + ((row >> 7) * sf_atoms + (blk >> 2)) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4 + (blk & 3));
      s[j] = s_row != nullptr ? __ldg(s_row + row) : 1.0f;
    }
#pragma unroll
    for (int j = 0; j < DEQ_RUNS; ++j) {
      const int64_t i = i0 + 256 * j;
      if (i >= n) continue;
      uint32_t d2 = 0;                     // NV: d twice, fp16
      float d = 0.0f;
      if (NV) asm("{\n\t.reg .b16 l, h;\n\tcvt.rn.f16x2.e4m3x2 %0, %1;\n\tmov.b32 {l, h}, %0;\n\tmov.b32 %0, {l, l};\n\t}" : "=r"(d2) : "h"(static_cast<uint16_t>(byte[j])));
      else d = byte[j] == 255u ? __uint_as_float(0x7fc00000u) : pow2i(static_cast<int>(byte[j]) - 127);
      const uint64_t s2 = pack_f2(s[j], s[j]), df2 = pack_f2(d, d);
      uint32_t o[8];
#pragma unroll
      for (int h = 0; h < 8; ++h) {
        const uint32_t b = ((h < 4 ? c[j].x : c[j].y) >> (8 * (h & 3))) & 0xffu;
        uint32_t h2;
        asm("{\n\t.reg .b8 t;\n\tcvt.u8.u32 t, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, t;\n\t}" : "=r"(h2) : "r"(b));
        if (NV) asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(h2) : "r"(d2));
        float lo, hi;
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
            : "=f"(lo), "=f"(hi)
            : "r"(h2));
        uint64_t p = pack_f2(lo, hi);
        if (!NV) p = mul_f2(p, df2);
        unpack_f2(mul_f2(p, s2), lo, hi);
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o[h]) : "f"(hi), "f"(lo));
      }
      uint16_t* dst = out + i * 16;
      if (WIDE) {
        asm volatile("st.global.L1::no_allocate.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(o[0]),
                     "r"(o[1]), "r"(o[2]), "r"(o[3]), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7])
                     : "memory");
      } else {
        __stcs(reinterpret_cast<uint4*>(dst), make_uint4(o[0], o[1], o[2], o[3]));
        __stcs(reinterpret_cast<uint4*>(dst) + 1, make_uint4(o[4], o[5], o[6], o[7]));
      }
    }
  }
}

// Block scales [rows, blocks] -> tiles of 128 rows x 4 blocks, zero padded.
__global__ void __launch_bounds__(256) fp4_tile_kernel(const uint8_t* __restrict__ src, int64_t rows, int64_t blocks,
                                                       int64_t atoms, int64_t total, uint8_t* __restrict__ dst) {
  griddep_launch_dependents();
  griddep_wait();
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < total; i += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t tile = i >> 9;
    const int in = static_cast<int>(i & 511);
    const int64_t r = (tile / atoms) * 128 + (in >> 4) + ((in >> 2) & 3) * 32;
    const int64_t b = (tile % atoms) * 4 + (in & 3);
    dst[i] = r < rows && b < blocks ? src[r * blocks + b] : 0;
  }
}

// Programmatic (early) launch: every kernel here executes griddep_wait()
// before its first global access.
template <typename... P, typename... A>
dq_status launch(void (*kernel)(P...), int64_t blocks, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
  return e == cudaSuccess ? DQ_OK : cuda_fail(e);
}

constexpr int64_t kMaxGrid = 1 << 20;

template <typename T, bool NV, int VPT>
auto rows_kernel(bool wide) {
  return wide ? fp4_rows_kernel<T, NV, VPT, true> : fp4_rows_kernel<T, NV, VPT, false>;
}

template <typename T, bool NV>
dq_status quantize(const T* x, int64_t M, int64_t K, int64_t ldx, uint8_t* q, int64_t ldq, uint8_t* sf, float* s_row,
                   int sm_count, cudaStream_t stream) {
  const int64_t rows = (M + 127) / 128 * 128;
  const int64_t atoms = fp4_atoms(K, NV ? DQ_FP4_NV : DQ_FP4_MX);
  constexpr int V = 16 / sizeof(T);                      // elements per 16 bytes
  if (K <= 4096 * V && ldx % V == 0 && aligned(x, 16) && ldq % 8 == 0 && aligned(q, 8)) {
    // Runs per thread: four for NV and bf16 (fewer threads share the row maximum: 16384 x 8192 53.4 us against 57.5
    // with two), two for MX (49.1 against 53.9 with four) and for fp32 (28672 x 8192 nv 151 against 179 with four),
    // more where 256 threads would not hold the row; three, or for NV and bf16 five, where that leaves fewer idle
    // places (65792 x 1280: nv 34.4 us with five, 44.3 with four; mx 33.0 with three, 37.9 with two) and still gives
    // each SM two blocks (the layer of 1799 x 1280 -> 5120 nv, whose product starts beside the last blocks: 20.2 us
    // with five, 17.5 with four).  Fewer runs where there would be fewer blocks than that (512 x 4096 nv 2.9 us, 3.2
    // with four; with its product of 4096 channels 13.1, 14.2). Short rows share a warp (65792 x 64: 5.0 us, 14.8 with
    // a warp per row).
    const int64_t nu = K / 16;
    constexpr bool four = NV && sizeof(T) == 2;
    auto threads_log2 = [nu](int v) {
      int lg = 3;
      while (lg < 8 && (static_cast<int64_t>(v) << lg) < nu) ++lg;
      return lg;
    };
    int vpt = nu <= 32 ? 1 : four && nu > 64 ? 4 : 2;
    while ((static_cast<int64_t>(vpt) << 8) < nu) vpt *= 2;
    int lg = threads_log2(vpt);
    while (vpt > 1 && vpt <= 4 && lg < 8 && rows >> (8 - lg) < 2 * sm_count) lg = threads_log2(vpt /= 2);
    for (int v = four ? 5 : 3; v >= 3 && nu > 32; v -= 2) {
      const int l = threads_log2(v);
      if ((static_cast<int64_t>(v) << l) >= nu && 10 * (v << l) < 9 * (vpt << lg) && rows >> (8 - l) >= 2 * sm_count) {
        vpt = v;
        lg = l;
      }
    }
    const int64_t blocks = (rows + (256 >> lg) - 1) / (256 >> lg);
    const bool wide = aligned(x, 32) && ldx % (2 * V) == 0;
    auto k = vpt == 1 ? rows_kernel<T, NV, 1>(wide) : vpt == 2 ? rows_kernel<T, NV, 2>(wide)
             : vpt == 3 ? rows_kernel<T, NV, 3>(wide) : rows_kernel<T, NV, 4>(wide);
    if constexpr (four) {
      if (vpt == 5) k = rows_kernel<T, NV, 5>(wide);
    }
    if constexpr (sizeof(T) == 2) {                      // (fp32 rows end at four)
      if (vpt == 8) k = rows_kernel<T, NV, 8>(wide);
    }
    return launch(k, blocks, stream, x, M, K, ldx, q, ldq, sf, atoms, s_row, lg);
  }
  return launch(fp4_generic_kernel<T, NV>, rows < kMaxGrid ? rows : kMaxGrid, stream, x, M, rows, K, ldx, q, ldq, sf,
                atoms, s_row);
}

template <typename T>
dq_status quantize_entry(const T* x, int64_t M, int64_t K, int64_t ldx, int fmt, uint8_t* q, int64_t ldq, uint8_t* sf,
                         float* s, dq_stream_t stream) {
  const bool nv = fmt == DQ_FP4_NV;
  if ((!nv && fmt != DQ_FP4_MX) || M < 0 || K < 1 || ldx < K || ldq < K / 2) return DQ_ERR_INVALID_ARG;
  if (M > 0 && (x == nullptr || q == nullptr || sf == nullptr || (nv && s == nullptr))) return DQ_ERR_INVALID_ARG;
  if (K % 32 != 0 || M > kMxMaxDim || K > kMxMaxDim) return DQ_ERR_UNSUPPORTED;
  if (!aligned(sf, 16) || !aligned(s, 4) || !aligned(x, sizeof(T))) return DQ_ERR_UNSUPPORTED;
  DeviceInfo* d = nullptr;
  const dq_status st = current_device(&d);
  if (st != DQ_OK) return st;
  if (M == 0) return DQ_OK;
  auto cs = reinterpret_cast<cudaStream_t>(stream);
  return nv ? quantize<T, true>(x, M, K, ldx, q, ldq, sf, s, d->sm_count, cs)
            : quantize<T, false>(x, M, K, ldx, q, ldq, sf, s, d->sm_count, cs);
}

}  // namespace
}  // namespace dq

using namespace dq;

extern "C" {

size_t dq_fp4_scales_size(int64_t rows, int64_t K, int fmt) {
  if ((fmt != DQ_FP4_MX && fmt != DQ_FP4_NV) || rows < 0 || K < 1 || K % 32 != 0 || rows > kMxMaxDim || K > kMxMaxDim)
    return 0;
  return static_cast<size_t>((rows + 127) / 128 * fp4_atoms(K, fmt) * 512);
}

dq_status dq_quantize_rows_fp4(const void* x_bf16, int64_t M, int64_t K, int64_t ldx, int fmt, uint8_t* q, int64_t ldq,
                               uint8_t* sf, float* s_row, dq_stream_t stream) {
  return quantize_entry(static_cast<const uint16_t*>(x_bf16), M, K, ldx, fmt, q, ldq, sf, s_row, stream);
}

dq_status dq_quantize_weight_fp4(const float* w, int64_t N, int64_t K, int64_t ldw, int fmt, uint8_t* wq, int64_t ldwq,
                                 uint8_t* sf, float* s_col, dq_stream_t stream) {
  return quantize_entry(w, N, K, ldw, fmt, wq, ldwq, sf, s_col, stream);
}

dq_status dq_fp4_dequantize(const uint8_t* q, const uint8_t* sf, const float* s, int64_t M, int64_t K, int fmt,
                            void* out_bf16, dq_stream_t stream) {
  if ((fmt != DQ_FP4_MX && fmt != DQ_FP4_NV) || M < 0 || K < 1) return DQ_ERR_INVALID_ARG;
  if (M > 0 && (q == nullptr || sf == nullptr || out_bf16 == nullptr)) return DQ_ERR_INVALID_ARG;
  if (K % 32 != 0 || M > kMxMaxDim || K > kMxMaxDim) return DQ_ERR_UNSUPPORTED;
  if (!aligned(q, 16) || !aligned(sf, 16) || !aligned(out_bf16, 16) || !aligned(s, 4)) return DQ_ERR_UNSUPPORTED;
  DeviceInfo* d = nullptr;
  const dq_status st = current_device(&d);
  if (st != DQ_OK) return st;
  if (M == 0) return DQ_OK;
  const int64_t want = (M * (K / 16) + 256 * DEQ_RUNS - 1) / (256 * DEQ_RUNS);
  const int64_t blocks = want < kMaxGrid ? want : kMaxGrid;
  auto cs = reinterpret_cast<cudaStream_t>(stream);
  const bool wide = aligned(out_bf16, 32);
  auto k = fmt == DQ_FP4_NV ? (wide ? fp4_dequant_kernel<true, true> : fp4_dequant_kernel<true, false>)
                            : (wide ? fp4_dequant_kernel<false, true> : fp4_dequant_kernel<false, false>);
  const uint64_t per_row = static_cast<uint64_t>(K / 16);   // (2 at least: K % 32 == 0)
  return launch(k, blocks, cs, q, sf, s, M * (K / 16), per_row, ~uint64_t(0) / per_row + 1, fp4_atoms(K, fmt),
                static_cast<uint16_t*>(out_bf16));
}

dq_status dq_fp4_tile_scales(const uint8_t* scales, int64_t rows, int64_t K, int fmt, uint8_t* sf, dq_stream_t stream) {
  if ((fmt != DQ_FP4_MX && fmt != DQ_FP4_NV) || rows < 0 || K < 1) return DQ_ERR_INVALID_ARG;
  if (rows > 0 && (scales == nullptr || sf == nullptr)) return DQ_ERR_INVALID_ARG;
  if (K % 32 != 0 || rows > kMxMaxDim || K > kMxMaxDim) return DQ_ERR_UNSUPPORTED;
  if (!aligned(sf, 16)) return DQ_ERR_UNSUPPORTED;
  DeviceInfo* d = nullptr;
  const dq_status st = current_device(&d);
  if (st != DQ_OK) return st;
  if (rows == 0) return DQ_OK;
  const int64_t total = static_cast<int64_t>(dq_fp4_scales_size(rows, K, fmt));
  const int64_t want = (total + 255) / 256;
  return launch(fp4_tile_kernel, want < kMaxGrid ? want : kMaxGrid, reinterpret_cast<cudaStream_t>(stream), scales, rows,
                K / (fmt == DQ_FP4_NV ? 16 : 32), fp4_atoms(K, fmt), total, sf);
}

}  // extern "C"
