// act8.cu -- 8-bit activation checkpoints: a layer's bf16 input kept for the
// backward pass in half the bytes, and read back.
//
// Format: blocks of 32 consecutive tokens of ONE feature share a ue8m0 scale
// byte E = floor(log2 a) + 127 (a the block's largest magnitude, E clamped to
// 0..254); code q = rint(64 x / 2^(E - 127)), ties to even, clamped to +-127;
// the value is q 2^(E - 133) (the element and scale types of the OCP
// Microscaling int8 format).  A block that holds a NaN or an infinity has
// E = 255 and codes 0 and reads back as NaN.
//  - Blocks run along the tokens because outliers in a layer's input sit in a
//    few features: a feature's block keeps its own scale, where a block along
//    the features would lose the 31 neighbours' low bits to the outlier.
//  - The scale is a power of two, so q 2^(E - 133) has at most 7 significant
//    bits and IS a bf16 number: the weight gradient multiplies the checkpoint
//    on the bf16 tensor cores without a further rounding.
//  - bf16 input: x 2^(133 - E) is at most 127.5, so clamping to 127 costs no
//    more than rounding does (half a step).
// Layout: codes [2 ceil(M / 32)][K][16]: 16 tokens of a feature are 16
// contiguous bytes, so the gradient kernel's thread, which owns a feature,
// reads its contraction axis in 16-byte words; scales [ceil(M / 32)][K].
// Tokens past M in the last block hold code 0.
#include <cuda_bf16.h>

#include "internal.h"
#include "mx.h"
#include "sm100.cuh"

namespace dq {
namespace {

// Single-warp blocks: the blocks tile a row exactly for more row lengths
// (2048 x 4096, unpack: 6.2 us against 7.9 with 128 threads).
constexpr int ACT8_THREADS = 32;

// 2^(E - 133) as bf16 bits, NaN for E = 255.
__device__ __forceinline__ uint32_t act8_scale_bf16(uint32_t e) {
  if (e == 255u) return 0x7fc0u;
  return e >= 7u ? (e - 6u) << 7 : 1u << e;
}

// HBM bound: 2 bytes read, 33/32 written per element (65792 x 1280: 41.0 us,
// 6.22 TB/s, 0.96 of the copy rate).  Lane l holds 8 features x 16 tokens (half l
// / 16 of the block: 16 loads of 16 bytes, half a warp covering 256 contiguous
// bytes of a row); the halves' maxima meet in one exchange, and a lane writes
// its half block as 128 contiguous bytes, 32 at a time: whole sectors
// (with 16-byte stores 49.0 us; 4 features x 32 tokens per lane 46.7).
// LOAD: bytes per load, 16 or 8 by the rows' alignment, else 2; WIDE: 32-byte
// aligned codes (as an argument instead: 43.1 us).
template <int LOAD, bool WIDE>
__global__ void __launch_bounds__(ACT8_THREADS) act8_pack_kernel(const uint16_t* __restrict__ x, int64_t M, int K,
                                                                 int64_t ldx, uint8_t* __restrict__ codes,
                                                                 uint8_t* __restrict__ scales) {
  griddep_launch_dependents();
  griddep_wait();
  const int h = threadIdx.x >> 4;
  const int k = blockIdx.x * 128 + (threadIdx.x & 15) * 8;
  const bool in = k < K;
  for (int64_t blk = blockIdx.y; blk * 32 < M; blk += gridDim.y) {
    const int64_t m0 = blk * 32 + 16 * h;
    uint4 v[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      v[j] = make_uint4(0u, 0u, 0u, 0u);
      if (in && m0 + j < M) {
        const uint16_t* p = x + (m0 + j) * ldx + k;
        if (LOAD == 16) {
          v[j] = __ldcs(reinterpret_cast<const uint4*>(p));
        } else if (LOAD == 8) {
          const uint2 a = __ldcs(reinterpret_cast<const uint2*>(p)), b = __ldcs(reinterpret_cast<const uint2*>(p) + 1);
          v[j] = make_uint4(a.x, a.y, b.x, b.y);
        } else {
          v[j].x = static_cast<uint32_t>(p[0]) | (static_cast<uint32_t>(p[1]) << 16);
          v[j].y = static_cast<uint32_t>(p[2]) | (static_cast<uint32_t>(p[3]) << 16);
          v[j].z = static_cast<uint32_t>(p[4]) | (static_cast<uint32_t>(p[5]) << 16);
          v[j].w = static_cast<uint32_t>(p[6]) | (static_cast<uint32_t>(p[7]) << 16);
        }
      }
    }
    uint32_t top[4] = {};                  // largest magnitudes of features (2i, 2i + 1)
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      top[0] = __vmaxu2(top[0], v[j].x & 0x7fff7fffu);
      top[1] = __vmaxu2(top[1], v[j].y & 0x7fff7fffu);
      top[2] = __vmaxu2(top[2], v[j].z & 0x7fff7fffu);
      top[3] = __vmaxu2(top[3], v[j].w & 0x7fff7fffu);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) top[i] = __vmaxu2(top[i], __shfl_xor_sync(0xffffffffu, top[i], 16));
    if (!in) continue;
    const uint64_t magic = pack_f2(12582912.0f, 12582912.0f);
    uint32_t bytes[2] = {};                // the scales
    uint4* dst = reinterpret_cast<uint4*>(codes + ((blk * 2 + h) * K + k) * 16);
    uint32_t even[4];
#pragma unroll
    for (int f = 0; f < 8; ++f) {
      // the codes' magnitudes are integer bits: bf16 exponent field = E (0 for
      // subnormals, whose block scale is 2^-127 like the least normal's)
      const uint32_t e = ((f & 1) ? top[f >> 1] >> 16 : top[f >> 1] & 0xffffu) >> 7;
      bytes[f >> 2] |= e << (8 * (f & 3));
      // 2^(133 - E) as two factors (one would overflow for E < 6)
      const int s = 133 - static_cast<int>(e);            // -122 .. 133
      const int s1 = s > 127 ? 127 : s;
      const float u1 = e >= 255u ? 0.0f : __uint_as_float(static_cast<uint32_t>(s1 + 127) << 23);
      const float u2 = __uint_as_float(static_cast<uint32_t>(s - s1 + 127) << 23);
      const uint64_t up = pack_f2(u1, u1), up2 = pack_f2(u2, u2);
      uint32_t w[4];
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        uint32_t c[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {      // tokens 2u, 2u + 1 of the four
          const uint4 v0 = v[4 * g + 2 * u], v1 = v[4 * g + 2 * u + 1];
          const uint32_t b0 = f < 2 ? v0.x : f < 4 ? v0.y : f < 6 ? v0.z : v0.w;
          const uint32_t b1 = f < 2 ? v1.x : f < 4 ? v1.y : f < 6 ? v1.z : v1.w;
          const uint64_t x2 = (f & 1) ? pack_f2(__uint_as_float(b0 & 0xffff0000u), __uint_as_float(b1 & 0xffff0000u))
                                      : pack_f2(__uint_as_float(b0 << 16), __uint_as_float(b1 << 16));
          // the scaling is exact; adding 1.5 * 2^23 leaves rint(y), -128 .. 128, in the low 16 bits
          const uint64_t t = add_f2(mul_f2(mul_f2(x2, up), up2), magic);
          const uint32_t r = __byte_perm(static_cast<uint32_t>(t), static_cast<uint32_t>(t >> 32), 0x5410);
          c[u] = __vmaxs2(__vmins2(r, 0x007f007fu), 0xff81ff81u);
        }
        w[g] = e >= 255u ? 0u : __byte_perm(c[0], c[1], 0x6420);
      }
      if (f & 1) {
        if (WIDE) {
          asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst + f - 1), "r"(even[0]),
                       "r"(even[1]), "r"(even[2]), "r"(even[3]), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                       : "memory");
        } else {
          dst[f - 1] = make_uint4(even[0], even[1], even[2], even[3]);
          dst[f] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      } else {
#pragma unroll
        for (int g = 0; g < 4; ++g) even[g] = w[g];
      }
    }
    if (h == 0) *reinterpret_cast<uint2*>(scales + blk * K + k) = make_uint2(bytes[0], bytes[1]);
  }
}

// Two bf16 values q * scale from two codes held as 16-bit lanes of `u` (the
// byte in each lane's low 8 bits): 128 + low 7 bits and -128 (or -256 for a
// negative code) are exact bf16 numbers made from the bits, their sum is the
// code, and the product with a power of two is exact.
__device__ __forceinline__ uint32_t act8_pair(uint32_t u, uint32_t s2) {
  const uint32_t a = (u & 0x007f007fu) | 0x43004300u;
  const uint32_t b = (u & 0x00800080u) | 0xc300c300u;
  uint32_t q, r;
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(q) : "r"(a), "r"(b));
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(q), "r"(s2));
  return r;
}

// A thread restores 8 features x 16 tokens: eight 16-byte loads, a register
// transpose by byte selection, sixteen 16-byte stores (512 contiguous bytes
// of a row per warp).  HBM bound (65792 x 1280: 40.0 us, 0.99 of the copy rate).
__global__ void __launch_bounds__(ACT8_THREADS) act8_unpack_kernel(const uint8_t* __restrict__ codes,
                                                          const uint8_t* __restrict__ scales, int64_t M, int K,
                                                          uint16_t* __restrict__ out) {
  griddep_launch_dependents();
  griddep_wait();
  const int k = (blockIdx.x * ACT8_THREADS + threadIdx.x) * 8;
  if (k >= K) return;
  for (int64_t half = blockIdx.y; half * 16 < M; half += gridDim.y) {
    uint4 c[8];
    const uint4* src = reinterpret_cast<const uint4*>(codes + (half * K + k) * 16);
#pragma unroll
    for (int f = 0; f < 8; ++f) c[f] = __ldcs(src + f);
    const uint2 e = *reinterpret_cast<const uint2*>(scales + (half >> 1) * K + k);
    uint32_t s2[4];                        // scale pairs of features (2i, 2i + 1)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = (i < 2 ? e.x : e.y) >> (16 * (i & 1));
      s2[i] = act8_scale_bf16(w & 0xffu) | (act8_scale_bf16((w >> 8) & 0xffu) << 16);
    }
#pragma unroll
    for (int t = 0; t < 16; ++t) {
      if (half * 16 + t < M) {
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 a = c[2 * i], b = c[2 * i + 1];
          const uint32_t wa = t < 4 ? a.x : t < 8 ? a.y : t < 12 ? a.z : a.w;
          const uint32_t wb = t < 4 ? b.x : t < 8 ? b.y : t < 12 ? b.z : b.w;
          const uint32_t j = t & 3;
          // lanes: byte j of feature 2i, byte j of feature 2i + 1 (upper bytes ignored)
          o[i] = act8_pair(__byte_perm(wa, wb, j | (j << 4) | ((4 + j) << 8) | ((4 + j) << 12)), s2[i]);
        }
        __stcs(reinterpret_cast<uint4*>(out + (half * 16 + t) * K + k), make_uint4(o[0], o[1], o[2], o[3]));
      }
    }
  }
}

template <typename... P, typename... A>
dq_status launch(void (*kernel)(P...), dim3 grid, int threads, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
  return e == cudaSuccess ? DQ_OK : cuda_fail(e);
}

}  // namespace
}  // namespace dq

using namespace dq;

extern "C" {

size_t dq_act8_codes_size(int64_t M, int64_t K) {
  if (M < 0 || K < 1 || M > kMxMaxDim || K > kMxMaxDim) return 0;
  return static_cast<size_t>((M + 31) / 32 * 32 * K);
}

size_t dq_act8_scales_size(int64_t M, int64_t K) {
  if (M < 0 || K < 1 || M > kMxMaxDim || K > kMxMaxDim) return 0;
  return static_cast<size_t>((M + 31) / 32 * K);
}

dq_status dq_act8_pack(const void* x_bf16, int64_t M, int64_t K, int64_t ldx, int8_t* codes, uint8_t* scales,
                       dq_stream_t stream) {
  if (M < 0 || K < 1 || ldx < K) return DQ_ERR_INVALID_ARG;
  if (M > 0 && (x_bf16 == nullptr || codes == nullptr || scales == nullptr)) return DQ_ERR_INVALID_ARG;
  if (K % 16 != 0 || M > kMxMaxDim || K > kMxMaxDim) return DQ_ERR_UNSUPPORTED;
  if (!aligned(x_bf16, 2) || !aligned(codes, 16) || !aligned(scales, 16)) return DQ_ERR_UNSUPPORTED;
  DeviceInfo* d = nullptr;
  const dq_status st = current_device(&d);
  if (st != DQ_OK) return st;
  if (M == 0) return DQ_OK;
  const int64_t blks = (M + 31) / 32;
  const dim3 grid(static_cast<unsigned>((K + 127) / 128), static_cast<unsigned>(blks < 65535 ? blks : 65535));
  auto k = aligned(x_bf16, 16) && ldx % 8 == 0 ? (aligned(codes, 32) ? act8_pack_kernel<16, true> : act8_pack_kernel<16, false>)
           : aligned(x_bf16, 8) && ldx % 4 == 0 ? act8_pack_kernel<8, false>
                                                : act8_pack_kernel<2, false>;
  return launch(k, grid, ACT8_THREADS, reinterpret_cast<cudaStream_t>(stream),
                static_cast<const uint16_t*>(x_bf16), M, static_cast<int>(K), ldx, reinterpret_cast<uint8_t*>(codes),
                scales);
}

dq_status dq_act8_unpack(const int8_t* codes, const uint8_t* scales, int64_t M, int64_t K, void* out_bf16,
                         dq_stream_t stream) {
  if (M < 0 || K < 1) return DQ_ERR_INVALID_ARG;
  if (M > 0 && (out_bf16 == nullptr || codes == nullptr || scales == nullptr)) return DQ_ERR_INVALID_ARG;
  if (K % 16 != 0 || M > kMxMaxDim || K > kMxMaxDim) return DQ_ERR_UNSUPPORTED;
  if (!aligned(out_bf16, 16) || !aligned(codes, 16) || !aligned(scales, 16)) return DQ_ERR_UNSUPPORTED;
  DeviceInfo* d = nullptr;
  const dq_status st = current_device(&d);
  if (st != DQ_OK) return st;
  if (M == 0) return DQ_OK;
  const int64_t halves = (M + 15) / 16;
  const dim3 grid(static_cast<unsigned>((K / 8 + ACT8_THREADS - 1) / ACT8_THREADS), static_cast<unsigned>(halves < 65535 ? halves : 65535));
  return launch(act8_unpack_kernel, grid, ACT8_THREADS, reinterpret_cast<cudaStream_t>(stream),
                reinterpret_cast<const uint8_t*>(codes), scales, M, static_cast<int>(K),
                static_cast<uint16_t*>(out_bf16));
}

}  // extern "C"
