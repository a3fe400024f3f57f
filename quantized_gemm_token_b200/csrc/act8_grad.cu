// act8_grad.cu -- the gradients of a linear layer's weight and bias from the
// 8-bit checkpoint of its input (act8.cu describes the format):
//     dW[n, k] = sum_m dY[m, n] x8[m, k],   db[n] = sum_m dY[m, n],
// x8 = q 2^(E - 133).  Both factors are bf16 numbers, so the product runs on
// the bf16 tensor cores (tcgen05.mma kind::f16, fp32 accumulators) without any
// rounding before the sum.
//
// The contraction runs over the tokens, the slow axis of both operands:
//  - dY is loaded as it lies ([token][channel], 128B-swizzled boxes of 64
//    channels) and taken MN-major by the tensor core: no transposition.
//  - the checkpoint is the A operand, in TENSOR MEMORY: a converting thread
//    owns one feature (a TMEM lane), reads 16 of its tokens per 16-byte word
//    and writes them as bf16 pairs along its lane.  Keeping A out of shared
//    memory saves its write and the tensor core's read (2 x 16 KB per 64
//    tokens x 128 features), the bound of the kernels here that build an
//    operand in shared memory.
// Roles (448 threads): warp 0 TMA producer; warp 1 MMA issuer; warps 2..9
// converters, two groups of four taking alternate 64-token steps; warps
// 10..13 epilogue (lane = feature, column = channel).
// Few tiles: the tokens are split over a cluster of up to 8 CTAs whose fp32
// partial tiles are added through distributed shared memory in split order
// (no workspace, no atomics).
#include <cuda_bf16.h>
#include <cudaTypedefs.h>

#include <algorithm>

#include "gemm_common.cuh"
#include "internal.h"
#include "pipeline.cuh"
#include "sm100.cuh"

namespace dq {
namespace {

constexpr int WG_GROUPS = 3;                 // converter groups
constexpr int WG_CVT_WARPS = 4;              // per group
constexpr int WG_EPI_WARP0 = 2 + WG_GROUPS * WG_CVT_WARPS;
constexpr int WG_THREADS = 32 * (WG_EPI_WARP0 + 4);
constexpr int WG_STEP = 64;                  // tokens per step
constexpr int WG_CODES = 128 * WG_STEP;      // bytes: [4 x 16 tokens][128 features][16]
constexpr int WG_MAX_STAGES = 12;
constexpr int WG_BAR_BYTES = 512;
constexpr int WG_OUT_BUF = 4096;             // 32 x 32 fp32, or two 32 x 32 bf16
constexpr int WG_SLOT_COLS = WG_STEP / 2;    // TMEM columns of one converted step
constexpr int64_t kGradMaxDim = int64_t(1) << 30;

struct GradArgs {
  int M, N, K;
  int bn;                  // channels per tile (multiple of 64)
  int kt, nt;              // feature tiles (128), channel tiles
  int splits, units;
  int ks;                  // token steps: ceil(M / 64)
  int stages;
  int accs, acc_cols;      // accumulator buffers and their TMEM columns
  int slots, slot_col;     // converted-step slots and their first column
  int full_chunks;         // N / 64: chunks the 3-D map covers
  uint32_t off_out, off_bar;
  void* dw;
  int f32, accumulate;
  WaitCtl wait;
};

// kind::f16, bf16 A (tensor memory, K-major) and B (shared memory, MN-major),
// fp32 accumulator.
__host__ __device__ constexpr uint32_t idesc_grad(int N) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | (static_cast<uint32_t>(N >> 3) << 17) | (8u << 24);
}

__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// MN-major operand of 64-element (128-byte) chunks, 128B-swizzled: rows of one
// contraction index, 8-row groups 1024 B apart (stride), chunks `chunk` bytes
// apart (leading dimension).
__device__ __forceinline__ uint64_t smem_desc_mn(uint32_t addr, uint32_t chunk) {
  return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(chunk >> 4) << 16) |
         (static_cast<uint64_t>(1024u >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* tmap, uint32_t bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// dW += the staged fp32 block (each element has one writer per call).
__device__ __forceinline__ void tma_add_2d(const void* tmap, uint32_t src, int x, int y) {
  asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(tmap)),
               "r"(src), "r"(x), "r"(y)
               : "memory");
}

__device__ __forceinline__ void tmem_st_32x32b_x32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Two bf16 values q * scale from two codes, the bytes at bits 0 and 16 of `u`:
// 128 + low 7 bits and -128 (-256 for a negative code) are exact bf16 numbers
// made from the bits, their sum is the code, the product with a power of two
// is exact.
__device__ __forceinline__ uint32_t code_pair(uint32_t u, uint32_t s2) {
  const uint32_t a = (u & 0x007f007fu) | 0x43004300u;
  const uint32_t b = (u & 0x00800080u) | 0xc300c300u;
  uint32_t q, r;
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(q) : "r"(a), "r"(b));
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(q), "r"(s2));
  return r;
}
// 2^(E - 133) twice, NaN for E = 255.
__device__ __forceinline__ uint32_t code_scale2(uint32_t e) {
  const uint32_t b = e == 255u ? 0x7fc0u : e >= 7u ? (e - 6u) << 7 : 1u << e;
  return b | (b << 16);
}

struct GradUnit {
  int split, kt, nt, s0, s1;
};
__device__ __forceinline__ GradUnit grad_unit(const GradArgs& g, int u) {
  GradUnit t;
  const int tile = u / g.splits;
  t.split = u - tile * g.splits;
  t.nt = tile / g.kt;
  t.kt = tile - t.nt * g.kt;
  t.s0 = static_cast<int>(static_cast<int64_t>(t.split) * g.ks / g.splits);
  t.s1 = static_cast<int>(static_cast<int64_t>(t.split + 1) * g.ks / g.splits);
  return t;
}

__global__ void __launch_bounds__(WG_THREADS, 1)
    act8_grad_kernel(const __grid_constant__ CUtensorMap tm_y3, const __grid_constant__ CUtensorMap tm_y2,
                     const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_e,
                     const __grid_constant__ CUtensorMap tm_c, const GradArgs g) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const smem = smem_raw + (base - raw);
  // stage: dY (bn / 64 chunks of 64 tokens x 128 B), codes, scales [2][128]
  const uint32_t y_bytes = static_cast<uint32_t>(g.bn) * 128u;
  const uint32_t stage_bytes = y_bytes + WG_CODES + 1024u;
  uint64_t* const full = reinterpret_cast<uint64_t*>(smem + g.off_bar);
  uint64_t* const cvt = full + WG_MAX_STAGES;
  uint64_t* const empty = cvt + WG_MAX_STAGES;
  uint64_t* const accf = empty + WG_MAX_STAGES;
  uint64_t* const acce = accf + 2;
  uint64_t* const drain = acce + 2;
  uint32_t* const tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < g.stages; ++i) {
      mbar_init(smem_u32(full + i), 1);
      mbar_init(smem_u32(cvt + i), WG_CVT_WARPS);
      mbar_init(smem_u32(empty + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(accf + i), 1);
      mbar_init(smem_u32(acce + i), 4);
    }
    mbar_init(smem_u32(drain), 1);
    fence_barrier_init();
    tma_prefetch_desc(&tm_y3);
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_e);
    tma_prefetch_desc(&tm_c);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_holder), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  griddep_launch_dependents();
  griddep_wait();

  if (warp == 0) {
    // ---------------------------------------------------------- producer
    int stage = 0;
    uint32_t phase = 0;
    long long issued = 0;
    bool ok = true;
    const int chunks = g.bn / 64;
    for (int u = blockIdx.x; ok && u < g.units; u += gridDim.x) {
      const GradUnit t = grad_unit(g, u);
      const int c0 = t.nt * chunks;
      // the 3-D map covers whole chunks only: a tile that holds the ragged last one is loaded chunk by chunk
      const bool whole = c0 + chunks <= g.full_chunks || g.N % 64 == 0;
      for (int s = t.s0; s < t.s1; ++s) {
        if (!mbar_wait_warp(smem_u32(empty + stage), phase ^ 1, g.wait, abort_flag)) {
          ok = false;
          break;
        }
        const uint32_t fb = smem_u32(full + stage);
        const uint32_t sy = base + static_cast<uint32_t>(stage) * stage_bytes;
        if (elect_one()) {
          mbar_arrive_expect_tx(fb, y_bytes + WG_CODES + 256u);
          tma_load_2d(sy + y_bytes, &tm_q, fb, t.kt * 256, s * 4);
          tma_load_2d(sy + y_bytes + WG_CODES, &tm_e, fb, t.kt * 128, s * 2);
          if (whole)
            tma_load_3d(sy, &tm_y3, fb, 0, s * WG_STEP, c0);
          else
            for (int c = 0; c < chunks; ++c)
              tma_load_2d(sy + static_cast<uint32_t>(c) * 8192u, &tm_y2, fb, (c0 + c) * 64, s * WG_STEP);
        }
        __syncwarp();
        ++issued;
        if (++stage == g.stages) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    volatile int never = 0;
    for (long long i = issued > g.stages ? issued - g.stages : 0; i < issued; ++i)
      pipe::wait(smem_u32(full + static_cast<int>(i % g.stages)), static_cast<uint32_t>((i / g.stages) & 1), g.wait,
                 &never);
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    const uint32_t idesc = idesc_grad(g.bn);
    int stage = 0, acc = 0, slot = 0;
    uint32_t phase = 0, aphase = 0;
    bool ok = true;
    for (int u = blockIdx.x; ok && u < g.units; u += gridDim.x) {
      const GradUnit t = grad_unit(g, u);
      if (!mbar_wait_warp(smem_u32(acce + acc), aphase ^ 1, g.wait, abort_flag)) break;
      tc_fence_after();
      const uint32_t d = tmem + static_cast<uint32_t>(acc * g.acc_cols);
      for (int s = t.s0; s < t.s1; ++s) {
        // the converters waited for the copies
        if (!mbar_wait_warp(smem_u32(cvt + stage), phase, g.wait, abort_flag) ||
            !mbar_wait_warp(smem_u32(full + stage), phase, g.wait, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t bd = smem_desc_mn(base + static_cast<uint32_t>(stage) * stage_bytes, 8192u);
        const uint32_t a = tmem + static_cast<uint32_t>(g.slot_col + slot * WG_SLOT_COLS);
        if (elect_one()) {
#pragma unroll
          for (int j = 0; j < 4; ++j)        // 16 tokens: 8 columns of A, 2048 bytes of B
            mma_bf16_ts(d, a + 8 * j, bd + 128 * j, idesc, (s > t.s0 || j > 0) ? 1u : 0u);
          mma_commit(smem_u32(empty + stage));
        }
        __syncwarp();
        if (++slot == g.slots) slot = 0;
        if (++stage == g.stages) {
          stage = 0;
          phase ^= 1;
        }
      }
      if (!ok) break;
      if (elect_one()) mma_commit(smem_u32(accf + acc));
      __syncwarp();
      if (++acc == g.accs) {
        acc = 0;
        aphase ^= 1;
      }
    }
    if (elect_one()) mma_commit(smem_u32(drain));
    __syncwarp();
    volatile int never = 0;
    pipe::wait(smem_u32(drain), 0, g.wait, &never);
  } else if (warp < WG_EPI_WARP0) {
    // ---------------------------------------------------------- converters
    const int grp = (warp - 2) >> 2;
    const int q = warp & 3;                      // TMEM sub-partition
    const uint32_t feat = static_cast<uint32_t>(q * 32 + lane);
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(g.slot_col);
    int stage = 0, slot = 0, old = 0;            // ring positions of the CTA's current step, over its units
    uint32_t phase = 0, old_phase = 0;
    int warm = g.slots;                          // steps until a slot is used again
    int turn = 0;
    bool ok = true;
    auto advance = [&]() {
      if (++turn == WG_GROUPS) turn = 0;
      if (++stage == g.stages) {
        stage = 0;
        phase ^= 1;
      }
      if (++slot == g.slots) slot = 0;
      if (warm > 0) {
        --warm;
      } else if (++old == g.stages) {
        old = 0;
        old_phase ^= 1;
      }
    };
    for (int u = blockIdx.x; ok && u < g.units; u += gridDim.x) {
      const GradUnit t = grad_unit(g, u);
      for (int s = t.s0; s < t.s1; ++s, advance()) {
        if (turn != grp) continue;
        bool w = pipe::wait(smem_u32(full + stage), phase, g.wait, abort_flag);
        const uint32_t sq = base + static_cast<uint32_t>(stage) * stage_bytes + y_bytes;
        uint32_t r[32];
        if (w) {
          const uint32_t s2[2] = {code_scale2(pipe::lds8(sq + WG_CODES + feat)),
                                  code_scale2(pipe::lds8(sq + WG_CODES + 128u + feat))};
          uint4 c[4];
#pragma unroll
          for (int h = 0; h < 4; ++h) c[h] = pipe::lds128(sq + static_cast<uint32_t>(h) * 2048u + feat * 16u);
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            const uint32_t cw[4] = {c[h].x, c[h].y, c[h].z, c[h].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              r[8 * h + 2 * i] = code_pair(__byte_perm(cw[i], 0u, 0x0100), s2[h >> 1]);
              r[8 * h + 2 * i + 1] = code_pair(__byte_perm(cw[i], 0u, 0x0302), s2[h >> 1]);
            }
          }
          // the slot's previous MMAs have completed
          if (warm == 0) w = pipe::wait(smem_u32(empty + old), old_phase, g.wait, abort_flag);
        }
        if (!__all_sync(0xffffffffu, w)) {
          ok = false;
          break;
        }
        tc_fence_after();
        tmem_st_32x32b_x32(lane_base + static_cast<uint32_t>(slot) * WG_SLOT_COLS, r);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(cvt + stage));
      }
    }
  } else {
    // ---------------------------------------------------------- epilogue
    const int q = warp & 3;
    const uint32_t buf0 = base + g.off_out + static_cast<uint32_t>(warp - WG_EPI_WARP0) * WG_OUT_BUF;
    int acc = 0, flip = 0;
    uint32_t aphase = 0;
    for (int u = blockIdx.x; u < g.units; u += gridDim.x) {
      const GradUnit t = grad_unit(g, u);
      const bool w = pipe::wait(smem_u32(accf + acc), aphase, g.wait, abort_flag);
      if (!__all_sync(0xffffffffu, w)) break;
      tc_fence_after();
      const uint32_t tb = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(acc * g.acc_cols);
      const int k0 = t.kt * 128 + q * 32;
      const int n0 = t.nt * g.bn;
#pragma unroll 1
      for (int c0 = 0; c0 < g.bn; c0 += 32) {
        uint32_t r[32];
        tmem_ld_32x32b_x32(tb + c0, r);
        tmem_ld_wait();
        if (c0 + 32 == g.bn) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(acce + acc));
        }
        if (g.splits > 1) {
          // fp32 partial [channel][feature] at the start of the stage ring (the CTA's only unit: all consumed)
#pragma unroll
          for (int j = 0; j < 32; ++j)
            pipe::sts32(base + static_cast<uint32_t>((c0 + j) * 128 + q * 32 + lane) * 4u, r[j]);
          continue;
        }
        uint32_t buf = buf0;
        if (g.f32) {
          if (lane == 0) bulk_wait_group_read<0>();
          __syncwarp();
          // row j = channel, 128 bytes of features, 16-byte units XORed with j mod 8 (the map's 128B swizzle)
#pragma unroll
          for (int j = 0; j < 32; ++j)
            pipe::sts32(buf + static_cast<uint32_t>(j * 128 + (((lane >> 2) ^ (j & 7)) << 4) + (lane & 3) * 4), r[j]);
        } else {
          buf += static_cast<uint32_t>(flip) * (WG_OUT_BUF / 2);
          flip ^= 1;
          if (lane == 0) bulk_wait_group_read<1>();
          __syncwarp();
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i)
            pk[i] = pack_bf16x2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
          pipe::stage_bf16_pairs(buf, pk, 32, lane);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (k0 < g.K && n0 + c0 < g.N) {            // blocks wholly outside are not issued
            if (g.f32 && g.accumulate) tma_add_2d(&tm_c, buf, k0, n0 + c0);
            else tma_store_2d(&tm_c, buf, g.f32 ? k0 : 2 * k0, n0 + c0);
          }
          bulk_commit_group();
        }
      }
      if (++acc == g.accs) {
        acc = 0;
        aphase ^= 1;
      }
    }
    if (lane == 0) bulk_wait_group<0>();
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);

  if (g.splits > 1) {
    cluster_sync_all();
    const GradUnit t = grad_unit(g, blockIdx.x);
    const int rows = (g.bn + g.splits - 1) / g.splits;
    const int r0 = t.split * rows;
    const int r1 = min(g.bn, r0 + rows);
    for (int i = threadIdx.x; i < (r1 - r0) * 32; i += WG_THREADS) {
      const int ch = r0 + (i >> 5);
      const int quad = i & 31;
      const int n = t.nt * g.bn + ch;
      const int k = t.kt * 128 + 4 * quad;
      if (n >= g.N || k >= g.K) continue;              // K % 16 == 0: the quad is all in or all out
      const uint32_t off = base + static_cast<uint32_t>(ch * 128 + 4 * quad) * 4u;
      float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int sp = 0; sp < g.splits; ++sp) {
        const float4 v = ld_shared_cluster_f4(map_to_rank(off, static_cast<uint32_t>(sp)));
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
      }
      const int64_t o = static_cast<int64_t>(n) * g.K + k;
      if (g.f32) {
        float4* p = reinterpret_cast<float4*>(static_cast<float*>(g.dw) + o);
        if (g.accumulate) {
          const float4 v = *p;
          s = make_float4(v.x + s.x, v.y + s.y, v.z + s.z, v.w + s.w);
        }
        *p = s;
      } else {
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(g.dw) + o) =
            make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
      }
    }
    cluster_sync_all();
  }
}

// db[n] (+)= sum_m dY[m, n]: a cluster of CTAs shares 64 channels, each CTA a
// contiguous run of tokens; a thread sums 8 channels of every 32nd token in
// fp32, the 32 partial sums and then the CTAs' sums are added in order.  One
// read of dY at HBM rate.
constexpr int DB_THREADS = 256;
__global__ void __launch_bounds__(DB_THREADS) bias_grad_kernel(const uint16_t* __restrict__ dy, int M, int N, int64_t ld,
                                                               int accumulate, float* __restrict__ db) {
  __shared__ __align__(16) float part[32][64];
  __shared__ __align__(16) float tot[64];
  griddep_launch_dependents();
  griddep_wait();
  const int S = static_cast<int>(gridDim.y);
  const int split = static_cast<int>(blockIdx.y);
  const int n0 = blockIdx.x * 64 + (threadIdx.x & 7) * 8;
  const int r = threadIdx.x >> 3;
  const int m0 = static_cast<int>(static_cast<int64_t>(split) * M / S);
  const int m1 = static_cast<int>(static_cast<int64_t>(split + 1) * M / S);
  float a[8] = {};
  if (n0 < N) {                                          // N % 8 == 0
    for (int m = m0 + r; m < m1; m += 32) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(dy + m * ld + n0));
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[2 * i] += __uint_as_float(w[i] << 16);
        a[2 * i + 1] += __uint_as_float(w[i] & 0xffff0000u);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) part[r][(threadIdx.x & 7) * 8 + i] = a[i];
  __syncthreads();
  if (threadIdx.x < 64) {
    float s = 0.0f;
    for (int i = 0; i < 32; ++i) s += part[i][threadIdx.x];
    tot[threadIdx.x] = s;
  }
  if (S > 1) cluster_sync_all();
  else __syncthreads();
  if (split == 0 && threadIdx.x < 16) {
    const int n = blockIdx.x * 64 + threadIdx.x * 4;
    if (n < N) {
      const uint32_t off = smem_u32(tot) + threadIdx.x * 16u;
      float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int sp = 0; sp < S; ++sp) {
        float4 v;
        if (S > 1) v = ld_shared_cluster_f4(map_to_rank(off, static_cast<uint32_t>(sp)));
        else v = *reinterpret_cast<const float4*>(tot + threadIdx.x * 4);
        s = make_float4(s.x + v.x, s.y + v.y, s.z + v.z, s.w + v.w);
      }
      float4* p = reinterpret_cast<float4*>(db + n);
      if (accumulate) {
        const float4 v = *p;
        s = make_float4(v.x + s.x, v.y + s.y, v.z + s.z, v.w + s.w);
      }
      *p = s;
    }
  }
  if (S > 1) cluster_sync_all();                         // the sums have been read
}

template <typename... P, typename... A>
dq_status launch(void (*kernel)(P...), dim3 grid, int threads, int smem, dim3 cluster, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster.x;
  attr[1].val.clusterDim.y = cluster.y;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster.x * cluster.y > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
  return e == cudaSuccess ? DQ_OK : cuda_fail(e);
}

dq_status launch_bias_grad(const uint16_t* dy, int64_t M, int64_t N, int64_t ld, int accumulate, float* db, int sm_count,
                           cudaStream_t stream) {
  const int groups = static_cast<int>((N + 63) / 64);
  int S = 1;
  while (S < 8 && groups * S < 4 * sm_count && M / (2 * S) >= 64) S *= 2;
  return launch(bias_grad_kernel, dim3(groups, S), DB_THREADS, 0, dim3(1, S), stream, dy, static_cast<int>(M),
                static_cast<int>(N), ld, accumulate, db);
}

}  // namespace
}  // namespace dq

using namespace dq;

extern "C" {

dq_status dq_act8_weight_grad(const void* dy_bf16, int64_t M, int64_t N, int64_t lddy, const int8_t* codes,
                              const uint8_t* scales, int64_t K, void* dw, dq_out_dtype dw_dtype, int accumulate,
                              float* db, dq_stream_t stream) {
  if (M < 0 || N < 1 || K < 1 || lddy < N) return DQ_ERR_INVALID_ARG;
  if (dw_dtype != DQ_OUT_BF16 && dw_dtype != DQ_OUT_F32) return DQ_ERR_INVALID_ARG;
  if (dw == nullptr || (M > 0 && (dy_bf16 == nullptr || codes == nullptr || scales == nullptr))) return DQ_ERR_INVALID_ARG;
  if (accumulate && dw_dtype != DQ_OUT_F32) return DQ_ERR_INVALID_ARG;
  if (K % 16 != 0 || N % 8 != 0 || lddy % 8 != 0 || M > kGradMaxDim || N > kGradMaxDim || K > kGradMaxDim ||
      lddy > (int64_t(1) << 37))
    return DQ_ERR_UNSUPPORTED;
  if (!aligned(dy_bf16, 16) || !aligned(codes, 16) || !aligned(scales, 16) || !aligned(dw, 16) || !aligned(db, 16))
    return DQ_ERR_UNSUPPORTED;
  DeviceInfo* dev = nullptr;
  dq_status st = current_device(&dev);
  if (st != DQ_OK) return st;
  const auto cs = reinterpret_cast<cudaStream_t>(stream);
  const bool f32 = dw_dtype == DQ_OUT_F32;
  if (M == 0) {                                           // an empty sum
    if (accumulate) return DQ_OK;
    cudaError_t e = cudaMemsetAsync(dw, 0, static_cast<size_t>(N) * K * (f32 ? 4 : 2), cs);
    if (e == cudaSuccess && db != nullptr) e = cudaMemsetAsync(db, 0, static_cast<size_t>(N) * 4, cs);
    return e == cudaSuccess ? DQ_OK : cuda_fail(e);
  }
  const auto* dy = static_cast<const uint16_t*>(dy_bf16);
  if (db != nullptr && (st = launch_bias_grad(dy, M, N, lddy, accumulate, db, dev->sm_count, cs)) != DQ_OK) return st;

  GradArgs g = {};
  g.M = static_cast<int>(M);
  g.N = static_cast<int>(N);
  g.K = static_cast<int>(K);
  g.bn = N > 128 ? 192 : N > 64 ? 128 : 64;
  g.kt = static_cast<int>((K + 127) / 128);
  g.nt = static_cast<int>((N + g.bn - 1) / g.bn);
  g.ks = static_cast<int>((M + WG_STEP - 1) / WG_STEP);
  const int64_t tiles = static_cast<int64_t>(g.kt) * g.nt;
  if (tiles > 0x3fffffff) return DQ_ERR_UNSUPPORTED;
  g.splits = 1;
  while (g.splits < 8 && tiles * g.splits * 2 <= dev->sm_count && g.ks >= 4 * g.splits) g.splits *= 2;
  g.units = static_cast<int>(tiles) * g.splits;
  g.accs = 2;
  g.acc_cols = g.bn;
  g.slot_col = 2 * g.bn;
  g.slots = std::min(8, (512 - g.slot_col) / WG_SLOT_COLS);
  g.full_chunks = static_cast<int>(N / 64);
  const int stage_bytes = g.bn * 128 + WG_CODES + 1024;
  const int fixed = 1024 + 4 * WG_OUT_BUF + WG_BAR_BYTES;
  g.stages = std::min(WG_MAX_STAGES, (227 * 1024 - fixed) / stage_bytes);
  g.slots = std::min(g.slots, g.stages);   // a slot's wait looks back less than one lap of the ring
  g.off_out = static_cast<uint32_t>(g.stages * stage_bytes);
  g.off_bar = g.off_out + 4 * WG_OUT_BUF;
  const int smem = static_cast<int>(g.off_bar) + WG_BAR_BYTES + 1024;
  g.dw = dw;
  g.f32 = f32;
  g.accumulate = accumulate != 0;
  g.wait = WaitCtl{dev->err_word, wait_timeout_ns()};

  const int64_t groups = (M + 31) / 32;
  CUtensorMap y3, y2, tq, te, tc;
  if ((st = make_tmap_2d(&y2, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, dy, N, M, static_cast<uint64_t>(lddy) * 2, 64, WG_STEP,
                         128)) != DQ_OK)
    return st;
  y3 = y2;
  if (g.full_chunks > 0 &&
      (st = make_tmap_chunks(&y3, dy, M, g.full_chunks, static_cast<uint64_t>(lddy) * 2, WG_STEP, g.bn / 64)) != DQ_OK)
    return st;
  if ((st = make_tmap_2d(&tq, CU_TENSOR_MAP_DATA_TYPE_UINT64, codes, static_cast<uint64_t>(K) * 2, 2 * groups,
                         static_cast<uint64_t>(K) * 16, 256, 4, 0)) != DQ_OK)
    return st;
  if ((st = make_tmap_2d(&te, CU_TENSOR_MAP_DATA_TYPE_UINT8, scales, K, groups, K, 128, 2, 0)) != DQ_OK) return st;
  if (f32) {
    st = make_tmap_2d(&tc, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, dw, K, N, static_cast<uint64_t>(K) * 4, 32, 32, 128);
  } else {
    st = make_tmap_2d(&tc, CU_TENSOR_MAP_DATA_TYPE_UINT8, dw, static_cast<uint64_t>(K) * 2, N,
                      static_cast<uint64_t>(K) * 2, 64, 32, 0);
  }
  if (st != DQ_OK) return st;
  if ((st = smem_limit_once(reinterpret_cast<const void*>(&act8_grad_kernel), smem)) != DQ_OK) return st;
  const unsigned grid = g.splits > 1 ? static_cast<unsigned>(g.units)
                                     : static_cast<unsigned>(std::min<int64_t>(tiles, dev->sm_count));
  return launch(act8_grad_kernel, dim3(grid), WG_THREADS, smem, dim3(g.splits, 1), cs, y3, y2, tq, te, tc, g);
}

}  // extern "C"
