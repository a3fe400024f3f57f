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
// Roles (five warpgroups): warp 0 dY producer, warp 1 MMA issuer, warp 2 code
// producer; two warpgroups of converters taking alternate 64-token steps; two
// warpgroups of accumulating epilogue warps (lane = feature, a warp holds half
// of the tile's channels in registers).
// Three rings, each as deep as its own round trip asks: dY in shared memory
// (freed by the MMAs), codes in shared memory (freed by the converters), and
// converted steps in tensor memory.  With one ring for both loads a step's
// slot waited for copy, conversion AND product in turn (0.34 us per step with
// neither arithmetic nor MMAs in it).
// Sums: the tensor core truncates when it adds to its accumulator, so a chain
// of MMAs loses about 2^-26 of the sum per instruction, all in one direction
// (65792 tokens in one chain: 4.4e-5 of the result).  Every 1024 tokens the
// epilogue adds the accumulator to fp32 registers (rounding to nearest) and
// the chain starts anew; the eight converted steps in flight cover the read.
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

constexpr int WG_THREADS = 640;
constexpr int WG_CVT_WARP0 = 4;              // warps 4..11: two converter groups
constexpr int WG_EPI_WARP0 = 12;             // warps 12..19
constexpr int WG_EPI_WARPS = 8;
// registers per thread of the five warpgroups: 40 + 2 * 56 + 2 * 160 = 472, of
// the 5 * 96 = 480 that the block is launched with; at the end all go back to 96
constexpr int WG_REGS = 96;
constexpr int WG_REGS_ISSUE = 40, WG_REGS_CVT = 56, WG_REGS_EPI = 160;
constexpr int WG_STEP = 64;                  // tokens per step
constexpr int WG_SEG = 16;                   // steps per accumulator chain
constexpr int WG_CODES = 128 * WG_STEP;      // bytes: [4 x 16 tokens][128 features][16]
constexpr int WG_MAX_RING = 8;               // stages or slots of each ring
constexpr int WG_CODE_STAGE = WG_CODES + 256;
constexpr int WG_BAR_BYTES = 512;
constexpr int WG_OUT_BUF = 2048;             // per epilogue warp: 32 x 32 bf16 or 16 x 32 fp32
constexpr int WG_SLOT_COLS = WG_STEP / 2;    // TMEM columns of one converted step
constexpr int64_t kGradMaxDim = int64_t(1) << 30;

struct GradArgs {
  int M, N, K;
  int bn;                  // channels per tile (64, 128, 192 or 256)
  int kt, nt;              // feature tiles (128), channel tiles
  int splits, units;
  int ks;                  // token steps: ceil(M / 64)
  int stages, code_stages; // dY and code rings
  int slots;               // converted-step slots in tensor memory, after the accumulator
  int full_chunks;         // N / 64: chunks the 3-D map covers
  uint32_t off_q, off_out, off_bar;
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

__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void set_regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void set_regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// A word of four codes -> two pairs of bf16 values q 2^(E - 133).  With v =
// q + 128 (the code's sign bit flipped), the byte v at the foot of a 16-bit
// lane IS the bf16 number v 2^-133 (subnormal, or of the least exponent);
// times 2^127 it is v 2^-6, and fma(v 2^-6, 2^(E - 127), -2^(E - 126)) =
// (v - 128) 2^(E - 133) exactly.  s2 = 2^(E - 127) and c2 = -2^(E - 126) twice.
__device__ __forceinline__ void codes4(uint32_t w, uint32_t s2, uint32_t c2, uint32_t& r0, uint32_t& r1) {
  const uint32_t v = w ^ 0x80808080u;
  const uint32_t u0 = __byte_perm(v, 0u, 0x4140), u1 = __byte_perm(v, 0u, 0x4342);
  uint32_t t0, t1;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(t0) : "r"(u0), "r"(0x7f007f00u));
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(t1) : "r"(u1), "r"(0x7f007f00u));
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r0) : "r"(t0), "r"(s2), "r"(c2));
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r1) : "r"(t1), "r"(s2), "r"(c2));
}
__device__ __forceinline__ uint32_t code_s2(uint32_t e) { return (e == 0u ? 0x0040u : e << 7) * 0x00010001u; }
__device__ __forceinline__ uint32_t code_c2(uint32_t e) { return (0x8000u | ((e + 1u) << 7)) * 0x00010001u; }
// The same for E = 254, whose -2^128 is not a bf16 number (two halves of the
// scale), and E = 255 (NaN).
__device__ __forceinline__ void codes4_top(uint32_t w, uint32_t e, uint32_t& r0, uint32_t& r1) {
  uint32_t a, b;
  codes4(w, code_s2(253u), code_c2(253u), a, b);
  const uint32_t two = e == 255u ? 0x7fc07fc0u : 0x40004000u;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r0) : "r"(a), "r"(two));
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r1) : "r"(b), "r"(two));
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
                     const __grid_constant__ CUtensorMap tm_c, const __grid_constant__ GradArgs g) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const smem = smem_raw + (base - raw);
  // rings: dY (bn / 64 chunks of 64 tokens x 128 B); codes, then their scales [2][128]
  const uint32_t y_bytes = static_cast<uint32_t>(g.bn) * 128u;
  uint64_t* const yfull = reinterpret_cast<uint64_t*>(smem + g.off_bar);
  uint64_t* const yempty = yfull + WG_MAX_RING;
  uint64_t* const qfull = yempty + WG_MAX_RING;
  uint64_t* const qempty = qfull + WG_MAX_RING;
  uint64_t* const afull = qempty + WG_MAX_RING;    // a slot holds a converted step
  uint64_t* const aempty = afull + WG_MAX_RING;
  uint64_t* const accf = aempty + WG_MAX_RING;
  uint64_t* const acce = accf + 1;
  uint64_t* const drain = acce + 1;
  uint32_t* const tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < WG_MAX_RING; ++i) {
      mbar_init(smem_u32(yfull + i), 1);
      mbar_init(smem_u32(yempty + i), 1);
      mbar_init(smem_u32(qfull + i), 1);
      mbar_init(smem_u32(qempty + i), 4);
      mbar_init(smem_u32(afull + i), 4);
      mbar_init(smem_u32(aempty + i), 1);
    }
    mbar_init(smem_u32(accf), 1);
    mbar_init(smem_u32(acce), WG_EPI_WARPS);
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
  griddep_wait();
  griddep_launch_dependents();

  if (warp < WG_CVT_WARP0) {
    set_regs_down<WG_REGS_ISSUE>();
    if (warp == 0 || warp == 2) {
      // -------------------------------------------------------- producers
      const bool codes = warp == 2;
      uint64_t* const full = codes ? qfull : yfull;
      uint64_t* const empty = codes ? qempty : yempty;
      const int ring = codes ? g.code_stages : g.stages;
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
          const uint32_t sy = base + static_cast<uint32_t>(stage) * y_bytes;
          const uint32_t sq = base + g.off_q + static_cast<uint32_t>(stage) * WG_CODE_STAGE;
          if (elect_one()) {
            if (codes) {
              mbar_arrive_expect_tx(fb, WG_CODE_STAGE);
              tma_load_2d(sq, &tm_q, fb, t.kt * 256, s * 4);
              tma_load_2d(sq + WG_CODES, &tm_e, fb, t.kt * 128, s * 2);
            } else {
              mbar_arrive_expect_tx(fb, y_bytes);
              if (whole)
                tma_load_3d(sy, &tm_y3, fb, 0, s * WG_STEP, c0);
              else
                for (int c = 0; c < chunks; ++c)
                  tma_load_2d(sy + static_cast<uint32_t>(c) * 8192u, &tm_y2, fb, (c0 + c) * 64, s * WG_STEP);
            }
          }
          __syncwarp();
          ++issued;
          if (++stage == ring) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      // every copy issued lands before the CTA can exit
      volatile int never = 0;
      for (long long i = issued > ring ? issued - ring : 0; i < issued; ++i)
        pipe::wait(smem_u32(full + static_cast<int>(i % ring)), static_cast<uint32_t>((i / ring) & 1), g.wait, &never);
    } else if (warp == 1) {
      // -------------------------------------------------------- MMA issuer
      const uint32_t idesc = idesc_grad(g.bn);
      int stage = 0, slot = 0;
      uint32_t phase = 0, sphase = 0, aphase = 0;
      bool ok = true, tested = false;             // tested: the next step's operands were found ready
      for (int u = blockIdx.x; ok && u < g.units; u += gridDim.x) {
        const GradUnit t = grad_unit(g, u);
        for (int s = t.s0; ok && s < t.s1;) {
          const int end = min(t.s1, s + WG_SEG);
          if (!mbar_wait_warp(smem_u32(acce), aphase ^ 1, g.wait, abort_flag)) {
            ok = false;
            break;
          }
          aphase ^= 1;
          tc_fence_after();
          for (int first = s; s < end; ++s) {
            if (!mbar_wait_warp2(tested, smem_u32(yfull + stage), phase, smem_u32(afull + slot), sphase, g.wait,
                                 abort_flag)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint64_t bd = smem_desc_mn(base + static_cast<uint32_t>(stage) * y_bytes, 8192u);
            const uint32_t a = tmem + static_cast<uint32_t>(g.bn + slot * WG_SLOT_COLS);
            const uint32_t yb = smem_u32(yempty + stage), ab = smem_u32(aempty + slot);
            if (++slot == g.slots) {
              slot = 0;
              sphase ^= 1;
            }
            if (++stage == g.stages) {
              stage = 0;
              phase ^= 1;
            }
            const bool ty = mbar_test(smem_u32(yfull + stage), phase), ta = mbar_test(smem_u32(afull + slot), sphase);
            if (elect_one()) {
#pragma unroll
              for (int j = 0; j < 4; ++j)      // 16 tokens: 8 columns of A, 2048 bytes of B
                mma_bf16_ts(tmem, a + 8 * j, bd + 128 * j, idesc, (s > first || j > 0) ? 1u : 0u);
              mma_commit(yb);
              mma_commit(ab);
            }
            __syncwarp();
            tested = ty && ta;
          }
          if (!ok) break;
          if (elect_one()) mma_commit(smem_u32(accf));
          __syncwarp();
        }
      }
      if (elect_one()) mma_commit(smem_u32(drain));
      __syncwarp();
      volatile int never = 0;
      pipe::wait(smem_u32(drain), 0, g.wait, &never);
    }
  } else if (warp < WG_EPI_WARP0) {
    // ---------------------------------------------------------- converters
    set_regs_down<WG_REGS_CVT>();
    const int grp = (warp - WG_CVT_WARP0) >> 2;
    const int q = warp & 3;                      // TMEM sub-partition
    const uint32_t feat = static_cast<uint32_t>(q * 32 + lane);
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(g.bn);
    int stage = 0, slot = 0;                     // ring positions of the CTA's current step, over its units
    uint32_t phase = 0, sphase = 0;
    int turn = 0;
    bool ok = true;
    auto advance = [&]() {
      turn ^= 1;
      if (++stage == g.code_stages) {
        stage = 0;
        phase ^= 1;
      }
      if (++slot == g.slots) {
        slot = 0;
        sphase ^= 1;
      }
    };
    for (int u = blockIdx.x; ok && u < g.units; u += gridDim.x) {
      const GradUnit t = grad_unit(g, u);
      for (int s = t.s0; s < t.s1; ++s, advance()) {
        if (turn != grp) continue;
        // the step's codes have landed, its slot's previous MMAs completed
        const bool tq = mbar_test(smem_u32(qfull + stage), phase), ta = mbar_test(smem_u32(aempty + slot), sphase ^ 1);
        if (!mbar_wait_warp2(tq && ta, smem_u32(qfull + stage), phase, smem_u32(aempty + slot), sphase ^ 1, g.wait,
                             abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t sq = base + g.off_q + static_cast<uint32_t>(stage) * WG_CODE_STAGE + feat * 16u;
        const uint32_t se = base + g.off_q + static_cast<uint32_t>(stage) * WG_CODE_STAGE + WG_CODES + feat;
#pragma unroll
        for (int b = 0; b < 2; ++b) {            // 32 tokens with one scale
          const uint32_t e = pipe::lds8(se + 128u * b);
          const uint4 c0 = pipe::lds128(sq + 4096u * b), c1 = pipe::lds128(sq + 4096u * b + 2048u);
          const uint32_t cw[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
          uint32_t r[16];
          const uint32_t s2 = code_s2(e), c2 = code_c2(e);
#pragma unroll
          for (int i = 0; i < 8; ++i) codes4(cw[i], s2, c2, r[2 * i], r[2 * i + 1]);
          if (e >= 254u) {
#pragma unroll
            for (int i = 0; i < 8; ++i) codes4_top(cw[i], e, r[2 * i], r[2 * i + 1]);
          }
          __syncwarp();
          tmem_st_32x32b_x16(lane_base + static_cast<uint32_t>(slot * WG_SLOT_COLS + 16 * b), r);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(qempty + stage));   // the codes are in registers
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(afull + slot));
      }
    }
  } else {
    // ---------------------------------------------------------- accumulation and epilogue
    set_regs_up<WG_REGS_EPI>();
    const int ew = warp - WG_EPI_WARP0;
    const int q = warp & 3;
    const int half = g.bn / 2;                   // channels of this warp: [h0, h0 + half) of the tile
    const int h0 = (ew >> 2) * half;
    const uint32_t buf = base + g.off_out + static_cast<uint32_t>(ew) * WG_OUT_BUF;
    const uint32_t tb = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(h0);
    uint32_t aphase = 0;
    bool ok = true;
    for (int u = blockIdx.x; ok && u < g.units; u += gridDim.x) {
      const GradUnit t = grad_unit(g, u);
      float sum[128];
#pragma unroll
      for (int j = 0; j < 128; ++j) sum[j] = 0.0f;
      for (int s = t.s0; s < t.s1; s += WG_SEG) {
        if (!mbar_wait_warp(smem_u32(accf), aphase, g.wait, abort_flag)) {
          ok = false;
          break;
        }
        aphase ^= 1;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          if (16 * c < half) {
            uint32_t r[16];
            tmem_ld_32x32b_x16(tb + 16 * c, r);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j) sum[16 * c + j] += __uint_as_float(r[j]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(acce));
      }
      if (!ok) break;
      const int k0 = t.kt * 128 + q * 32;
      const int n0 = t.nt * g.bn + h0;
      if (g.splits > 1) {
        // fp32 partial [channel][feature] over the dY ring (the CTA's only unit: its last accumulator is
        // complete, so every stage has been consumed)
#pragma unroll
        for (int j = 0; j < 128; ++j)
          if (j < half)
            pipe::sts32(base + static_cast<uint32_t>((h0 + j) * 128 + q * 32 + lane) * 4u, __float_as_uint(sum[j]));
        continue;
      }
#pragma unroll
      for (int c = 0; c < 8; ++c) {              // 16 channels at a time
        if (16 * c < half) {
          const bool issue = g.f32 || (c & 1);   // bf16 blocks hold 32 channels
          if (g.f32 || !(c & 1)) {
            if (lane == 0) bulk_wait_group_read<0>();
            __syncwarp();
          }
          if (g.f32) {
            // row j = channel, 128 bytes of features, 16-byte units XORed with j mod 8 (the map's 128B swizzle)
#pragma unroll
            for (int j = 0; j < 16; ++j)
              pipe::sts32(buf + static_cast<uint32_t>(j * 128 + (((lane >> 2) ^ (j & 7)) << 4) + (lane & 3) * 4),
                          __float_as_uint(sum[16 * c + j]));
          } else {
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 8; ++i) pk[i] = pack_bf16x2(sum[16 * c + 2 * i], sum[16 * c + 2 * i + 1]);
#pragma unroll
            for (int i = 8; i < 16; ++i) pk[i] = 0u;
            pipe::stage_bf16_pairs(buf + (c & 1) * 1024u, pk, 16, lane);
          }
          if (issue) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              const int n = n0 + (g.f32 ? 16 * c : 16 * (c - 1));
              if (k0 < g.K && n < g.N) {         // blocks wholly outside are not issued
                if (g.f32 && g.accumulate) tma_add_2d(&tm_c, buf, k0, n);
                else tma_store_2d(&tm_c, buf, g.f32 ? k0 : 2 * k0, n);
                bulk_commit_group();
              }
            }
          }
        }
      }
    }
    if (lane == 0) bulk_wait_group<0>();
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // Every thread takes its launch share of the registers again, but not before
  // all roles have ended: a warp that grew earlier (one without a role would
  // at once) could take what the epilogue's own growth still waits for.
  if (warp < WG_EPI_WARP0) set_regs_up<WG_REGS>();
  else set_regs_down<WG_REGS>();
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
  g.kt = static_cast<int>((K + 127) / 128);
  g.ks = static_cast<int>((M + WG_STEP - 1) / WG_STEP);
  // Tile width and split with the least estimated time: waves of steps, a step
  // costing about 0.25 + bn / 1280 us, plus a few us per unit for its ends.
  int64_t tiles = 0;
  double best = 1e300;
  for (int bn = 64; bn <= 256; bn += 64) {
    const int64_t nt = (N + bn - 1) / bn, n = nt * g.kt;
    for (int sp = 1; sp <= 8; sp *= 2) {
      if (sp > 1 && (n * sp > dev->sm_count || g.ks < 2 * sp)) break;
      const double waves = static_cast<double>((n * sp + dev->sm_count - 1) / dev->sm_count);
      const double cost = waves * (((g.ks + sp - 1) / sp) * (0.25 + bn / 1280.0) + 2.0) + (sp > 1 ? 1.0 + 0.2 * sp : 0.0);
      if (cost < best) {
        best = cost;
        g.bn = bn;
        g.nt = static_cast<int>(nt);
        g.splits = sp;
        tiles = n;
      }
    }
  }
  if (tiles > 0x3fffffff) return DQ_ERR_UNSUPPORTED;
  g.units = static_cast<int>(tiles) * g.splits;
  g.full_chunks = static_cast<int>(N / 64);
  // Five stages of dY at 256 channels, the rest of the shared memory for codes.
  // The rings that the two converter groups share have an even length, so that
  // a stage belongs to one group: a parity wait cannot tell a lap from the one
  // two before it, and a group that ran ahead of the other could take its
  // stage's next lap for landed.
  const int room = 227 * 1024 - 1024 - WG_EPI_WARPS * WG_OUT_BUF - WG_BAR_BYTES;
  g.stages = std::min(WG_MAX_RING, (room - 6 * WG_CODE_STAGE) / (g.bn * 128));
  g.code_stages = std::min(WG_MAX_RING, (room - g.stages * g.bn * 128) / WG_CODE_STAGE) & ~1;
  g.slots = std::min(WG_MAX_RING, (512 - g.bn) / WG_SLOT_COLS) & ~1;
  // (the swizzle of the output blocks counts from 1024-byte boundaries)
  g.off_out = static_cast<uint32_t>(g.stages * g.bn * 128);
  g.off_q = g.off_out + WG_EPI_WARPS * WG_OUT_BUF;
  g.off_bar = g.off_q + static_cast<uint32_t>(g.code_stages * WG_CODE_STAGE);
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
    st = make_tmap_2d(&tc, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, dw, K, N, static_cast<uint64_t>(K) * 4, 32, 16, 128);
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
