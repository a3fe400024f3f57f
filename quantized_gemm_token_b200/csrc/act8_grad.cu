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
// A pair of SMs (cta_group::2) per tile of 256 features x 256 (or 128)
// channels: each CTA converts its own 128 features into its own tensor memory
// and loads half of the channels, which the pair's tensor cores share.  Alone,
// a CTA loads 41 KB per 64-token step, 640 cycles at the 64 bytes per cycle an
// SM takes from L2, against 512 cycles of MMAs; in a pair 25 KB.
// Roles (five warpgroups per CTA): warp 0 dY producer, warp 1 MMA issuer (rank
// 0 only), warp 2 code producer; two warpgroups of converters taking
// alternate 64-token steps; two warpgroups of accumulating epilogue warps
// (lane = feature, a warp holds half of the tile's channels in registers).
// Three rings, each as deep as its own round trip asks: dY in shared memory
// (freed by the MMAs), codes in shared memory (freed by the converters), and
// converted steps in tensor memory.
// Sums: the tensor core truncates when it adds an MMA's 16 tokens to its
// accumulator, less than 2^-23 of the sum so far, all in one direction (65792
// tokens in one chain: 4.4e-5 of the result).  Every 2048 tokens (128 MMAs) the
// epilogue adds the accumulator to fp32 registers (rounding to nearest) and
// the chain starts anew; the converted steps in flight cover the read.  So
// |dW - exact| <= (min(ceil(M / 16), 128) 2^-23 + (ceil(M / 2048) + 4) 2^-24)
// sum |dY x|.  The length is a choice between error and time.  Measured, chains
// of 2048 against 1024 tokens: operands of one sign, 8192 tokens, 2.4e-6 against
// 1.0e-6 of the sum (a library fp32 product 0.3e-6); zero-mean ones, relative
// norm, 4.5e-7 against 2.1e-7 (1e-7 to 2e-7); 2048 x 4096 x 4096 57.4 against 61.5
// us, 8192 x 4096 x 4096 198 against 209, 65792 x 1280 -> 5120 with db 655 against
// 693.  dY itself carries bf16's 2^-9 per element.
// db: in the tiles of the first 256 features the epilogue warps also add up
// the dY tile that lies in shared memory (each lane eight channels), so dY is
// not read again: there a stage's MMAs hand it to them, and they free it.
// A partial wave of tiles: they are halved (128 channels) where the halves fit
// in one wave (2048 x 2560 x 2048, 80 tiles on 74 pairs: 26.8 us, whole 29.1), or
// their tokens are split over a cluster of 2 or 4 pairs whose fp32 partial
// tiles are added through distributed shared memory in split order (no
// workspace, no atomics), in a second launch where whole waves come first.
// Measured (bound: the MMAs' 512 cycles per step, about 590 reached): 8192 x
// 4096 x 4096 197 us, 1393 TFLOP/s (0.82 of the measured bf16 burst, 0.97 of
// the sustained rate); 65792 tokens, 1280 -> 5120, fp32: 611 us, 641 us with db
// (dY read again by a kernel of its own: 790 - 870 us); 2048 x 4096 x 4096 53.5 us
// (256 tiles on 74 pairs; 5 us of it are launch, prologue and ends).
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>

#include "gemm_common.cuh"
#include "internal.h"
#include "mx.cuh"
#include "mx.h"
#include "pipeline.cuh"
#include "sm100.cuh"

namespace dq {
namespace {

constexpr int WG_THREADS = 640;
constexpr int WG_CVT_WARP0 = 4;              // warps 4..11: two converter groups
constexpr int WG_EPI_WARP0 = 12;             // warps 12..19
constexpr int WG_EPI_WARPS = 8;
// registers per thread of the five warpgroups: 32 + 2 * 56 + 2 * 168 = 480, of
// the 5 * 96 = 480 that the block is launched with; at the end all go back to 96
constexpr int WG_REGS = 96;
constexpr int WG_REGS_ISSUE = 32, WG_REGS_CVT = 56, WG_REGS_EPI = 168;
static_assert(WG_REGS_ISSUE + 2 * WG_REGS_CVT + 2 * WG_REGS_EPI <= 5 * WG_REGS, "register split");
constexpr int WG_STEP = 64;                  // tokens per step
constexpr int WG_SEG = 32;                   // steps per accumulator chain
constexpr int WG_CODES = 128 * WG_STEP;      // bytes: [4 x 16 tokens][128 features][16]
constexpr int WG_RING = 8;                   // stages or slots of each ring
constexpr int WG_CODE_STAGE = WG_CODES + 256;
constexpr int WG_BAR_BYTES = 512;
constexpr int WG_OUT_BUF = 2048;             // per epilogue warp: 32 x 32 bf16 or 16 x 32 fp32
constexpr int WG_SLOT_COLS = WG_STEP / 2;    // TMEM columns of one converted step
constexpr int WG_MAX_SMEM = WG_RING * 256 * 64 + WG_EPI_WARPS * WG_OUT_BUF + WG_RING * WG_CODE_STAGE + WG_BAR_BYTES + 1024;
static_assert(WG_MAX_SMEM <= 227 * 1024, "shared memory");

struct GradArgs {
  int M, N, K;
  int bn;                  // channels per tile (128 or 256), half of them per CTA
  int kt, nt;              // feature tiles (256), channel tiles
  int t1;                  // tiles from here on are halved (128 channels each)
  int tile0;               // first tile of this launch
  int splits, units;
  int ks;                  // token steps: ceil(M / 64)
  int full_chunks;         // N / 64: chunks the 3-D map covers
  uint32_t off_q, off_out, off_bar;
  void* dw;
  float* db;               // or null
  int f32, accumulate;
  WaitCtl wait;
};

// kind::f16, bf16 A (tensor memory, K-major) and B (shared memory, MN-major),
// fp32 accumulator, M = 256 over the pair.
__host__ __device__ constexpr uint32_t idesc_grad(int N) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | (static_cast<uint32_t>(N >> 3) << 17) | (16u << 24);
}

__device__ __forceinline__ void mma_bf16_ts_pair(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
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

// Arrive once on the mbarrier at shared::cta offset `bar` in both CTAs of the
// pair (`mask`: their bits in the cluster) when all MMAs issued so far by this
// thread have completed.
__device__ __forceinline__ void commit_pair(uint32_t bar, uint16_t mask) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                   bar),
               "h"(mask)
               : "memory");
}

// Arrive on the mbarrier at shared::cluster address `bar` for tensor-memory
// accesses (waited for, and fenced by tcgen05.fence::before_thread_sync): they
// are not ordered by the arrive itself, so it needs no release (which at
// cluster scope takes more than the 512 cycles of a step).
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// 3-D tiled load into this CTA's shared memory, completing on the pair
// leader's mbarrier.
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const void* tmap, uint32_t bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
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

// Two fp32 sums take a pair of bf16 values (each addition rounds in fp32; the
// mixed addition saves the conversion: db above 664 us, 679 with shifts and
// masks; four tokens to one address the rest).
__device__ __forceinline__ void add_bf16x2(float& lo, float& hi, uint32_t v) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tadd.rn.f32.bf16 %0, l, %0;\n\tadd.rn.f32.bf16 %1, h, %1;\n\t}"
      : "+f"(lo), "+f"(hi)
      : "r"(v));
}

struct GradUnit {
  int split, kt, n0, bn, s0, s1;
};
__device__ __forceinline__ GradUnit grad_unit(const GradArgs& g, int u) {
  GradUnit t;
  int tile = u / g.splits;
  t.split = u - tile * g.splits;
  tile += g.tile0;
  t.bn = g.bn;
  t.n0 = 0;
  if (tile >= g.t1) {
    t.bn = 128;
    t.n0 = ((tile - g.t1) & 1) * 128;
    tile = g.t1 + ((tile - g.t1) >> 1);
  }
  if (g.db != nullptr) {
    // the tiles that also sum columns (kt = 0, the slowest) come last, where a
    // partial wave is split
    t.kt = g.kt - 1 - tile / g.nt;
    t.n0 += tile % g.nt * g.bn;
  } else {
    const int nt = tile / g.kt;
    t.kt = tile - nt * g.kt;
    t.n0 += nt * g.bn;
  }
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
  // rings: this CTA's half of dY (bn / 128 chunks of 64 tokens x 128 B); codes, then their scales [2][128]
  const uint32_t y_bytes = static_cast<uint32_t>(g.bn) * 64u;
  uint64_t* const yfull = reinterpret_cast<uint64_t*>(smem + g.off_bar);   // leader: both halves of dY
  uint64_t* const yempty = yfull + WG_RING;
  uint64_t* const qfull = yempty + WG_RING;
  uint64_t* const qempty = qfull + WG_RING;
  uint64_t* const afull = qempty + WG_RING;        // leader: both CTAs' slots hold a converted step
  uint64_t* const aempty = afull + WG_RING;
  uint64_t* const ydone = aempty + WG_RING;        // the MMAs are done with a stage that column sums still read
  uint64_t* const accf = ydone + WG_RING;
  uint64_t* const acce = accf + 1;
  uint64_t* const drain = acce + 1;
  uint32_t* const tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t crank = cluster_ctarank();
  const uint32_t rank = crank & 1u;                // in the pair
  const uint32_t lead = crank & ~1u;               // the pair's leader in the cluster
  const uint16_t mask = static_cast<uint16_t>(3u << lead);
  const int G = static_cast<int>(gridDim.x) >> 1;
  const int u0 = static_cast<int>(blockIdx.x) >> 1;
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < WG_RING; ++i) {
      mbar_init(smem_u32(yfull + i), 1);
      mbar_init(smem_u32(yempty + i), g.db != nullptr ? 2 : 1);
      mbar_init(smem_u32(qfull + i), 1);
      mbar_init(smem_u32(qempty + i), 4);
      mbar_init(smem_u32(afull + i), 8);
      mbar_init(smem_u32(aempty + i), 1);
      mbar_init(smem_u32(ydone + i), 1);
    }
    mbar_init(smem_u32(accf), 1);
    mbar_init(smem_u32(acce), 2 * WG_EPI_WARPS);
    mbar_init(smem_u32(drain), 1);
    fence_barrier_init();
    tma_prefetch_desc(&tm_y3);
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_e);
    tma_prefetch_desc(&tm_c);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_holder), 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync_all();            // the barriers are initialised before any remote use
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
      int stage = 0;
      uint32_t phase = 0;
      long long issued = 0;
      bool ok = true;
      for (int u = u0; ok && u < g.units; u += G) {
        const GradUnit t = grad_unit(g, u);
        const int chunks = t.bn / 128;
        const int c0 = t.n0 / 64 + static_cast<int>(rank) * chunks;
        const int f0 = t.kt * 256 + static_cast<int>(rank) * 128;
        // the 3-D map covers whole chunks only, a whole tile's at a time: a tile that holds the ragged last one and
        // a halved tile are loaded chunk by chunk
        const bool whole = t.bn == g.bn && (c0 + chunks <= g.full_chunks || g.N % 64 == 0);
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
              tma_load_2d(sq, &tm_q, fb, f0 * 2, s * 4);
              tma_load_2d(sq + WG_CODES, &tm_e, fb, f0, s * 2);
            } else {
              if (rank == 0) mbar_arrive_expect_tx(fb, static_cast<uint32_t>(t.bn) * 128u);
              const uint32_t fl = map_to_rank(fb, lead);
              if (whole)
                tma_load_3d_pair(sy, &tm_y3, fl, 0, s * WG_STEP, c0);
              else
                for (int c = 0; c < chunks; ++c)
                  tma_load_2d_pair(sy + static_cast<uint32_t>(c) * 8192u, &tm_y2, fl, (c0 + c) * 64, s * WG_STEP);
            }
          }
          __syncwarp();
          ++issued;
          if (++stage == WG_RING) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      // Every copy issued lands before the CTA can exit: the leader's barriers
      // tell; rank 1, whose dY copies complete on the leader's, exits after the
      // leader's MMAs (drain), and after a failed wait a while later.
      volatile int never = 0;
      if (codes || rank == 0) {
        for (long long i = issued > WG_RING ? issued - WG_RING : 0; i < issued; ++i)
          pipe::wait(smem_u32(full + static_cast<int>(i % WG_RING)), static_cast<uint32_t>((i / WG_RING) & 1), g.wait,
                     &never);
      } else {
        pipe::wait(smem_u32(drain), 0, g.wait, &never);
        if (!ok) {
          const uint64_t w0 = globaltimer();
          while (globaltimer() - w0 < 100000ull) {
          }
        }
      }
    } else if (warp == 1 && rank == 0) {
      // -------------------------------------------------------- MMA issuer
      int stage = 0;
      uint32_t phase = 0, aphase = 0;
      bool ok = true, tested = false;             // tested: the next step's operands were found ready
      for (int u = u0; ok && u < g.units; u += G) {
        const GradUnit t = grad_unit(g, u);
        const uint32_t idesc = idesc_grad(t.bn);
        // a stage is freed by the MMAs, or in db tiles by the two warps that sum it
        uint64_t* const ynext = g.db != nullptr && t.kt == 0 ? ydone : yempty;
        const bool twice = g.db != nullptr && t.kt != 0;
        for (int s = t.s0; ok && s < t.s1;) {
          const int end = min(t.s1, s + WG_SEG);
          if (!mbar_wait_warp(smem_u32(acce), aphase ^ 1, g.wait, abort_flag)) {
            ok = false;
            break;
          }
          aphase ^= 1;
          tc_fence_after();
          for (int first = s; s < end; ++s) {
            if (!mbar_wait_warp2(tested, smem_u32(yfull + stage), phase, smem_u32(afull + stage), phase, g.wait,
                                 abort_flag)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint64_t bd = smem_desc_mn(base + static_cast<uint32_t>(stage) * y_bytes, 8192u);
            const uint32_t a = tmem + static_cast<uint32_t>(256 + stage * WG_SLOT_COLS);
            const uint32_t yb = smem_u32(ynext + stage), ab = smem_u32(aempty + stage);
            if (++stage == WG_RING) {
              stage = 0;
              phase ^= 1;
            }
            const bool ty = mbar_test(smem_u32(yfull + stage), phase), ta = mbar_test(smem_u32(afull + stage), phase);
            if (elect_one()) {
#pragma unroll
              for (int j = 0; j < 4; ++j)      // 16 tokens: 8 columns of A, 2048 bytes of B
                mma_bf16_ts_pair(tmem, a + 8 * j, bd + 128 * j, idesc, (s > first || j > 0) ? 1u : 0u);
              commit_pair(yb, mask);
              if (twice) commit_pair(yb, mask);
              commit_pair(ab, mask);
            }
            __syncwarp();
            tested = __all_sync(0xffffffffu, ty && ta);
          }
          if (!ok) break;
          if (elect_one()) commit_pair(smem_u32(accf), mask);
          __syncwarp();
        }
      }
      if (elect_one()) commit_pair(smem_u32(drain), mask);
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
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(q * 32) << 16) + 256u;
    int stage = 0;                               // ring position of the CTA's current step, over its units
    uint32_t phase = 0;
    int turn = 0;
    bool ok = true;
    auto advance = [&]() {
      turn ^= 1;
      if (++stage == WG_RING) {
        stage = 0;
        phase ^= 1;
      }
    };
    for (int u = u0; ok && u < g.units; u += G) {
      const GradUnit t = grad_unit(g, u);
      for (int s = t.s0; s < t.s1; ++s, advance()) {
        if (turn != grp) continue;
        // the step's codes have landed, its slot's previous MMAs completed
        const bool tq = mbar_test(smem_u32(qfull + stage), phase), ta = mbar_test(smem_u32(aempty + stage), phase ^ 1);
        if (!mbar_wait_warp2(tq && ta, smem_u32(qfull + stage), phase, smem_u32(aempty + stage), phase ^ 1, g.wait,
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
          tmem_st_32x32b_x16(lane_base + static_cast<uint32_t>(stage * WG_SLOT_COLS + 16 * b), r);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(qempty + stage));   // the codes are in registers
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_relaxed(map_to_rank(smem_u32(afull + stage), lead));
      }
    }
  } else {
    // ---------------------------------------------------------- accumulation and epilogue
    set_regs_up<WG_REGS_EPI>();
    const int ew = warp - WG_EPI_WARP0;
    const int q = warp & 3;
    const uint32_t buf = base + g.off_out + static_cast<uint32_t>(ew) * WG_OUT_BUF;
    int stage = 0;
    uint32_t aphase = 0;
    uint32_t dphase = 0;                         // bit s: the phase of ydone[s], which only db tiles use
    bool ok = true;
    for (int u = u0; ok && u < g.units; u += G) {
      const GradUnit t = grad_unit(g, u);
      const int half_n = t.bn / 2;                 // channels of this CTA's half of dY, and of
      const int half = half_n;                     // this warp: [h0, h0 + half) of the tile
      const int h0 = (ew >> 2) * half;
      const uint32_t tb = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(h0);
      float sum[128];
#pragma unroll
      for (int j = 0; j < 128; ++j) sum[j] = 0.0f;
      const bool with_db = g.db != nullptr && t.kt == 0;
      // Column sums: warps w and w + 4 take the steps of ring stages w and w + 4,
      // half of a step's tokens each (so four steps are summed at a time), a
      // lane the 8 channels of 16-byte unit lane % (units per row) of every
      // second (or fourth) token of eight.
      const int unit = lane & (half_n / 8 - 1);
      const int tstep = 256 / half_n;
      const int tok0 = lane / (half_n / 8);
      float col[8] = {};
      auto sum_stage = [&](int st) {             // false: the wait failed
        if (!mbar_wait_warp(smem_u32(ydone + st), (dphase >> st) & 1u, g.wait, abort_flag)) return false;
        dphase ^= 1u << st;
        const uint32_t sy = base + static_cast<uint32_t>(st) * y_bytes + static_cast<uint32_t>(unit >> 3) * 8192u +
                            static_cast<uint32_t>(ew >> 2) * (WG_STEP / 2 * 128);
        for (int tok = tok0; tok < 8; tok += tstep) {
          // (rows eight apart share their swizzle)
          const uint32_t row = sy + pipe::sw128_off(tok, unit & 7);
#pragma unroll
          for (int i = 0; i < WG_STEP / 16; ++i) {
            const uint4 v = pipe::lds128(row + 1024u * i);
            add_bf16x2(col[0], col[1], v.x);
            add_bf16x2(col[2], col[3], v.y);
            add_bf16x2(col[4], col[5], v.z);
            add_bf16x2(col[6], col[7], v.w);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(yempty + st));
        return true;
      };
      for (int s = t.s0; s < t.s1;) {
        const int end = min(t.s1, s + WG_SEG);
        // this warp's steps of the chain: all but its last now, that one after the accumulator is read
        int last = -1;
        if (with_db) {
          for (int i = s + ((ew - stage) & 3); ok && i < end; i += 4) {
            const int st = (stage + i - s) & (WG_RING - 1);
            if (i + 4 < end) ok = sum_stage(st);
            else last = st;
          }
        }
        stage = (stage + end - s) & (WG_RING - 1);
        s = end;
        ok = ok && mbar_wait_warp(smem_u32(accf), aphase, g.wait, abort_flag);
        if (!pipe::bar_and(1, 32 * WG_EPI_WARPS, ok)) {
          ok = false;
          break;
        }
        aphase ^= 1;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (32 * c < half) {
            uint32_t r[32];
            tmem_ld_32x32b_x32(tb + 32 * c, r);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; ++j) sum[32 * c + j] += __uint_as_float(r[j]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_relaxed(map_to_rank(smem_u32(acce), lead));
        if (last >= 0) ok = sum_stage(last);
      }
      if (!pipe::bar_and(1, 32 * WG_EPI_WARPS, ok)) {
        ok = false;
        break;
      }
      const int k0 = t.kt * 256 + static_cast<int>(rank) * 128 + q * 32;
      const int n0 = t.n0 + h0;
      if (with_db) {
        // the lanes of a unit, then the eight warps in order; the sums of this CTA's channels go to db, or for
        // a split beside the partial tile
        for (int o = half_n / 8; o < 32; o *= 2) {
#pragma unroll
          for (int i = 0; i < 8; ++i) col[i] += __shfl_xor_sync(0xffffffffu, col[i], o);
        }
        if (lane == 0) bulk_wait_group_read<0>();     // the staging buffer is free
        __syncwarp();
        if (lane < half_n / 8) {
#pragma unroll
          for (int i = 0; i < 8; ++i) pipe::sts32(buf + static_cast<uint32_t>(lane * 8 + i) * 4u, __float_as_uint(col[i]));
        }
        named_bar_sync(1, 32 * WG_EPI_WARPS);
        const int c = threadIdx.x - 32 * WG_EPI_WARP0;     // channel of this CTA's half
        float v = 0.0f;
        if (c < half_n)
          for (int w = 0; w < WG_EPI_WARPS; ++w)
            v += __uint_as_float(pipe::lds32(base + g.off_out + static_cast<uint32_t>(w * WG_OUT_BUF + c * 4)));
        named_bar_sync(1, 32 * WG_EPI_WARPS);              // read before the buffers are used again
        if (c < half_n) {
          const int n = t.n0 + static_cast<int>(rank) * half_n + c;
          if (g.splits > 1) pipe::sts32(base + g.off_out + static_cast<uint32_t>(c) * 4u, __float_as_uint(v));
          else if (n < g.N) g.db[n] = g.accumulate ? g.db[n] + v : v;
        }
      }
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
  cluster_sync_all();            // no CTA leaves while its peer may still signal it; partials are in place
  if (warp == 1) tmem_dealloc_pair(tmem, 512);

  if (g.splits > 1) {
    // split s of the tile and this rank of its pair is the cluster's CTA 2 s + rank
    const GradUnit t = grad_unit(g, u0);
    const int rows = (g.bn + g.splits - 1) / g.splits;
    const int r0 = t.split * rows;
    const int r1 = min(g.bn, r0 + rows);
    for (int i = threadIdx.x; i < (r1 - r0) * 32; i += WG_THREADS) {
      const int ch = r0 + (i >> 5);
      const int quad = i & 31;
      const int n = t.n0 + ch;
      const int k = t.kt * 256 + static_cast<int>(rank) * 128 + 4 * quad;
      if (n >= g.N || k >= g.K) continue;              // K % 16 == 0: the quad is all in or all out
      const uint32_t off = base + static_cast<uint32_t>(ch * 128 + 4 * quad) * 4u;
      float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int sp = 0; sp < g.splits; ++sp) {
        const float4 v = ld_shared_cluster_f4(map_to_rank(off, static_cast<uint32_t>(2 * sp) + rank));
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
    if (g.db != nullptr && t.kt == 0 && t.split == 0 && static_cast<int>(threadIdx.x) < g.bn / 8) {
      const int n = t.n0 + static_cast<int>(rank) * (g.bn / 2) + 4 * static_cast<int>(threadIdx.x);
      if (n < g.N) {                                   // N % 8 == 0
        const uint32_t off = base + g.off_out + threadIdx.x * 16u;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int sp = 0; sp < g.splits; ++sp) {
          const float4 v = ld_shared_cluster_f4(map_to_rank(off, static_cast<uint32_t>(2 * sp) + rank));
          s = make_float4(s.x + v.x, s.y + v.y, s.z + v.z, s.w + v.w);
        }
        float4* p = reinterpret_cast<float4*>(g.db + n);
        if (g.accumulate) {
          const float4 v = *p;
          s = make_float4(v.x + s.x, v.y + s.y, v.z + s.z, v.w + s.w);
        }
        *p = s;
      }
    }
    cluster_sync_all();
  }
}

std::atomic<int> g_grad_clusters[64][3] = {};

cudaLaunchConfig_t grad_config(cudaLaunchAttribute (&attr)[2], int splits, int smem, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(WG_THREADS);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(2 * splits);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cfg;
}

// Clusters of `splits` (1, 2 or 4) pairs that fit on the device at once, one
// CTA per SM (an SM count that is no multiple of the cluster size in a GPC
// leaves SMs idle).
dq_status grad_clusters(const DeviceInfo& d, int splits, int* out) {
  std::atomic<int>& slot = g_grad_clusters[d.device & 63][splits == 1 ? 0 : splits == 2 ? 1 : 2];
  int n = slot.load(std::memory_order_relaxed);
  if (n == 0) {
    // the register split must fit what the block is launched with
    cudaFuncAttributes fa;
    cudaError_t fe = cudaFuncGetAttributes(&fa, act8_grad_kernel);
    if (fe != cudaSuccess) return cuda_fail(fe);
    if (fa.numRegs < WG_REGS) return DQ_ERR_UNSUPPORTED;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = grad_config(attr, splits, WG_MAX_SMEM, nullptr);
    cfg.numAttrs = 1;                                     // the cluster shape only
    cfg.gridDim = dim3(static_cast<unsigned>(2 * splits * (d.sm_count / (2 * splits))));
    const cudaError_t e = cudaOccupancyMaxActiveClusters(&n, act8_grad_kernel, &cfg);
    if (e != cudaSuccess) return cuda_fail(e);
    n = n < 1 ? 1 : n;
    slot.store(n, std::memory_order_relaxed);
  }
  *out = n;
  return DQ_OK;
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
  if (K % 16 != 0 || N % 8 != 0 || lddy % 8 != 0 || M > kMxMaxDim || N > kMxMaxDim || K > kMxMaxDim ||
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

  GradArgs g = {};
  g.M = static_cast<int>(M);
  g.N = static_cast<int>(N);
  g.K = static_cast<int>(K);
  g.kt = static_cast<int>((K + 255) / 256);
  g.ks = static_cast<int>((M + WG_STEP - 1) / WG_STEP);
  if ((st = smem_limit_once(reinterpret_cast<const void*>(&act8_grad_kernel), WG_MAX_SMEM)) != DQ_OK) return st;
  int fit[3];                                             // clusters of 1, 2 and 4 pairs
  for (int i = 0; i < 3; ++i)
    if ((st = grad_clusters(*dev, 1 << i, fit + i)) != DQ_OK) return st;
  const int pairs = fit[0];
  // The plan with the least estimated time: whole waves of tiles, then the
  // remaining ones as they are, halved (128 channels), or with their tokens
  // split over 2 or 4 pairs (a launch of its own), where that still fits in one
  // wave.
  int64_t tiles = 0;
  int rest = 0, rest_splits = 1;
  bool halved = false;
  double best = 1e300;
  for (int bn = 128; bn <= 256; bn += 128) {
    const int64_t nt = (N + bn - 1) / bn, n = nt * g.kt;
    const double step = bn == 256 ? 0.31 : 0.24, ends = 4.0;       // us
    const int64_t waves = n / pairs, r = n % pairs;
    auto take = [&](double cost, int sp, bool hv) {
      if (cost >= 0.98 * best) return;
      best = cost;
      g.bn = bn;
      g.nt = static_cast<int>(nt);
      tiles = n;
      rest = sp > 1 || hv ? static_cast<int>(r) : 0;
      rest_splits = sp;
      halved = hv;
    };
    if (bn == 256 && waves > 0 && r > 0 && 2 * r <= pairs)
      take(static_cast<double>(waves) * (g.ks * step + ends) + g.ks * 0.24 + ends, 1, true);
    for (int sp = 1; sp <= 4; sp *= 2) {
      if (sp > 1 && (r == 0 || r > fit[sp / 2] || g.ks < 4 * sp)) break;
      const double cost = static_cast<double>(waves) * (g.ks * step + ends) +
                          (r > 0 ? (g.ks + sp - 1) / sp * step + ends : 0.0) +
                          (sp > 1 ? (waves > 0 ? 10.0 : 5.0) : 0.0);   // the join, and a second launch
      take(cost, sp, false);
    }
  }
  if (tiles > 0x1fffffff) return DQ_ERR_UNSUPPORTED;
  g.full_chunks = static_cast<int>(N / 64);
  // (the swizzle of the output blocks counts from 1024-byte boundaries)
  g.off_out = static_cast<uint32_t>(WG_RING * g.bn * 64);
  g.off_q = g.off_out + WG_EPI_WARPS * WG_OUT_BUF;
  g.off_bar = g.off_q + WG_RING * WG_CODE_STAGE;
  const int smem = static_cast<int>(g.off_bar) + WG_BAR_BYTES + 1024;
  static_assert(256 + WG_RING * WG_SLOT_COLS <= 512, "tensor memory");
  // The converter groups share the code and slot rings: with an even length a
  // stage belongs to one group (a parity wait cannot tell a lap from the one
  // two before it, and a group that ran ahead of the other could take its
  // stage's next lap for landed).
  static_assert(WG_RING % 2 == 0, "ring length");
  g.dw = dw;
  g.db = db;
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
      (st = make_tmap_chunks(&y3, dy, M, g.full_chunks, static_cast<uint64_t>(lddy) * 2, WG_STEP, g.bn / 128)) != DQ_OK)
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
  auto run = [&](int tile0, int count, int splits) {
    g.tile0 = tile0;
    g.splits = splits;
    g.units = count * splits;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = grad_config(attr, splits, smem, cs);
    cfg.gridDim = dim3(static_cast<unsigned>(2 * (splits > 1 ? g.units : std::min(pairs, g.units))));
    const cudaError_t e = cudaLaunchKernelEx(&cfg, act8_grad_kernel, y3, y2, tq, te, tc, g);
    return e == cudaSuccess ? DQ_OK : cuda_fail(e);
  };
  const int whole = static_cast<int>(tiles) - rest;
  g.t1 = whole;
  if (halved) return run(0, whole + 2 * rest, 1);
  g.t1 = static_cast<int>(tiles);
  if (whole > 0 && (st = run(0, whole, 1)) != DQ_OK) return st;
  return rest > 0 ? run(whole, rest, rest_splits) : DQ_OK;
}

}  // extern "C"
