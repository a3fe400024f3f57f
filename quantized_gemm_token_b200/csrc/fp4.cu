// fp4.cu -- the microscaled 4-bit linear layer's product: e2m1 codes with
// block scales on both sides (fp4_quant.cu describes the formats),
//     acc[m, n] = sum over blocks b of sfa[m, b] sfw[n, b] sum_{k in b} a[m, k] w[n, k]
//     out = bf16(((acc * s_row[m]) * s_col[n]) + bias[n])
// on tcgen05.mma kind::mxf4nvf4.block_scale: the tensor core applies the block
// scales itself, out of tensor memory, and accumulates in fp32.
//
// Operand layout: codes K-major, 256 features (128 bytes, 128B-swizzled) per
// pipeline stage, four MMAs of K = 64 each.  Block scales arrive as the
// 512-byte tiles the quantizer writes (128 rows x 4 blocks: byte 16 (r % 32) +
// 4 (r / 32) + b), which one tcgen05.cp.32x128b.warpx4 puts into four columns
// of tensor memory as the MMA wants them (column r / 32, lane r % 32,
// replicated to the four sub-partitions); a tile serves one MMA (NV) or two
// (MX, selected by the descriptor's scale id).
//
// Sums: the tensor core truncates when it adds an MMA's products (64 features)
// to its fp32 accumulator: it loses less than 2^-23 of the sum so far, always
// downwards.  A row is one chain, so |acc - exact| <= (ceil(K / 64) 2^-23 +
// 2^-21) sum |a w| (2^-21: the additions of a split row).  Operands of one sign,
// nv, pair kernel: 1.9e-6 of the sum at K = 8192, 8.8e-6 at 28672, 9.3e-5 at
// 262144.  A chain taken to registers every 8192 features would lose 1.9e-6 at
// any length and cost 1 us each time, the MMAs standing still (2048 x 16384 ->
// 4096 58.3 -> 60.5 us): far below bf16 output's 2^-9, so it is not done.
#include <cuda_bf16.h>

#include <algorithm>

#include "gemm_common.cuh"
#include "internal.h"
#include "mx.cuh"
#include "mx.h"
#include "pipeline.cuh"
#include "sm100.cuh"

namespace dq {
namespace {

constexpr int F4_KB = 128;           // code bytes per row and stage (256 features)
constexpr int F4_KE = 256;           // features per stage

// Scale tiles per stage (per 128 rows): NV 4 (64 features each), MX 2 (128).
__host__ __device__ constexpr int f4_tiles(bool nv) { return nv ? 4 : 2; }

// Instruction descriptor for kind::mxf4nvf4 with e2m1 A and B, both K-major:
// scale type (0 ue4m3, 1 ue8m0) at bit 23, A / B scale ids at 29 / 4 (which
// half of the four scale bytes a block-32 MMA takes: 0 or 2).
__host__ __device__ constexpr uint32_t idesc_fp4(int M, int N, bool nv, int half) {
  return (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) | (nv ? 0u : 1u << 23) |
         (static_cast<uint32_t>(M >> 4) << 24) | (static_cast<uint32_t>(2 * half) << 29) |
         (static_cast<uint32_t>(2 * half) << 4);
}

// Shared-memory descriptor of one 512-byte scale tile: 32 rows of 16 bytes, no
// swizzle, 8-row groups 128 bytes apart.
__device__ __forceinline__ uint64_t sf_desc(uint32_t addr) {
  return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(128u >> 4) << 16) |
         (static_cast<uint64_t>(128u >> 4) << 32) | (1ull << 46);
}

template <int CG>
__device__ __forceinline__ void cp_sf(uint32_t taddr, uint64_t desc) {
  if constexpr (CG == 1)
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

template <int CG, bool NV>
__device__ __forceinline__ void mma_fp4(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t sfa,
                                        uint32_t sfb, uint32_t accumulate) {
#define DQ_FP4_MMA(CGS, VEC)                                                                               \
  asm volatile(                                                                                            \
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"                                                    \
      "tcgen05.mma.cta_group::" CGS ".kind::mxf4nvf4.block_scale.scale_vec::" VEC                          \
      " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),                                                   \
      "l"(ad), "l"(bd), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)                                    \
      : "memory")
  if constexpr (CG == 1 && NV) DQ_FP4_MMA("1", "4X");
  else if constexpr (CG == 1) DQ_FP4_MMA("1", "2X");
  else if constexpr (NV) DQ_FP4_MMA("2", "4X");
  else DQ_FP4_MMA("2", "2X");
#undef DQ_FP4_MMA
}

// fp32 output: the sum itself, but NaN where a row scale is: an NV row with a
// NaN or an infinity has its NaN there alone (codes and block scales are 0).
__device__ __forceinline__ float raw_sum(float acc, float s_row, float s_col) {
  return isnan(s_row) || isnan(s_col) ? __uint_as_float(0x7fc00000u) : acc;
}

// The same for one row's 32 columns, whose scales lie at shared address `sc`.
// One load and one vote per lane unless there is a NaN among the 32.
__device__ __forceinline__ void raw_sums(uint32_t (&r)[32], float s_row, uint32_t sc, int lane) {
  const uint32_t cols = __ballot_sync(0xffffffffu, isnan(__uint_as_float(pipe::lds32(sc + 4u * lane))));
  const uint32_t bad = isnan(s_row) ? 0xffffffffu : cols;
  if (__any_sync(0xffffffffu, bad != 0u)) {
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if ((bad >> j) & 1u) r[j] = 0x7fc00000u;
  }
}

// ---------------------------------------------------------------- few tokens
// The weight stream is the bound (0.53 - 0.56 bytes per weight at HBM rate),
// so the weight's 128 channels sit on the MMA's M and the tokens on its N, one
// work unit per CTA, two CTAs per SM: their loads overlap each other's
// prologue, pipeline ends and epilogue.  Few channel tiles: the features are
// split over a cluster of up to 8 CTAs, whose fp32 partial tiles are added
// through distributed shared memory in split order.  Measured, K = 8192, N =
// 28672: 24.2 us at one token (NV, 132 MB, 5.47 TB/s, 0.85 of the measured copy
// rate), 23.8 us at 16 (MX).
//   warp 0 producer, warp 1 scale copies and MMAs, warps 2..5 drain the
//   accumulator, all six write the output.
constexpr int FS_THREADS = 192;
constexpr int FS_MAX_STAGES = 8;
constexpr int FS_PREFETCH = 4;
constexpr int FS_BAR_BYTES = 256;

struct FewArgs {
  int M, N;
  int ks_total;            // 64-feature MMA steps: ceil(K / 64)
  int kb_total;            // stages: ceil(K / 256)
  int bn;                  // token columns (M rounded up to 16, <= 64)
  int nt, splits;          // channel tiles, feature splits
  int stages;
  int tmem_cols, sf_col;   // allocation; first column of the scale slots
  int sf_slots;            // tensor-memory scale slots
  uint32_t off_bar;
  const float* s_row;
  const float* s_col;
  const uint16_t* bias;
  void* out;
  int raw;                 // fp32 accumulators instead of bf16
  WaitCtl wait;
};

template <bool NV>
__global__ void __launch_bounds__(FS_THREADS) fp4_few_kernel(const __grid_constant__ CUtensorMap tm_w,
                                                             const __grid_constant__ CUtensorMap tm_x,
                                                             const __grid_constant__ CUtensorMap tm_sw,
                                                             const __grid_constant__ CUtensorMap tm_sx,
                                                             const FewArgs g) {
  constexpr int T = f4_tiles(NV);
  constexpr uint32_t W_BYTES = 128 * F4_KB;
  constexpr uint32_t S_BYTES = T * 512;
  constexpr int SF_COLS = 2 * T * 4;                 // A and B scale columns per stage
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const smem = smem_raw + (base - raw);
  // stage: weight codes, token codes, weight scales, token scales
  const uint32_t x_bytes = static_cast<uint32_t>(g.bn) * F4_KB;
  const uint32_t stage_bytes = W_BYTES + x_bytes + 2 * S_BYTES;   // a multiple of 1024 (bn % 8 == 0)
  uint64_t* const full = reinterpret_cast<uint64_t*>(smem + g.off_bar);
  uint64_t* const empty = full + FS_MAX_STAGES;
  uint64_t* const accf = empty + FS_MAX_STAGES;
  uint32_t* const tmem_holder = reinterpret_cast<uint32_t*>(accf + 1);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < g.stages; ++i) {
      mbar_init(smem_u32(full + i), 1);
      mbar_init(smem_u32(empty + i), 1);
    }
    mbar_init(smem_u32(accf), 1);
    fence_barrier_init();
    tma_prefetch_desc(&tm_w);
    tma_prefetch_desc(&tm_x);
    tma_prefetch_desc(&tm_sw);
    tma_prefetch_desc(&tm_sx);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_holder), static_cast<uint32_t>(g.tmem_cols));
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  griddep_launch_dependents();

  // unit: (channel tile, split), splits neighbouring (one cluster)
  const int nt = blockIdx.x / g.splits;
  const int split = blockIdx.x - nt * g.splits;
  const int kb0 = static_cast<int>(static_cast<int64_t>(split) * g.kb_total / g.splits);
  const int kb1 = static_cast<int>(static_cast<int64_t>(split + 1) * g.kb_total / g.splits);

  // while the kernel before this one (which quantizes the tokens) still runs,
  // the first stages' weights come to L2
  if (warp == 0 && elect_one())
    for (int kb = kb0; kb < min(kb1, kb0 + FS_PREFETCH); ++kb) {
      tma_prefetch_2d(&tm_w, kb * F4_KB, nt * 128);
      tma_prefetch_2d(&tm_sw, kb * T * 64, nt);
    }
  __syncwarp();
  griddep_wait();

  if (warp == 0) {
    int stage = 0;
    uint32_t phase = 0;
    int issued = 0;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!mbar_wait_warp(smem_u32(empty + stage), phase ^ 1, g.wait, abort_flag)) break;
      const uint32_t fb = smem_u32(full + stage);
      const uint32_t sw = base + static_cast<uint32_t>(stage) * stage_bytes;
      if (elect_one()) {
        mbar_arrive_expect_tx(fb, stage_bytes);
        tma_load_2d(sw, &tm_w, fb, kb * F4_KB, nt * 128);
        tma_load_2d(sw + W_BYTES + x_bytes, &tm_sw, fb, kb * T * 64, nt);
        tma_load_2d(sw + W_BYTES, &tm_x, fb, kb * F4_KB, 0);
        tma_load_2d(sw + W_BYTES + x_bytes + S_BYTES, &tm_sx, fb, kb * T * 64, 0);
      }
      __syncwarp();
      ++issued;
      if (++stage == g.stages) {
        stage = 0;
        phase ^= 1;
      }
    }
    // every copy issued lands before the CTA can exit
    volatile int never = 0;
    for (int i = issued > g.stages ? issued - g.stages : 0; i < issued; ++i)
      pipe::wait(smem_u32(full + i % g.stages), static_cast<uint32_t>((i / g.stages) & 1), g.wait, &never);
  } else if (warp == 1) {
    int stage = 0, slot = 0, old = 0;
    uint32_t phase = 0, old_phase = 0;
    for (int kb = kb0, i = 0; kb < kb1; ++kb, ++i) {
      if (!mbar_wait_warp(smem_u32(full + stage), phase, g.wait, abort_flag)) break;
      if (i >= g.sf_slots) {               // the scale slot's previous user has completed
        if (!mbar_wait_warp(smem_u32(empty + old), old_phase, g.wait, abort_flag)) break;
        if (++old == g.stages) {
          old = 0;
          old_phase ^= 1;
        }
      }
      tc_fence_after();
      const uint32_t sw = base + static_cast<uint32_t>(stage) * stage_bytes;
      const uint32_t sfa = tmem + static_cast<uint32_t>(g.sf_col + slot * SF_COLS);
      if (++slot == g.sf_slots) slot = 0;
      const uint32_t sfb = sfa + T * 4;
      const int steps = min(4, g.ks_total - 4 * kb);
      const uint64_t da = sf_desc(sw + W_BYTES + x_bytes), db = sf_desc(sw + W_BYTES + x_bytes + S_BYTES);
      const uint64_t ad = smem_desc_kmajor<128>(sw);
      const uint64_t bd = smem_desc_kmajor<128>(sw + W_BYTES);
      if (elect_one()) {
#pragma unroll
        for (int t = 0; t < T; ++t) {
          cp_sf<1>(sfa + 4 * t, da + 32 * t);
          cp_sf<1>(sfb + 4 * t, db + 32 * t);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (k < steps) {
            const int t = NV ? k : k >> 1;
            mma_fp4<1, NV>(tmem, ad + 2 * k, bd + 2 * k, idesc_fp4(128, g.bn, NV, NV ? 0 : k & 1), sfa + 4 * t,
                           sfb + 4 * t, (i > 0 || k > 0) ? 1u : 0u);
          }
        mma_commit(smem_u32(empty + stage));
      }
      __syncwarp();
      if (++stage == g.stages) {
        stage = 0;
        phase ^= 1;
      }
    }
    // every MMA issued has completed once this flips
    if (elect_one()) mma_commit(smem_u32(accf));
    __syncwarp();
    volatile int never = 0;
    pipe::wait(smem_u32(accf), 0, g.wait, &never);
  }
  __syncwarp();
  // ------------------------------------------------------------ epilogue
  // The accumulator goes to shared memory as [token][channel] fp32 (the
  // consumed stage ring), from where the split's CTAs add their shares.
  const bool ok = pipe::wait(smem_u32(accf), 0, g.wait, abort_flag);
  tc_fence_after();
  if (warp >= 2 && __all_sync(0xffffffffu, ok)) {
    const int q = warp & 3;
    const uint32_t tb = tmem + (static_cast<uint32_t>(q * 32) << 16);
    for (int c0 = 0; c0 < g.bn; c0 += 16) {
      uint32_t r[16];
      tmem_ld_32x32b_x16(tb + c0, r);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 16; ++j)
        pipe::sts32(base + static_cast<uint32_t>((c0 + j) * 128 + q * 32 + lane) * 4u, r[j]);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, static_cast<uint32_t>(g.tmem_cols));
  if (g.splits > 1) cluster_sync_all();
  const int rows = (g.bn + g.splits - 1) / g.splits;
  const int r0 = split * rows;
  const int r1 = min(g.bn, r0 + rows);
  for (int i = threadIdx.x; i < (r1 - r0) * 32; i += FS_THREADS) {
    const int m = r0 + (i >> 5);
    const int quad = i & 31;
    const int ch = nt * 128 + 4 * quad;
    if (m >= g.M || ch >= g.N) continue;              // N % 8 == 0: the quad is all in or all out
    const uint32_t off = base + static_cast<uint32_t>(m * 128 + 4 * quad) * 4u;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (g.splits > 1) {
      for (int sp = 0; sp < g.splits; ++sp) {
        const float4 v = ld_shared_cluster_f4(map_to_rank(off, static_cast<uint32_t>(sp)));
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
      }
    } else {
      const uint4 v = pipe::lds128(off);
      s = make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
    }
    const int64_t o = static_cast<int64_t>(m) * g.N + ch;
    const float sr = g.s_row != nullptr ? __ldg(g.s_row + m) : 1.0f;
    float4 sc = make_float4(1.f, 1.f, 1.f, 1.f);
    if (g.s_col != nullptr) sc = __ldg(reinterpret_cast<const float4*>(g.s_col + ch));
    if (g.raw) {
      *reinterpret_cast<float4*>(static_cast<float*>(g.out) + o) =
          make_float4(raw_sum(s.x, sr, sc.x), raw_sum(s.y, sr, sc.y), raw_sum(s.z, sr, sc.z), raw_sum(s.w, sr, sc.w));
      continue;
    }
    float y[4] = {__fmul_rn(__fmul_rn(s.x, sr), sc.x), __fmul_rn(__fmul_rn(s.y, sr), sc.y),
                  __fmul_rn(__fmul_rn(s.z, sr), sc.z), __fmul_rn(__fmul_rn(s.w, sr), sc.w)};
    if (g.bias != nullptr) {
      const uint2 b = __ldg(reinterpret_cast<const uint2*>(g.bias + ch));
      y[0] = __fadd_rn(y[0], __uint_as_float(b.x << 16));
      y[1] = __fadd_rn(y[1], __uint_as_float(b.x & 0xffff0000u));
      y[2] = __fadd_rn(y[2], __uint_as_float(b.y << 16));
      y[3] = __fadd_rn(y[3], __uint_as_float(b.y & 0xffff0000u));
    }
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(g.out) + o) =
        make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
  }
  if (g.splits > 1) cluster_sync_all();               // peers have read this CTA's partials
}

// ---------------------------------------------------------------- many tokens
// A pair of SMs per 256 x 256 (or narrower) tile (cta_group::2), as the int8
// pair kernel: each CTA loads its 128 token rows and half of the tile's weight
// rows, plus its own rows' scale tiles and ALL of the tile's weight scale tiles
// (each SM's tensor core multiplies its rows with every column, so both tensor
// memories need every column's scales).
//   warp 0 producer, warp 1 (leader) scale copies and MMAs, warps 2..9
//   epilogue, two per TMEM sub-partition on alternate 32-column chunks.
// What bounds it: a 256-feature stage is 512 cycles of MMAs, and a CTA loads
// 38.9 KB for it (NV), 608 cycles at the 64 bytes per cycle an SM takes from L2;
// measured 660 - 680.  Narrower tiles load more per MMA (192 columns: 34.8 KB
// for 384 cycles).  Measured: 8192^3 196 us (NV, 5.62 PFLOP/s, 0.83 of four
// times the measured bf16 rate), 184 us (MX); 2048 x 4096 x 4096 19.0 us, of
// which 5.7 us are launch, prologue and the pipeline's ends and 3.4 us the
// last tiles' epilogue (16.8 MB of output).
template <bool NV>
struct CfgP {
  static constexpr int BN = 256;
  static constexpr int T = f4_tiles(NV);
  static constexpr int RB = 2;                          // weight scale row blocks of a tile
  static constexpr int A_BYTES = 128 * F4_KB;
  static constexpr int B_BYTES = (BN / 2) * F4_KB;
  static constexpr int SA_BYTES = T * 512;
  static constexpr int SB_BYTES = RB * T * 512;
  static constexpr int CTA_BYTES = A_BYTES + B_BYTES + SA_BYTES + SB_BYTES;
  static constexpr int EPI_WARPS = 8;
  static constexpr int CHUNKS = BN / 32 / (EPI_WARPS / 4);   // 32-column chunks per epilogue warp
  static constexpr int OUT_BUF_BYTES = 32 * 32 * 4;
  static constexpr int OUT_BYTES = EPI_WARPS * OUT_BUF_BYTES;
  static constexpr int BAR_BYTES = 512;
  static constexpr int SLACK = 1024;
  static constexpr int STAGES = (227 * 1024 - SLACK - BAR_BYTES - OUT_BYTES - kScSlotBytes) / CTA_BYTES;
  static constexpr int SF_A = T * 4, SF_B = T * RB * 4; // scale columns per stage
  static constexpr int SF_COLS = SF_A + SF_B;
  static constexpr int SF_COL0 = BN;                    // after the accumulator
  static constexpr int THREADS = 64 + 32 * EPI_WARPS;
  static constexpr int OFF_SA = STAGES * (A_BYTES + B_BYTES);
  static constexpr int OFF_SB = OFF_SA + STAGES * SA_BYTES;
  static constexpr int OFF_OUT = OFF_SB + STAGES * SB_BYTES;
  static constexpr int OFF_SC = OFF_OUT + OUT_BYTES;
  static constexpr int OFF_BARS = OFF_SC + kScSlotBytes;
  static constexpr int SMEM_BYTES = OFF_BARS + BAR_BYTES + SLACK;
  static_assert(STAGES >= 3 && SMEM_BYTES <= 227 * 1024, "shared memory");
  // every stage has a scale slot of its own, so a slot is free when its stage is
  static_assert(SF_COL0 + STAGES * SF_COLS <= 512, "tensor memory");
  static_assert((2 * STAGES + 5) * 8 + 8 <= BAR_BYTES, "barrier area");
};

// RAW: fp32 output (a template switch: as a run-time test before each block's
// store it cost bf16 output 0.4 - 0.8 us).
template <bool NV, bool RAW>
__global__ void __launch_bounds__(CfgP<NV>::THREADS, 1)
    fp4_pair_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                    const __grid_constant__ CUtensorMap tm_b2, const __grid_constant__ CUtensorMap tm_sa,
                    const __grid_constant__ CUtensorMap tm_sb, const __grid_constant__ CUtensorMap tm_c,
                    const __grid_constant__ GemmArgs g) {
  using C = CfgP<NV>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sA = smem_u32(smem);
  const uint32_t sB = sA + C::STAGES * C::A_BYTES;
  const uint32_t sSA = sA + C::OFF_SA;
  const uint32_t sSB = sA + C::OFF_SB;
  uint8_t* sOut = smem + C::OFF_OUT;
  const uint32_t sc_slot = sA + C::OFF_SC;
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(smem + C::OFF_BARS);
  uint64_t* empty_bar = full_bar + C::STAGES;
  uint64_t* accf_bar = empty_bar + C::STAGES;
  uint64_t* acce_bar = accf_bar + 1;
  uint64_t* drain_bar = acce_bar + 1;
  uint64_t* sc_full = drain_bar + 1;
  uint64_t* sc_free = sc_full + 1;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(sc_free + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int G = gridDim.x >> 1;
  const int pair = blockIdx.x >> 1;

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(smem_u32(full_bar + s), 1);
      mbar_init(smem_u32(empty_bar + s), 1);
    }
    mbar_init(smem_u32(accf_bar), 1);
    mbar_init(smem_u32(acce_bar), 2 * C::EPI_WARPS);
    mbar_init(smem_u32(drain_bar), 1);
    mbar_init(smem_u32(sc_full), 1);
    mbar_init(smem_u32(sc_free), C::EPI_WARPS);
    fence_barrier_init();
    tma_prefetch_desc(&tm_a);
    tma_prefetch_desc(&tm_b);
    tma_prefetch_desc(&tm_b2);
    tma_prefetch_desc(&tm_sa);
    tma_prefetch_desc(&tm_sb);
    tma_prefetch_desc(&tm_c);
  }
  // no column scales (MX): the slot holds ones for the whole launch
  if (g.s_col == nullptr)
    for (int i = threadIdx.x; i < 256; i += C::THREADS) pipe::sts32(sc_slot + 4u * i, __float_as_uint(1.0f));
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_holder), 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  griddep_launch_dependents();

  // while the kernel before this one (which quantizes the tokens) still runs,
  // the first tile's first stages of weights come to L2, one ring's worth (the
  // layer of 2048 x 4096 x 4096 with its quantizer 24.7 us, 25.2 without; twice
  // the ring 25.1, all 16 stages 26.3)
  if (warp == 0 && pair < g.num_tiles && elect_one()) {
    const TileGeom geo = tile_geom(g, pair, C::BN, true);
    const void* const tmb = geo.narrow ? &tm_b2 : &tm_b;
    for (int kb = 0; kb < min(g.kb_total, C::STAGES); ++kb) {
      tma_prefetch_2d(tmb, kb * F4_KB, geo.n0 + static_cast<int>(rank) * (geo.width / 2));
      if (leader) tma_prefetch_2d(&tm_sb, kb * C::T * 64, geo.n0 / 128);
    }
  }
  __syncwarp();
  griddep_wait();

  if (warp == 0) {
    // ------------------------------------------------------------ producer (both CTAs)
    int stage = 0;
    uint32_t phase = 0;
    long long issued = 0;
    bool ok = true, tested = true;       // tested: the next stage was found free
    for (int t = pair; ok && t < g.num_tiles; t += G) {
      const TileGeom geo = tile_geom(g, t, C::BN, true);
      const int ta = geo.ta, n0 = geo.n0, half = geo.width / 2;
      const uint32_t stage_tx = 2u * static_cast<uint32_t>(C::CTA_BYTES - C::B_BYTES + half * F4_KB);
      const void* const tmb = geo.narrow ? &tm_b2 : &tm_b;
      for (int kb = 0; kb < g.kb_total; ++kb) {
        if (!tested && !mbar_wait_warp(smem_u32(empty_bar + stage), phase ^ 1, g.wait, abort_flag)) {
          ok = false;
          break;
        }
        const uint32_t fb = smem_u32(full_bar + stage);
        const uint32_t fbl = map_to_rank(fb, 0);
        const int now = stage;
        ++issued;
        if (++stage == C::STAGES) {
          stage = 0;
          phase ^= 1;
        }
        const bool te = mbar_test(smem_u32(empty_bar + stage), phase ^ 1);
        if (elect_one()) {
          if (leader) mbar_arrive_expect_tx(fb, stage_tx);
          tma_load_2d_pair(sA + now * C::A_BYTES, &tm_a, fbl, kb * F4_KB, ta * 256 + static_cast<int>(rank) * 128);
          tma_load_2d_pair(sB + now * C::B_BYTES, tmb, fbl, kb * F4_KB, n0 + static_cast<int>(rank) * half);
          tma_load_2d_pair(sSA + now * C::SA_BYTES, &tm_sa, fbl, kb * C::T * 64, ta * 2 + static_cast<int>(rank));
          tma_load_2d_pair(sSB + now * C::SB_BYTES, &tm_sb, fbl, kb * C::T * 64, n0 / 128);
        }
        __syncwarp();
        tested = __all_sync(0xffffffffu, te);
      }
    }
    if (!ok) {
      // Loads already issued land before the CTA leaves (see gemm2sm.cu).
      if (leader) {
        WaitCtl quick = g.wait;
        quick.timeout_ns = quick.timeout_ns < 50000000ull ? quick.timeout_ns : 50000000ull;
        volatile int never = 0;
        for (long long i = 0; i < issued && i < C::STAGES; ++i) {
          if (--stage < 0) {
            stage = C::STAGES - 1;
            phase ^= 1;
          }
          mbar_wait(smem_u32(full_bar + stage), phase, quick, &never);
        }
      } else {
        const uint64_t t0 = globaltimer();
        while (globaltimer() - t0 < 100000ull) {
        }
      }
      __syncwarp();
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (leader)
    if (leader) {
      int stage = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true, tested = false;     // tested: the next stage was found landed
      const int ks_total = (g.K + 63) / 64;
      for (int t = pair; ok && t < g.num_tiles; t += G) {
        const TileGeom geo = tile_geom(g, t, C::BN, true);
        // a tile may start in the middle of a scale row block (widths of 64 and 192)
        const uint32_t col_b = static_cast<uint32_t>((geo.n0 % 128) / 32);
        const uint32_t id0 = idesc_fp4(256, geo.width, NV, 0), id1 = NV ? id0 : idesc_fp4(256, geo.width, NV, 1);
        if (!mbar_wait_warp(smem_u32(acce_bar), acc_phase ^ 1, g.wait, abort_flag)) break;
        acc_phase ^= 1;
        tc_fence_after();
        for (int kb = 0; kb < g.kb_total; ++kb) {
          if (!tested && !mbar_wait_warp(smem_u32(full_bar + stage), phase, g.wait, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sfa = tmem_base + C::SF_COL0 + static_cast<uint32_t>(stage) * C::SF_COLS;
          const uint32_t sfb = sfa + C::SF_A;
          const uint64_t da = sf_desc(sSA + stage * C::SA_BYTES), db = sf_desc(sSB + stage * C::SB_BYTES);
          const uint64_t ad = smem_desc_kmajor<128>(sA + stage * C::A_BYTES);
          const uint64_t bd = smem_desc_kmajor<128>(sB + stage * C::B_BYTES);
          const uint32_t eb = smem_u32(empty_bar + stage);
          const int steps = min(4, ks_total - 4 * kb);
          if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1;
          }
          // the next stage's barrier is tested before this stage's MMAs are issued
          const bool tf = mbar_test(smem_u32(full_bar + stage), phase);
          if (elect_one()) {
#pragma unroll
            for (int s = 0; s < C::T; ++s) {
              cp_sf<2>(sfa + 4 * s, da + 32 * s);
#pragma unroll
              for (int r = 0; r < C::RB; ++r) cp_sf<2>(sfb + 4 * (s * C::RB + r), db + 32 * (r * C::T + s));
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (k < steps) {
                const int s = NV ? k : k >> 1;
                mma_fp4<2, NV>(tmem_base, ad + 2 * k, bd + 2 * k, (k & 1) ? id1 : id0, sfa + 4 * s,
                               sfb + 4 * C::RB * s + col_b, (kb > 0 || k > 0) ? 1u : 0u);
              }
            mma_commit_pair_both(eb);
          }
          __syncwarp();
          tested = __all_sync(0xffffffffu, tf);
        }
        if (!ok) break;
        if (elect_one()) mma_commit_pair_both(smem_u32(accf_bar));
        __syncwarp();
      }
      if (elect_one()) mma_commit_pair(map_to_rank(smem_u32(drain_bar), 0));
      __syncwarp();
      volatile int never = 0;
      mbar_wait(smem_u32(drain_bar), 0, g.wait, &never);
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ epilogue (both CTAs)
    constexpr int GROUPS = C::EPI_WARPS / 4;
    const int ew = warp - 2;
    const int sp = warp & 3;
    const int grp = ew / 4;
    const int ep_tid = threadIdx.x - 64;
    uint8_t* my_out = sOut + ew * C::OUT_BUF_BYTES;
    int out_flip = 0;
    auto next_buf = [&]() -> uint8_t* {
      if (g.out_s32) {
        if (lane == 0) bulk_wait_group_read<0>();
        __syncwarp();
        return my_out;
      }
      if (lane == 0) bulk_wait_group_read<1>();
      __syncwarp();
      uint8_t* b = my_out + out_flip * (C::OUT_BUF_BYTES / 2);
      out_flip ^= 1;
      return b;
    };
    uint32_t acc_phase = 0;
    uint32_t sc_phase = 0;
    for (int t = pair; t < g.num_tiles; t += G) {
      const TileGeom geo = tile_geom(g, t, C::BN, true);
      const int n0 = geo.n0, nch = geo.width / 32;
      const int m_slab = geo.ta * 256 + static_cast<int>(rank) * 128 + sp * 32;
      const int m = m_slab + lane;
      bool free_slot = true;
      if (ep_tid == 0) {
        free_slot = t == pair || mbar_wait(smem_u32(sc_free), sc_phase ^ 1, g.wait, abort_flag);
        if (free_slot) {
          // the tile's column scales (unless there are none) and bias
          const int ncols = min(geo.width, g.N - n0);
          const uint32_t sb = g.s_col != nullptr ? static_cast<uint32_t>(ncols) * 4u : 0u;
          const uint32_t bb = !g.out_s32 && g.bias != nullptr ? static_cast<uint32_t>(ncols) * 2u : 0u;
          mbar_arrive_expect_tx(smem_u32(sc_full), sb + bb);
          if (sb) bulk_load_1d(sc_slot, g.s_col + n0, sb, smem_u32(sc_full));
          if (bb) bulk_load_1d(sc_slot + kScBiasOff, g.bias + n0, bb, smem_u32(sc_full));
        }
      }
      if (!__all_sync(0xffffffffu, free_slot)) break;    // (a warp leaves whole)
      const float srow = (g.s_row != nullptr && m < g.M) ? __ldg(g.s_row + m) : 1.0f;
      if (!mbar_wait_warp(smem_u32(accf_bar), acc_phase, g.wait, abort_flag)) break;
      if (!mbar_wait_warp(smem_u32(sc_full), sc_phase, g.wait, abort_flag)) break;
      acc_phase ^= 1;
      sc_phase ^= 1;
      tc_fence_after();
      // The one accumulator (256 columns leave tensor memory only for the
      // scales beside it) is taken into registers whole and handed back before
      // any of it is scaled and stored, so the next tile's MMAs wait for the
      // reads alone.
      const uint32_t tbase = tmem_base + (static_cast<uint32_t>(sp * 32) << 16);
      uint32_t r[C::CHUNKS][32];
#pragma unroll
      for (int i = 0; i < C::CHUNKS; ++i)
        if (grp + i * GROUPS < nch) tmem_ld_32x32b_x32(tbase + (grp + i * GROUPS) * 32, r[i]);
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(map_to_rank(smem_u32(acce_bar), 0));
#pragma unroll
      for (int i = 0; i < C::CHUNKS; ++i) {
        const int c = grp + i * GROUPS;
        // a block wholly past the matrix is not stored and takes no buffer: the wait for a buffer counts stores
        if (c < nch && n0 + c * 32 < g.N && m_slab < g.M) {
          if constexpr (RAW) raw_sums(r[i], srow, sc_slot + static_cast<uint32_t>(c) * 128u, lane);
          store_row_chunk_staged<true>(g, &tm_c, next_buf(), lane, m_slab, n0 + c * 32, r[i], srow, sc_slot, c * 32);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(sc_free));
    }
    if (lane == 0) bulk_wait_group<0>();
    __syncwarp();
  }

  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem_base, 512);
}

// ---------------------------------------------------------------- host

// Scale tiles [row blocks][tiles x 512 B] as 8-byte elements, box one stage
// (64 elements per tile) x `box_rows` row blocks; zero fill past the end.
dq_status make_tmap_sf(CUtensorMap* map, const uint8_t* sf, int64_t row_blocks, int64_t atoms, int tiles, int box_rows) {
  return make_tmap_2d(map, CU_TENSOR_MAP_DATA_TYPE_UINT64, sf, static_cast<uint64_t>(atoms) * 64,
                      static_cast<uint64_t>(row_blocks), static_cast<uint64_t>(atoms) * 512,
                      static_cast<uint32_t>(tiles) * 64, static_cast<uint32_t>(box_rows), 0);
}

// Two CTAs per SM.  All units resident at once share the memory's bandwidth
// evenly and end together, whatever their number per SM, so only too few of
// them call for a split, and not one of less than eight stages (K = 1280, N =
// 5120, one token: 4.1 us whole, 4.8 in two; K = 2048, N = 512: 4.1 in four, 4.7
// in two).
int few_splits(int nt, int kb_total, int sm_count) {
  int splits = 1;
  if (kb_total < 8) return 1;
  while (splits < 8 && nt * splits <= sm_count && kb_total / (2 * splits) >= 2) splits *= 2;
  return splits;
}

template <bool NV>
dq_status launch_few(const uint8_t* A, const uint8_t* sfa, int64_t M, int64_t K, const uint8_t* W, const uint8_t* sfw,
                     int64_t N, FewArgs g, int sm_count, cudaStream_t stream) {
  constexpr int T = f4_tiles(NV);
  const int64_t atoms = fp4_atoms(K, NV ? DQ_FP4_NV : DQ_FP4_MX);
  g.bn = static_cast<int>((M + 15) / 16 * 16);
  g.nt = static_cast<int>((N + 127) / 128);
  g.kb_total = static_cast<int>((K + F4_KE - 1) / F4_KE);
  g.ks_total = static_cast<int>((K + 63) / 64);
  g.splits = few_splits(g.nt, g.kb_total, sm_count);
  const int stage_bytes = 128 * F4_KB + g.bn * F4_KB + 2 * T * 512;
  const int limit = (227 * 1024 - 2 * 1024) / 2;      // two CTAs per SM
  g.stages = (limit - 1024 - FS_BAR_BYTES) / stage_bytes;
  const int max_need = (g.kb_total + g.splits - 1) / g.splits;
  g.stages = std::min({g.stages, FS_MAX_STAGES, max_need});
  // the fp32 tile reuses the ring
  const int ring = std::max(g.stages * stage_bytes, g.bn * 512);
  g.off_bar = static_cast<uint32_t>((ring + 15) / 16 * 16);
  const int smem = static_cast<int>(g.off_bar) + FS_BAR_BYTES + 1024;
  constexpr int SF_COLS = 2 * T * 4;
  g.sf_col = g.bn <= 32 ? 32 : 64;
  g.tmem_cols = 128;
  g.sf_slots = std::min((g.tmem_cols - g.sf_col) / SF_COLS, g.stages);
  CUtensorMap tw, tx, tsw, tsx;
  dq_status st;
  if ((st = make_tmap_u8_2d(&tw, W, K / 2, N, K / 2, F4_KB, 128, 128)) != DQ_OK) return st;
  if ((st = make_tmap_u8_2d(&tx, A, K / 2, M, K / 2, F4_KB, g.bn, 128)) != DQ_OK) return st;
  if ((st = make_tmap_sf(&tsw, sfw, (N + 127) / 128, atoms, T, 1)) != DQ_OK) return st;
  if ((st = make_tmap_sf(&tsx, sfa, (M + 127) / 128, atoms, T, 1)) != DQ_OK) return st;
  auto k = fp4_few_kernel<NV>;
  if ((st = smem_limit_once(reinterpret_cast<const void*>(k), limit)) != DQ_OK) return st;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(g.nt * g.splits));
  cfg.blockDim = dim3(FS_THREADS);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(g.splits);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = g.splits > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, k, tw, tx, tsw, tsx, g);
  return e == cudaSuccess ? DQ_OK : cuda_fail(e);
}

// Tiles for `pairs` CTA pairs: 256 columns wide, or all of one narrower
// width, or whole waves of 256 and the rest in one wave of a narrower width;
// whichever takes the fewest stage times.  A stage's time follows the bytes
// that a CTA loads for it (the bound: 38.9 KB at 256 columns against 512 cycles
// of MMAs), a tile's ends cost about 2.5 stages.
struct PairPlan {
  int t1, bn2, mb0, c_start, first_cnt, per_row, num_tiles;
};
bool plan_pair(int64_t M, int64_t N, int kb_total, int64_t pairs, PairPlan& out) {
  const int64_t at = (M + 255) / 256, bt = (N + 255) / 256, T = at * bt;
  if (T > 0x3fffff) return false;                    // (64 columns: at most four times as many)
  auto cost = [&](int w) { return kb_total * (0.51 + 0.49 * w / 256) + 2.5 * w / 256; };
  double best = static_cast<double>((T + pairs - 1) / pairs) * cost(256);
  out = PairPlan{static_cast<int>(T), 0, 0, 0, 0, 0, static_cast<int>(T)};
  for (int w = 192; w >= 64; w -= 64) {
    const int64_t row = (N + w - 1) / w, n = at * row;
    const double c = static_cast<double>((n + pairs - 1) / pairs) * cost(w);
    if (c < 0.98 * best) {
      best = c;
      out = PairPlan{0, w, 0, 0, static_cast<int>(row), static_cast<int>(row), static_cast<int>(n)};
    }
    const int64_t t1 = T / pairs * pairs;            // whole waves
    if (t1 == 0 || t1 == T) continue;
    const int64_t mb0 = t1 / bt, c0 = (t1 % bt) * 256;
    const int64_t first = (N - c0 + w - 1) / w, t2 = first + (at - mb0 - 1) * row;
    if (t2 > pairs) continue;
    const double c2 = static_cast<double>(t1 / pairs) * cost(256) + cost(w);
    if (c2 < 0.98 * best) {
      best = c2;
      out = PairPlan{static_cast<int>(t1), w, static_cast<int>(mb0), static_cast<int>(c0), static_cast<int>(first),
                     static_cast<int>(row), static_cast<int>(t1 + t2)};
    }
  }
  return true;
}

template <bool NV>
dq_status launch_pair(const uint8_t* A, const uint8_t* sfa, const uint8_t* W, const uint8_t* sfw, GemmArgs g, int pairs,
                      cudaStream_t stream) {
  using C = CfgP<NV>;
  const int64_t K = g.K;
  const int64_t atoms = fp4_atoms(K, NV ? DQ_FP4_NV : DQ_FP4_MX);
  g.a_tiles = (g.M + 255) / 256;
  g.b_tiles = (g.N + C::BN - 1) / C::BN;
  g.kb_total = static_cast<int>((K + F4_KE - 1) / F4_KE);
  PairPlan p;
  if (!plan_pair(g.M, g.N, g.kb_total, pairs, p)) return DQ_ERR_UNSUPPORTED;
  g.t1 = p.t1;
  g.bn2 = p.bn2;
  g.mb0 = p.mb0;
  g.c_start = p.c_start;
  g.first_cnt = p.first_cnt;
  g.per_row = p.per_row;
  g.num_tiles = p.num_tiles;
  CUtensorMap ta, tb, tb2, tsa, tsb, tc;
  dq_status st;
  if ((st = make_tmap_u8_2d(&ta, A, K / 2, g.M, K / 2, F4_KB, 128, 128)) != DQ_OK) return st;
  if ((st = make_tmap_u8_2d(&tb, W, K / 2, g.N, K / 2, F4_KB, C::BN / 2, 128)) != DQ_OK) return st;
  tb2 = tb;
  if (g.bn2 > 0 && (st = make_tmap_u8_2d(&tb2, W, K / 2, g.N, K / 2, F4_KB, g.bn2 / 2, 128)) != DQ_OK) return st;
  if ((st = make_tmap_sf(&tsa, sfa, (g.M + 127) / 128, atoms, C::T, 1)) != DQ_OK) return st;
  if ((st = make_tmap_sf(&tsb, sfw, (g.N + 127) / 128, atoms, C::T, C::RB)) != DQ_OK) return st;
  if ((st = make_tmap_out_2d(&tc, g.out, g.N, g.M, g.out_s32 ? 4 : 2)) != DQ_OK) return st;
  auto k = g.out_s32 ? fp4_pair_kernel<NV, true> : fp4_pair_kernel<NV, false>;
  if ((st = smem_limit_once(reinterpret_cast<const void*>(k), C::SMEM_BYTES)) != DQ_OK) return st;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * std::min(pairs, g.num_tiles)));
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM_BYTES;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, k, ta, tb, tb2, tsa, tsb, tc, g);
  return e == cudaSuccess ? DQ_OK : cuda_fail(e);
}

}  // namespace
}  // namespace dq

using namespace dq;

extern "C" {

dq_status dq_fp4_linear(const uint8_t* A, const uint8_t* sfa, const float* s_row, int64_t M, int64_t K,
                        const uint8_t* W, const uint8_t* sfw, const float* s_col, int64_t N, int fmt,
                        const void* bias_bf16, void* out, dq_out_dtype out_dtype, dq_stream_t stream) {
  if ((fmt != DQ_FP4_MX && fmt != DQ_FP4_NV) || M < 0 || N < 1 || K < 1) return DQ_ERR_INVALID_ARG;
  if (out_dtype != DQ_OUT_BF16 && out_dtype != DQ_OUT_F32) return DQ_ERR_INVALID_ARG;
  if (W == nullptr || sfw == nullptr || (M > 0 && (A == nullptr || sfa == nullptr || out == nullptr)))
    return DQ_ERR_INVALID_ARG;
  if (K % 32 != 0 || N % 8 != 0 || M > kMxMaxDim || N > kMxMaxDim || K > kMxMaxDim) return DQ_ERR_UNSUPPORTED;
  if (!aligned(A, 16) || !aligned(sfa, 16) || !aligned(W, 16) || !aligned(sfw, 16) || !aligned(out, 16) ||
      !aligned(s_row, 4) || !aligned(s_col, 16) || !aligned(bias_bf16, 16))
    return DQ_ERR_UNSUPPORTED;
  DeviceInfo* d = nullptr;
  dq_status st = current_device(&d);
  if (st != DQ_OK) return st;
  if (M == 0) return DQ_OK;
  const auto cs = reinterpret_cast<cudaStream_t>(stream);
  const bool nv = fmt == DQ_FP4_NV;
  const WaitCtl wait{d->err_word, wait_timeout_ns()};
  // Few tokens: up to 32, or 64 where the pair kernel's tiles would leave SMs idle (long rows) or their ends would
  // show (many channel tiles).  64 tokens, this kernel against the pair kernel: K = 8192, N = 512 6.6 us against
  // 12.1, N = 4096 9.7 against 13.6, N = 28672 27.5 against 31.9; K = 4096, N = 4096 8.9 against 8.9; K = 1280, N =
  // 28672 9.0 against 11.1, but N = 5120 6.9 against 6.1; 32 tokens: 5.4 against 5.9.
  const int64_t nt = (N + 127) / 128;
  if (M <= 32 || (M <= 64 && (K > 7 * F4_KE || nt >= d->sm_count))) {
    FewArgs f = {};
    f.M = static_cast<int>(M);
    f.N = static_cast<int>(N);
    f.s_row = s_row;
    f.s_col = s_col;
    f.bias = static_cast<const uint16_t*>(bias_bf16);
    f.out = out;
    f.raw = out_dtype == DQ_OUT_F32;
    f.wait = wait;
    return nv ? launch_few<true>(A, sfa, M, K, W, sfw, N, f, d->sm_count, cs)
              : launch_few<false>(A, sfa, M, K, W, sfw, N, f, d->sm_count, cs);
  }
  GemmArgs g = {};
  g.M = static_cast<int>(M);
  g.N = static_cast<int>(N);
  g.K = static_cast<int>(K);
  g.s_row = s_row;
  g.s_col = s_col;
  g.bias = static_cast<const uint16_t*>(bias_bf16);
  g.out = out;
  g.out_s32 = out_dtype == DQ_OUT_F32;
  g.wait = wait;
  int pairs = 0;
  if ((st = pair_slots(*d, &pairs)) != DQ_OK) return st;
  return nv ? launch_pair<true>(A, sfa, W, sfw, g, pairs, cs) : launch_pair<false>(A, sfa, W, sfw, g, pairs, cs);
}

}  // extern "C"
