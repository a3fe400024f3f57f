// mx.h -- sizes and host helpers shared by the microscaled translation units.
#pragma once

#include <cstdint>

#include "internal.h"

namespace dq {

// Largest row or feature count accepted (tile and tensor-map coordinates are
// 32-bit).
constexpr int64_t kMxMaxDim = int64_t(1) << 30;

// Scale tiles (4 blocks each) along the features.
constexpr int64_t fp4_atoms(int64_t K, int fmt) { return (K + (fmt == DQ_FP4_NV ? 63 : 127)) / (fmt == DQ_FP4_NV ? 64 : 128); }

// 2-D tensor map of any element type (boxes of up to 256 elements per
// dimension), zero fill out of bounds; swizzle_bytes 128, or none.
dq_status make_tmap_2d(CUtensorMap* map, CUtensorMapDataType type, const void* base, uint64_t inner, uint64_t outer,
                       uint64_t stride_bytes, uint32_t box_inner, uint32_t box_outer, int swizzle_bytes);

// 3-D tensor map over a row-major bf16 matrix as [chunk][row][64 columns], 128B
// swizzle: one copy of box_rows x box_chunks lays 64-column chunks out one
// after the other.  `chunks` counts whole chunks of 64 columns only.
dq_status make_tmap_chunks(CUtensorMap* map, const void* base, uint64_t rows, uint64_t chunks, uint64_t stride_bytes,
                           uint32_t box_rows, uint32_t box_chunks);

}  // namespace dq
