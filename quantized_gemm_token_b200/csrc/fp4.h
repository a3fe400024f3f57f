// fp4.h -- sizes shared by the microscaled 4-bit translation units.
#pragma once

#include <cstdint>

#include "../../include/dq.h"

namespace dq {

// Largest row or feature count accepted (tile and tensor-map coordinates are
// 32-bit).
constexpr int64_t kFp4MaxDim = int64_t(1) << 30;

// Scale tiles (4 blocks each) along the features.
constexpr int64_t fp4_atoms(int64_t K, int fmt) { return (K + (fmt == DQ_FP4_NV ? 63 : 127)) / (fmt == DQ_FP4_NV ? 64 : 128); }

}  // namespace dq
