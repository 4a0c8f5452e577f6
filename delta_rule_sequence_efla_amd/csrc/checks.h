// checks.h -- argument checks shared by the C entry points.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "efla.h"

namespace {

inline bool valid_dim(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }
inline bool valid_chunk(int c) { return c == 16 || c == 32 || c == 64; }
inline bool valid_dtype(efla_dtype dt) { return dt == EFLA_F32 || dt == EFLA_BF16; }
inline bool valid_rule(efla_rule r) { return r == EFLA_RULE_EXACT || r == EFLA_RULE_EULER; }
inline size_t elem_bytes(efla_dtype dt) { return dt == EFLA_BF16 ? 2 : 4; }
constexpr int64_t kMaxGrid = (int64_t(1) << 31) - 1;

inline efla_status from_hip(hipError_t e) { return e == hipSuccess ? EFLA_OK : EFLA_ERR_HIP; }

inline size_t al256(size_t x) { return (x + 255) / 256 * 256; }

// The kernels move q, k, v, T and states with 16-byte vector accesses.
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Shape checks shared by the chunked entry points (pointer checks are separate).
inline efla_status check_chunk_shape(int B, int H, int64_t L, int d_k, int d_v, int chunk, efla_dtype dt) {
  if (B < 1 || H < 1 || L < 0 || !valid_dtype(dt)) return EFLA_ERR_INVALID_ARG;
  if (!valid_dim(d_k) || !valid_dim(d_v) || !valid_chunk(chunk)) return EFLA_ERR_UNSUPPORTED;
  const int64_t bh = int64_t(B) * H;
  const int64_t nc = (L + chunk - 1) / chunk;
  if (bh * (d_v / 16) > kMaxGrid || bh * nc > kMaxGrid || nc > kMaxGrid) return EFLA_ERR_UNSUPPORTED;
  return EFLA_OK;
}

}  // namespace
