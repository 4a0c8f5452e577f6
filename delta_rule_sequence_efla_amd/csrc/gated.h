// gated.h -- what the kernels of the gated delta rule share.
//
// The recurrence (per value head; a from beta and lambda = ||k||^2 under either
// rule, common.h; g the log-decay):
//     S_t = e^{g_t} (I - a_t k_t k_t^T) S_{t-1} + a_t k_t v_t^T,   o_t = S_t^T q_t.
// With u_t = a_t (v_t - e^{g_t} S_{t-1}^T k_t) it is S_t = e^{g_t} S_{t-1} + k_t u_t^T.
// Over a chunk with G_i = g_1 + .. + g_i and Gam_ij = e^{G_i - G_j} (i >= j, so
// no exponent of a decaying gate is positive):
//     A  = tril(diag(a) (Gam * K K^T), -1),   T = (I + A)^{-1} diag(a)
//     U  = T (V - diag(e^G) K S)
//     O  = diag(e^G) Q S + (Gam * tril(Q K^T)) U
//     S <- e^{G_C} S + K^T diag(e^{G_C - G_j}) U
// Query and key heads may be fewer than value heads: value head h reads query
// and key head h / (H / Hk).
#pragma once

#include <type_traits>

#include "common.h"

namespace efla {

// Chunks of 2^shift tokens in a sequence of `tokens` >= 0, up to 2^31 - 1 of them:
// the sum is formed unsigned, since a signed one is negative in the last chunk
// below 2^31.
__host__ __device__ constexpr int chunk_count(int tokens, int shift) {
  return int((uint32_t(tokens) + (1u << shift) - 1u) >> shift);
}

// Log-decays below -128 act as -128: e^{-128} is zero in fp32 already, and
// sums of a chunk's gates stay finite (G_i - G_j of two infinities would be
// NaN), so g = -inf resets the state.  NaN passes through.
__device__ __forceinline__ float gate_floor(float g) { return g < -128.0f ? -128.0f : g; }

// G of a chunk's tokens, lane by lane: the inclusive sum of their gates in 64
// bits.  What is needed of G are differences, and after a reset (-128) or much
// decay the float sum is too coarse for them: 1.5e-5 apart behind one reset,
// 1e-3 behind a chunk of them.
__device__ __forceinline__ double wave_scan_gate(float g, int lane) {
  double x = double(g);
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const double y = __shfl_up(x, d);
    if (lane >= d) x += y;
  }
  return x;
}

// Sum over the 16 lanes of a DPP row, in every lane.
__device__ __forceinline__ float row_sum16(float s) {
  s += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, s), 0x128, 0xF, 0xF, false));
  s += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, s), 0x124, 0xF, 0xF, false));
  s += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, s), 0x122, 0xF, 0xF, false));
  s += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, s), 0x121, 0xF, 0xF, false));
  return s;
}

// Sum over the four lanes li, li + 16, li + 32, li + 48, in each of them: by the
// row and half exchanges of the vector unit, no LDS round trips.
__device__ __forceinline__ float row_sum4(float s) {
  const uint32_t a = __float_as_uint(s);
  const auto x = __builtin_amdgcn_permlane16_swap(a, a, false, false);
  const float t = __uint_as_float(x[0]) + __uint_as_float(x[1]);
  const uint32_t b = __float_as_uint(t);
  const auto y = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  return __uint_as_float(y[0]) + __uint_as_float(y[1]);
}

// Inclusive sum over the lanes, by DPP: within rows of 16, then the rows' ends.
__device__ __forceinline__ float wave_scan_dpp(float s) {
  auto add = [&](auto ctrl, auto rows) {  // lanes without a source, and rows not named, add zero
    s += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, s), decltype(ctrl)::value,
                                                               decltype(rows)::value, 0xF, false));
  };
  add(std::integral_constant<int, 0x111>{}, std::integral_constant<int, 0xF>{});  // row_shr:1, 2, 4, 8
  add(std::integral_constant<int, 0x112>{}, std::integral_constant<int, 0xF>{});
  add(std::integral_constant<int, 0x114>{}, std::integral_constant<int, 0xF>{});
  add(std::integral_constant<int, 0x118>{}, std::integral_constant<int, 0xF>{});
  add(std::integral_constant<int, 0x142>{}, std::integral_constant<int, 0xA>{});  // row_bcast:15 into rows 1, 3
  add(std::integral_constant<int, 0x143>{}, std::integral_constant<int, 0xC>{});  // row_bcast:31 into rows 2, 3
  return s;
}

// slot_chunk (common.h) by all 64 lanes, uniform arguments but for the lane:
// each step of the search tests 64 sequences, one load's latency instead of six.
template <int C>
__device__ __forceinline__ bool gated_slot_chunk(const int32_t* __restrict__ cu, int N, int64_t j, int64_t h, int H,
                                                 int64_t L, int NC, int lane, SeqSpan& sp, int& n) {
  int lo = 0, left = N;
  while (left > 1) {
    const int step = (left + kWave - 1) / kWave, u = lane * step;
    const bool before = u < left && clamp_offset(cu[lo + u], 0, L) / C + lo + u <= j;
    const int cnt = __popcll(__ballot(before));
    const int at = cnt > 1 ? (cnt - 1) * step : 0;
    lo += at;
    left = left - at < step ? left - at : step;
  }
  lo = __builtin_amdgcn_readfirstlane(lo);
  sp = seq_span<C>(cu, lo, h, H, L, NC);
  const int64_t nn = h * NC + j - sp.slot0;
  n = int(nn);
  return nn >= 0 && nn < sp.nc;
}

// State a sequence starts from and ends in: row `seq` of the state tensor, or
// row slots[seq] of a pool of P states; -1 (no row) for an entry outside it.
__device__ __forceinline__ int64_t state_row(const int32_t* __restrict__ slots, int seq, int P) {
  if (slots == nullptr) return seq;
  const int s = slots[seq];
  return s >= 0 && s < P ? s : -1;
}

// dg of a token: float32, or rounded to the inputs' type.
template <typename T>
__device__ __forceinline__ void store_gate_grad(void* dg, int64_t at, float x, int dg32) {
  if (dg32) static_cast<float*>(dg)[at] = x;
  else static_cast<T*>(dg)[at] = from_f32<T>(x);
}

}  // namespace efla
