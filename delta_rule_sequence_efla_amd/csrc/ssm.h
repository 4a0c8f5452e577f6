// ssm.h -- what the kernels of the selective state space scan share.
//
// The recurrence (per value head; state S of d_k x d_v, rate a, skip d):
//     D_t = softplus(dt_t + bias),   S_t = e^{a D_t} S_{t-1} + D_t k_t v_t^T,
//     o_t = S_t^T q_t + d v_t.
// Over a chunk with G_i = a (D_1 + .. + D_i) and start state S, for i >= j
// (no exponent positive for a decaying rate):
//     P_ij = e^{G_i - G_j} D_j (q_i . k_j)
//     O    = diag(e^G) Q S + P V + d V
//     S   <- e^{G_C} S + K^T diag(w) V,          w_j = e^{G_C - G_j} D_j
// Backward, with X the gradient with respect to the state at the chunk's end and
// dP_ij = (dO_i . V_j) e^{G_i - G_j}:
//     dQ = (dP D) K + diag(e^G) dO S^T
//     dK = diag(D) (dP^T Q) + diag(w) V X^T
//     dV = P^T dO + diag(w) K X + d dO
//     X <- e^{G_C} X + Q^T diag(e^G) dO         (at the chunk's start)
// and the gradient of the decay exponent a D_t is the sum over all pairs it
// stands between: with M_ij = dP_ij (q_i . k_j) D_j, r_i = e^{G_i} q_i . (S dO_i)
// and p_j = w_j k_j . (X v_j),
//     gd_t = sum_{i >= t > j} M_ij + sum_{i >= t} r_i + sum_{j < t} p_j + e^{G_C} <X, S>,
// whose first term is taken tile by tile (16 x 16): of t's own diagonal tile the pairs
// around t, of the tiles left of it row sums, of those below it column sums, of those
// between whole tiles.  Then
//     dD_t = (column sum of M + p)_t / D_t + a gd_t,   ddt = dD sigmoid(dt + bias),
//     da = sum D_t gd_t,   dbias = sum ddt,   dd = sum v . dO.
// Query and key heads may be fewer than value heads: value head h reads query
// and key head h / (H / Hk).
#pragma once

#include "gated.h"

namespace efla {

__device__ __forceinline__ float softplus(float x) { return fmaxf(x, 0.0f) + log1pf(expf(-fabsf(x))); }

// Inclusive sums over the lanes in 64 bits, by DPP (wave_scan_dpp for doubles).
__device__ __forceinline__ double wave_scan_dpp64(double s) {
  auto add = [&](auto ctrl, auto rows) {
    const uint64_t u = __builtin_bit_cast(uint64_t, s);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, int(uint32_t(u)), decltype(ctrl)::value, decltype(rows)::value, 0xF, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, int(uint32_t(u >> 32)), decltype(ctrl)::value, decltype(rows)::value, 0xF, false);
    s += __builtin_bit_cast(double, (uint64_t(hi) << 32) | lo);
  };
  add(std::integral_constant<int, 0x111>{}, std::integral_constant<int, 0xF>{});
  add(std::integral_constant<int, 0x112>{}, std::integral_constant<int, 0xF>{});
  add(std::integral_constant<int, 0x114>{}, std::integral_constant<int, 0xF>{});
  add(std::integral_constant<int, 0x118>{}, std::integral_constant<int, 0xF>{});
  add(std::integral_constant<int, 0x142>{}, std::integral_constant<int, 0xA>{});
  add(std::integral_constant<int, 0x143>{}, std::integral_constant<int, 0xC>{});
  return s;
}

// The gates of a chunk of C tokens, in log2 units: G as the sum of two floats (what
// is needed of it are differences, and e^{G_i - G_j} is then good to float32 however
// far G has fallen), D, e^{G}, w.
template <int C>
struct GatesOf {
  float hi[C], lo[C], D[C], e[C], w[C];
  // e^{G_i - G_j}, by token i's own hi and lo
  __device__ __forceinline__ float between(float hi_i, float lo_i, int j) const {
    return __builtin_amdgcn_exp2f((hi_i - hi[j]) + (lo_i - lo[j]));
  }
};
using ChunkGates = GatesOf<64>;

// By one wavefront, a lane a token; raw: dt + bias.
template <int C>
__device__ __forceinline__ void put_chunk_gates(GatesOf<C>& gt, float raw, float rate, bool real, int lane) {
  constexpr double kLog2E = 1.4426950408889634;
  const float D = real ? softplus(raw) : 0.0f;
  const double G = wave_scan_dpp64(real ? double(gate_floor(rate * D)) * kLog2E : 0.0);
  const uint64_t u = __builtin_bit_cast(uint64_t, G);
  const uint32_t el = __builtin_amdgcn_readlane(int(uint32_t(u)), 63), eh = __builtin_amdgcn_readlane(int(uint32_t(u >> 32)), 63);
  const double end = __builtin_bit_cast(double, (uint64_t(eh) << 32) | el);
  if (lane >= C) return;
  gt.hi[lane] = float(G);
  gt.lo[lane] = float(G - double(float(G)));
  gt.D[lane] = D;
  gt.e[lane] = __builtin_amdgcn_exp2f(float(G));
  gt.w[lane] = __builtin_amdgcn_exp2f(float(end - G)) * D;
}

// Sequence handled in rank r of a packed batch: by the caller's order, or, for up
// to 64 sequences without one, the r-th longest by chunks of C tokens (ties by
// index), found by every wavefront for itself; larger batches go by index.
// Workgroups start in index order, so the longest chains start first.
template <int C>
__device__ __forceinline__ int ranked_seq(const int32_t* __restrict__ cu, const int32_t* __restrict__ order, int r, int N,
                                          int64_t T) {
  if (order != nullptr) return seq_of_rank(order, r, N);
  if (N > kWave) return r;
  const int lane = threadIdx.x & 63, mine = lane < N ? seq_chunks<C>(cu, lane, T) : -1;
  int rank = 0;
  for (int u = 0; u < N; ++u) {
    const int n = __builtin_amdgcn_readlane(mine, u);
    rank += n > mine || (n == mine && u < lane) ? 1 : 0;
  }
  return __builtin_amdgcn_readfirstlane(__builtin_ctzll(__ballot(lane < N && rank == r)));
}

// What workgroup unit x (of the sequences' or their segments') has to do for head h.
struct SsmUnit {
  int seq;            // sequence; < 0: nothing to do
  int64_t bos, len;   // its tokens
  int64_t slot;       // its segment's place in seg_s and seg_e; those of the sequence are H apart
  int64_t first, end; // the places of the sequence's first and last segment
  int before;         // segments before it
  bool last;          // the sequence ends in it
  // Where the unit's first state comes from.  The launch that brings the segments' ends
  // (local) starts a sequence's first segment from s0, and keeps s0 at the place of the
  // last, which it has no use for: the final state may be written over s0, and in the
  // second launch the last segment may end before the first one begins.
  __device__ __forceinline__ const float* start(bool local, const float* s0, const float* seg_s, int64_t state) const {
    if (before == 0 && (local || last)) return s0;
    return local ? nullptr : seg_s + (before == 0 ? end : first) * state;
  }
};
template <int C, typename Args>
__device__ __forceinline__ SsmUnit ssm_unit(const Args& a, int x, int h, int lane) {
  SsmUnit u{x, 0, 0, 0, 0, 0, 0, true};
  if (a.seg == 0) {
    u.bos = int64_t(x) * a.L;
    u.len = a.L;
    if (a.cu != nullptr) {
      u.seq = ranked_seq<C>(a.cu, a.order, x, a.N, a.L);
      u.bos = clamp_offset(a.cu[u.seq], 0, a.L);
      u.len = clamp_offset(a.cu[u.seq + 1], u.bos, a.L) - u.bos;
    }
    return u;
  }
  int64_t end;
  if (a.cu == nullptr) {
    const int per = int((a.L + a.seg - 1) / a.seg);
    u.seq = x / per;
    u.before = x % per;
    u.bos = int64_t(u.seq) * a.L;
    end = u.bos + a.L;
  } else {
    // slots floor(offset / seg) + u, as those of chunks (common.h); a sequence
    // without tokens has one, to copy its state
    int lo = 0, left = a.N;
    while (left > 1) {
      const int step = (left + kWave - 1) / kWave, at = lane * step;
      const bool before = at < left && clamp_offset(a.cu[lo + at], 0, a.L) / a.seg + lo + at <= x;
      const int cnt = __popcll(__ballot(before)), by = cnt > 1 ? (cnt - 1) * step : 0;
      lo += by;
      left = left - by < step ? left - by : step;
    }
    u.seq = __builtin_amdgcn_readfirstlane(lo);
    u.bos = clamp_offset(a.cu[u.seq], 0, a.L);
    end = clamp_offset(a.cu[u.seq + 1], u.bos, a.L);
    const int64_t n = x - (u.bos / a.seg + u.seq);
    if (n < 0 || n * a.seg >= (end > u.bos ? end - u.bos : 1)) {
      u.seq = -1;
      return u;
    }
    u.before = int(n);
  }
  u.slot = int64_t(x) * a.H + h;
  u.first = u.slot - int64_t(u.before) * a.H;
  u.end = u.first + (end > u.bos ? (end - u.bos - 1) / a.seg : 0) * a.H;
  u.bos += u.before * a.seg;
  u.last = u.bos + a.seg >= end;
  u.len = u.last ? end - u.bos : a.seg;
  return u;
}

// Of a diagonal tile with x[qq] = M_ij D_j at row i = li and column j = 4 g + qq: in
// lanes li = 0, out[qq] = sum_{i >= t > j} M_ij D_j for t = 4 g + qq, the tile's own share
// of gd_t.  Formed from the pairs around t alone: as differences of row and column
// sums, whose diagonals and whose pairs on one side of t cancel, da was off by 1e-5.
__device__ __forceinline__ f32x4 tile_between(const f32x4& x, int li, int g) {
  float sum = (x[0] + x[1]) + (x[2] + x[3]);
  const float one = __shfl_up(sum, 16);
  sum += g >= 1 ? one : 0.0f;
  const float two = __shfl_up(sum, 32);
  sum += g >= 2 ? two : 0.0f;
  const float left = __shfl_up(sum, 16);
  float before = g >= 1 ? left : 0.0f;  // of the row's columns below t
  f32x4 out;
#pragma unroll
  for (int qq = 0; qq < 4; ++qq) {
    out[qq] = row_sum16(li >= 4 * g + qq ? before : 0.0f);
    before += x[qq];
  }
  return out;
}

// The same with the tile the other way round: x[qq] at row i = 4 g + qq, column j = li.
__device__ __forceinline__ f32x4 tile_between_tr(const f32x4& x, int li, int g) {
  float sum = (x[0] + x[1]) + (x[2] + x[3]);
  const float one = __shfl_down(sum, 16);
  sum += g <= 2 ? one : 0.0f;
  const float two = __shfl_down(sum, 32);
  sum += g <= 1 ? two : 0.0f;
  const float right = __shfl_down(sum, 16);
  float from = g <= 2 ? right : 0.0f;  // of the column's rows from t on
  f32x4 out;
#pragma unroll
  for (int qq = 3; qq >= 0; --qq) {
    from += x[qq];
    out[qq] = row_sum16(li < 4 * g + qq ? from : 0.0f);
  }
  return out;
}

// Sums over the lane's row of 16: of itself and the lanes above, and of the lanes below.
__device__ __forceinline__ float row_suffix16(float x, int li) {
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) {
    const float y = __shfl_down(x, d, 16);
    x += li + d < 16 ? y : 0.0f;
  }
  return x;
}
__device__ __forceinline__ float row_before16(float x, int li) {
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) {
    const float y = __shfl_up(x, d, 16);
    x += li >= d ? y : 0.0f;
  }
  const float y = __shfl_up(x, 1, 16);
  return li > 0 ? y : 0.0f;
}

}  // namespace efla
