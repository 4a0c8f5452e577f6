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
// whose first term is sum_{i >= t} (row sum - column sum) of M.  Then
//     dD_t = (column sum of M + p)_t / D_t + a gd_t,   ddt = dD sigmoid(dt + bias),
//     da = sum D_t gd_t,   dbias = sum ddt,   dd = sum v . dO.
// Query and key heads may be fewer than value heads: value head h reads query
// and key head h / (H / Hk).
#pragma once

#include "gated.h"

namespace efla {

__device__ __forceinline__ float softplus(float x) { return fmaxf(x, 0.0f) + log1pf(expf(-fabsf(x))); }

// e^x for differences of the log-decay's sums, which are held in 64 bits: their
// difference is exact to float32, and so is the decay.
__device__ __forceinline__ float decay_between(double hi, double lo) { return expf(float(hi - lo)); }

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

}  // namespace efla
