// plan.hip -- the tables of a packed batch, from the requests' lengths in
// device memory: offsets, the longest-first order of the recurrence, and the
// sequence and position of every packed row.
//
// With l_u = max(lengths[u], 0): cu[u] = min(l_0 + .. + l_{u-1}, T); order by
// chunk count as rank_sequences (common.h) writes it; a row t belongs to the
// first sequence that ends after it (sequences without tokens own no row), at
// position t - cu[u] + starts[u].
//
// Up to kPlanSeqs sequences one launch does it all: every workgroup sums the
// lengths for itself into LDS (16 KiB at most, read from L2) rather than wait
// for another launch's sums; the first N / 16 then rank 16 sequences each, the
// others fill their rows by binary search there.  At these sizes the time is
// launch and load latency (2000 sequences and 65536 rows: 7.9 us, 16 sequences:
// 4.4; ranks and rows by the same workgroups: 14).  More sequences take a launch
// for the offsets (order is then the index order) and one for the rows.
#include "gated.h"
#include "launchers.h"

namespace efla {

namespace {
constexpr int kPlanSeqs = 4096;   // sequences whose offsets fit the LDS copy
constexpr int kPlanRows = 1024;   // packed rows per workgroup
constexpr int kPlanRank = 16;     // sequences ranked per workgroup, 16 lanes each

// Sums are clamped at T as they grow: with T < 2^31 and partial sums clamped
// to T, min(a + b, T) needs a + b < 2^32, so it is formed unsigned.
__device__ __forceinline__ int sat_add(int a, int b, int T) {
  const uint32_t s = uint32_t(a) + uint32_t(b);
  return s > uint32_t(T) ? T : int(s);
}
__device__ __forceinline__ int wave_scan_sat(int x, int lane, int T) {
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const int y = __shfl_up(x, d);
    if (lane >= d) x = sat_add(x, y, T);
  }
  return x;
}
__device__ __forceinline__ int plan_length(const int32_t* __restrict__ lengths, int u, int T) {
  const int l = lengths[u];
  return l < 0 ? 0 : (l > T ? T : l);
}

// end[u] (u < N) = min(l_0 + .. + l_u, T) in place of l_u, by all kThreads
// threads, thread t on `per` consecutive entries; end: LDS; wsum: kThreads / 64
// ints of LDS.
__device__ __forceinline__ void scan_lds(int N, int T, int32_t* end, int* wsum) {
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int per = (N + kThreads - 1) / kThreads, a = tid * per, z = a + per < N ? a + per : N;
  int sum = 0;
  for (int u = a; u < z; ++u) end[u] = sum = sat_add(sum, end[u], T);
  const int x = wave_scan_sat(sum, lane, T);
  if (lane == kWave - 1) wsum[w] = x;
  __syncthreads();
  int before = __shfl_up(x, 1);
  if (lane == 0) before = 0;
  for (int j = 0; j < w; ++j) before = sat_add(before, wsum[j], T);
  for (int u = a; u < z; ++u) end[u] = sat_add(before, end[u], T);
  __syncthreads();
}

// sequence of row t: the first u with end[u] > t; N past the last
__device__ __forceinline__ int plan_seq(const int32_t* end, int N, int t) {
  int lo = 0, hi = N;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (end[mid] > t) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}
// Rows blk * kPlanRows ..: a thread's four rows follow each other, so the search
// is made for the first, and again where a row lies past the next sequence too.
__device__ __forceinline__ void plan_rows(const int32_t* end, int N, int T, int64_t blk,
                                          const int32_t* __restrict__ starts, int32_t* __restrict__ seq,
                                          int32_t* __restrict__ pos) {
  static_assert(kPlanRows == 4 * kThreads, "four rows a thread");
  const int64_t t0 = blk * kPlanRows + 4 * threadIdx.x;
  if (t0 >= T) return;
  int u = plan_seq(end, N, int(t0));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t t = t0 + i;
    if (t >= T) return;
    if (u < N && end[u] <= t && ++u < N && end[u] <= t) u = plan_seq(end, N, int(t));
    const bool in = u < N;
    if (seq != nullptr) seq[t] = in ? u : -1;
    if (pos != nullptr)
      pos[t] = in ? int(uint32_t(t) - uint32_t(u > 0 ? end[u - 1] : 0) + uint32_t(starts != nullptr ? starts[u] : 0)) : -1;
  }
}
}  // namespace

// The first rank_wgs workgroups rank kPlanRank sequences each (the very first
// also writes the offsets), the others fill kPlanRows rows each.
__global__ __launch_bounds__(kThreads) void plan_kernel(const int32_t* __restrict__ lengths,
                                                        const int32_t* __restrict__ starts, int N, int T, int shift,
                                                        int rank_wgs, int32_t* __restrict__ cu,
                                                        int32_t* __restrict__ order, int32_t* __restrict__ seq,
                                                        int32_t* __restrict__ pos) {
  __shared__ __align__(16) int32_t end[kPlanSeqs];
  __shared__ __align__(16) int32_t chunks[kPlanSeqs];
  __shared__ int wsum[kThreads / kWave];
  const int tid = threadIdx.x, blk = blockIdx.x;
  for (int u = tid; u < N; u += kThreads) end[u] = plan_length(lengths, u, T);
  __syncthreads();
  scan_lds(N, T, end, wsum);
  if (blk >= rank_wgs) {
    if (seq != nullptr || pos != nullptr) plan_rows(end, N, T, blk - rank_wgs, starts, seq, pos);
    return;
  }
  if (blk == 0)
    for (int u = tid; u <= N; u += kThreads) cu[u] = u > 0 ? end[u - 1] : 0;
  if (order == nullptr) return;
  // chunk counts, padded with -1 (below every count) to whole steps of 64
  const int padded = (N + 63) / 64 * 64;
  for (int u = tid; u < padded; u += kThreads)
    chunks[u] = u < N ? chunk_count(end[u] - (u > 0 ? end[u - 1] : 0), shift) : -1;
  __syncthreads();
  // rank(u) = #{v : n(v) > n(u)} + #{v < u : n(v) = n(u)}, 16 lanes a sequence, four v a step
  typedef int i32x4 __attribute__((ext_vector_type(4)));
  const int u = blk * kPlanRank + (tid >> 4);
  const int nu = u < N ? chunks[u] : 0;
  int rank = 0;
#pragma unroll 4
  for (int x = 4 * (tid & 15); x < padded; x += 64) {
    const i32x4 nv = *reinterpret_cast<const i32x4*>(chunks + x);
#pragma unroll
    for (int i = 0; i < 4; ++i) rank += nv[i] + (x + i < u ? 1 : 0) > nu ? 1 : 0;
  }
#pragma unroll
  for (int d = 8; d > 0; d >>= 1) rank += __shfl_xor(rank, d);
  if ((tid & 15) == 0 && u < N) order[rank] = u;
}

__global__ __launch_bounds__(kThreads) void plan_offsets_kernel(const int32_t* __restrict__ lengths, int N, int T,
                                                                int32_t* __restrict__ cu, int32_t* __restrict__ order) {
  __shared__ int32_t end[kPlanSeqs];
  __shared__ int wsum[kThreads / kWave];
  if (threadIdx.x == 0) cu[0] = 0;
  int carry = 0;  // the same in every thread
  for (int base = 0; base < N; base += kPlanSeqs) {
    const int n = N - base < kPlanSeqs ? N - base : kPlanSeqs;
    for (int u = threadIdx.x; u < n; u += kThreads) end[u] = plan_length(lengths, base + u, T);
    __syncthreads();
    scan_lds(n, T, end, wsum);
    for (int u = threadIdx.x; u < n; u += kThreads) cu[1 + base + u] = sat_add(carry, end[u], T);
    carry = sat_add(carry, end[n - 1], T);
    __syncthreads();
  }
  if (order != nullptr)
    for (int u = threadIdx.x; u < N; u += kThreads) order[u] = u;
}

__global__ __launch_bounds__(kThreads) void plan_rows_kernel(const int32_t* __restrict__ cu,
                                                             const int32_t* __restrict__ starts, int N, int T,
                                                             int32_t* __restrict__ seq, int32_t* __restrict__ pos) {
  plan_rows(cu + 1, N, T, blockIdx.x, starts, seq, pos);
}

hipError_t launch_plan(const int32_t* lengths, const int32_t* starts, int N, int T, int C, int32_t* cu,
                       int32_t* order, int32_t* seq, int32_t* pos, hipStream_t s) {
  const int shift = C == 64 ? 6 : C == 32 ? 5 : 4;
  const int row_wgs = seq != nullptr || pos != nullptr ? int((int64_t(T) + kPlanRows - 1) / kPlanRows) : 0;
  if (N <= kPlanSeqs) {
    const int rank_wgs = order != nullptr && N > 0 ? (N + kPlanRank - 1) / kPlanRank : 1;
    hipLaunchKernelGGL(plan_kernel, dim3(unsigned(rank_wgs + row_wgs)), dim3(kThreads), 0, s, lengths, starts, N, T,
                       shift, rank_wgs, cu, order, seq, pos);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(plan_offsets_kernel, dim3(1), dim3(kThreads), 0, s, lengths, N, T, cu, order);
  if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  if (row_wgs > 0)
    hipLaunchKernelGGL(plan_rows_kernel, dim3(unsigned(row_wgs)), dim3(kThreads), 0, s, cu, starts, N, T, seq, pos);
  return hipGetLastError();
}

}  // namespace efla
