// pool.hip -- moves of whole rows of state pools: copies to other rows (a
// request forked into several), rows cleared (a request that starts anew), and
// compaction of the rows in use to the front.  A row is the state of one request
// in one layer; all layers' pools move in one launch.
#include "common.h"
#include "launchers.h"

namespace efla {

constexpr int kPieceVecs = 8;                              // 16-byte vectors a thread
constexpr int kPieceBytes = kThreads * kPieceVecs * 16;    // of a row, a workgroup
// Whether entries that name one source share a read of it.  A workgroup that reads for
// others saves reads from memory and makes their writes wait for one another, and
// every one runs over the list.  us without / with it, rows copied to 1, 2, 8, 32 or
// 500 others (500: to all of a list of 500), from 32 MiB written and up to 512 entries:
//   500 x 4 KiB (below it)   3.5 / 5.2, 3.6 / 5.2, 3.6 / 6.5, 3.6 / 10, 3.5 / 16
//   500 x 64 KiB (below it)  14 / 16.5, 14 / 12.4, 11 / 11.8, 10 / 18, 10 / 33
//   64 x 1 MiB   25 / 25.5, 25 / 19, 15.7 / 15.4, 15.5 / 16.1
//   256 x 1 MiB  103 / 111, 87 / 85, 82 / 53, 45 / 49
//   500 x 1 MiB  201 / 220, 201 / 171, 167 / 129, 129 / 115, 120 / 107
//   1024 x 512 KiB (above)  183 / 313, 159 / 273, 183 / 179;  8192 x 64 KiB  181 / 1395, 166 / 1425, 181 / 1475
constexpr uint64_t kMinShareBytes = uint64_t(32) << 20;
constexpr int kMaxShare = 512;
// Destinations a workgroup writes, of those in 64 entries: with all of them one piece of
// a row that goes to 500 was 500 writes one after the other (500 x 64 KiB: 132 us).
constexpr int kShared = 8;

// The lowest n of the bits set in m.
__device__ __forceinline__ uint64_t lowest(uint64_t m, int n) {
  while (__popcll(m) > n) m &= ~(uint64_t(1) << (63 - __builtin_clzll(m)));
  return m;
}

int64_t pool_pieces(uint64_t row_bytes) { return int64_t((row_bytes + kPieceBytes - 1) / kPieceBytes); }

// One workgroup moves one 32 KiB piece of one row, entry i's.  With `share` it writes the
// piece to the destinations of the first `served` entries with the same source in
// every 64 from i + 1 on, up to `end`, as well.
template <typename V>
__device__ __forceinline__ void pool_piece(const PoolSet& set, int p, uint32_t piece, const int32_t* __restrict__ src,
                                           const int32_t* __restrict__ dst, int i, int P, bool share, int served,
                                           int end) {
  const uint64_t bytes = set.bytes[p], at = uint64_t(piece) * kPieceBytes;
  const int from = src[i];
  const bool clear = from < 0 || from >= P;
  constexpr int PER = 16 * kPieceVecs / int(sizeof(V));
  V val[PER];
  const char* base = static_cast<const char*>(set.base[p]);
  const char* in = base + uint64_t(clear ? 0 : from) * bytes;
#pragma unroll
  for (int e = 0; e < PER; ++e) {
    const uint64_t off = at + (uint64_t(e) * kThreads + threadIdx.x) * sizeof(V);
    val[e] = V{};
    if (!clear && off < bytes) val[e] = *reinterpret_cast<const V*>(in + off);
  }
  auto put = [&](int to) {
    char* out = static_cast<char*>(set.base[p]) + uint64_t(to) * bytes;
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      const uint64_t off = at + (uint64_t(e) * kThreads + threadIdx.x) * sizeof(V);
      if (off < bytes) *reinterpret_cast<V*>(out + off) = val[e];
    }
  };
  const int to = dst[i];
  if (to >= 0 && to < P) put(to);
  if (!share || clear) return;
  const int lane = threadIdx.x & 63;
  for (int j0 = i + 1; j0 < end; j0 += kWave) {
    const int j = j0 + lane;
    const bool same = j < end && src[j] == from;
    const int tj = same ? dst[j] : -1;
    uint64_t todo = __ballot(tj >= 0 && tj < P);
    const uint64_t all = __ballot(same);
    if (__popcll(all) > served) todo &= lowest(all, served);
    while (todo != 0) {
      const int l = __builtin_ctzll(todo);
      todo &= todo - 1;
      put(__builtin_amdgcn_readlane(tj, l));
    }
  }
}

__global__ __launch_bounds__(kThreads) void pool_copy_kernel(PoolSet set, const int32_t* __restrict__ src,
                                                             const int32_t* __restrict__ dst, int N, int P, int share) {
  const uint32_t pieces = set.first[set.count];
  const int i = int(blockIdx.x / pieces);
  const uint32_t at = blockIdx.x % pieces;
  const int from = src[i], to = dst[i], lane = threadIdx.x & 63;
  const bool clear = from < 0 || from >= P;
  int served = kShared, end = N;
  if (share && !clear) {
    // The first entry f with a source writes for the first kShared others in every 64
    // entries behind it, and of the rest of those 64 every kShared-th for the ones up to
    // the next: a fork into eight costs nine row moves, not sixteen.
    for (int j0 = 0; j0 < i; j0 += kWave) {
      const uint64_t same = __ballot(j0 + lane < i && src[j0 + lane] == from);
      if (same == 0) continue;
      const int f = j0 + __builtin_ctzll(same), first = i - (i - f - 1) % kWave;  // of i's 64
      const int rank = i <= j0 + kWave ? __popcll(same) - 1
                                       : __popcll(__ballot(first + lane < i && src[first + lane] == from));
      if (rank == 0 || rank % kShared != 0) return;
      served = kShared - 1;
      end = first + kWave < N ? first + kWave : N;
      break;
    }
  } else if (to < 0 || to >= P) {
    return;
  }
  int p = 0;
  while (set.first[p + 1] <= at) ++p;
  const uint64_t odd = set.bytes[p] | reinterpret_cast<uintptr_t>(set.base[p]);
  if ((odd & 15) == 0) pool_piece<u32x4>(set, p, at - set.first[p], src, dst, i, P, share, served, end);
  else if ((odd & 3) == 0) pool_piece<uint32_t>(set, p, at - set.first[p], src, dst, i, P, share, served, end);
  else pool_piece<uint16_t>(set, p, at - set.first[p], src, dst, i, P, share, served, end);
}

hipError_t launch_pool_copy(const PoolSet& set, const int32_t* src, const int32_t* dst, int N, int P, bool share,
                            hipStream_t s) {
  const int64_t wgs = int64_t(set.first[set.count]) * N;
  uint64_t row = 0;  // bytes in all pools
  for (int p = 0; p < set.count; ++p) row += set.bytes[p];
  if (wgs == 0) return hipSuccess;
  hipLaunchKernelGGL(pool_copy_kernel, dim3(unsigned(wgs)), dim3(kThreads), 0, s, set, src, dst, N, P,
                     share && N <= kMaxShare && row * uint64_t(N) >= kMinShareBytes ? 1 : 0);
  return hipGetLastError();
}

// The moves of a compaction, by one workgroup over a bitmap of the rows in use:
// with K of them, the j-th row in use at or above K goes to the j-th unused row
// below K.  There are as many of one as of the other, and no row is both a source
// and a destination, so the copies may run in any order.
constexpr int kPlanThreads = 1024;
__global__ __launch_bounds__(kPlanThreads) void pool_plan_kernel(const int32_t* slots, int N, int P, int32_t* out,
                                                                 int32_t* __restrict__ live, int32_t* __restrict__ src,
                                                                 int32_t* __restrict__ dst) {
  extern __shared__ uint32_t used[];  // a bit a row, then the ones before each word
  const int words = (P + 31) / 32;
  uint32_t* before = used + words;
  __shared__ uint32_t sums[kPlanThreads / kWave];
  const int tid = threadIdx.x, lane = tid & 63, w = wave_id();
  for (int i = tid; i < words; i += kPlanThreads) used[i] = 0;
  __syncthreads();
  for (int i = tid; i < N; i += kPlanThreads) {
    const int r = slots[i];
    if (r >= 0 && r < P) atomicOr(&used[r >> 5], 1u << (r & 31));
    src[i] = dst[i] = -1;
  }
  __syncthreads();
  // exclusive sums of the words' counts: each thread a run of words
  const int per = (words + kPlanThreads - 1) / kPlanThreads;
  const int w0 = tid * per < words ? tid * per : words, w1 = w0 + per < words ? w0 + per : words;
  uint32_t mine = 0;
  for (int i = w0; i < w1; ++i) mine += __popc(used[i]);
  uint32_t scan = mine;
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const uint32_t y = __shfl_up(scan, d);
    if (lane >= d) scan += y;
  }
  if (lane == kWave - 1) sums[w] = scan;
  __syncthreads();
  uint32_t base = scan - mine, K = 0;
  for (int i = 0; i < kPlanThreads / kWave; ++i) {
    if (i < w) base += sums[i];
    K += sums[i];
  }
  for (int i = w0; i < w1; ++i) {
    before[i] = base;
    base += __popc(used[i]);
  }
  __syncthreads();
  // rows in use below r
  auto rank = [&](uint32_t r) { return before[r >> 5] + __popc(used[r >> 5] & ((1u << (r & 31)) - 1u)); };
  const uint32_t below = K < uint32_t(P) ? rank(K) : K;  // in use below K
  for (int r = tid; r < P; r += kPlanThreads) {
    const bool in_use = used[r >> 5] >> (r & 31) & 1;
    const uint32_t before_r = rank(uint32_t(r));
    if (in_use && uint32_t(r) >= K) src[before_r - below] = r;
    if (!in_use && uint32_t(r) < K) dst[uint32_t(r) - before_r] = r;
  }
  if (tid == 0) *live = int32_t(K);
  __threadfence_block();
  __syncthreads();
  for (int i = tid; i < N; i += kPlanThreads) {
    const int r = slots[i];
    out[i] = r >= 0 && r < P && uint32_t(r) >= K ? dst[rank(uint32_t(r)) - below] : r;
  }
}

hipError_t launch_pool_plan(const int32_t* slots, int N, int P, int32_t* out, int32_t* live, int32_t* src, int32_t* dst,
                            hipStream_t s) {
  const size_t lds = size_t((P + 31) / 32) * 8;
  hipLaunchKernelGGL(pool_plan_kernel, dim3(1), dim3(kPlanThreads), lds, s, slots, N, P, out, live, src, dst);
  return hipGetLastError();
}

}  // namespace efla
