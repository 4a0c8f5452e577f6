// gated_fwd.hip -- launches of the chunked gated forward pass for bf16 inputs:
// the UT transform (gated_ut.h), then the recurrence (gated_split.h).
// Workspace, regions 256-byte aligned: X fragments [slots][12 KiB], gate blocks
// [slots][1 KiB], and for packed batches the schedule (int32 per sequence).
#include "gated_split.h"

namespace efla {

namespace {
size_t align256(size_t x) { return (x + 255) / 256 * 256; }
constexpr int kGatedChunk = 64;
// Packed batches of at most this many sequences run longest first (the ranking
// compares every pair of sequences).
constexpr int kGatedOrderedSeqs = 4096;

template <int DK, bool BWD>
hipError_t ut_impl(const GatedFwd& a, uint16_t* xfr, float* gws, const GatedUtBwd& b, int32_t* order, hipStream_t s) {
  const int NC = a.cu == nullptr ? int((a.L + kGatedChunk - 1) / kGatedChunk) : int(a.L / kGatedChunk) + a.N;
  const int64_t nchunks = int64_t(a.cu == nullptr ? a.B : 1) * a.H * NC;
  constexpr int W = UtWaveShape<DK, kGatedChunk>::WAVES;
  static_assert(64 * W == kThreads && W * UtWaveShape<DK, kGatedChunk>::SCRATCH >= int(kRankSeqs * sizeof(int)),
                "ranking workgroups reuse the kernel's shape and LDS");
  const int64_t nwg = (nchunks + W - 1) / W;
  const int64_t nrank = order != nullptr ? (a.N + kRankSeqs - 1) / kRankSeqs : 0;
  if (nwg + nrank == 0) return hipSuccess;
  hipLaunchKernelGGL((gated_ut_wave_kernel<DK, BWD>), dim3(unsigned(nwg + nrank)), dim3(kThreads), 0, s,
                     static_cast<const uint16_t*>(a.k), static_cast<const uint16_t*>(a.beta), a.g, xfr, gws, a.H, a.Hk,
                     a.L, NC, nchunks, a.rule, a.cu, a.N, nwg, order, b);
  return hipGetLastError();
}

template <int DK>
hipError_t split_impl(const GatedFwd& a, const uint16_t* xfr, const float* gws, const int32_t* order, hipStream_t s) {
  const int NC = a.cu == nullptr ? int((a.L + kGatedChunk - 1) / kGatedChunk) : int(a.L / kGatedChunk) + a.N;
  const int64_t bh = int64_t(a.cu == nullptr ? a.B : a.N) * a.H;
  const int NVB = a.DV / 32;
  hipLaunchKernelGGL((gated_split_kernel<DK>), dim3(unsigned(bh * NVB)), dim3(GatedSplitShape<DK>::THREADS), 0, s, a,
                     xfr, gws, order, NC, NVB, bh % 8 == 0 ? 1 : 0);
  return hipGetLastError();
}
}  // namespace

bool gated_chunk_supported(int DK, int DV) { return (DK == 64 || DK == 128) && DV % 32 == 0; }

GatedFwdLayout gated_fwd_layout(int B, int N, int H, int64_t L, bool packed) {
  const size_t slots = packed ? size_t(H) * (L / kGatedChunk + N) : size_t(B) * H * ((L + kGatedChunk - 1) / kGatedChunk);
  GatedFwdLayout w{};
  w.x = 0;
  w.g = align256(slots * kGatedX * 2);
  w.order = w.g + align256(slots * kGatedG * 4);
  w.total = w.order + (packed ? align256(size_t(N) * 4) : 0);
  return w;
}

int64_t gated_chunk_threads(int64_t seqs, int H, int64_t L, bool packed, int DK, int DV) {
  const int64_t slots = packed ? H * (L / kGatedChunk + seqs) : seqs * H * ((L + kGatedChunk - 1) / kGatedChunk);
  const int64_t split = seqs * H * (DV / 32) * (DK == 64 ? GatedSplitShape<64>::THREADS : GatedSplitShape<128>::THREADS);
  return split > slots * kWave ? split : slots * kWave;
}

hipError_t launch_gated_ut_bwd(const GatedFwd& a, uint16_t* xfr, float* gws, uint16_t* p, uint16_t* qe, hipStream_t s) {
  const GatedUtBwd b{static_cast<const uint16_t*>(a.q), p, qe};
  return a.DK == 64 ? ut_impl<64, true>(a, xfr, gws, b, nullptr, s) : ut_impl<128, true>(a, xfr, gws, b, nullptr, s);
}

hipError_t launch_gated_chunk(const GatedFwd& a, void* workspace, hipStream_t s) {
  const bool packed = a.cu != nullptr;
  const GatedFwdLayout lay = gated_fwd_layout(a.B, a.N, a.H, a.L, packed);
  auto* ws = static_cast<unsigned char*>(workspace);
  auto* xfr = reinterpret_cast<uint16_t*>(ws + lay.x);
  auto* gws = reinterpret_cast<float*>(ws + lay.g);
  // packed: the caller's schedule, or one ranked by workgroups of the UT launch
  int32_t* mine = packed && a.order == nullptr && a.N <= kGatedOrderedSeqs ? reinterpret_cast<int32_t*>(ws + lay.order) : nullptr;
  const GatedUtBwd none{};
  const hipError_t e = a.DK == 64 ? ut_impl<64, false>(a, xfr, gws, none, mine, s) : ut_impl<128, false>(a, xfr, gws, none, mine, s);
  if (e != hipSuccess) return e;
  const int32_t* order = mine != nullptr ? mine : a.order;
  return a.DK == 64 ? split_impl<64>(a, xfr, gws, order, s) : split_impl<128>(a, xfr, gws, order, s);
}

}  // namespace efla
