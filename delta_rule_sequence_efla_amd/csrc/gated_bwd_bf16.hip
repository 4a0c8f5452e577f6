// gated_bwd_bf16.hip -- launches of the gated backward's passes for bf16 inputs
// (gated_reverse.h, gated_bwd_chunk.h), in a translation unit of its own so that
// it builds in parallel with the others.
#include "launchers.h"
#include "gated_bwd_chunk.h"
#include "gated_reverse.h"

namespace efla {

int gated_chains_threads(int DK) { return DK == 64 ? GatedSplitShape<64>::STATE_THREADS : GatedSplitShape<128>::STATE_THREADS; }
int gated_bwd_chunk_threads(int DK) { return DK == 64 ? GatedTrShape<64>::NTH : GatedTrShape<128>::NTH; }

template <int DK>
static hipError_t chains_impl(const GatedFwd& a, const GatedBwd& b, const uint16_t* xfr, const uint16_t* qe,
                              const float* gws, uint16_t* statesT, uint16_t* dstatesT, hipStream_t s) {
  const int NC = int((b.L + 63) / 64), NVB = b.DV / 32;
  const int64_t bh = int64_t(b.B) * b.H;
  hipLaunchKernelGGL((gated_chains_kernel<DK>), dim3(unsigned(2 * bh * NVB)), dim3(GatedSplitShape<DK>::STATE_THREADS),
                     0, s, a, b, qe, xfr, gws, statesT, dstatesT, NC, NVB, bh % 8 == 0 ? 1 : 0);
  return hipGetLastError();
}

hipError_t launch_gated_chains(const GatedFwd& a, const GatedBwd& b, const uint16_t* xfr, const uint16_t* qe,
                               const float* gws, uint16_t* statesT, uint16_t* dstatesT, hipStream_t s) {
  return b.DK == 64 ? chains_impl<64>(a, b, xfr, qe, gws, statesT, dstatesT, s)
                    : chains_impl<128>(a, b, xfr, qe, gws, statesT, dstatesT, s);
}

template <int DK, bool SHARED>
static hipError_t chunk_impl(const GatedBwd& b, const uint16_t* xfr, const uint16_t* p, const float* gws,
                             const uint16_t* statesT, const uint16_t* dstatesT, float* dqh, float* dkh, hipStream_t s) {
  const int NC = int((b.L + 63) / 64);
  hipLaunchKernelGGL((gated_bwd_tr_kernel<DK, SHARED>), dim3(unsigned(int64_t(b.B) * b.H * NC)),
                     dim3(GatedTrShape<DK>::NTH), 0, s, b, xfr, p, gws, statesT, dstatesT, dqh, dkh, NC);
  return hipGetLastError();
}

hipError_t launch_gated_bwd_chunk(const GatedBwd& b, const uint16_t* xfr, const uint16_t* p, const float* gws,
                                  const uint16_t* statesT, const uint16_t* dstatesT, float* dqh,
                                  float* dkh, hipStream_t s) {
  if (b.DK == 64)
    return dqh != nullptr ? chunk_impl<64, true>(b, xfr, p, gws, statesT, dstatesT, dqh, dkh, s)
                          : chunk_impl<64, false>(b, xfr, p, gws, statesT, dstatesT, dqh, dkh, s);
  return dqh != nullptr ? chunk_impl<128, true>(b, xfr, p, gws, statesT, dstatesT, dqh, dkh, s)
                        : chunk_impl<128, false>(b, xfr, p, gws, statesT, dstatesT, dqh, dkh, s);
}

}  // namespace efla
