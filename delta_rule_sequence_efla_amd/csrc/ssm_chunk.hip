// ssm_chunk.hip -- launches of the chunked scan for bf16 inputs (ssm_chunk.h).
#include "launchers.h"
#include "ssm_chunk.h"

namespace efla {

bool ssm_chunk_supported(int DK, int DV) { return (DK == 64 || DK == 128) && DV % 32 == 0; }

int64_t ssm_chunk_threads(int64_t seqs, int H, int DV) { return seqs * H * (DV / 32) * SsmShape<64>::THREADS; }

template <int DK>
static hipError_t chunk_impl(const SsmFwd& a, bool local, hipStream_t s) {
  const int NVB = a.DV / 32;
  const int64_t bh = (a.seg > 0 ? a.seg_slots : a.N) * a.H;
  // packed sequences differ in length, and segments in what they fold: there only a head's own value blocks go together
  const int remap = ssm_remap(bh, a.cu == nullptr && a.seg == 0 ? a.H / a.Hk : 1);
  if (local)
    hipLaunchKernelGGL((ssm_chunk_kernel<DK, true>), dim3(unsigned(bh * NVB)), dim3(SsmShape<DK>::LOCAL_THREADS), 0, s, a,
                       NVB, remap);
  else
    hipLaunchKernelGGL((ssm_chunk_kernel<DK, false>), dim3(unsigned(bh * NVB)), dim3(SsmShape<DK>::THREADS), 0, s, a, NVB, remap);
  return hipGetLastError();
}

hipError_t launch_ssm_chunk(const SsmFwd& a, bool local, hipStream_t s) {
  return a.DK == 64 ? chunk_impl<64>(a, local, s) : chunk_impl<128>(a, local, s);
}

}  // namespace efla
