// ssm_bwd_chunk.hip -- launches of the scan's backward pass for bf16 inputs
// (ssm_bwd_chunk.h).
#include "launchers.h"
#include "ssm_bwd_chunk.h"

namespace efla {

namespace {

struct Layout {
  size_t state, gates, sums, part, total;  // bytes of one of the two state arrays; offsets behind them
};
Layout layout(int B, int H, int64_t L, int DK, int DV) {
  const size_t slots = size_t(B) * H * size_t((L + 63) / 64);
  Layout w{};
  w.state = slots * DK * DV * sizeof(float);
  w.gates = 2 * w.state;
  w.sums = w.gates + slots * sizeof(ChunkGates);
  w.part = w.sums + slots * sizeof(ChunkSums);
  w.total = w.part + slots * 3 * sizeof(float);
  return w;
}

template <int DK>
hipError_t bwd_impl(const SsmBwd& b, void* ws, hipStream_t s) {
  const Layout w = layout(b.B, b.H, b.L, DK, b.DV);
  auto* at = static_cast<unsigned char*>(ws);
  const SsmStates st{reinterpret_cast<float*>(at), reinterpret_cast<float*>(at + w.state), reinterpret_cast<ChunkGates*>(at + w.gates),
                     reinterpret_cast<ChunkSums*>(at + w.sums)};
  float* part = reinterpret_cast<float*>(at + w.part);
  const int NC = int((b.L + 63) / 64), NVB = b.DV / 32, half = b.B * b.H * NVB;
  const int64_t slots = int64_t(b.B) * b.H * NC;
  hipLaunchKernelGGL(ssm_gates_kernel, dim3(unsigned((slots + 3) / 4)), dim3(kThreads), 0, s, b, st.gates, NC, slots);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((ssm_chain_kernel<DK>), dim3(unsigned(2 * half)), dim3(SsmChainShape<DK>::THREADS), 0, s, b, NVB, half,
                     ssm_remap(int64_t(b.B) * b.H, b.H / b.Hk), st);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  const dim3 grid(unsigned(int64_t(b.B) * b.Hk * NC)), wg(SsmGradShape<DK, 64>::THREADS);
  switch (b.DV) {
    case 32: hipLaunchKernelGGL((ssm_grad_kernel<DK, 32>), grid, wg, 0, s, b, st, NC); break;
    case 64: hipLaunchKernelGGL((ssm_grad_kernel<DK, 64>), grid, wg, 0, s, b, st, NC); break;
    case 128: hipLaunchKernelGGL((ssm_grad_kernel<DK, 128>), grid, wg, 0, s, b, st, NC); break;
    default: return hipErrorInvalidValue;
  }
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(ssm_steps_kernel, dim3(unsigned((slots + 3) / 4)), dim3(kThreads), 0, s, b, st, part, NC, slots, DK / 16);
  e = hipGetLastError();
  return e != hipSuccess ? e : launch_ssm_sums(part, b.da, b.dbias, b.dd, int64_t(b.B) * NC, b.H, s);
}

}  // namespace

size_t ssm_bwd_chunk_workspace(int B, int H, int64_t L, int DK, int DV) { return layout(B, H, L, DK, DV).total; }

int64_t ssm_bwd_chunk_threads(int B, int H, int64_t L, int DV) {
  const int64_t chains = 2 * int64_t(B) * H * (DV / 32) * SsmChainShape<64>::THREADS;
  const int64_t grads = int64_t(B) * H * ((L + 63) / 64) * SsmGradShape<64, 64>::THREADS;
  return chains > grads ? chains : grads;
}

hipError_t launch_ssm_bwd_chunk(const SsmBwd& b, void* ws, hipStream_t s) {
  return b.DK == 64 ? bwd_impl<64>(b, ws, s) : bwd_impl<128>(b, ws, s);
}

}  // namespace efla
