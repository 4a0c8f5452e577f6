// ssm_step.hip -- the selective state space scan (ssm.h) for one token a
// request: S <- e^{a D} S + D k v^T, o = S^T q + d v, in float32.
#include "launchers.h"
#include "ssm.h"

namespace efla {

// Each state is read once and written once (8 d_k d_v bytes a head), which is
// the whole cost.  One workgroup per request, head and DVW value columns; thread
// (rg, cq) keeps columns 4 cq .. 4 cq + 3 of rows rg, rg + NRG, ..: the loads of
// the state are issued before anything else, the new state leaves without a wait
// for the others' rows, and only o is summed over the rows through the LDS.
// A row of the batch whose slot lies outside the pool has no request: its
// state does not exist and its row of o is left as it was.
template <typename T, int DK, int DVW>
__global__ __launch_bounds__(kThreads) void ssm_step_kernel(SsmStep a, int NVB) {
  constexpr int NCQ = DVW / 4;
  constexpr int NRG = kThreads / NCQ < DK ? kThreads / NCQ : DK;  // rows in flight
  constexpr int RPT = DK / NRG;
  __shared__ __align__(16) float red[NRG * DVW];

  const uint32_t wg = blockIdx.x, unit = wg / uint32_t(NVB);  // 32-bit divisions: the 64-bit ones cost a microsecond
  const int v0 = int(wg % uint32_t(NVB)) * DVW;
  const int n = int(unit / uint32_t(a.H)), h = int(unit % uint32_t(a.H));
  const int64_t row = state_row(a.slots, n, a.P);
  if (row < 0) return;
  const int hk = h / (a.H / a.Hk);
  const int tid = threadIdx.x, cq = tid % NCQ, rg = tid / NCQ;
  const bool on = NRG * NCQ == kThreads || rg < NRG;
  float* Su = a.state + (row * a.H + h) * DK * a.DV + v0;

  f32x4 S[RPT];
#pragma unroll
  for (int i = 0; i < RPT; ++i)
    S[i] = on ? *reinterpret_cast<const f32x4*>(Su + int64_t(rg + i * NRG) * a.DV + 4 * cq) : zero4();
  const T* k = static_cast<const T*>(a.k) + n * a.k_row + hk * DK;
  const T* q = static_cast<const T*>(a.q) + n * a.q_row + hk * DK;
  const T* v = static_cast<const T*>(a.v) + n * a.v_row + int64_t(h) * a.DV + v0;
  T* o = static_cast<T*>(a.o) + n * a.o_row + int64_t(h) * a.DV + v0;
  float kk[RPT], qq[RPT];
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    kk[i] = on ? to_f32(k[rg + i * NRG]) : 0.0f;
    qq[i] = on ? to_f32(q[rg + i * NRG]) : 0.0f;
  }
  f32x4 vv;
#pragma unroll
  for (int c = 0; c < 4; ++c) vv[c] = to_f32(v[4 * cq + c]);
  const float raw = to_f32(static_cast<const T*>(a.dt)[n * a.dt_row + h]) + (a.bias != nullptr ? a.bias[h] : 0.0f);
  const float delta = softplus(raw), e = expf(gate_floor(a.a[h] * delta));
  f32x4 sum = zero4();
  if (on) {
    vv = delta * vv;
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      f32x4 x;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        x[c] = fmaf(kk[i], vv[c], e * S[i][c]);
        sum[c] = fmaf(qq[i], x[c], sum[c]);
      }
      __builtin_nontemporal_store(x, reinterpret_cast<f32x4*>(Su + int64_t(rg + i * NRG) * a.DV + 4 * cq));
    }
    *reinterpret_cast<f32x4*>(red + rg * DVW + 4 * cq) = sum;
  }
  __syncthreads();
  if (tid < DVW) {
    float x = 0.0f;
#pragma unroll 8
    for (int p = 0; p < NRG; ++p) x += red[p * DVW + tid];
    const float skip = a.d != nullptr ? a.d[h] : 0.0f;
    o[tid] = from_f32<T>(a.d != nullptr ? fmaf(skip, to_f32(v[tid]), x) : x);
  }
}

template <typename T, int DK, int DVW>
static hipError_t ssm_step_impl(const SsmStep& a, hipStream_t s) {
  const int NVB = a.DV / DVW;
  hipLaunchKernelGGL((ssm_step_kernel<T, DK, DVW>), dim3(unsigned(int64_t(a.N) * a.H * NVB)), dim3(kThreads), 0, s, a, NVB);
  return hipGetLastError();
}

// 64 value columns a workgroup, as the gated step; where that gives the compute
// units less than four workgroups each, 32.
static bool cut_columns(int N, int H, int DV) { return int64_t(N) * H * (DV / 64) < 1024; }

int64_t ssm_step_threads(int N, int H, int DV) {
  return int64_t(N) * H * (DV < 64 ? 1 : DV / (cut_columns(N, H, DV) ? 32 : 64)) * kThreads;
}

template <typename T, int DK>
static hipError_t ssm_step_dv(const SsmStep& a, hipStream_t s) {
  const bool cut = cut_columns(a.N, a.H, a.DV);
  switch (a.DV) {
    case 16: return ssm_step_impl<T, DK, 16>(a, s);
    case 32: return ssm_step_impl<T, DK, 32>(a, s);
    case 64:
    case 128: return cut ? ssm_step_impl<T, DK, 32>(a, s) : ssm_step_impl<T, DK, 64>(a, s);
  }
  return hipErrorInvalidValue;
}

template <typename T>
hipError_t launch_ssm_step(const SsmStep& a, hipStream_t s) {
  switch (a.DK) {
    case 16: return ssm_step_dv<T, 16>(a, s);
    case 32: return ssm_step_dv<T, 32>(a, s);
    case 64: return ssm_step_dv<T, 64>(a, s);
    case 128: return ssm_step_dv<T, 128>(a, s);
  }
  return hipErrorInvalidValue;
}
template hipError_t launch_ssm_step<float>(const SsmStep&, hipStream_t);
template hipError_t launch_ssm_step<uint16_t>(const SsmStep&, hipStream_t);

}  // namespace efla
