// gated_bwd.hip -- launches of the gated backward pass (gated_bwd.h).
// Workspace, every region 256-byte aligned, per chunk slot ((b H + h) NC + n),
// all fp32: T, X, P [C][C]; a, G [C]; S, dS [d_k][d_v]; and where key heads are
// shared dq and dk per value head, [B L][H][d_k].
#include "gated_bwd.h"

namespace efla {

namespace {
size_t align256(size_t x) { return (x + 255) / 256 * 256; }
}  // namespace

static GatedBwdLayout gated_bwd_layout(int B, int H, int Hk, int64_t L, int DK, int DV, int C) {
  const size_t slots = size_t(B) * H * ((L + C - 1) / C);
  GatedBwdLayout w{};
  w.t = 0;
  w.x = w.t + align256(slots * C * C * 4);
  w.p = w.x + align256(slots * C * C * 4);
  w.a = w.p + align256(slots * C * C * 4);
  w.gc = w.a + align256(slots * C * 4);
  w.s = w.gc + align256(slots * C * 4);
  w.ds = w.s + align256(slots * size_t(DK) * DV * 4);
  w.dqh = w.ds + align256(slots * size_t(DK) * DV * 4);
  const size_t heads = Hk < H ? align256(size_t(B) * L * H * DK * 4) : 0;
  w.dkh = w.dqh + heads;
  w.total = w.dkh + heads;
  return w;
}

size_t gated_bwd_workspace(int B, int H, int Hk, int64_t L, int DK, int DV, int C, size_t) {
  return gated_bwd_layout(B, H, Hk, L, DK, DV, C).total;
}

template <typename T, int DK, int C>
static hipError_t gated_bwd_impl(const GatedBwd& b, unsigned char* ws, hipStream_t s) {
  const int NC = int((b.L + C - 1) / C);
  const int64_t bh = int64_t(b.B) * b.H, slots = bh * NC;
  const GatedBwdLayout lay = gated_bwd_layout(b.B, b.H, b.Hk, b.L, DK, b.DV, C);
  auto f = [&](size_t off) { return reinterpret_cast<float*>(ws + off); };
  if (slots > 0) {
    hipLaunchKernelGGL((gated_ut_kernel<T, DK, C>), dim3(unsigned(slots)), dim3(kThreads), 0, s, b, f(lay.t), f(lay.x),
                       f(lay.p), f(lay.a), f(lay.gc), NC);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    GatedFwd a{};
    a.q = b.q;
    a.k = b.k;
    a.v = b.v;
    a.beta = b.beta;
    a.g = b.g;
    a.s0 = b.s0;
    a.B = b.B;
    a.H = b.H;
    a.Hk = b.Hk;
    a.P = b.B;
    a.L = b.L;
    a.DK = DK;
    a.DV = b.DV;
    a.rule = b.rule;
    if (hipError_t e = launch_gated_recurrent<T>(a, f(lay.s), C, s); e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((gated_bwd_state_kernel<T, DK, C>), dim3(unsigned(bh * (b.DV / 16))), dim3(kThreads), 0, s, b,
                     f(lay.t), f(lay.p), f(lay.gc), f(lay.ds), NC, b.DV / 16);
  if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  if (slots == 0) return hipSuccess;
  const bool shared = b.Hk < b.H;
  hipLaunchKernelGGL((gated_bwd_chunk_kernel<T, DK, C>), dim3(unsigned(slots)), dim3(kThreads), 0, s, b, f(lay.t),
                     f(lay.x), f(lay.p), f(lay.a), f(lay.gc), f(lay.s), f(lay.ds), shared ? f(lay.dqh) : nullptr,
                     shared ? f(lay.dkh) : nullptr, NC);
  if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  if (shared) {
    const int64_t rows = int64_t(b.B) * b.L * b.Hk, n = rows * (DK / 4);
    hipLaunchKernelGGL((gated_head_sum_kernel<T>), dim3(unsigned((n + kThreads - 1) / kThreads)), dim3(kThreads), 0, s,
                       f(lay.dqh), f(lay.dkh), static_cast<T*>(b.dq), static_cast<T*>(b.dk), rows, b.H / b.Hk, DK);
  }
  return hipGetLastError();
}

template <typename T, int DK>
static hipError_t gated_bwd_c(const GatedBwd& b, int C, unsigned char* ws, hipStream_t s) {
  switch (C) {
    case 16: return gated_bwd_impl<T, DK, 16>(b, ws, s);
    case 32: return gated_bwd_impl<T, DK, 32>(b, ws, s);
    case 64: return gated_bwd_impl<T, DK, 64>(b, ws, s);
  }
  return hipErrorInvalidValue;
}

template <typename T>
hipError_t launch_gated_bwd(const GatedBwd& b, int C, void* workspace, hipStream_t s) {
  auto* ws = static_cast<unsigned char*>(workspace);
  switch (b.DK) {
    case 16: return gated_bwd_c<T, 16>(b, C, ws, s);
    case 32: return gated_bwd_c<T, 32>(b, C, ws, s);
    case 64: return gated_bwd_c<T, 64>(b, C, ws, s);
    case 128: return gated_bwd_c<T, 128>(b, C, ws, s);
  }
  return hipErrorInvalidValue;
}
template hipError_t launch_gated_bwd<float>(const GatedBwd&, int, void*, hipStream_t);
template hipError_t launch_gated_bwd<uint16_t>(const GatedBwd&, int, void*, hipStream_t);

}  // namespace efla
