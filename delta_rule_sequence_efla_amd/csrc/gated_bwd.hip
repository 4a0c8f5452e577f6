// gated_bwd.hip -- the gated backward pass: which kernels run, and its
// workspace, every region 256-byte aligned, per chunk slot ((b H + h) NC + n).
//   fp32 arithmetic (gated_bwd.h; every type and size), all fp32:
//     T, X, P [C][C]; a [C], G [C] in 64 bits; S, dS [d_k][d_v]
//   bf16 matrix cores (bf16 inputs, d_k 64 or 128, d_v % 32 == 0; chunks of 64
//   whatever chunk the caller names):
//     X fragments (12 KiB) and gate block (1 KiB) as the forward's, P fragments
//     (6 KiB), Qe bf16 [C][d_k], S and dS bf16 [d_v][d_k]
// and for both, where key heads are shared, dq and dk per value head in fp32,
// [B L][H][d_k].
#include "gated_bwd.h"

namespace efla {

namespace {
size_t align256(size_t x) { return (x + 255) / 256 * 256; }
}  // namespace

// Sequences this short run in fp32 (chunk 16) for bf16 inputs too: dq and dk of
// a few tokens are keys and queries times single scalar products dO_i . U_j,
// which cancel by chance, so the bf16 rounding of U shows in them (8e-3 of dq
// at two tokens and two key heads; from some tens of scalars on, 4e-3 at most).
// Either way the call is four or five launches of a few microseconds.
constexpr int64_t kShort = 16;
static bool gated_bwd_fast(int64_t L, int DK, int DV, size_t esz) {
  return esz == 2 && L > kShort && gated_chunk_supported(DK, DV);
}
// Chunk of the fp32 kernels: 32 tokens.  A workgroup's products with S cost as
// much a token at any chunk, so half the chunk is twice the workgroups at half the
// time each; at 16 the chains over the chunks outweigh it.  Measured, 16 / 32 / 64
// (us, float32): 8 heads d 64, 200 tokens 75 / 61 / 91, 3 x 1100 323 / 210 / 246;
// d 128, 200 tokens 118 / 97 / 156, 3 x 1100 633 / 392 / 421.
static int fp32_chunk(int64_t L) { return L <= kShort ? 16 : 32; }

static GatedBwdLayout gated_bwd_layout(int B, int H, int Hk, int64_t L, int DK, int DV, size_t esz) {
  const bool fast = gated_bwd_fast(L, DK, DV, esz);
  const int C = fast ? 64 : fp32_chunk(L);
  const size_t slots = size_t(B) * H * ((L + C - 1) / C);
  size_t at = 0;
  auto region = [&](size_t bytes) {
    const size_t here = at;
    at += align256(bytes);
    return here;
  };
  GatedBwdLayout w{};
  const size_t e = fast ? 2 : 4;
  w.s = region(slots * size_t(DK) * DV * e);
  w.ds = region(slots * size_t(DK) * DV * e);
  if (fast) {
    w.xfr = region(slots * 12 * 1024);
    w.p = region(slots * 6 * 1024);
    w.gc = region(slots * 1024);
    w.qe = region(slots * size_t(C) * DK * 2);
  } else {
    w.x = region(slots * C * C * 4);
    w.t = region(slots * C * C * 4);
    w.p = region(slots * C * C * 4);
    w.a = region(slots * C * 4);
    w.gc = region(slots * C * 8);
  }
  const size_t heads = Hk < H ? size_t(B) * L * H * DK * 4 : 0;
  w.dqh = region(heads);
  w.dkh = region(heads);
  w.total = at;
  return w;
}

size_t gated_bwd_workspace(int B, int H, int Hk, int64_t L, int DK, int DV, size_t esz) {
  return gated_bwd_layout(B, H, Hk, L, DK, DV, esz).total;
}

int64_t gated_bwd_threads(int B, int H, int Hk, int64_t L, int DK, int DV, size_t esz) {
  const bool fast = gated_bwd_fast(L, DK, DV, esz);
  const int C = fast ? 64 : fp32_chunk(L);
  const int64_t bh = int64_t(B) * H, slots = bh * ((L + C - 1) / C);
  const int64_t chains = fast ? 2 * bh * (DV / 32) * gated_chains_threads(DK) : gated_recurrent_threads(B, H, L, false, DK, DV);
  const int64_t chunks = slots * (fast ? gated_bwd_chunk_threads(DK) : kThreads);
  const int64_t heads = Hk < H ? int64_t(B) * L * Hk * (DK / 4) : 0;
  const int64_t most = chains > chunks ? chains : chunks;
  return most > heads ? most : heads;
}

// The forward's inputs, for the backward's recomputation.
static GatedFwd forward_of(const GatedBwd& b) {
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
  a.DK = b.DK;
  a.DV = b.DV;
  a.rule = b.rule;
  return a;
}

// dq and dk of shared key heads from those of their value heads.
template <typename T>
static hipError_t sum_heads(const GatedBwd& b, const float* dqh, const float* dkh, hipStream_t s) {
  const int64_t rows = int64_t(b.B) * b.L * b.Hk, n = rows * (b.DK / 4);
  hipLaunchKernelGGL((gated_head_sum_kernel<T>), dim3(unsigned((n + kThreads - 1) / kThreads)), dim3(kThreads), 0, s,
                     dqh, dkh, static_cast<T*>(b.dq), static_cast<T*>(b.dk), rows, b.H / b.Hk, b.DK);
  return hipGetLastError();
}

static hipError_t gated_bwd_bf16(const GatedBwd& b, unsigned char* ws, hipStream_t s) {
  const GatedBwdLayout lay = gated_bwd_layout(b.B, b.H, b.Hk, b.L, b.DK, b.DV, 2);
  auto f = [&](size_t off) { return reinterpret_cast<float*>(ws + off); };
  auto u = [&](size_t off) { return reinterpret_cast<uint16_t*>(ws + off); };
  const GatedFwd a = forward_of(b);
  const bool shared = b.Hk < b.H;
  hipError_t e = launch_gated_ut_bwd(a, u(lay.xfr), f(lay.gc), u(lay.p), u(lay.qe), s);
  if (e == hipSuccess) e = launch_gated_chains(a, b, u(lay.xfr), u(lay.qe), f(lay.gc), u(lay.s), u(lay.ds), s);
  if (e == hipSuccess)
    e = launch_gated_bwd_chunk(b, u(lay.xfr), u(lay.p), f(lay.gc), u(lay.s), u(lay.ds),
                               shared ? f(lay.dqh) : nullptr, shared ? f(lay.dkh) : nullptr, s);
  if (e == hipSuccess && shared) e = sum_heads<uint16_t>(b, f(lay.dqh), f(lay.dkh), s);
  return e;
}

template <typename T, int DK, int C>
static hipError_t gated_bwd_impl(const GatedBwd& b, unsigned char* ws, hipStream_t s) {
  const int NC = int((b.L + C - 1) / C);
  const int64_t bh = int64_t(b.B) * b.H, slots = bh * NC;
  const GatedBwdLayout lay = gated_bwd_layout(b.B, b.H, b.Hk, b.L, DK, b.DV, sizeof(T));
  auto f = [&](size_t off) { return reinterpret_cast<float*>(ws + off); };
  if (slots > 0) {
    hipLaunchKernelGGL((gated_ut_kernel<T, DK, C>), dim3(unsigned(slots)), dim3(kThreads), 0, s, b, f(lay.t), f(lay.x),
                       f(lay.p), f(lay.a), reinterpret_cast<double*>(ws + lay.gc), NC);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    if (hipError_t e = launch_gated_recurrent<T>(forward_of(b), f(lay.s), C, s); e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((gated_bwd_state_kernel<T, DK, C>), dim3(unsigned(bh * (b.DV / 16))), dim3(kThreads), 0, s, b,
                     f(lay.t), f(lay.p), reinterpret_cast<double*>(ws + lay.gc), f(lay.ds), NC, b.DV / 16);
  if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  if (slots == 0) return hipSuccess;
  const bool shared = b.Hk < b.H;
  hipLaunchKernelGGL((gated_bwd_chunk_kernel<T, DK, C>), dim3(unsigned(slots)), dim3(kThreads), 0, s, b, f(lay.t),
                     f(lay.x), f(lay.p), f(lay.a), reinterpret_cast<double*>(ws + lay.gc), f(lay.s), f(lay.ds), shared ? f(lay.dqh) : nullptr,
                     shared ? f(lay.dkh) : nullptr, NC);
  if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  return shared ? sum_heads<T>(b, f(lay.dqh), f(lay.dkh), s) : hipSuccess;
}

template <typename T, int DK>
static hipError_t gated_bwd_c(const GatedBwd& b, unsigned char* ws, hipStream_t s) {
  return fp32_chunk(b.L) == 16 ? gated_bwd_impl<T, DK, 16>(b, ws, s) : gated_bwd_impl<T, DK, 32>(b, ws, s);
}

template <typename T>
hipError_t launch_gated_bwd(const GatedBwd& b, void* workspace, hipStream_t s) {
  auto* ws = static_cast<unsigned char*>(workspace);
  if (gated_bwd_fast(b.L, b.DK, b.DV, sizeof(T))) return gated_bwd_bf16(b, ws, s);
  switch (b.DK) {
    case 16: return gated_bwd_c<T, 16>(b, ws, s);
    case 32: return gated_bwd_c<T, 32>(b, ws, s);
    case 64: return gated_bwd_c<T, 64>(b, ws, s);
    case 128: return gated_bwd_c<T, 128>(b, ws, s);
  }
  return hipErrorInvalidValue;
}
template hipError_t launch_gated_bwd<float>(const GatedBwd&, void*, hipStream_t);
template hipError_t launch_gated_bwd<uint16_t>(const GatedBwd&, void*, hipStream_t);

}  // namespace efla
