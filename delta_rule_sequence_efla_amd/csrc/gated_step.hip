// gated_step.hip -- the gated delta rule token by token (gated.h): one decode
// token per request, and whole sequences for the inputs that the chunked
// kernels do not take.  All arithmetic is fp32.
#include "gated.h"
#include "launchers.h"

namespace efla {

// ---------------------------------------------------------------------------
// Decode.  With r = S^T k, p = S^T q and a decay e = e^g:
//     u = a (v - e r),   S <- e S + k u^T,   o = e p + (k.q) u
// so each state is read once and written once, which is the whole cost: the
// step is bound by HBM (8 d_k d_v bytes a head).  One workgroup per request,
// head and DVW value columns; thread (rg, cq) keeps columns 4 cq .. 4 cq + 3 of
// rows rg, rg + NRG, .. in registers, and r and p are summed through LDS.
// States are read and written past the caches (nontemporal): a step touches
// each once, and a model's other layers run before the next one.  256 requests
// of 16 heads, d 128 (541 MB, three pools in turn): 106.7 us with ordinary
// accesses and whole states per workgroup, 99.4 us nontemporal, 96.3 us with 64
// columns a workgroup, 98.2 us with 32 (a large in-place copy's rate: 89 us).
// A row of the batch whose slot lies outside the pool has no request: its
// state does not exist and its row of o is left as it was.
template <typename T, int DK, int DVW>
__global__ __launch_bounds__(kThreads) void gated_step_kernel(
    const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v, const T* __restrict__ beta,
    const float* __restrict__ g, float* __restrict__ state, const int32_t* __restrict__ slots, T* __restrict__ o,
    int P, int H, int Hk, int DV, int NVB, int rule) {
  constexpr int NCQ = DVW / 4;
  constexpr int NRG = kThreads / NCQ < DK ? kThreads / NCQ : DK;  // rows in flight
  constexpr int RPT = DK / NRG;
  __shared__ float ks[DK], qs[DK], us[DVW];
  __shared__ __align__(16) float red_k[NRG * DVW];
  __shared__ __align__(16) float red_q[NRG * DVW];
  __shared__ float coef[3];

  const int64_t unit = blockIdx.x / NVB;
  const int v0 = int(blockIdx.x % NVB) * DVW;
  const int n = int(unit / H), h = int(unit % H);
  const int64_t row = state_row(slots, n, P);
  if (row < 0) return;
  const int64_t uk = int64_t(n) * Hk + h / (H / Hk);
  const int tid = threadIdx.x, cq = tid % NCQ, rg = tid / NCQ;
  const bool on = NRG * NCQ == kThreads || rg < NRG;
  float* Su = state + (row * H + h) * DK * DV + v0;

  f32x4 S[RPT];
#pragma unroll
  for (int i = 0; i < RPT; ++i)
    S[i] = on ? __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(Su + int64_t(rg + i * NRG) * DV + 4 * cq))
              : zero4();
  if (tid < DK) {
    ks[tid] = to_f32(k[uk * DK + tid]);
    qs[tid] = to_f32(q[uk * DK + tid]);
  }
  __syncthreads();
  if (tid < kWave) {
    float lam = 0.0f, kq = 0.0f;
    for (int d = tid; d < DK; d += kWave) {
      lam = fmaf(ks[d], ks[d], lam);
      kq = fmaf(ks[d], qs[d], kq);
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
      lam += __shfl_xor(lam, off);
      kq += __shfl_xor(kq, off);
    }
    if (tid == 0) {
      coef[0] = efla_alpha_rule(to_f32(beta[unit]), lam, rule);
      coef[1] = kq;
      coef[2] = expf(gate_floor(g[unit]));
    }
  }
  f32x4 pk = zero4(), pq = zero4();
  if (on) {
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      pk += ks[rg + i * NRG] * S[i];
      pq += qs[rg + i * NRG] * S[i];
    }
    *reinterpret_cast<f32x4*>(red_k + rg * DVW + 4 * cq) = pk;
    *reinterpret_cast<f32x4*>(red_q + rg * DVW + 4 * cq) = pq;
  }
  __syncthreads();
  const float e = coef[2];
  if (tid < DVW) {
    float rk = 0.0f, rq = 0.0f;
#pragma unroll 8
    for (int p = 0; p < NRG; ++p) {
      rk += red_k[p * DVW + tid];
      rq += red_q[p * DVW + tid];
    }
    const float u = coef[0] * (to_f32(v[unit * DV + v0 + tid]) - e * rk);
    us[tid] = u;
    o[unit * DV + v0 + tid] = from_f32<T>(fmaf(coef[1], u, e * rq));
  }
  __syncthreads();
  const f32x4 uq = *reinterpret_cast<const f32x4*>(us + 4 * cq);
  if (on) {
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const float kk = ks[rg + i * NRG];
      f32x4 x;
#pragma unroll
      for (int c = 0; c < 4; ++c) x[c] = fmaf(kk, uq[c], e * S[i][c]);
      __builtin_nontemporal_store(x, reinterpret_cast<f32x4*>(Su + int64_t(rg + i * NRG) * DV + 4 * cq));
    }
  }
}

template <typename T, int DK, int DVW>
static hipError_t gated_step_impl(const GatedStep& a, hipStream_t s) {
  const int NVB = a.DV / DVW;
  const int64_t nwg = int64_t(a.N) * a.H * NVB;
  hipLaunchKernelGGL((gated_step_kernel<T, DK, DVW>), dim3(unsigned(nwg)), dim3(kThreads), 0, s,
                     static_cast<const T*>(a.q), static_cast<const T*>(a.k), static_cast<const T*>(a.v),
                     static_cast<const T*>(a.beta), a.g, a.state, a.slots, static_cast<T*>(a.o), a.P, a.H, a.Hk, a.DV,
                     NVB, a.rule);
  return hipGetLastError();
}

template <typename T, int DK>
static hipError_t gated_step_dv(const GatedStep& a, hipStream_t s) {
  // 64 value columns a workgroup (above); where that gives the compute units
  // less than four workgroups each, 32, so that more of them share the loads.
  const bool cut = int64_t(a.N) * a.H * (a.DV / 64) < 1024;
  switch (a.DV) {
    case 16: return gated_step_impl<T, DK, 16>(a, s);
    case 32: return gated_step_impl<T, DK, 32>(a, s);
    case 64: return cut ? gated_step_impl<T, DK, 32>(a, s) : gated_step_impl<T, DK, 64>(a, s);
    case 128: return cut ? gated_step_impl<T, DK, 32>(a, s) : gated_step_impl<T, DK, 64>(a, s);
  }
  return hipErrorInvalidValue;
}

template <typename T>
hipError_t launch_gated_step(const GatedStep& a, hipStream_t s) {
  if (int64_t(a.N) * a.H == 0) return hipSuccess;
  switch (a.DK) {
    case 16: return gated_step_dv<T, 16>(a, s);
    case 32: return gated_step_dv<T, 32>(a, s);
    case 64: return gated_step_dv<T, 64>(a, s);
    case 128: return gated_step_dv<T, 128>(a, s);
  }
  return hipErrorInvalidValue;
}
template hipError_t launch_gated_step<float>(const GatedStep&, hipStream_t);
template hipError_t launch_gated_step<uint16_t>(const GatedStep&, hipStream_t);

// ---------------------------------------------------------------------------
// Whole sequences token by token, fp32 throughout: one workgroup per sequence,
// head and 16 value columns.  The 16 lanes of a DPP row share one column and
// split the key dims, NK each, so r = S^T k and o = S^T q are sums over a row
// (four DPP adds, no LDS); a wavefront carries four columns.  Blocks of 16
// tokens of q, k, v, beta and g are loaded into registers a block ahead (16
// threads per token), widened into one of two LDS buffers, with a and e^g
// formed on the way, so that a token costs LDS reads and the chain
// r -> u -> S alone.  With `states`, the state before every C-th token is
// stored, [chunk slot][d_k][d_v] fp32 (the backward's chunk starts; C % 16 == 0).
template <typename T, int N> struct alignas(N * sizeof(T) < 16 ? N * sizeof(T) : 16) Piece { T e[N]; };
template <int NK> struct Token {
  float k[NK], q[NK], v, a, e;
};

template <typename T, int DK>
__global__ __launch_bounds__(kThreads) void gated_recurrent_kernel(GatedFwd a, float* __restrict__ states, int C,
                                                                   int NC) {
  constexpr int NK = DK / 16, TB = 16;
  __shared__ __align__(16) float kS[2][TB][DK], qS[2][TB][DK];
  __shared__ float vS[2][TB][16], aS[2][TB], eS[2][TB], oS[2][TB][17];

  const int NVB = a.DV / 16, H = a.H, DV = a.DV;
  const int64_t unit = blockIdx.x / NVB;
  const int v0 = int(blockIdx.x % NVB) * 16;
  const int h = int(unit % H);
  int seq = int(unit / H);
  int64_t bos = int64_t(seq) * a.L, len = a.L;
  if (a.cu != nullptr) {
    if (a.order != nullptr) seq = seq_of_rank(a.order, seq, a.N);
    bos = clamp_offset(a.cu[seq], 0, a.L);
    len = clamp_offset(a.cu[seq + 1], bos, a.L) - bos;
  }
  const int64_t row = state_row(a.slots, seq, a.P);
  const int hk = h / (H / a.Hk);
  const T* q = static_cast<const T*>(a.q) + (bos * a.Hk + hk) * DK;
  const T* k = static_cast<const T*>(a.k) + (bos * a.Hk + hk) * DK;
  const T* v = static_cast<const T*>(a.v) + (bos * H + h) * DV + v0;
  const T* beta = static_cast<const T*>(a.beta) + bos * H + h;
  const float* g = a.g + bos * H + h;
  T* o = a.o == nullptr ? nullptr : static_cast<T*>(a.o) + (bos * H + h) * DV + v0;

  const int tid = threadIdx.x, lane = tid & 63, w = wave_id(), li = lane & 15, grp = lane >> 4;
  const int col = 4 * w + grp;            // this lane's value column of the block
  const int tok = tid >> 4, pc = tid & 15;  // staging: token of the block, piece of its row

  float S[NK];
  const float* s0 = a.s0 == nullptr || row < 0 ? nullptr : a.s0 + (row * H + h) * DK * DV + v0 + col;
#pragma unroll
  for (int e = 0; e < NK; ++e) S[e] = s0 == nullptr ? 0.0f : s0[int64_t(li * NK + e) * DV];

  Piece<T, NK> pk, pq;
  float pv = 0.0f, pb = 0.0f, pg = 0.0f;
  auto load = [&](int64_t t0) {
    const int64_t t = t0 + tok;
#pragma unroll
    for (int e = 0; e < NK; ++e) pk.e[e] = pq.e[e] = T(0);
    pv = pb = pg = 0.0f;
    if (t < len) {
      pk = *reinterpret_cast<const Piece<T, NK>*>(k + t * a.Hk * DK + pc * NK);
      pq = *reinterpret_cast<const Piece<T, NK>*>(q + t * a.Hk * DK + pc * NK);
      pv = to_f32(v[t * H * DV + pc]);
      pb = to_f32(beta[t * H]);
      pg = g[t * H];
    }
  };
  auto stage = [&](int b) {
    float lam = 0.0f;
#pragma unroll
    for (int e = 0; e < NK; ++e) {
      const float x = to_f32(pk.e[e]);
      lam = fmaf(x, x, lam);
      kS[b][tok][pc * NK + e] = x;
      qS[b][tok][pc * NK + e] = to_f32(pq.e[e]);
    }
    lam = row_sum16(lam);
    vS[b][tok][pc] = pv;
    if (pc == 0) {
      aS[b][tok] = efla_alpha_rule(pb, lam, a.rule);
      eS[b][tok] = expf(gate_floor(pg));
    }
  };
  auto store = [&](int64_t t0, int b) {
    const int64_t t = t0 + tok;
    if (o != nullptr && t < len) o[t * H * DV + pc] = from_f32<T>(oS[b][tok][pc]);
  };

  auto fetch = [&](Token<NK>& x, int b, int j) {
#pragma unroll
    for (int e = 0; e < NK; ++e) {
      x.k[e] = kS[b][j][li * NK + e];
      x.q[e] = qS[b][j][li * NK + e];
    }
    x.v = vS[b][j][col];
    x.a = aS[b][j];
    x.e = eS[b][j];
  };
  auto token = [&](const Token<NK>& x, int b, int j) {
    float r0 = 0.0f, r1 = 0.0f;
#pragma unroll
    for (int e = 0; e < NK; ++e) {
      if (e & 1) r1 = fmaf(x.k[e], S[e], r1);
      else r0 = fmaf(x.k[e], S[e], r0);
    }
    const float r = row_sum16(r0 + r1);
    const float u = x.a * fmaf(-x.e, r, x.v);
    float p0 = 0.0f, p1 = 0.0f;
#pragma unroll
    for (int e = 0; e < NK; ++e) {
      S[e] = fmaf(x.k[e], u, x.e * S[e]);
      if (e & 1) p1 = fmaf(x.q[e], S[e], p1);
      else p0 = fmaf(x.q[e], S[e], p0);
    }
    const float p = row_sum16(p0 + p1);
    if (li == 0) oS[b][j][col] = p;
  };

  const int64_t slot0 = int64_t(unit) * NC;  // dense batches only
  auto finish = [&]() {
    if (a.sfin == nullptr || row < 0) return;
    float* sf = a.sfin + (row * H + h) * DK * DV + v0 + col;
#pragma unroll
    for (int e = 0; e < NK; ++e) sf[int64_t(li * NK + e) * DV] = S[e];
  };
  if (len <= 0) {
    finish();
    return;
  }
  // (staging waits for the first block's loads and, in order, for S before
  // them: were the loop reachable with S in flight, every block would wait for
  // the next block's loads at its first token)
  load(0);
  stage(0);
  if (TB < len) load(TB);
  __syncthreads();
  for (int64_t t0 = 0; t0 < len; t0 += TB) {
    const int b = int(t0 / TB) & 1;
    if (states != nullptr && t0 % C == 0) {
      float* dst = states + (slot0 + t0 / C) * DK * DV + v0 + col;
#pragma unroll
      for (int e = 0; e < NK; ++e) dst[int64_t(li * NK + e) * DV] = S[e];
    }
    const int cnt = int(len - t0 < TB ? len - t0 : TB);
    // a token's values are read from the LDS while the one before is worked on
    Token<NK> now, next;
    fetch(now, b, 0);
    for (int j = 0; j < cnt; j += 2) {
      fetch(next, b, j + 1 < TB ? j + 1 : j);
      token(now, b, j);
      if (j + 1 >= cnt) break;
      fetch(now, b, j + 2 < TB ? j + 2 : j);
      token(next, b, j + 1);
    }
    if (t0 + TB < len) {
      stage(b ^ 1);  // last read two blocks ago, before the barrier below
      if (t0 + 2 * TB < len) load(t0 + 2 * TB);
    }
    __syncthreads();
    store(t0, b);  // oS[b] is written again two blocks on, after the next barrier
  }
  finish();
}

template <typename T>
hipError_t launch_gated_recurrent(const GatedFwd& a, float* states, int C, hipStream_t s) {
  const int64_t units = int64_t(a.cu == nullptr ? a.B : a.N) * a.H;
  const int64_t nwg = units * (a.DV / 16);
  if (nwg == 0) return hipSuccess;
  const int NC = int((a.L + C - 1) / C);
  const dim3 grid{unsigned(nwg)}, wg{kThreads};
  switch (a.DK) {
    case 16: hipLaunchKernelGGL((gated_recurrent_kernel<T, 16>), grid, wg, 0, s, a, states, C, NC); break;
    case 32: hipLaunchKernelGGL((gated_recurrent_kernel<T, 32>), grid, wg, 0, s, a, states, C, NC); break;
    case 64: hipLaunchKernelGGL((gated_recurrent_kernel<T, 64>), grid, wg, 0, s, a, states, C, NC); break;
    case 128: hipLaunchKernelGGL((gated_recurrent_kernel<T, 128>), grid, wg, 0, s, a, states, C, NC); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}
template hipError_t launch_gated_recurrent<float>(const GatedFwd&, float*, int, hipStream_t);
template hipError_t launch_gated_recurrent<uint16_t>(const GatedFwd&, float*, int, hipStream_t);

}  // namespace efla
