// gated_step.hip -- the gated delta rule without chunks (gated.h): one decode
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
// States are written past the caches (nontemporal): a step touches each once,
// and a model's other layers run before the next one.  Measured with three pools
// in turn, bf16, 16 heads, d 128, ordinary / nontemporal loads / stores / both:
// 256 requests (541 MB) 106.0 / 103.1 / 97.6 / 96.3 us (whole states per
// workgroup, ordinary: 106.7; a large in-place scale's rate: 89 us), 84 requests
// (177 MB) 31.6 / 30.8 / 30.5 / 33.6 us: part of a smaller pool stays in the
// last-level cache and is lost to nontemporal loads.
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
  __shared__ float ks[DK], qs[DK];
  __shared__ __align__(16) float us[DVW];
  __shared__ __align__(16) float red_k[NRG * DVW];
  __shared__ __align__(16) float red_q[NRG * DVW];
  __shared__ float coef[3];

  const uint32_t wg = blockIdx.x, unit32 = wg / uint32_t(NVB);  // 32-bit divisions: the 64-bit ones cost a microsecond
  const int64_t unit = unit32;
  const int v0 = int(wg % uint32_t(NVB)) * DVW;
  const int n = int(unit32 / uint32_t(H)), h = int(unit32 % uint32_t(H));
  const int64_t row = state_row(slots, n, P);
  if (row < 0) return;
  const int64_t uk = int64_t(n) * Hk + h / (H / Hk);
  const int tid = threadIdx.x, cq = tid % NCQ, rg = tid / NCQ;
  const bool on = NRG * NCQ == kThreads || rg < NRG;
  float* Su = state + (row * H + h) * DK * DV + v0;

  f32x4 S[RPT];
#pragma unroll
  for (int i = 0; i < RPT; ++i)
    S[i] = on ? *reinterpret_cast<const f32x4*>(Su + int64_t(rg + i * NRG) * DV + 4 * cq) : zero4();
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

// 64 value columns a workgroup (above); where that gives the compute units
// less than four workgroups each, 32, so that more of them share the loads.
static bool cut_columns(int N, int H, int DV) { return int64_t(N) * H * (DV / 64) < 1024; }

int64_t gated_step_threads(int N, int H, int DV) {
  return int64_t(N) * H * (DV < 64 ? 1 : DV / (cut_columns(N, H, DV) ? 32 : 64)) * kThreads;
}

template <typename T, int DK>
static hipError_t gated_step_dv(const GatedStep& a, hipStream_t s) {
  const bool cut = cut_columns(a.N, a.H, a.DV);
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
// Whole sequences in fp32 throughout, two tokens at a time: one workgroup per
// sequence, head and 16 value columns.  The 16 lanes of a DPP row share one
// column and split the key dims, NK each, so a product of a key or query with S
// is a sum over a row (four DPP adds, no LDS); a wavefront carries four columns.
// With S the state before tokens 0 and 1 of a pair and r = k^T S, p = q^T S:
//     u_0 = a_0 (v_0 - e_0 r_0)
//     u_1 = a_1 (v_1 - e_1 (e_0 r_1 + (k_1.k_0) u_0))
//     o_0 = e_0 p_0 + (q_0.k_0) u_0
//     o_1 = e_1 (e_0 p_1 + (q_1.k_0) u_0) + (q_1.k_1) u_1
//     S <- e_1 e_0 S + e_1 k_0 u_0 + k_1 u_1
// so the four sums over rows, each a chain of DPP adds with two wait states in
// between, run side by side.  Four more wavefronts stage blocks of 16 tokens, 16
// threads a token: they load two blocks ahead into registers, form a, e and the
// products of keys and queries among themselves, widen into one of two LDS
// buffers, and store the outputs of the block before.
// 2 x 777 tokens, 8 heads, d 64, fp32: 142 us token by token with the staging in
// the same wavefronts, 111 us by pairs, 82 us with wavefronts for each (and 49
// by 16 tokens, gated_blocks.hip, which takes the longer sequences).
// With `states`, the state before every C-th token is stored, [chunk
// slot][d_k][d_v] fp32 (the backward's chunk starts; C % 16 == 0).
template <typename T, int N> struct alignas(N * sizeof(T) < 16 ? N * sizeof(T) : 16) Piece { T e[N]; };
template <int NK> struct TokenPair {
  float k0[NK], k1[NK], q0[NK], q1[NK], v0, v1;
  f32x4 c, d;  // a_0, e_0, a_1, e_1; k_1.k_0, q_0.k_0, q_1.k_0, q_1.k_1
};

template <typename T, int DK>
__global__ __launch_bounds__(2 * kThreads) void gated_recurrent_kernel(GatedFwd a, float* __restrict__ states, int C,
                                                                   int NC) {
  constexpr int NK = DK / 16, TB = 16;
  __shared__ __align__(16) float kS[2][TB][DK], qS[2][TB][DK];
  __shared__ __align__(16) float cS[2][TB / 2][4], dS[2][TB / 2][4];  // per pair: TokenPair's c and d
  __shared__ float vS[2][TB][16];
  __shared__ float oS[2][TB * 17 + kThreads];  // behind the tile: where lanes without an output write

  const int NVB = a.DV / 16, H = a.H, DV = a.DV;
  const uint32_t wg = blockIdx.x, unit = wg / uint32_t(NVB);
  const int v0 = int(wg % uint32_t(NVB)) * 16;
  const int h = int(unit % uint32_t(H));
  int seq = int(unit / uint32_t(H));
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

  const int tid = threadIdx.x & (kThreads - 1), lane = tid & 63, w = wave_id() & 3, li = lane & 15, grp = lane >> 4;
  const bool stager = wave_id() >= 4;
  const int col = 4 * w + grp;            // this lane's value column of the block
  const int tok = tid >> 4, pc = tid & 15;  // staging: token of the block, piece of its row
  const int blocks = int((len + TB - 1) / TB);

  if (stager) {
    if (len <= 0) return;
    struct Regs {
      Piece<T, NK> k, q;
      float v, b, g;
    } X, Y;
    auto load = [&](Regs& x, int n) {  // tokens past the end: zeros, which change nothing
      const int64_t t = int64_t(n) * TB + tok;
#pragma unroll
      for (int e = 0; e < NK; ++e) x.k.e[e] = x.q.e[e] = T(0);
      x.v = x.b = x.g = 0.0f;
      if (t < len) {
        x.k = *reinterpret_cast<const Piece<T, NK>*>(k + t * a.Hk * DK + pc * NK);
        x.q = *reinterpret_cast<const Piece<T, NK>*>(q + t * a.Hk * DK + pc * NK);
        x.v = to_f32(v[t * H * DV + pc]);
        x.b = to_f32(beta[t * H]);
        x.g = g[t * H];
      }
    };
    auto stage = [&](const Regs& r, int b) {
      float lam = 0.0f, qk = 0.0f, kk1 = 0.0f, qk1 = 0.0f;
#pragma unroll
      for (int e = 0; e < NK; ++e) {
        const float x = to_f32(r.k.e[e]), y = to_f32(r.q.e[e]);
        const float other = __shfl_xor(x, 16);  // the key of the pair's other token
        lam = fmaf(x, x, lam);
        qk = fmaf(y, x, qk);
        kk1 = fmaf(x, other, kk1);
        qk1 = fmaf(y, other, qk1);
        kS[b][tok][pc * NK + e] = x;
        qS[b][tok][pc * NK + e] = y;
      }
      lam = row_sum16(lam);
      qk = row_sum16(qk);
      kk1 = row_sum16(kk1);
      qk1 = row_sum16(qk1);
      vS[b][tok][pc] = r.v;
      if (pc == 0) {
        cS[b][tok >> 1][2 * (tok & 1)] = efla_alpha_rule(r.b, lam, a.rule);
        cS[b][tok >> 1][2 * (tok & 1) + 1] = expf(gate_floor(r.g));
        if (tok & 1) {
          dS[b][tok >> 1][0] = kk1;
          dS[b][tok >> 1][2] = qk1;
          dS[b][tok >> 1][3] = qk;
        } else {
          dS[b][tok >> 1][1] = qk;
        }
      }
    };
    auto store = [&](int n) {
      const int64_t t = int64_t(n) * TB + tok;
      if (o != nullptr && t < len) o[t * H * DV + pc] = from_f32<T>(oS[n & 1][tok * 17 + pc]);
    };
    // iteration n (block n is worked on): block n + 1 goes into the other
    // buffer, block n - 1's outputs leave; loads past the end bring zeros
    load(X, 0);
    load(Y, 1);
    stage(X, 0);
    load(X, 2);
    __syncthreads();
    auto step = [&](Regs& r, int n) {
      stage(r, (n + 1) & 1);
      load(r, n + 3);
      if (n > 0) store(n - 1);
      __syncthreads();
    };
    for (int n = 0;;) {
      step(Y, n);
      if (++n >= blocks) break;
      step(X, n);
      if (++n >= blocks) break;
    }
    store(blocks - 1);
    return;
  }

  float S[NK];
  const float* s0 = a.s0 == nullptr || row < 0 ? nullptr : a.s0 + (row * H + h) * DK * DV + v0 + col;
#pragma unroll
  for (int e = 0; e < NK; ++e) S[e] = s0 == nullptr ? 0.0f : s0[int64_t(li * NK + e) * DV];
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

  auto fetch = [&](TokenPair<NK>& x, int b, int j) {
#pragma unroll
    for (int e = 0; e < NK; ++e) {
      x.k0[e] = kS[b][j][li * NK + e];
      x.k1[e] = kS[b][j + 1][li * NK + e];
      x.q0[e] = qS[b][j][li * NK + e];
      x.q1[e] = qS[b][j + 1][li * NK + e];
    }
    x.v0 = vS[b][j][col];
    x.v1 = vS[b][j + 1][col];
    x.c = *reinterpret_cast<const f32x4*>(cS[b][j >> 1]);
    x.d = *reinterpret_cast<const f32x4*>(dS[b][j >> 1]);
  };
  // lane 0 of a row writes o of the pair's first token, lane 1 of its second,
  // the others a place of their own
  const int o_at = li < 2 ? li * 17 + col : TB * 17 + tid, o_step = li < 2 ? 17 : 0;
  auto pair = [&](const TokenPair<NK>& x, int b, int j) {
    float r0 = 0.0f, r1 = 0.0f, p0 = 0.0f, p1 = 0.0f;
#pragma unroll
    for (int e = 0; e < NK; ++e) {
      r0 = fmaf(x.k0[e], S[e], r0);
      r1 = fmaf(x.k1[e], S[e], r1);
      p0 = fmaf(x.q0[e], S[e], p0);
      p1 = fmaf(x.q1[e], S[e], p1);
    }
    r0 = row_sum16(r0);
    r1 = row_sum16(r1);
    p0 = row_sum16(p0);
    p1 = row_sum16(p1);
    const float e0 = x.c[1], e1 = x.c[3];
    const float u0 = x.c[0] * fmaf(-e0, r0, x.v0);
    const float u1 = x.c[2] * fmaf(-e1, fmaf(x.d[0], u0, e0 * r1), x.v1);
    const float o0 = fmaf(x.d[1], u0, e0 * p0);
    const float o1 = fmaf(x.d[3], u1, e1 * fmaf(x.d[2], u0, e0 * p1));
    const float e01 = e0 * e1, w0 = e1 * u0;
#pragma unroll
    for (int e = 0; e < NK; ++e) S[e] = fmaf(x.k1[e], u1, fmaf(x.k0[e], w0, e01 * S[e]));
    oS[b][o_at + j * o_step] = li == 0 ? o0 : o1;
  };

  const int64_t slot0 = int64_t(unit) * NC;  // dense batches only
  __syncthreads();
  for (int64_t t0 = 0; t0 < len; t0 += TB) {
    const int b = int(t0 / TB) & 1;
    const uint32_t blk = uint32_t(t0 / TB), per = uint32_t(C) / TB;
    if (states != nullptr && blk % per == 0) {
      float* dst = states + (slot0 + blk / per) * DK * DV + v0 + col;
#pragma unroll
      for (int e = 0; e < NK; ++e) dst[int64_t(li * NK + e) * DV] = S[e];
    }
    const int cnt = int(len - t0 < TB ? len - t0 : TB);
    // a pair's values are read from the LDS while the pair before is worked on
    TokenPair<NK> now, next;
    fetch(now, b, 0);
    for (int j = 0; j < cnt; j += 4) {
      fetch(next, b, j + 2 < TB ? j + 2 : j);
      pair(now, b, j);
      if (j + 2 >= cnt) break;
      fetch(now, b, j + 4 < TB ? j + 4 : j);
      pair(next, b, j + 2);
    }
    __syncthreads();
  }
  finish();
}

// By 16 tokens (gated_blocks.hip) the chain is shorter, but it starts four
// blocks late and fewer of its workgroups share a compute unit.  Measured (fp32,
// us, pairs / blocks):
//   d 64,   256 workgroups: 16 tokens 5.8 / 6.0, 32 7.5 / 7.1, 128 17.7 / 13.0, 512 57 / 38
//   d 64,  1024:            32 18.3 / 24.7, 128 49.1 / 50.4, 512 160 / 142
//   d 128,   64:            16 7.2 / 6.5, 32 9.6 / 8.0, 128 23.6 / 16.8, 512 80 / 52
//   d 128,  512:            32 14.7 / 16.1, 64 24.1 / 25.1, 128 38.8 / 36.6, 512 126 / 105
//   d 128, 8192:            32 155 / 231, 128 508 / 525, 512 1963 / 1613
// Packed batches go by their mean length: most of their workgroups are about that
// long, and both forms take any length.  Measured (sequences x tokens, same units):
//   d 64, 8 heads:   64 x 8 18.4 / 37.5, 200 x 1 43 / 112, 4 x 100 15.0 / 11.3
//   d 128, 16 heads: 64 x 8 92 / 169, 32 x 32 85 / 115, 8 x 64 41.5 / 45.1
//   and one long among short ones: 300 and 15 x 1 at d 64 35 / 22, at d 128 51 / 58
static bool by_blocks(int64_t nwg, int64_t tokens, int DK) { return DK >= 64 && tokens >= (nwg <= 256 ? 32 : 160); }

int64_t gated_recurrent_threads(int64_t seqs, int H, int64_t L, bool packed, int DK, int DV) {
  const int64_t nwg = seqs * H * (DV / 16);
  return nwg * (by_blocks(nwg, packed ? L / seqs : L, DK) ? kGatedBlocksThreads : 2 * kThreads);
}

template <typename T>
hipError_t launch_gated_recurrent(const GatedFwd& a, float* states, int C, hipStream_t s) {
  const int64_t units = int64_t(a.cu == nullptr ? a.B : a.N) * a.H;
  const int64_t nwg = units * (a.DV / 16);
  if (nwg == 0) return hipSuccess;
  if (by_blocks(nwg, a.cu == nullptr ? a.L : a.L / a.N, a.DK)) return launch_gated_blocks<T>(a, states, C, s);
  const int NC = int((a.L + C - 1) / C);
  const dim3 grid{unsigned(nwg)}, wg{2 * kThreads};
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
