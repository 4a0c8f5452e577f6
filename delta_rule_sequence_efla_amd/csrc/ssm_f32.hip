// ssm_f32.hip -- the selective state space scan (ssm.h) in float32 throughout:
// chunks of 32 tokens whose products run on the fp32 matrix cores.  Takes every
// head size and both input types (bf16 is widened on its way into the LDS): the
// forward pass, the chains of states and of state gradients that the backward
// pass reads, and the backward pass's gradients chunk by chunk.
#include <type_traits>

#include "launchers.h"
#include "ssm.h"

namespace efla {

namespace {

constexpr int kC = 32, kBV = 16;  // tokens a chunk, value columns a workgroup of a chain
constexpr int kFwd = 0, kStates = 1, kReverse = 2, kLocal = 3;
constexpr int kChain = 2 * kThreads;  // threads of a workgroup of a chain

// ROWS x COLS values of T (row t at src + t * stride) on their way to the LDS:
// fetched into registers, widened and stored with a pitch; rows at or past
// `valid` are zero.  Columns from COLS on, which products over a head size of 16 read,
// are left as they are: a kernel zeroes them, behind a barrier, before the first put.
template <typename T, int COLS, int THREADS = kThreads>
struct Tile {
  static constexpr int VE = 16 / sizeof(T), VPR = COLS / VE, N = kC * VPR, PER = cdiv(N, THREADS);
  struct alignas(16) Vec {
    T e[VE];
  };
  Vec x[PER];
  __device__ __forceinline__ void fetch(const T* __restrict__ src, int64_t stride, int valid, int tid) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int at = tid + i * THREADS, r = at / VPR, c = at % VPR;
#pragma unroll
      for (int e = 0; e < VE; ++e) x[i].e[e] = T(0);
      if (at < N && r < valid) x[i] = *reinterpret_cast<const Vec*>(src + r * stride + c * VE);
    }
  }
  __device__ __forceinline__ void put(float* dst, int pitch, int tid) const {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int at = tid + i * THREADS, r = at / VPR, c = at % VPR;
      if (at < N) {
#pragma unroll
        for (int e = 0; e < VE; e += 4)
          *reinterpret_cast<f32x4*>(dst + r * pitch + c * VE + e) =
              f32x4{to_f32(x[i].e[e]), to_f32(x[i].e[e + 1]), to_f32(x[i].e[e + 2]), to_f32(x[i].e[e + 3])};
      }
    }
  }
};

using Gates = GatesOf<kC>;

// ---------------------------------------------------------------------------
// One workgroup carries 16 value columns of one sequence and head through its
// chunks.
//   kFwd:     o and the final state
//   kStates:  the state before every chunk, [slot][d_k][d_v]
//   kReverse: the chunks from last to first, X <- e^{G_C} X + Q^T diag(e^G) dO,
//             and X after every chunk (k = q, v = dO here)
//   kLocal:   a segment's end state (the first's from s0, the others' from zero) and
//             its decay
// A chunk takes two barriers.  Behind the first, side by side: three wavefronts the
// tiles of P, two S^T Q^T for half of the tokens each, two (the chains: four) the
// state's tiles, which stay in their accumulators, one the gates of the next chunk.
// Behind the second: O = diag(e^G) S^T Q^T + V^T P^T and its store, the new state
// into the LDS for the next readout, and the next chunk's tokens into the other
// buffer.  Bound by that chain: 777 tokens, d 64, 25 chunks in one go, 52 us; one after the other
// with three barriers and the gates in line, on four wavefronts, 77 us.
template <typename T, int DK, int MODE>
__global__ __launch_bounds__(kChain) void ssm_f32_kernel(SsmFwd a, float* __restrict__ states, int NC) {
  constexpr bool FWD = MODE == kFwd;
  constexpr int DKP = DK < 32 ? 32 : DK, KP = DKP + 4, VP = kBV + 4, PP = kC + 4;
  constexpr int KU = DKP / 32, DT = DK / 16, SW = FWD ? 2 : 4, OWN = cdiv(DT, SW);  // S waves: the last SW
  __shared__ __align__(16) float Qs[FWD ? 2 : 1][FWD ? kC : 1][KP];
  __shared__ __align__(16) float Ks[2][kC][KP];
  __shared__ __align__(16) float Vs[2][kC][VP];
  __shared__ __align__(16) float Ps[kC][PP];
  __shared__ __align__(16) float St[kBV][KP];  // S^T, for the readout
  __shared__ Gates gates[2];

  const int NVB = a.DV / kBV, H = a.H;
  const uint32_t wg = blockIdx.x, unit = wg / uint32_t(NVB);
  const int v0 = int(wg % uint32_t(NVB)) * kBV, h = int(unit % uint32_t(H));
  const SsmUnit sp = ssm_unit<kC>(a, int(unit / uint32_t(H)), h, int(threadIdx.x) & 63);
  if (sp.seq < 0 || (MODE == kLocal && sp.last)) return;
  const int64_t bos = sp.bos, len = sp.len, row = state_row(a.slots, sp.seq, a.P);
  const int hk = h / (H / a.Hk);
  const T* q = static_cast<const T*>(a.q) + bos * a.q_row + hk * DK;
  const T* k = static_cast<const T*>(a.k) + bos * a.k_row + hk * DK;
  const T* v = static_cast<const T*>(a.v) + bos * a.v_row + int64_t(h) * a.DV + v0;
  const T* dt = static_cast<const T*>(a.dt) + bos * a.dt_row + h;
  T* o = static_cast<T*>(a.o) + bos * a.o_row + int64_t(h) * a.DV + v0;
  const float rate = a.a[h], bias = a.bias != nullptr ? a.bias[h] : 0.0f, skip = a.d != nullptr ? a.d[h] : 0.0f;
  const int tid = threadIdx.x, lane = tid & 63, w = wave_id(), li = lane & 15, g = lane >> 4;
  const int sw = w - (8 - SW);  // >= 0: an S wave, tiles sw, sw + SW, ..

  f32x4 S[OWN];
  const float* s0 = a.s0 == nullptr || row < 0 ? nullptr : a.s0 + (row * H + h) * DK * a.DV;
  s0 = sp.start(MODE == kLocal, s0, a.seg_s, int64_t(DK) * a.DV);
#pragma unroll
  for (int i = 0; i < OWN; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = 16 * (sw + SW * i) + 4 * g + e;
      S[i][e] = sw >= 0 && s0 != nullptr && r < DK ? s0[int64_t(r) * a.DV + v0 + li] : 0.0f;
    }
  auto store = [&](float* dst) {
#pragma unroll
    for (int i = 0; i < OWN; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = 16 * (sw + SW * i) + 4 * g + e;
        if (r < DK) dst[int64_t(r) * a.DV + v0 + li] = S[i][e];
      }
  };
  if (MODE == kLocal && sw >= 0 && sp.before == 0) store(a.seg_s + sp.end * DK * a.DV);
  if (FWD && sw >= 0) {
    for (int64_t slot = sp.first + H; slot < sp.slot; slot += H) {  // the segments before, in order
      const float d = a.seg_e[slot];
      const float* src = a.seg_s + slot * DK * a.DV + v0 + li;
#pragma unroll
      for (int i = 0; i < OWN; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = 16 * (sw + SW * i) + 4 * g + e;
          if (r < DK) S[i][e] = fmaf(d, S[i][e], src[int64_t(r) * a.DV]);
        }
    }
  }
  float decay = 1.0f;  // of all chunks
  auto publish = [&]() {
#pragma unroll
    for (int i = 0; i < OWN; ++i)
      if (sw + SW * i < DT) st4(&St[li][16 * (sw + SW * i) + 4 * g], S[i]);
  };

  const int chunks = int((len + kC - 1) / kC);
  for (int at = tid; at < kC * KP; at += kChain) {  // columns past d_k
    Ks[0][at / KP][at % KP] = Ks[1][at / KP][at % KP] = 0.0f;
    if constexpr (FWD) Qs[0][at / KP][at % KP] = Qs[1][at / KP][at % KP] = 0.0f;
    if (at < kBV * KP) St[at / KP][at % KP] = 0.0f;
    if (at < kC * PP) Ps[at / PP][at % PP] = 0.0f;  // above the diagonal
  }
  Tile<T, DK, kChain> tk, tq;
  Tile<T, kBV, kChain> tv;
  float raw = 0.0f;
  auto chunk_at = [&](int n) { return MODE == kReverse ? chunks - 1 - n : n; };
  auto valid_of = [&](int n) {
    const int64_t t = int64_t(chunk_at(n)) * kC;
    return int(len - t < kC ? len - t : kC);
  };
  auto fetch = [&](int n) {
    const int64_t t = int64_t(chunk_at(n)) * kC;
    const int valid = valid_of(n);
    tk.fetch(k + t * a.k_row, a.k_row, valid, tid);
    if constexpr (FWD) tq.fetch(q + t * a.q_row, a.q_row, valid, tid);
    tv.fetch(v + t * a.v_row, a.v_row, valid, tid);
  };
  auto stage = [&](int b) {
    tk.put(Ks[b][0], KP, tid);
    if constexpr (FWD) tq.put(Qs[b][0], KP, tid);
    tv.put(Vs[b][0], VP, tid);
  };
  auto fetch_dt = [&](int n) {
    raw = n < chunks && lane < valid_of(n) ? to_f32(dt[(int64_t(chunk_at(n)) * kC + lane) * a.dt_row]) + bias : 0.0f;
  };
  if (chunks > 0) {
    fetch(0);
    __syncthreads();  // the zeros
    stage(0);
    if (chunks > 1) fetch(1);
    if (w == 3) {
      fetch_dt(0);
      put_chunk_gates(gates[0], raw, rate, lane < valid_of(0), lane);
      fetch_dt(1);
    }
    if (FWD && sw >= 0) publish();
    __syncthreads();
  }
  for (int n = 0; n < chunks; ++n) {
    const int b = n & 1;
    const int64_t t = int64_t(chunk_at(n)) * kC;
    const int valid = valid_of(n);
    const Gates& gt = gates[b];
    f32x4 x = zero4();  // of the Z waves: diag(e^G) S^T Q^T, 16 tokens
    if (FWD && w < 3) {  // P, lower triangle: tiles (0, 0), (1, 0), (1, 1)
      const int it = (w + 1) / 2, jt = w / 2, i = 16 * it + li;
      f32x4 p = zero4();
#pragma unroll
      for (int ku = 0; ku < KU; ++ku)
        mma(p, lds_frag(Ks[b][0], KP, 16 * jt + li, ku, g), lds_frag(Qs[b][0], KP, i, ku, g));
      const float hi = gt.hi[i], lo = gt.lo[i];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = 16 * jt + 4 * g + e;
        p[e] = i >= j ? p[e] * (gt.between(hi, lo, j) * gt.D[j]) : 0.0f;
      }
      st4(&Ps[i][16 * jt + 4 * g], p);
    } else if (w == 3) {
      put_chunk_gates(gates[b ^ 1], raw, rate, n + 1 < chunks && lane < valid_of(n + 1), lane);
      fetch_dt(n + 2);
    } else if (FWD && sw < 0) {  // wavefronts 4 and 5
      const int i = 16 * (w - 4) + li;
#pragma unroll
      for (int ku = 0; ku < KU; ++ku) mma(x, lds_frag(St[0], KP, li, ku, g), lds_frag(Qs[b][0], KP, i, ku, g));
      x = gt.e[i] * x;
    } else if (sw >= 0) {  // S <- e^{G_C} S + K^T diag(w) V
      if constexpr (MODE == kStates || MODE == kReverse) store(states + (int64_t(unit) * NC + chunk_at(n)) * DK * a.DV);
      Frag<float> wv = lds_frag_t(Vs[b][0], VP, li, 0, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) wv.v[e] *= (MODE == kReverse ? gt.e : gt.w)[16 * (e / 4) + 4 * g + e % 4];
      const float all = gt.e[kC - 1];
      decay *= all;
#pragma unroll
      for (int i = 0; i < OWN; ++i)
        if (sw + SW * i < DT) {
          f32x4 own = zero4();  // added once: eight steps onto S would round it eight times
          mma(own, lds_frag_t(Ks[b][0], KP, 16 * (sw + SW * i) + li, 0, g), wv);
#pragma unroll
          for (int e = 0; e < 4; ++e) S[i][e] = fmaf(all, S[i][e], own[e]);
        }
    }
    __syncthreads();
    if (n + 1 < chunks) {
      stage(b ^ 1);
      if (n + 2 < chunks) fetch(n + 2);
    }
    if constexpr (FWD) {
      if (w == 4 || w == 5) {
        const int i = 16 * (w - 4) + li;
        mma(x, lds_frag_t(Vs[b][0], VP, li, 0, g), lds_frag(Ps[0], PP, i, 0, g));
        if (a.d != nullptr) {
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = fmaf(skip, Vs[b][i][4 * g + e], x[e]);
        }
        if (i < valid) st4(o + (t + i) * a.o_row + 4 * g, x);
      }
      if (sw >= 0) publish();
    }
    __syncthreads();
  }
  if constexpr (MODE == kLocal) {
    if (sw >= 0) store(a.seg_s + sp.slot * DK * a.DV);
    if (v0 == 0 && sw == 0 && lane == 0) a.seg_e[sp.slot] = decay;
  } else {
    if (a.sfin != nullptr && row >= 0 && sw >= 0 && sp.last) store(a.sfin + (row * H + h) * DK * a.DV);
  }
}

// ---------------------------------------------------------------------------
// Gradients of one chunk of 32 tokens for one query and key head: its value
// heads one after the other, dQ and dK summed over them in registers, in order.
// The states S and X are read from memory as operand fragments.
template <typename T, int DK, int DV>
__global__ __launch_bounds__(kThreads) void ssm_bwd_f32_kernel(SsmBwd b, const float* __restrict__ states,
                                                               const float* __restrict__ dstates,
                                                               float* __restrict__ part, int NC) {
  constexpr int DKP = DK < 32 ? 32 : DK, DVP = DV < 32 ? 32 : DV, KP = DKP + 4, VP = DVP + 4, PP = kC + 4;
  constexpr int KU = DKP / 32, VU = DVP / 32, DT = DK / 16, VT = DV / 16;
  constexpr int KOWN = cdiv(2 * DT, 4), VOWN = cdiv(2 * VT, 4);  // tiles (token half, column tile) a wavefront
  __shared__ __align__(16) float Qs[kC][KP], Ks[kC][KP], Vs[kC][VP], Os[kC][VP];
  __shared__ __align__(16) float Pm[kC][PP], Dm[kC][PP];  // e^{G_i - G_j} times q_i . k_j and dO_i . v_j
  // rowM: of the diagonal tiles what tile_between has
  __shared__ __align__(16) float rowM[3][16];
  __shared__ float colM[3][16], rin[4][kC], pin[4][kC], red[3][4];
  __shared__ Gates gt;

  const int r = b.H / b.Hk;
  const uint32_t wg = blockIdx.x;
  const int n = int(wg % uint32_t(NC));
  const uint32_t bk = wg / uint32_t(NC);
  const int hk = int(bk % uint32_t(b.Hk));
  const int64_t bb = bk / uint32_t(b.Hk);
  const int tid = threadIdx.x, lane = tid & 63, w = wave_id(), li = lane & 15, g = lane >> 4;
  const int64_t t = int64_t(n) * kC, tok = bb * b.L + t;
  const int valid = int(b.L - t < kC ? b.L - t : kC);

  for (int at = tid; at < kC * (KP > VP ? KP : VP); at += kThreads) {
    if (at < kC * KP) Qs[at / KP][at % KP] = Ks[at / KP][at % KP] = 0.0f;
    if (at < kC * VP) Vs[at / VP][at % VP] = Os[at / VP][at % VP] = 0.0f;
    if (at < kC * PP) Pm[at / PP][at % PP] = Dm[at / PP][at % PP] = 0.0f;
  }
  __syncthreads();
  {
    Tile<T, DK> x;
    x.fetch(static_cast<const T*>(b.q) + tok * b.q_row + hk * DK, b.q_row, valid, tid);
    x.put(Qs[0], KP, tid);
    x.fetch(static_cast<const T*>(b.k) + tok * b.k_row + hk * DK, b.k_row, valid, tid);
    x.put(Ks[0], KP, tid);
  }
  __syncthreads();
  const int it = (w + 1) / 2, jt = w / 2;  // this wavefront's tile of the lower triangle (w < 3)
  f32x4 raw = zero4();                     // raw[i = 16 it + 4 g + e][j = 16 jt + li]
  if (w < 3)
#pragma unroll
    for (int ku = 0; ku < KU; ++ku)
      mma(raw, lds_frag(Qs[0], KP, 16 * it + li, ku, g), lds_frag(Ks[0], KP, 16 * jt + li, ku, g));
  f32x4 dQ[KOWN], dK[KOWN];
#pragma unroll
  for (int i = 0; i < KOWN; ++i) dQ[i] = dK[i] = zero4();

  for (int hh = 0; hh < r; ++hh) {
    const int h = hk * r + hh;
    const int64_t slot = (bb * b.H + h) * NC + n;
    const float* S = states + slot * DK * DV;
    const float* X = dstates + slot * DK * DV;
    const float rate = b.a[h], skip = b.d != nullptr ? b.d[h] : 0.0f;
    __syncthreads();  // the head before is done with the LDS
    float skips = 0.0f, dot = 0.0f;
    {
      Tile<T, DV> x, y;
      x.fetch(static_cast<const T*>(b.v) + tok * b.v_row + int64_t(h) * DV, b.v_row, valid, tid);
      y.fetch(static_cast<const T*>(b.d_o) + tok * b.do_row + int64_t(h) * DV, b.do_row, valid, tid);
      x.put(Vs[0], VP, tid);
      y.put(Os[0], VP, tid);
#pragma unroll
      for (int i = 0; i < Tile<T, DV>::PER; ++i)
#pragma unroll
        for (int e = 0; e < Tile<T, DV>::VE; ++e) skips = fmaf(to_f32(x.x[i].e[e]), to_f32(y.x[i].e[e]), skips);
    }
    for (int at = tid; at < DK * DV / 4; at += kThreads) {
      const f32x4 x = reinterpret_cast<const f32x4*>(X)[at], s = reinterpret_cast<const f32x4*>(S)[at];
#pragma unroll
      for (int e = 0; e < 4; ++e) dot = fmaf(x[e], s[e], dot);
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
      skips += __shfl_xor(skips, off);
      dot += __shfl_xor(dot, off);
    }
    if (lane == 0) {
      red[0][w] = skips;
      red[1][w] = dot;
    }
    if (w == 3)
      put_chunk_gates(gt, lane < valid ? to_f32(static_cast<const T*>(b.dt)[(tok + lane) * b.dt_row + h]) +
                                             (b.bias != nullptr ? b.bias[h] : 0.0f)
                                       : 0.0f,
                      rate, lane < valid, lane);
    __syncthreads();
    if (w < 3) {
      f32x4 p = zero4();
#pragma unroll
      for (int ku = 0; ku < VU; ++ku)
        mma(p, lds_frag(Os[0], VP, 16 * it + li, ku, g), lds_frag(Vs[0], VP, 16 * jt + li, ku, g));
      const int j = 16 * jt + li;
      float col = 0.0f;
      f32x4 md;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = 16 * it + 4 * g + e;
        const float f = i >= j ? gt.between(gt.hi[i], gt.lo[i], j) : 0.0f;
        p[e] = i >= j ? p[e] * f : 0.0f;
        Pm[i][j] = i >= j ? raw[e] * f : 0.0f;
        Dm[i][j] = p[e];
        const float m = i >= j ? p[e] * raw[e] : 0.0f;
        col += m;
        md[e] = m * gt.D[j];
      }
      if (it == jt) {
        md = tile_between_tr(md, li, g);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) md[e] = row_sum16(md[e]);
      }
      if (li == 0) st4(&rowM[w][4 * g], md);
      col = row_sum4(col);
      if (g == 0) colM[w][li] = col;
    }
    __syncthreads();
    const float end_hi = gt.hi[kC - 1], end_lo = gt.lo[kC - 1];
    auto del = [&](int ku, Frag<float>& f) {  // times D of the k index
#pragma unroll
      for (int e = 0; e < 8; ++e) f.v[e] *= gt.D[32 * ku + 16 * (e / 4) + 4 * g + e % 4];
    };
    auto state_rows = [&](const float* M, int dk, int ku) {  // operand row dk, k index over d_v
      Frag<float> f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = 32 * ku + 16 * (e / 4) + 4 * g + e % 4;
        f.v[e] = c < DV ? M[int64_t(dk) * DV + c] : 0.0f;
      }
      return f;
    };
    auto state_cols = [&](const float* M, int dv, int ku) {  // operand row dv, k index over d_k
      Frag<float> f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = 32 * ku + 16 * (e / 4) + 4 * g + e % 4;
        f.v[e] = c < DK ? M[int64_t(c) * DV + dv] : 0.0f;
      }
      return f;
    };
    float rsum[2][4] = {}, psum[2][4] = {};
#pragma unroll
    for (int i = 0; i < KOWN; ++i) {  // dQ and dK: tile (half, dt)
      const int at = w + 4 * i, half = at & 1, dt = at >> 1;
      if (at < 2 * DT) {
        f32x4 x = zero4(), y = zero4();
#pragma unroll
        for (int ku = 0; ku < VU; ++ku) {
          mma(x, lds_frag(Os[0], VP, 16 * half + li, ku, g), state_rows(S, 16 * dt + li, ku));
          mma(y, lds_frag(Vs[0], VP, 16 * half + li, ku, g), state_rows(X, 16 * dt + li, ku));
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int tk = 16 * half + 4 * g + e, c = 16 * dt + li;
          x[e] *= gt.e[tk];
          y[e] *= gt.between(end_hi, end_lo, tk);
          rsum[half][e] += x[e] * Qs[tk][c];
          psum[half][e] += y[e] * Ks[tk][c];
        }
        Frag<float> d = lds_frag(Dm[0], PP, 16 * half + li, 0, g);
        del(0, d);
        mma(dQ[i], d, lds_frag_t(Ks[0], KP, 16 * dt + li, 0, g));
        mma(y, lds_frag_t(Dm[0], PP, 16 * half + li, 0, g), lds_frag_t(Qs[0], KP, 16 * dt + li, 0, g));
        dQ[i] += x;
#pragma unroll
        for (int e = 0; e < 4; ++e) dK[i][e] = fmaf(gt.D[16 * half + 4 * g + e], y[e], dK[i][e]);
      }
    }
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = row_sum16(rsum[half][e]), y = row_sum16(psum[half][e]);
        if (li == 0) {
          rin[w][16 * half + 4 * g + e] = x;
          pin[w][16 * half + 4 * g + e] = y;
        }
      }
    T* dv = static_cast<T*>(b.dv) + tok * b.dv_row + int64_t(h) * DV;
#pragma unroll
    for (int i = 0; i < VOWN; ++i) {  // dV: tile (half, vt)
      const int at = w + 4 * i, half = at & 1, vt = at >> 1;
      if (at < 2 * VT) {
        f32x4 x = zero4();
#pragma unroll
        for (int ku = 0; ku < KU; ++ku)
          mma(x, lds_frag(Ks[0], KP, 16 * half + li, ku, g), state_cols(X, 16 * vt + li, ku));
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] *= gt.between(end_hi, end_lo, 16 * half + 4 * g + e);
        mma(x, lds_frag_t(Pm[0], PP, 16 * half + li, 0, g), lds_frag_t(Os[0], VP, 16 * vt + li, 0, g));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = 16 * half + 4 * g + e;
          if (j < valid)
            dv[j * b.dv_row + 16 * vt + li] = from_f32<T>(fmaf(skip, Os[j][16 * vt + li], gt.D[j] * x[e]));
        }
      }
    }
    __syncthreads();
    if (w == 0) {
      const bool real = lane < valid;
      const int l = lane < kC ? lane : kC - 1, half = l >> 4, i = l & 15;
      // tiles: 0 (0, 0), 1 (1, 0), 2 (1, 1)
      const float ci = !real ? 0.0f : half ? colM[2][i] : colM[0][i] + colM[1][i];
      float rr = rin[0][l] + rin[1][l] + rin[2][l] + rin[3][l], pp = pin[0][l] + pin[1][l] + pin[2][l] + pin[3][l];
      if (!real) rr = pp = 0.0f;
      const float D = gt.D[l];
      const float left = row_suffix16(rowM[1][i], i), below = row_before16(D * colM[1][i], i);
      const float own = half ? rowM[2][i] + left : rowM[0][i] + below;
      float suf = rr, pre = D * pp;  // to be summed over i >= t, and over j < t
#pragma unroll
      for (int d = 1; d < kC; d <<= 1) {
        const float y = __shfl_down(suf, d), z = __shfl_up(pre, d);
        if (lane + d < kC) suf += y;
        if (lane >= d) pre += z;
      }
      const float xs = gt.e[kC - 1] * (red[1][0] + red[1][1] + red[1][2] + red[1][3]);
      const float before = __shfl_up(pre, 1);  // not pre less its own term, which may be far larger than the others
      const float gd = own + (suf + (lane > 0 ? before : 0.0f) + xs);
      const float dD = ci + pp + rate * gd;
      float raw_dt = b.bias != nullptr ? b.bias[h] : 0.0f;
      if (real) raw_dt += to_f32(static_cast<const T*>(b.dt)[(tok + lane) * b.dt_row + h]);
      const float ddt = dD * (1.0f / (1.0f + expf(-raw_dt)));
      if (real) static_cast<T*>(b.ddt)[(tok + lane) * b.ddt_row + h] = from_f32<T>(ddt);
      float sa = real ? D * gd : 0.0f, sb = real ? ddt : 0.0f;
#pragma unroll
      for (int off = 32; off > 0; off >>= 1) {
        sa += __shfl_xor(sa, off);
        sb += __shfl_xor(sb, off);
      }
      if (lane == 0) {
        const int64_t M = int64_t(b.B) * NC, at = int64_t(h) * M + bb * NC + n, all = int64_t(b.H) * M;
        part[at] = sa;
        part[all + at] = sb;
        part[2 * all + at] = red[0][0] + red[0][1] + red[0][2] + red[0][3];
      }
    }
  }
  T* dq = static_cast<T*>(b.dq) + tok * b.dq_row + hk * DK;
  T* dk = static_cast<T*>(b.dk) + tok * b.dk_row + hk * DK;
#pragma unroll
  for (int i = 0; i < KOWN; ++i) {
    const int at = w + 4 * i, half = at & 1, dt = at >> 1;
    if (at < 2 * DT)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int tk = 16 * half + 4 * g + e;
        if (tk < valid) {
          dq[tk * b.dq_row + 16 * dt + li] = from_f32<T>(dQ[i][e]);
          dk[tk * b.dk_row + 16 * dt + li] = from_f32<T>(dK[i][e]);
        }
      }
  }
}

// da, dbias and dd of a head from the M partial sums of its chunks, in a fixed order.
__global__ __launch_bounds__(kThreads) void ssm_sum_kernel(const float* __restrict__ part, float* __restrict__ da,
                                                           float* __restrict__ dbias, float* __restrict__ dd, int64_t M,
                                                           int H) {
  __shared__ float red[4];
  const int which = int(blockIdx.x) / H, h = int(blockIdx.x) % H, lane = threadIdx.x & 63;
  float* out = which == 0 ? da : which == 1 ? dbias : dd;
  if (out == nullptr) return;
  const float* src = part + (int64_t(which) * H + h) * M;
  float s = 0.0f;
  for (int64_t i = threadIdx.x; i < M; i += kThreads) s += src[i];
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) s += __shfl_xor(s, off);
  if (lane == 0) red[wave_id()] = s;
  __syncthreads();
  if (threadIdx.x == 0) out[h] = red[0] + red[1] + red[2] + red[3];
}

template <typename F>
hipError_t by_dim(int d, F&& f) {
  switch (d) {
    case 16: return f(std::integral_constant<int, 16>{});
    case 32: return f(std::integral_constant<int, 32>{});
    case 64: return f(std::integral_constant<int, 64>{});
    case 128: return f(std::integral_constant<int, 128>{});
  }
  return hipErrorInvalidValue;
}

template <typename T, int MODE>
hipError_t launch_chain(const SsmFwd& a, float* states, int NC, hipStream_t s) {
  const int64_t wgs = (a.seg > 0 ? a.seg_slots : a.N) * a.H * (a.DV / kBV);
  return by_dim(a.DK, [&](auto dk) {
    hipLaunchKernelGGL((ssm_f32_kernel<T, decltype(dk)::value, MODE>), dim3(unsigned(wgs)), dim3(kChain), 0, s, a,
                       states, NC);
    return hipGetLastError();
  });
}

}  // namespace

int64_t ssm_f32_threads(int64_t seqs, int H, int DV) { return seqs * H * (DV / kBV) * kChain; }

template <typename T>
hipError_t launch_ssm_f32(const SsmFwd& a, bool local, hipStream_t s) {
  return local ? launch_chain<T, kLocal>(a, nullptr, 0, s) : launch_chain<T, kFwd>(a, nullptr, 0, s);
}
template hipError_t launch_ssm_f32<float>(const SsmFwd&, bool, hipStream_t);
template hipError_t launch_ssm_f32<uint16_t>(const SsmFwd&, bool, hipStream_t);

hipError_t launch_ssm_sums(const float* part, float* da, float* dbias, float* dd, int64_t M, int H, hipStream_t s) {
  hipLaunchKernelGGL(ssm_sum_kernel, dim3(unsigned(3 * H)), dim3(kThreads), 0, s, part, da, dbias, dd, M, H);
  return hipGetLastError();
}

int64_t ssm_bwd_f32_threads(int B, int H, int64_t L, int DV) {
  const int64_t chains = ssm_f32_threads(B, H, DV), grads = int64_t(B) * H * ((L + kC - 1) / kC) * kThreads;
  return chains > grads ? chains : grads;
}

// Workspace: the chunks' states, their gradients, and the partial sums of da,
// dbias and dd.
size_t ssm_bwd_f32_workspace(int B, int H, int64_t L, int DK, int DV) {
  const size_t slots = size_t(B) * H * size_t((L + kC - 1) / kC);
  return slots * (2 * size_t(DK) * DV + 3) * sizeof(float);
}

template <typename T>
hipError_t launch_ssm_bwd_f32(const SsmBwd& b, void* ws, hipStream_t s) {
  const int NC = int((b.L + kC - 1) / kC);
  const size_t slots = size_t(b.B) * b.H * NC, state = size_t(b.DK) * b.DV;
  float* states = static_cast<float*>(ws);
  float* dstates = states + slots * state;
  float* part = dstates + slots * state;
  hipError_t e = hipSuccess;
  if (b.L > 0) {
    const SsmFwd f{b.q,     b.k,     b.v,     b.dt,     b.a,     nullptr, b.bias, b.s0, nullptr, nullptr, nullptr, nullptr,
                   nullptr, b.q_row, b.k_row, b.v_row, b.dt_row, 0,       b.B,    b.B,  b.H,     b.Hk,    b.DK,    b.DV,
                   b.L};
    e = launch_chain<T, kStates>(f, states, NC, s);
    if (e != hipSuccess) return e;
  }
  // the chain of state gradients reads q for k and dO for v; a sequence without tokens copies
  const SsmFwd x{nullptr, b.q,     b.d_o,   b.dt,     b.a,     nullptr, b.bias, b.dsf, nullptr, b.ds0, nullptr, nullptr,
                 nullptr, 0,       b.q_row, b.do_row, b.dt_row, 0,      b.B,    b.B,   b.H,     b.Hk,  b.DK,    b.DV,
                 b.L};
  e = launch_chain<T, kReverse>(x, dstates, NC, s);
  if (e != hipSuccess) return e;
  if (b.L > 0) {
    e = by_dim(b.DK, [&](auto dk) {
      return by_dim(b.DV, [&](auto dv) {
        hipLaunchKernelGGL((ssm_bwd_f32_kernel<T, decltype(dk)::value, decltype(dv)::value>),
                           dim3(unsigned(int64_t(b.B) * b.Hk * NC)), dim3(kThreads), 0, s, b, states, dstates, part, NC);
        return hipGetLastError();
      });
    });
    if (e != hipSuccess) return e;
  }
  return launch_ssm_sums(part, b.da, b.dbias, b.dd, int64_t(b.B) * NC, b.H, s);
}
template hipError_t launch_ssm_bwd_f32<float>(const SsmBwd&, void*, hipStream_t);
template hipError_t launch_ssm_bwd_f32<uint16_t>(const SsmBwd&, void*, hipStream_t);

}  // namespace efla
