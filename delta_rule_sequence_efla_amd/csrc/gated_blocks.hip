// gated_blocks.hip -- whole sequences of the gated delta rule in fp32, 16 tokens
// at a time on fp32 matrix cores (gated.h's chunk algebra with chunks of 16).
//
// One workgroup per sequence, head and 16 value columns.  What one block of 16
// tokens hands to the next is S alone, so everything else is done ahead or
// behind by wavefronts of their own, and the chain per block is
//     K S (summed over the key dims of four wavefronts through the LDS)
//     -> D = a (V - e K S) -> U = X D -> S <- e^{G_C} S + K^T (w U).
//   waves 0-3  S: a quarter of the key dims each, S in accumulator registers;
//              K S of the next block, D and U (all four, from the summed parts),
//              the update; also their parts of Q S
//   waves 4-7  load q, k, v six or seven blocks ahead into registers and widen
//              them into the LDS three blocks ahead
//   waves 8, 9    A = tril(a Gam K K^T) and X = (I + A)^{-1} by turns, a block in
//   waves 10, 11  two periods; P = Gam tril(Q K^T) likewise
//   wave 12    O = e Q S + P U, a block behind
// One barrier a block, where the parts of K S are exchanged; every other buffer
// is written a period or more before it is read, so it rides on that barrier.
// Products use the accumulator layout on both sides: of the 16x16x4 products that
// sum over 16 values, step r takes values 4 g + r, so rows 4 g .. 4 g + 3 of an
// accumulator are an operand as they stand.
// 2 x 777 tokens of 8 heads, d 64: 49 us, 0.95 us a block (token pairs,
// gated_step.hip: 83 us).  Bound by issue and latency about evenly: the chain, X's
// two halves, P's first and O each take 2000 to 2400 cycles of a block's 2450,
// thirteen wavefronts on four SIMDs.  X by all 16 rows of substitution and the
// gates' factors in the same wavefront: 81 us; factors moved to P's: 65 to 53.
#include "gated.h"
#include "launchers.h"
#include "lds_ring.h"
#include "ut_wave.h"

namespace efla {

namespace {
template <typename T, int N> struct alignas(N * sizeof(T) < 16 ? N * sizeof(T) : 16) Row { T e[N]; };
}  // namespace

// With `states`, the state before every C-th token is stored, [chunk
// slot][d_k][d_v] fp32 (dense batches; C % 16 == 0).
template <typename T, int DK>
__global__ __launch_bounds__(kGatedBlocksThreads) void gated_blocks_kernel(GatedFwd a, float* __restrict__ states, int C, int NC) {
  constexpr int TB = 16, NK = DK / 16, NT = DK / 64, KP = DK + 4;  // tokens a block, ...; key tiles a wave; row pitch
  constexpr int RING = 4;                                          // blocks of q, k, v, gates and P in the LDS
  __shared__ __align__(16) float kS[RING][TB * KP], qS[RING][TB * KP];
  __shared__ __align__(16) f32x4 vS[RING][kWave], pS[RING][kWave];  // lane (li, g): V[4 g ..][li], P[li][4 g ..]
  __shared__ __align__(16) float gS[RING][4][TB];                   // a, e, w; e^{G_C} in all of the last row
  __shared__ __align__(16) float aS[2][TB * 20], xdS[2][TB * 20];   // A and the diagonal blocks of X, by parity
  __shared__ __align__(16) f32x4 gamS[2][kWave];                    // Gam[li][4 g ..], j <= i
  __shared__ float bS[RING][2][TB];                                 // beta and gates as given
  __shared__ __align__(16) f32x4 xS[2][kWave];                      // X[li][4 g ..]
  __shared__ __align__(16) f32x4 ksS[2][4][kWave], qsS[2][4][kWave], uS[2][kWave];

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
  const int role = wave_id(), lane = threadIdx.x & 63, li = lane & 15, g = lane >> 4;
  const int nb = int((len + TB - 1) / TB);
  // Three or four wavefronts share a SIMD; the longest path issues first: X, then
  // S, then P and O, the loads last (all alike: 52.8 us for 49.0).
  if (role == 8 || role == 9) __builtin_amdgcn_s_setprio(3);
  else if (role < 4) __builtin_amdgcn_s_setprio(2);
  else if (role >= 10) __builtin_amdgcn_s_setprio(1);
  auto sync = [&]() {
    wait_lgkm0();
    barrier_nowait();
  };
  // period p lies between barriers p and p + 1, periods -3 .. nb
  auto periods = [&](auto&& work) {
    if (nb == 0) return;
    for (int p = -3; p <= nb; ++p) {
      work(p);
      if (p < nb) sync();
    }
  };

  if (role < 4) {
    // ----------------------------------------------------------------- S
    // St[t][r] = S[kb + 16 t + 4 g + r][v0 + li]
    const int kb = 16 * NT * role;
    f32x4 St[NT];
    const float* s0 = a.s0 == nullptr || row < 0 ? nullptr : a.s0 + (row * H + h) * DK * DV + v0 + li;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) St[t][r] = s0 == nullptr ? 0.0f : s0[int64_t(kb + 16 * t + 4 * g + r) * DV];
    auto part = [&](const float* X) {  // this wave's part of X S, X rows of K or Q
      f32x4 acc = zero4();
#pragma unroll
      for (int t = 0; t < NT; ++t)
        mma16_f32(acc, *reinterpret_cast<const f32x4*>(X + li * KP + kb + 16 * t + 4 * g), St[t]);
      return acc;
    };
    auto store = [&](float* dst) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) dst[int64_t(kb + 16 * t + 4 * g + r) * DV] = St[t][r];
    };
    const uint32_t per = uint32_t(C) / TB;
    periods([&](int p) {
      if (p >= 0 && p < nb) {
        if (states != nullptr && uint32_t(p) % per == 0)
          store(states + (int64_t(unit) * NC + uint32_t(p) / per) * DK * DV + v0 + li);
        const int s = p & (RING - 1), b = p & 1;
        f32x4 ks[4];
#pragma unroll
        for (int w = 0; w < 4; ++w) ks[w] = ksS[b][w][lane];
        const f32x4 av = *reinterpret_cast<const f32x4*>(&gS[s][0][4 * g]), ev = *reinterpret_cast<const f32x4*>(&gS[s][1][4 * g]);
        const f32x4 wv = *reinterpret_cast<const f32x4*>(&gS[s][2][4 * g]);
        const float end = gS[s][3][li];
        const f32x4 x = xS[b][lane], v = vS[s][lane];
        f32x4 kt[NT];  // K[4 g + r][kb + 16 t + li]
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r) kt[t][r] = kS[s][(4 * g + r) * KP + kb + 16 * t + li];
        qsS[b][role][lane] = part(qS[s]);
        const f32x4 sum = (ks[0] + ks[1]) + (ks[2] + ks[3]);
        f32x4 d, u = zero4();
#pragma unroll
        for (int r = 0; r < 4; ++r) d[r] = av[r] * fmaf(-ev[r], sum[r], v[r]);
        mma16_f32(u, x, d);
        if (role == 0) uS[b][lane] = u;
        u *= wv;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          St[t] *= end;
          mma16_f32(St[t], kt[t], u);
        }
      }
      if (p >= -1 && p + 1 < nb) ksS[(p + 1) & 1][role][lane] = part(kS[(p + 1) & (RING - 1)]);
    });
    if (a.sfin != nullptr && row >= 0) store(a.sfin + (row * H + h) * DK * DV + v0 + li);
  } else if (role < 8) {
    // -------------------------------------------------------------- loads
    const int tid = threadIdx.x - 4 * kWave, tok = tid >> 4, pc = tid & 15;
    const T* q = static_cast<const T*>(a.q) + (bos * a.Hk + hk) * DK + pc * NK;
    const T* k = static_cast<const T*>(a.k) + (bos * a.Hk + hk) * DK + pc * NK;
    const T* v = static_cast<const T*>(a.v) + (bos * H + h) * DV + v0 + pc;
    const T* beta = static_cast<const T*>(a.beta) + bos * H + h;
    const float* gate = a.g + bos * H + h;
    // register sets of blocks on the way (at d_k 128 in fp32 a fourth would spill)
    constexpr int NR = DK == 128 && sizeof(T) == 4 ? 3 : 4;
    struct Regs {
      Row<T, NK> k, q;
      T v, b;
      float g;
    } R[NR];
    // Loads and stores to the LDS run whether the block exists or not, tokens past
    // the end reading the last one: behind a branch the compiler could not count
    // the loads in flight and would wait for all of them in every period.
    const int64_t k_stride = int64_t(a.Hk) * DK, k_block = TB * k_stride, h_block = int64_t(TB) * H;
    auto load = [&](Regs& x, int m) {
      const int left = int(len - int64_t(m) * TB) - 1;  // the block's last token
      const int t = tok < left ? tok : left;            // may lie before the block
      const int64_t kt = m * k_block + t * k_stride, ht = m * h_block + int64_t(t) * H;
      x.k = *reinterpret_cast<const Row<T, NK>*>(k + kt);
      x.q = *reinterpret_cast<const Row<T, NK>*>(q + kt);
      x.v = v[ht * DV];
      x.b = beta[ht];
      x.g = gate[ht];
    };
    auto stage = [&](const Regs& x, int m) {  // tokens past the end: zeros, which change nothing
      const int s = m & (RING - 1);
      const bool in = int64_t(m) * TB + tok < len;
#pragma unroll
      for (int e = 0; e < NK; e += 4) {
        f32x4 kk, qq;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          kk[r] = in ? to_f32(x.k.e[e + r]) : 0.0f;
          qq[r] = in ? to_f32(x.q.e[e + r]) : 0.0f;
        }
        *reinterpret_cast<f32x4*>(&kS[s][tok * KP + pc * NK + e]) = kk;
        *reinterpret_cast<f32x4*>(&qS[s][tok * KP + pc * NK + e]) = qq;
      }
      reinterpret_cast<float*>(&vS[s][(tok >> 2) * 16 + pc])[tok & 3] = in ? to_f32(x.v) : 0.0f;
      if (pc == 0) {
        bS[s][0][tok] = in ? to_f32(x.b) : 0.0f;
        bS[s][1][tok] = in ? gate_floor(x.g) : 0.0f;
      }
    };
    if (nb == 0) return;
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      load(R[i], i);
      __builtin_amdgcn_sched_barrier(0);  // in this order: the waits count on it
    }
    auto period = [&](Regs& x, int p) {
      stage(x, p + 3);
      load(x, p + 3 + NR);
      if (p < nb) sync();
    };
    for (int p = -3;;) {
      bool more = true;
#pragma unroll
      for (int i = 0; i < NR; ++i)
        if (more) {
          period(R[i], p);
          more = ++p <= nb;
        }
      if (!more) break;
    }
  } else if (role < 12) {
    // ------------------------------------------------------------ X and P
    auto gate_sums = [&](int s) {  // G of token li
      double G = double(bS[s][1][li]);
      auto add = [&](auto ctrl) {  // lanes without a source add zero
        const uint64_t x = __builtin_bit_cast(uint64_t, G);
        const uint32_t lo = __builtin_amdgcn_update_dpp(0, int(uint32_t(x)), decltype(ctrl)::value, 0xF, 0xF, false);
        const uint32_t hi = __builtin_amdgcn_update_dpp(0, int(uint32_t(x >> 32)), decltype(ctrl)::value, 0xF, 0xF, false);
        G += __builtin_bit_cast(double, uint64_t(hi) << 32 | lo);
      };
      add(std::integral_constant<int, 0x111>{});  // row_shr:1, 2, 4, 8
      add(std::integral_constant<int, 0x112>{});
      add(std::integral_constant<int, 0x114>{});
      add(std::integral_constant<int, 0x118>{});
      return G;
    };
    auto gram = [&](const float* A, const float* B) {  // rows of A times rows of B
      f32x4 acc = zero4();
#pragma unroll
      for (int t = 0; t < NK; ++t)
        mma16_f32(acc, *reinterpret_cast<const f32x4*>(A + li * KP + 16 * t + 4 * g),
                  *reinterpret_cast<const f32x4*>(B + li * KP + 16 * t + 4 * g));
      return acc;
    };
    const int odd = role & 1;
    // What the halves hand on in registers: K_{4 g + r} . K_li (of a P wave: . Q_li),
    // and a of token li (Gam[li][4 g + r] for j <= i, else 0)
    f32x4 gr = zero4(), gam = zero4();
    float al = 0.0f;
    // e^x of a difference of gate sums: its base-2 logarithm in 64 bits, then v_exp_f32
    auto decay = [](double x) { return __builtin_amdgcn_exp2f(float(x * 1.4426950408889634)); };
    // block m by the waves of its parity: first half in period m - 2, second in m - 1
    auto first = [&](int m) {
      const int s = m & (RING - 1);
      if (role >= 10) {
        gr = gram(kS[s], qS[s]);
        const double G = gate_sums(s), last = __shfl(G, 15);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const double Gj = __shfl(G, 4 * g + r);
          gam[r] = 4 * g + r <= li ? decay(G - Gj) : 0.0f;
        }
        gamS[m & 1][lane] = gam;
        if (g == 0) {
          gS[s][1][li] = decay(G);
          gS[s][2][li] = decay(last - G);
          gS[s][3][li] = decay(last);
        }
        return;
      }
      gr = gram(kS[s], kS[s]);
      const float mine = li & 2 ? (li & 1 ? gr[3] : gr[2]) : (li & 1 ? gr[1] : gr[0]);
      const float lam = __shfl(mine, (li >> 2) * 16 + li);
      al = efla_alpha_rule(bS[s][0][li], lam, a.rule);
      if (g == 0) gS[s][0][li] = al;
    };
    auto second = [&](int m) {
      if (role >= 10) {
        pS[m & (RING - 1)][lane] = gam * gr;
      } else {
        // A[li][4 g + r] = a_li Gam K_li . K_{4 g + r}, strictly lower
        gam = gamS[m & 1][lane];
        f32x4 below;
#pragma unroll
        for (int r = 0; r < 4; ++r) below[r] = 4 * g + r < li ? al * gam[r] * gr[r] : 0.0f;
        *reinterpret_cast<f32x4*>(&aS[odd][li * 20 + 4 * g]) = below;
        wave_lds_order();
        // The two diagonal 8x8 blocks of X by forward substitution, a column to
        // each lane of 16 (the four groups alike), then the block below them as
        // -X_2 A_21 X_1 by two products (all 16 rows by substitution took as long
        // again).  The rows are read before the first is used.
        float* Al = aS[odd];
        float* Xd = xdS[odd];
        const int hb = li & 8;
        f32x4 ar[8][2];
#pragma unroll
        for (int r = 1; r < 8; ++r) {
          ar[r][0] = *reinterpret_cast<const f32x4*>(Al + (hb + r) * 20 + hb);
          if (r > 4) ar[r][1] = *reinterpret_cast<const f32x4*>(Al + (hb + r) * 20 + hb + 4);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) below[r] = li >= 8 && g < 2 ? below[r] : 0.0f;
        float x[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          float s0 = r == (li & 7) ? 1.0f : 0.0f, s1 = 0.0f;
#pragma unroll
          for (int m = 0; m < r; ++m) {
            if (m & 1) s1 = fmaf(-ar[r][m >> 2][m & 3], x[m], s1);
            else s0 = fmaf(-ar[r][m >> 2][m & 3], x[m], s0);
          }
          x[r] = s0 + s1;
        }
#pragma unroll
        for (int r = 0; r < 8; ++r)
          if ((r >> 1) == g) Xd[(hb + r) * 20 + li] = x[r];
        wave_lds_order();
        const f32x4 rows = *reinterpret_cast<const f32x4*>(Xd + li * 20 + 4 * g);
        f32x4 cols, R = zero4(), W = zero4();
#pragma unroll
        for (int r = 0; r < 4; ++r) cols[r] = Xd[(4 * g + r) * 20 + li];
        mma16_f32(R, below, cols);  // A_21 X_1
        mma16_f32(W, R, rows);      // (X_d R)^T: W[r] = (X_d R)[li][4 g + r]
        xS[m & 1][lane] = rows - W;
      }
    };
    if (role < 10)  // what the diagonal blocks leave stays zero
      for (int i = lane; i < TB * 20; i += kWave) xdS[odd][i] = 0.0f;
    periods([&](int p) {
      if (p + 2 >= 0 && p + 2 < nb && ((p + 2) & 1) == odd) first(p + 2);
      if (p + 1 >= 0 && p + 1 < nb && ((p + 1) & 1) == odd) second(p + 1);
    });
  } else {
    // ----------------------------------------------------------------- O
    T* o = a.o == nullptr ? nullptr : static_cast<T*>(a.o) + (bos * H + h) * DV + v0 + li;
    periods([&](int p) {
      const int m = p - 1;
      if (m < 0 || o == nullptr) return;
      const int s = m & (RING - 1), b = m & 1;
      const f32x4 ev = *reinterpret_cast<const f32x4*>(&gS[s][1][4 * g]);
      f32x4 acc = ev * ((qsS[b][0][lane] + qsS[b][1][lane]) + (qsS[b][2][lane] + qsS[b][3][lane]));
      mma16_f32(acc, pS[s][lane], uS[b][lane]);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int64_t t = int64_t(m) * TB + 4 * g + r;
        if (t < len) o[t * H * DV] = from_f32<T>(acc[r]);
      }
    });
  }
}

template <typename T>
hipError_t launch_gated_blocks(const GatedFwd& a, float* states, int C, hipStream_t s) {
  const int64_t nwg = int64_t(a.cu == nullptr ? a.B : a.N) * a.H * (a.DV / 16);
  if (nwg == 0) return hipSuccess;
  const int NC = int((a.L + C - 1) / C);
  const dim3 grid{unsigned(nwg)}, wg{kGatedBlocksThreads};
  if (a.DK == 64) hipLaunchKernelGGL((gated_blocks_kernel<T, 64>), grid, wg, 0, s, a, states, C, NC);
  else hipLaunchKernelGGL((gated_blocks_kernel<T, 128>), grid, wg, 0, s, a, states, C, NC);
  return hipGetLastError();
}
template hipError_t launch_gated_blocks<float>(const GatedFwd&, float*, int, hipStream_t);
template hipError_t launch_gated_blocks<uint16_t>(const GatedFwd&, float*, int, hipStream_t);

}  // namespace efla
