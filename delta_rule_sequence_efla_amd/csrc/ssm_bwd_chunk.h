// ssm_bwd_chunk.h -- the backward pass of the selective state space scan (ssm.h)
// for bf16 inputs on the matrix cores: the chains of states and of their
// gradients, and the gradients chunk by chunk, 64 tokens each.
//
// Precision.  dq, dk and dv are rounded to bf16, and the operands that lead to
// them alone (P, dP and the gradient of the state where it meets a key) once.  The gradients
// of the decays are sums of products r, p and M (ssm.h) over all tokens, which
// end in float32: M comes from exact products in float32, and in r and p the
// states go in as three bf16 parts (24 bits); so do the float32 operands that feed
// a state.
#pragma once

#include <type_traits>

#include "ssm_chunk.h"

namespace efla {

// What is kept of every (sequence, head, chunk): its gates, formed by a launch of
// their own (a wavefront a chunk: formed along the chains, they were half of the
// chains' time), the state S before it and the gradient X of the state behind it.
// The arrays are cut into k-units of 32, [slot][d_v / 32][d_k][32], so that what one
// workgroup of the chains writes of a chunk is one piece of memory, and so is the
// operand fragment that a wavefront of the gradients reads.  (Rows of d_v values, of
// which four workgroups on four dies write a part each: 188 us instead of 151 for
// the chains of 8 x 2048 tokens, 8 heads, d 128.)  Both are float32, and three bf16 parts
// where they become operands of sums that da and dbias are formed from: of 2 x 2048
// tokens these are off by 1.2e-7 and 3.2e-7, with two parts by 2.6e-7 and 6.8e-7 (8 x 2048
// tokens, whole pass 268 us, 262).
struct SsmStates {
  float *s, *x;
  ChunkGates* gates;
  struct ChunkSums* sums;
};

// What the gradients of a chunk's steps are formed from (ssm_steps_kernel), each
// written by the wavefront that has it: row sums of M (of a diagonal tile the sums
// of tile_between) and its column sums by D, a tile each; r and p / D by 16 key dims;
// <X, S> and v . dO by wavefront.
struct ChunkSums {
  float row[10][16], col[10][16], r[8][64], p[8][64], xs[16], vo[16];
};

// The gates of every chunk, a wavefront each; slot (b H + h) NC + n.
__global__ __launch_bounds__(kThreads) void ssm_gates_kernel(SsmBwd b, ChunkGates* __restrict__ gates, int NC, int64_t slots) {
  const int64_t slot = int64_t(blockIdx.x) * 4 + wave_id();
  if (slot >= slots) return;
  const int lane = threadIdx.x & 63, n = int(slot % NC), h = int(slot / NC % b.H);
  const int64_t t = int64_t(n) * 64 + lane;
  const bool real = t < b.L;
  float raw = b.bias != nullptr ? b.bias[h] : 0.0f;
  if (real) raw += to_f32(static_cast<const uint16_t*>(b.dt)[(slot / NC / b.H * b.L + t) * b.dt_row + h]);
  put_chunk_gates(gates[slot], raw, b.a[h], real, lane);
}

// The matrix cores round sums of bf16 products down, not to nearest (of the elements of
// X half an ulp on average, of either sign): a bias that sums over tokens collect where
// the other factor keeps its sign, as keys and values behind a SiLU do.  Products that lead
// to da and dbias have every second row of their first operand negated, so that the
// bias goes both ways; a lane's operand row is li, the rows of its results are
// 4 g .. 4 g + 3.  da of 2 x 2048 tokens was off by up to 99 half steps of its terms' root of
// squares, growing with the length, and is by 7; the pass takes the same time.
__device__ __forceinline__ constexpr float row_sign(int row) { return row & 1 ? -1.0f : 1.0f; }
__device__ __forceinline__ Frag<uint16_t> row_signed(const Frag<uint16_t>& x, int li) {
  const uint32_t flip = li & 1 ? 0x80008000u : 0u;
  u32x4 u = __builtin_bit_cast(u32x4, x.v);
#pragma unroll
  for (int e = 0; e < 4; ++e) u[e] ^= flip;
  Frag<uint16_t> f;
  f.v = __builtin_bit_cast(bf16x8, u);
  return f;
}
__device__ __forceinline__ f32x4 rows_unsigned(const f32x4& x) { return f32x4{x[0], -x[1], x[2], -x[3]}; }

template <int DK>
struct SsmChainShape {
  static constexpr int C = 64, BV = 32, NDT = DK / 16, ND = NDT / 4;  // state tiles of key dims, of an S wave
  static constexpr int SLOT = C * DK;
  using TK = DmaTile<C, DK, 1, true>;
  static constexpr int PK = TK::PER_WAVE;
  static constexpr int kW = 4, kDma = 8, THREADS = 9 * kWave;
};

// One chain: S <- e^{G_C} S + A^T diag(w) B over the chunks, storing S before each.
//   forward   A = k, B = v, w = e^{G_C - G} D
//   REV       the chunks from last to first, A = q, B = dO, w = e^G
// A workgroup owns 32 value columns of one (sequence, head).  Four S waves keep a
// quarter of the key dims each, transposed (a lane's rows are value columns, so that the
// states leave in whole 16-byte pieces); four W waves form the parts of diag(w) B of
// the next chunk, from rows they have asked for three chunks before; one wavefront
// fetches A into a ring of three slots.  One barrier a chunk; two workgroups share a
// compute unit and cover each other's waits.  A chunk's products are summed apart and
// added to S once, six roundings of S less.  (With B through the ring as well, one
// chunk ahead, the chains waited for it: 110 us.)
template <int DK, bool REV, typename Lds>
__device__ __forceinline__ void ssm_chain_run(Lds& lds, const SsmBwd& b, int x, int NVB, int remap,
                                              const SsmStates& st) {
  using S = SsmChainShape<DK>;
  constexpr int C = S::C, BV = S::BV, ND = S::ND;
  int bh, vb;
  ssm_block(x, NVB, remap, bh, vb);
  const int H = b.H, DV = b.DV, h = bh % H, hk = h / (H / b.Hk);
  const int64_t seq = bh / H;
  const int nc = int((b.L + C - 1) / C), v0 = vb * BV;
  const int lane = threadIdx.x & 63, role = wave_id(), li = lane & 15, g = lane >> 4;
  auto chunk_of = [&](int n) { return REV ? nc - 1 - n : n; };  // n in the chain's order
  auto valid_of = [&](int n) {
    const int64_t t = int64_t(chunk_of(n)) * C;
    return int(b.L - t < C ? b.L - t : C);
  };
  auto tok_of = [&](int n) { return seq * b.L + int64_t(chunk_of(n)) * C; };
  auto sync = [&]() {
    wait_lgkm0();
    barrier_nowait();
  };
  const int64_t krow = REV ? b.q_row : b.k_row, vrow = REV ? b.do_row : b.v_row;

  // A barrier before every chunk n: its A is in the ring and its W in the LDS.
  if (role == S::kDma) {
    using U = const uint16_t*;
    const U k = static_cast<U>(REV ? b.q : b.k) + hk * DK;
    typename S::TK tk;
    tk.init(krow, lane, 0);
    auto issue = [&](int m) {
      const U ks = (U)uniform_ptr(k + tok_of(m) * krow);
      const int valid = valid_of(m);
      const uint32_t addr = lds_addr_of(lds.ring + (m % 3) * S::SLOT);
      auto body = [&](auto ragged) {
#pragma unroll
        for (int j = 0; j < S::PK; ++j) tk.template issue<decltype(ragged)::value>(j, addr, ks, valid);
      };
      if (valid == C) body(std::false_type{});
      else body(std::true_type{});
    };
    auto wait_for = [&](bool more) {  // all but the transfers issued last, where there are such
      if (more) wait_vmcnt<S::PK>();
      else wait_vmcnt<0>();
    };
    issue(0);
    if (nc > 1) issue(1);
    wait_for(nc > 1);
    for (int n = 0; n < nc; ++n) {
      barrier_nowait();  // chunk n is there
      if (n + 2 < nc) issue(n + 2);  // into chunk n - 1's slot
      wait_for(n + 2 < nc);
    }
  } else if (role >= S::kW) {
    const int c = role & 1, ku = (role >> 1) & 1;
    // rows (tokens) 32 ku + lane / 4 and 16 further on, the columns 8 (lane % 4) + 4 c .. of the block
    const auto* v = static_cast<const uint16_t*>(REV ? b.d_o : b.v) + int64_t(h) * DV + v0 + 8 * (lane & 3) + 4 * c;
    uint16_t* const tile = lds.tile[role & 3];
    const float sign = row_sign(li);
    struct Rows {
      bf16x4 v[2];
      f32x4 w[2];  // weights of tokens 32 ku + 16 e + 4 g ..
      float all;
    } at[3];
    auto load = [&](Rows& x, int n) {
#pragma unroll
      for (int e = 0; e < 2; ++e) x.v[e] = bf16x4{};
      if (n >= nc) return;
      const int valid = valid_of(n);
      const uint16_t* rows = v + tok_of(n) * vrow;
      const ChunkGates& gt = st.gates[int64_t(bh) * nc + chunk_of(n)];
      x.all = gt.e[63];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int t = 32 * ku + 16 * e + (lane >> 2);
        if (t < valid) x.v[e] = *reinterpret_cast<const bf16x4*>(rows + t * vrow);
        x.w[e] = *reinterpret_cast<const f32x4*>((REV ? gt.e : gt.w) + 32 * ku + 16 * e + 4 * g);
      }
    };
    auto weigh = [&](Rows& x, int n) {  // into W of chunk n
#pragma unroll
      for (int e = 0; e < 2; ++e) *reinterpret_cast<bf16x4*>(tile + (16 * e + (lane >> 2)) * 16 + 4 * (lane & 3)) = x.v[e];
      wait_lgkm0();
      f32x4 y[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const bf16x4 t = lds_read_tr(tile + (16 * e + 4 * g + (li >> 2)) * 16 + 4 * (li & 3));
#pragma unroll
        for (int qq = 0; qq < 4; ++qq) y[e][qq] = sign * x.w[e][qq] * static_cast<float>(t[qq]);
      }
      Frag<uint16_t> p[3];
      split3_frag(y[0], y[1], p);
#pragma unroll
      for (int i = 0; i < 3; ++i) lds.bW[n & 1][i][c][ku][lane] = p[i].v;
      if (role == S::kW && lane == 0) lds.all[n & 1] = x.all;
      load(x, n + 3);
    };
#pragma unroll
    for (int i = 0; i < 3; ++i) load(at[i], i);
    weigh(at[0], 0);
    for (int n = 0; n < nc; n += 3) {
      sync();
      weigh(at[1], n + 1);  // past the last chunk: zeros or stale values that nothing uses
      if (n + 1 >= nc) break;
      sync();
      weigh(at[2], n + 2);
      if (n + 2 >= nc) break;
      sync();
      weigh(at[0], n + 3);
    }
  } else {
    const int sw = role;
    f32x4 T[ND][2];  // T[d][c][qq]: key dim key_phys(16 (ND sw + d) + li), value column v0 + 8 g + 4 c + qq
    const float* s0 = REV ? b.dsf : b.s0;
    const int64_t row0 = (seq * H + h) * DK;
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        T[d][c] = zero4();
        if (s0 != nullptr)
          T[d][c] = *reinterpret_cast<const f32x4*>(s0 + (row0 + key_phys(16 * (ND * sw + d) + li)) * DV + v0 + 8 * g + 4 * c);
      }
    float* const out = REV ? st.x : st.s;
    for (int n = 0; n < nc; ++n) {
      sync();
      const uint16_t* cur = lds.ring + (n % 3) * S::SLOT;
      Frag<uint16_t> KT[ND][2];
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int ku = 0; ku < 2; ++ku) KT[d][ku] = wide_frag_tr<DK>(cur, ND * sw + d, ku, lane);
      const int64_t slot = int64_t(bh) * nc + chunk_of(n);
#pragma unroll
      for (int d = 0; d < ND; ++d) {
        float* const to = out + ((slot * (DV / 32) + vb) * DK + key_phys(16 * (ND * sw + d) + li)) * 32 + 8 * g;
#pragma unroll
        for (int c = 0; c < 2; ++c) *reinterpret_cast<f32x4*>(to + 4 * c) = T[d][c];
      }
      const float all = lds.all[n & 1];
      f32x4 own[ND][2];
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int c = 0; c < 2; ++c) own[d][c] = zero4();
#pragma unroll
      for (int ku = 0; ku < 2; ++ku)
#pragma unroll
        for (int part = 2; part >= 0; --part)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            Frag<uint16_t> W;
            W.v = lds.bW[n & 1][part][c][ku][lane];
#pragma unroll
            for (int d = 0; d < ND; ++d) mma(own[d][c], W, KT[d][ku]);
          }
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int qq = 0; qq < 4; ++qq) T[d][c][qq] = fmaf(all, T[d][c][qq], row_sign(qq) * own[d][c][qq]);
    }
    if (REV && b.ds0 != nullptr) {
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int c = 0; c < 2; ++c)
          *reinterpret_cast<f32x4*>(b.ds0 + (row0 + key_phys(16 * (ND * sw + d) + li)) * DV + v0 + 8 * g + 4 * c) = T[d][c];
    }
  }
}

template <int DK>
__global__ __launch_bounds__((SsmChainShape<DK>::THREADS), 5) void ssm_chain_kernel(SsmBwd b, int NVB, int half, int remap,
                                                                                    SsmStates st) {
  using S = SsmChainShape<DK>;
  __shared__ __align__(1024) uint16_t ring[3 * S::SLOT];
  __shared__ __align__(16) bf16x8 bW[2][3][2][2][kWave];  // [buffer][part][column tile][k-unit]
  __shared__ __align__(16) uint16_t tile[4][32 * 16];     // a W wave's rows on their way to its operands
  __shared__ float all[2];                                // e^{G_C} of the chunk in bW
  struct Refs {
    uint16_t* ring;
    decltype(bW)& bW;
    decltype(tile)& tile;
    decltype(all)& all;
  };
  Refs lds{ring, bW, tile, all};
  if (int(blockIdx.x) < half) ssm_chain_run<DK, true>(lds, b, blockIdx.x, NVB, remap, st);
  else ssm_chain_run<DK, false>(lds, b, blockIdx.x - half, NVB, remap, st);
}

// ---------------------------------------------------------------------------
// Gradients of one chunk for one query and key head: its value heads one after
// the other, dQ and dK summed over them in registers, in order.  Sixteen wavefronts:
//   ten of them a tile each of the lower triangle of Q K^T and dO V^T: P and dP with
//   their decays and D into the LDS, row and column sums of M
//   then the first half key dims of dQ^T each (all tokens), the other half of dK^T,
//   states as operands straight from memory, and all of them a share of dV^T
// The gradients of the 64 steps follow in a launch of their own.
// All products have tokens as columns, so a lane's four rows are adjacent values
// of one token.
template <int DK, int DV>
struct SsmGradShape {
  static constexpr int C = 64, KU = DK / 32, VU = DV / 32, NW = 16, THREADS = NW * kWave;
  static constexpr int DT = DK / 16, VT = DV / 16;
  static constexpr int KTOK = DT / 2;              // token tiles of dQ or dK a wavefront: 8 wavefronts, DT x 4 tiles
  static constexpr int VSPLIT = NW / VT > 4 ? 4 : NW / VT, VTOK = 4 / VSPLIT;  // of dV: VT VSPLIT wavefronts
  using TK = DmaTile<C, DK, NW, true>;
  using TV = DmaTile<C, DV, NW, true>;
};

// Tile t (0 .. 9) of the lower triangle: row tile, column tile.
__host__ __device__ constexpr int tri_row(int t) { return t < 1 ? 0 : t < 3 ? 1 : t < 6 ? 2 : 3; }
__host__ __device__ constexpr int tri_at(int r, int c) { return r * (r + 1) / 2 + c; }

// P and dP live tile by tile, [tile][16][16] row-major with rows i and columns j.
// Operand row i (k index j) ...
__device__ __forceinline__ Frag<uint16_t> tri_rows(const uint16_t* X, int rt, int ku, int lane) {
  const int li = lane & 15, g = lane >> 4;
  Frag<uint16_t> f;
  const bf16x4 lo = *reinterpret_cast<const bf16x4*>(X + (tri_at(rt, 2 * ku) * 16 + li) * 16 + 4 * g);
  bf16x4 hi{};
  if (2 * ku + 1 <= rt) hi = *reinterpret_cast<const bf16x4*>(X + (tri_at(rt, 2 * ku + 1) * 16 + li) * 16 + 4 * g);
  f.v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  return f;
}
// ... and operand row j (k index i).
__device__ __forceinline__ Frag<uint16_t> tri_cols(const uint16_t* X, int ct, int ku, int lane) {
  const int j = lane & 15, g = lane >> 4, at = (4 * g + (j >> 2)) * 16 + 4 * (j & 3);
  Frag<uint16_t> f;
  bf16x4 lo{};
  if (2 * ku >= ct) lo = lds_read_tr(X + tri_at(2 * ku, ct) * 256 + at);
  const bf16x4 hi = lds_read_tr(X + tri_at(2 * ku + 1, ct) * 256 + at);
  f.v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  return f;
}

// Operand row m0 + li of the transpose of a tile in the 16-byte layout, k index
// over its rows.
template <int ROWE>
__device__ __forceinline__ Frag<uint16_t> sw_frag_tr_wide(const uint16_t* X, int m0, int ku, int lane) {
  const int j = lane & 15, g = lane >> 4;
  const int r = 32 * ku + 4 * g + (j >> 2), c = m0 + 4 * (j & 3);
  const bf16x4 lo = lds_read_tr(X + swzw_off<ROWE>(r, c));
  const bf16x4 hi = lds_read_tr(X + swzw_off<ROWE>(r + 16, c));
  Frag<uint16_t> f;
  f.v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  return f;
}

// Operand row `row` of a tile in the 16-byte layout with the k index in the plain
// order of common.h, as a transposing read's rows are.
template <int ROWE>
__device__ __forceinline__ Frag<uint16_t> key_frag(const uint16_t* X, int row, int ku, int g) {
  const bf16x4 lo = *reinterpret_cast<const bf16x4*>(X + swzw_off<ROWE>(row, 32 * ku + 4 * g));
  const bf16x4 hi = *reinterpret_cast<const bf16x4*>(X + swzw_off<ROWE>(row, 32 * ku + 16 + 4 * g));
  Frag<uint16_t> f;
  f.v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  return f;
}

// Sum of the products of eight pairs of bf16 values, added to c.
__device__ __forceinline__ float dot8(const u32x4& x, const u32x4& y, float c) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
#pragma unroll
  for (int e = 0; e < 4; ++e)
    c = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, uint32_t(x[e])), __builtin_bit_cast(bf16x2, uint32_t(y[e])), c, false);
  return c;
}

template <int DK, int DV>
__global__ __launch_bounds__((SsmGradShape<DK, DV>::THREADS)) void ssm_grad_kernel(SsmBwd b, SsmStates st, int NC) {
  using S = SsmGradShape<DK, DV>;
  constexpr int C = S::C, KU = S::KU, VU = S::VU, VT = S::VT, KTOK = S::KTOK, VTOK = S::VTOK;
  __shared__ __align__(1024) uint16_t Qs[C * DK], Ks[C * DK], VO[2][2][C * DV];  // V and dO of this head and the next
  __shared__ __align__(1024) uint16_t Xs[DK * DV];  // X's first part, from the wavefronts that hold it
  __shared__ __align__(16) uint16_t Pm[10 * 256], Dm[10 * 256];
  __shared__ __align__(16) ChunkGates gates[2];  // of this head and the next

  const int r = b.H / b.Hk;
  const uint32_t wg = blockIdx.x;
  const int n = int(wg % uint32_t(NC));
  const uint32_t bk = wg / uint32_t(NC);
  const int hk = int(bk % uint32_t(b.Hk));
  const int64_t bb = bk / uint32_t(b.Hk);
  const int w = wave_id();
  // The lane's index afresh, so that addresses formed from it belong to one stage:
  // kept over the heads, they were 43 registers a lane of scratch memory, 180 MB
  // of writes in all and half of the time.
  auto lane_now = [&]() {
    int x;
    asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=v"(x));
    return x;
  };
  const int64_t t0 = int64_t(n) * C, tok = bb * b.L + t0;
  const int valid = int(b.L - t0 < C ? b.L - t0 : C);
  auto sync = [&]() {
    wait_lgkm0();
    barrier_nowait();
  };
  using U = const uint16_t*;
  {
    typename S::TK tk;
    const U qs = (U)uniform_ptr(static_cast<U>(b.q) + tok * b.q_row + hk * DK);
    const U ks = (U)uniform_ptr(static_cast<U>(b.k) + tok * b.k_row + hk * DK);
    const int ln = lane_now();
    tk.init(b.q_row, ln, w);
#pragma unroll
    for (int i = 0; i < S::TK::PER_WAVE; ++i) tk.template issue<true>(i, lds_addr_of(Qs), qs, valid);
    tk.init(b.k_row, ln, w);
#pragma unroll
    for (int i = 0; i < S::TK::PER_WAVE; ++i) tk.template issue<true>(i, lds_addr_of(Ks), ks, valid);
  }
  auto fetch_head = [&](int hh) {
    const int h = hk * r + hh;
    typename S::TV tv;
    const U vs = (U)uniform_ptr(static_cast<U>(b.v) + tok * b.v_row + int64_t(h) * DV);
    const U os = (U)uniform_ptr(static_cast<U>(b.d_o) + tok * b.do_row + int64_t(h) * DV);
    const int ln = lane_now();
    tv.init(b.v_row, ln, w);
#pragma unroll
    for (int i = 0; i < S::TV::PER_WAVE; ++i) tv.template issue<true>(i, lds_addr_of(VO[hh & 1][0]), vs, valid);
    tv.init(b.do_row, ln, w);
#pragma unroll
    for (int i = 0; i < S::TV::PER_WAVE; ++i) tv.template issue<true>(i, lds_addr_of(VO[hh & 1][1]), os, valid);
  };
  fetch_head(0);

  const bool is_q = w < 8;                                                  // dQ, or dK
  const int dt = (w & 7) / (4 / KTOK), ktok = (w & 7) % (4 / KTOK) * KTOK;  // its key dims 16 dt .., token tiles from ktok on
  const int vt = w % VT, vtok = w / VT * VTOK;                              // the same of dV
  const bool do_v = vtok < 4;
  f32x4 dA[KTOK];  // dQ^T or dK^T
#pragma unroll
  for (int t = 0; t < KTOK; ++t) dA[t] = zero4();
  f32x4 raw = zero4();  // of tile w: raw[qq] = k_j . q_i, j = 16 ct + 4 g + qq, i = 16 rt + li
  const int tile = w < 10 ? w : 9, rt = tri_row(tile), ct = tile - tri_at(rt, 0);

  // This wavefront's state rows (values 8 g .. of every k-unit, as in wide_frag's
  // operands), S for dQ, X for dK, and a head's gates.  They are asked for as soon as
  // the head before has used its own.
  f32x4 A[VU][2];
  auto fetch_state = [&](int hh) {
    const int64_t slot = (bb * b.H + hk * r + hh) * NC + n;
    const int ln = lane_now();
    const int64_t row = ((slot * VU) * DK + 16 * dt + (ln & 15)) * 32 + 8 * (ln >> 4);
    const float* const src = (is_q ? st.s : st.x) + row;
#pragma unroll
    for (int ku = 0; ku < VU; ++ku)
#pragma unroll
      for (int e = 0; e < 2; ++e) A[ku][e] = *reinterpret_cast<const f32x4*>(src + ku * DK * 32 + 4 * e);
    if (w == 14) {
      const ChunkGates& src = st.gates[slot];
      ChunkGates& gt = gates[hh & 1];
      gt.hi[ln] = src.hi[ln];
      gt.lo[ln] = src.lo[ln];
      gt.D[ln] = src.D[ln];
      gt.e[ln] = src.e[ln];
      gt.w[ln] = src.w[ln];
    }
  };
  fetch_state(0);
  wait_vmcnt<0>();  // Q, K and the first head's V and dO

  for (int hh = 0; hh < r; ++hh) {
    const int h = hk * r + hh, u = hh & 1;
    const int64_t slot = (bb * b.H + h) * NC + n;
    const float skip = b.d != nullptr ? b.d[h] : 0.0f;
    uint16_t* const Vs = VO[u][0];
    uint16_t* const Os = VO[u][1];
    const ChunkGates& gt = gates[u];
    ChunkSums& sums = st.sums[slot];
    const int64_t sbase = (slot * VU * DK + 16 * dt) * 32;
    sync();  // this head's V, dO and gates are there, the one before is done with the LDS
    if (valid < C) {  // rows past the end repeat row 0: zeros
      if (hh == 0) {
        for (int at = w * kWave + lane_now(); at < (C - valid) * DK / 8; at += S::THREADS)
          reinterpret_cast<u32x4*>(Qs)[valid * DK / 8 + at] = reinterpret_cast<u32x4*>(Ks)[valid * DK / 8 + at] = u32x4{};
      }
      for (int at = w * kWave + lane_now(); at < (C - valid) * DV / 8; at += S::THREADS)
        reinterpret_cast<u32x4*>(Vs)[valid * DV / 8 + at] = reinterpret_cast<u32x4*>(Os)[valid * DV / 8 + at] = u32x4{};
      sync();
    }
    if (hh + 1 < r) fetch_head(hh + 1);
    if (w < 10) {
      const int ln = lane_now(), li = ln & 15, g = ln >> 4, i = 16 * rt + li;
      if (hh == 0) {
#pragma unroll
        for (int ku = 0; ku < KU; ++ku) mma(raw, row_signed(wide_frag<DK>(Ks, 16 * ct + li, ku, g), li), wide_frag<DK>(Qs, i, ku, g));
        raw = rows_unsigned(raw);
      }
      f32x4 dp = zero4();
#pragma unroll
      for (int ku = 0; ku < VU; ++ku) mma(dp, row_signed(wide_frag<DV>(Vs, 16 * ct + li, ku, g), li), wide_frag<DV>(Os, i, ku, g));
      dp = rows_unsigned(dp);
      const float hi = gt.hi[i], lo = gt.lo[i];
      const f32x4 ch = *reinterpret_cast<const f32x4*>(gt.hi + 16 * ct + 4 * g);
      const f32x4 cl = *reinterpret_cast<const f32x4*>(gt.lo + 16 * ct + 4 * g);
      const f32x4 D = *reinterpret_cast<const f32x4*>(gt.D + 16 * ct + 4 * g);
      f32x4 p, d, md;
#pragma unroll
      for (int qq = 0; qq < 4; ++qq) {
        const bool in = ct < rt || 4 * g + qq <= li;
        const float f = in ? __builtin_amdgcn_exp2f((hi - ch[qq]) + (lo - cl[qq])) : 0.0f;
        const float m = in ? dp[qq] * (raw[qq] * f) : 0.0f;
        p[qq] = in ? raw[qq] * f * D[qq] : 0.0f;
        d[qq] = in ? dp[qq] * f * D[qq] : 0.0f;
        md[qq] = m * D[qq];
        const float cs = row_sum16(m);
        if (li == 0) sums.col[tile][4 * g + qq] = cs;
      }
      if (rt == ct) {
        const f32x4 own = tile_between(md, li, g);
        if (li == 0) *reinterpret_cast<f32x4*>(sums.row[tile] + 4 * g) = own;
      } else {
        const float rs = row_sum4((md[0] + md[1]) + (md[2] + md[3]));
        if (g == 0) sums.row[tile][li] = rs;
      }
      st4(Pm + (tile * 16 + li) * 16 + 4 * g, p);
      st4(Dm + (tile * 16 + li) * 16 + 4 * g, d);
    }
    if (!is_q && ktok == 0) {
      const int ln = lane_now();
#pragma unroll
      for (int ku = 0; ku < VU; ++ku)
        *reinterpret_cast<bf16x8*>(Xs + swzw_off<DV>(16 * dt + (ln & 15), 32 * ku + 8 * (ln >> 4))) =
            acc_frag<uint16_t>(A[ku][0], A[ku][1]).v;
    }
    __builtin_amdgcn_sched_barrier(0);
    // v . dO of this chunk, and <X, S>: half of the value columns of both by the
    // wavefronts that hold S, the others by those that hold X (one of each key tile)
    float skips = 0.0f, dot = 0.0f;
    for (int at = w * kWave + lane_now(); at < C * DV / 8; at += S::THREADS)
      skips = dot8(reinterpret_cast<const u32x4*>(Vs)[at], reinterpret_cast<const u32x4*>(Os)[at], skips);
    if (ktok == 0) {
      const int ln = lane_now();
      const int64_t srow = sbase + (ln & 15) * 32 + 8 * (ln >> 4);
      const float* const other = (is_q ? st.x : st.s) + srow;
#pragma unroll
      for (int ku = 0; ku < VU; ++ku) {
        if (VU > 1 ? (ku < VU / 2) != is_q : !is_q) continue;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const f32x4 y = *reinterpret_cast<const f32x4*>(other + ku * DK * 32 + 4 * e);
#pragma unroll
          for (int qq = 0; qq < 4; ++qq) dot = fmaf(A[ku][e][qq], y[qq], dot);
        }
      }
    }
    skips = row_sum4(row_sum16(skips));
    dot = row_sum4(row_sum16(dot));
    if (lane_now() == 0) {
      sums.vo[w] = skips;
      sums.xs[w] = dot;
    }
    __builtin_amdgcn_sched_barrier(0);
    sync();  // P, dP and X
    // dQ^T = S (dO diag(e))^T + K^T dP, dK^T = X (V diag(w))^T + Q^T dP^T: tokens in columns
    auto key_grads = [&](auto qc) {
      constexpr bool Q = decltype(qc)::value;
      const int ln = lane_now(), li = ln & 15, g = ln >> 4;
      const uint16_t* rows = Q ? Os : Vs;
      const uint16_t* mine = Q ? Qs : Ks;
      Frag<uint16_t> T[2];
#pragma unroll
      for (int ku = 0; ku < 2; ++ku) T[ku] = sw_frag_tr_wide<DK>(Q ? Ks : Qs, 16 * dt, ku, ln);
      const float hi_end = gt.hi[63], lo_end = gt.lo[63];
      f32x4 xs[KTOK];
#pragma unroll
      for (int tt = 0; tt < KTOK; ++tt) xs[tt] = zero4();
#pragma unroll
      for (int ku = 0; ku < VU; ++ku) {  // the state in three parts: r and p go into sums that cancel
        Frag<uint16_t> p[3];
        split3_frag(row_sign(li) * A[ku][0], row_sign(li) * A[ku][1], p);
#pragma unroll
        for (int tt = 0; tt < KTOK; ++tt) {
          const Frag<uint16_t> f = wide_frag<DV>(rows, 16 * (ktok + tt) + li, ku, g);
#pragma unroll
          for (int i = 2; i >= 0; --i) mma(xs[tt], p[i], f);
        }
      }
#pragma unroll
      for (int tt = 0; tt < KTOK; ++tt) {
        const int t = ktok + tt, j = 16 * t + li;
        f32x4 x = (Q ? gt.e[j] : __builtin_amdgcn_exp2f((hi_end - gt.hi[j]) + (lo_end - gt.lo[j]))) * rows_unsigned(xs[tt]);
        const bf16x4 o = *reinterpret_cast<const bf16x4*>(mine + swzw_off<DK>(j, 16 * dt + 4 * g));
        float sum = 0.0f;
#pragma unroll
        for (int qq = 0; qq < 4; ++qq) sum = fmaf(x[qq], float(o[qq]), sum);
        sum = row_sum4(sum);
        if (g == 0) (Q ? sums.r : sums.p)[dt][j] = sum;
        if (!Q) x = gt.D[j] * x;
#pragma unroll
        for (int ku = 0; ku < 2; ++ku) {
          if (Q && 2 * ku <= t) mma(x, T[ku], tri_rows(Dm, t, ku, ln));
          if (!Q && 2 * ku + 1 >= t) mma(x, T[ku], tri_cols(Dm, t, ku, ln));
        }
        dA[tt] += x;
      }
    };
    if (is_q) key_grads(std::true_type{});
    else key_grads(std::false_type{});
    if (hh + 1 < r) {
      wait_vmcnt<0>();  // the next head's V and dO
      fetch_state(hh + 1);
    }
    __builtin_amdgcn_sched_barrier(0);
    if (do_v) {
      const int ln = lane_now(), li = ln & 15, g = ln >> 4;
      Frag<uint16_t> XT[KU];  // X^T: row 16 vt + li, k index over the key dims in the order of key_frag
#pragma unroll
      for (int ku = 0; ku < KU; ++ku) XT[ku] = sw_frag_tr_wide<DV>(Xs, 16 * vt, ku, ln);
      uint16_t* dv = static_cast<uint16_t*>(b.dv) + tok * b.dv_row + int64_t(h) * DV + 16 * vt + 4 * g;
      Frag<uint16_t> OT[2];
#pragma unroll
      for (int ku = 0; ku < 2; ++ku) OT[ku] = sw_frag_tr_wide<DV>(Os, 16 * vt, ku, ln);
#pragma unroll
      for (int tt = 0; tt < VTOK; ++tt) {
        const int t = vtok + tt, j = 16 * t + li;
        f32x4 x = zero4();
#pragma unroll
        for (int ku = 0; ku < KU; ++ku) mma(x, XT[ku], key_frag<DK>(Ks, j, ku, g));
        x = gt.w[j] * x;
#pragma unroll
        for (int ku = 0; ku < 2; ++ku)
          if (2 * ku + 1 >= t) mma(x, OT[ku], tri_cols(Pm, t, ku, ln));
        const bf16x4 o = *reinterpret_cast<const bf16x4*>(Os + swzw_off<DV>(j, 16 * vt + 4 * g));
#pragma unroll
        for (int qq = 0; qq < 4; ++qq) x[qq] = fmaf(skip, float(o[qq]), x[qq]);
        if (j < valid) st4(dv + j * b.dv_row, x);
      }
    }
  }
  const int ln = lane_now(), li = ln & 15, g = ln >> 4;
#pragma unroll
  for (int tt = 0; tt < KTOK; ++tt) {
    const int j = 16 * (ktok + tt) + li;
    if (j >= valid) continue;
    uint16_t* out = is_q ? static_cast<uint16_t*>(b.dq) + (tok + j) * b.dq_row : static_cast<uint16_t*>(b.dk) + (tok + j) * b.dk_row;
    st4(out + hk * DK + 16 * dt + 4 * g, dA[tt]);
  }
}

// ddt of every token and the chunks' shares of da, dbias and dd from their sums
// (ssm.h), a wavefront a chunk, a lane a token.  DT: key tiles of 16.
__global__ __launch_bounds__(kThreads) void ssm_steps_kernel(SsmBwd b, SsmStates st, float* __restrict__ part, int NC,
                                                             int64_t slots, int DT) {
  const int64_t slot = int64_t(blockIdx.x) * 4 + wave_id();
  if (slot >= slots) return;
  const int l = threadIdx.x & 63, lt = l >> 4, i = l & 15;
  const int n = int(slot % NC), h = int(slot / NC % b.H);
  const int64_t bb = slot / NC / b.H, t = int64_t(n) * 64 + l, tok = bb * b.L + t;
  const bool real = t < b.L;
  const ChunkSums& s = st.sums[slot];
  const ChunkGates& gt = st.gates[slot];
  // of M: t's own tile; rows and columns of the tiles left of it and below it; the tiles
  // between them; all columns by D
  float own = s.row[tri_at(lt, lt)][i], ri = 0.0f, cb = 0.0f, mid = 0.0f, ci = s.col[tri_at(lt, lt)][i], rr = 0.0f, pj = 0.0f;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    if (c < lt) ri += s.row[tri_at(lt, c)][i];
    if (c > lt) cb += s.col[tri_at(c, lt)][i];
#pragma unroll
    for (int r = c + 2; r < 4; ++r)
      if (c < lt && lt < r) mid += s.row[tri_at(r, c)][i];
  }
  ci += cb;
#pragma unroll
  for (int x = 0; x < 8; ++x) {
    if (x >= DT) break;
    rr += s.r[x][l];
    pj += s.p[x][l];
  }
  float xs = l < 16 ? s.xs[l] : 0.0f, vo = l < 16 ? s.vo[l] : 0.0f;
  const float D = gt.D[l], rate = b.a[h];
  float x = b.bias != nullptr ? b.bias[h] : 0.0f;
  if (real) x += to_f32(static_cast<const uint16_t*>(b.dt)[tok * b.dt_row + h]);
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) {
    xs += __shfl_xor(xs, off);
    vo += __shfl_xor(vo, off);
  }
  own += row_suffix16(ri, i) + row_before16(D * cb, i) + row_sum16(mid);
  float suf = real ? rr : 0.0f, pre = real ? D * pj : 0.0f;
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const float y = __shfl_down(suf, d), z = __shfl_up(pre, d);
    if (l + d < kWave) suf += y;
    if (l >= d) pre += z;
  }
  // the lane before's, not the lane's own less its term: a large last one would round the others away
  const float before = __shfl_up(pre, 1);
  const float gd = own + (suf + (l > 0 ? before : 0.0f) + gt.e[63] * xs);
  const float ddt = real ? (ci + pj + rate * gd) * (1.0f / (1.0f + expf(-x))) : 0.0f;
  if (real) static_cast<uint16_t*>(b.ddt)[tok * b.ddt_row + h] = from_f32<uint16_t>(ddt);
  float sa = real ? D * gd : 0.0f, sb = ddt;
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) {
    sa += __shfl_xor(sa, off);
    sb += __shfl_xor(sb, off);
  }
  if (l == 0) {
    const int64_t M = int64_t(b.B) * NC, at = int64_t(h) * M + bb * NC + n, all = int64_t(b.H) * M;
    part[at] = sa;
    part[all + at] = sb;
    part[2 * all + at] = vo;
  }
}

}  // namespace efla
