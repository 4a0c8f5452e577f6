// ssm_chunk.h -- the chunked pass of the selective state space scan (ssm.h) for
// bf16 inputs, in chunks of 64 tokens on the matrix cores.
//
// Per chunk (start state S; e = e^G, w = e^{G_C - G} D):
//     P = e^{G_i - G_j} D_j tril(Q K^T),   O = diag(e) Q S + P V + d V,
//     S <- e^{G_C} S + K^T diag(w) V
// Only the last line is sequential, one product deep, so a workgroup owns 32
// value columns of one (sequence, head), walks its chunks with S in registers,
// and everything else hangs off that chain, spread over thirteen wavefronts:
//   four S waves   S of a 16-column tile and half of the key dims; diag(w) V of
//                  the next chunk is split into operand parts beside the products
//                  of this one
//   four O waves   16 tokens: diag(e) Q S in the chunk's own iteration, P V in the
//                  next one, when P is there
//   three P waves  16 rows of P each (the first two tiles: one), from Q and K
//   gate wave      D, e, w and G two chunks ahead, its loads five
//   DMA wave       Q, K and V three chunks ahead into a ring of three slots
// with one barrier a chunk: S (bf16, for the readout), P and the gates are
// written to one buffer while another is read.  Every wavefront takes the next
// chunk's operands from the ring into registers behind its own products, so that
// the LDS works beside the matrix cores and a chunk's slot is free when the chunk
// begins; right behind the barrier only S and P are read.
//
// q, k and v are bf16, so Q K^T is exact in float32 sums.  diag(w) V, which
// feeds S, goes in as three bf16 parts (24 bits); S and P, which only feed o, are
// rounded once, as o itself is.
#pragma once

#include <type_traits>

#include "lds_ring.h"
#include "ssm.h"

namespace efla {

// Eight values (k-unit halves lo4, hi4) as a sum of three bf16 fragments.
__device__ __forceinline__ void split3_frag(const f32x4& lo4, const f32x4& hi4, Frag<uint16_t> (&p)[3]) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  u32x4 part[3];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const f32x4& src = e < 2 ? lo4 : hi4;
    f32x2 x{src[2 * (e & 1)], src[2 * (e & 1) + 1]};
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const uint32_t h = __builtin_bit_cast(uint32_t, __builtin_convertvector(x, bf16x2));
      part[i][e] = h;
      x = f32x2{x[0] - __uint_as_float(h << 16), x[1] - __uint_as_float(h & 0xffff0000u)};
    }
  }
#pragma unroll
  for (int i = 0; i < 3; ++i) p[i].v = __builtin_bit_cast(bf16x8, part[i]);
}

// (Sequence, head) and value block of workgroup x.  remap > 0: all value blocks of
// `remap` adjacent heads on one XCD (same x % 8), whose L2 then serves what they
// share; the (sequence, head)s are a multiple of 8 remap.
__device__ __forceinline__ void ssm_block(int x, int NVB, int remap, int& bh, int& vb) {
  if (remap > 0) {
    const int slot = x >> 3, in = slot % (remap * NVB);
    vb = in % NVB;
    bh = ((slot / (remap * NVB)) * 8 + (x & 7)) * remap + in / NVB;
  } else {
    bh = x / NVB;
    vb = x % NVB;
  }
}
// Heads that share their queries and keys together where that comes out even, else
// a head's own value blocks, else none.
inline int ssm_remap(int64_t bh, int r) { return bh / r % 8 == 0 ? r : bh % 8 == 0 ? 1 : 0; }

template <int DK>
struct SsmShape {
  static_assert(DK == 64 || DK == 128, "shapes of the chunked scan");
  static constexpr int C = 64, BV = 32, NKU = DK / 32, NDT = DK / 16, NPF = 6;
  static constexpr int QOFF = 0, KOFF = C * DK, VOFF = 2 * C * DK, SLOT = 2 * C * DK + C * BV;  // in elements
  using TQ = DmaTile<C, DK, 1, true>;
  using TV = DmaTile<C, BV, 1, true>;
  static constexpr int PQ = TQ::PER_WAVE, PV = TV::PER_WAVE, COUNT = 2 * PQ + PV;
  // wavefronts by index (SIMD = index % 4)
  static constexpr int kO = 4, kP = 8, kGate = 9, kP3 = 10, kP2 = 11, kDma = 12, THREADS = 13 * kWave;
  static constexpr int LOCAL_THREADS = 6 * kWave;  // S, gates, DMA
};

// Value columns of a block: row l of column tile c is column 8 (l / 4) + 4 c + l % 4,
// so that a lane's four rows 4 g .. of both tiles are eight adjacent columns of o.
__host__ __device__ constexpr int value_phys(int c, int l) { return 8 * (l / 4) + 4 * c + l % 4; }

// Operand row l of column tile c (k index over the tokens of k-unit ku) of a V tile.
template <int BV>
__device__ __forceinline__ Frag<uint16_t> value_frag(const uint16_t* X, int c, int ku, int lane) {
  const int j = lane & 15, g = lane >> 4, r = 32 * ku + 4 * g + (j >> 2), col = 8 * (j & 3) + 4 * c;
  const bf16x4 lo = lds_read_tr(X + swzw_off<BV>(r, col));
  const bf16x4 hi = lds_read_tr(X + swzw_off<BV>(r + 16, col));
  Frag<uint16_t> f;
  f.v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  return f;
}

// LOCAL: a segment's end state (the first's from s0, the others' from zero) and its
// decay alone, with the S, gate and DMA waves and neither Q nor o.
template <int DK, bool LOCAL>
__global__ __launch_bounds__((LOCAL ? SsmShape<DK>::LOCAL_THREADS : SsmShape<DK>::THREADS)) void ssm_chunk_kernel(
    SsmFwd a, int NVB, int remap) {
  using S = SsmShape<DK>;
  constexpr int C = S::C, BV = S::BV, NKU = S::NKU, NDT = S::NDT;
  __shared__ __align__(1024) uint16_t ring[3 * S::SLOT];
  __shared__ __align__(16) bf16x8 bS[2][2][NKU][kWave];  // S of a chunk's start, [buffer][column tile][k-unit]
  __shared__ __align__(16) bf16x8 bP[2][S::NPF][kWave];
  __shared__ __align__(16) ChunkGates gates[3];

  const int H = a.H, DV = a.DV;
  int bh, vb;
  ssm_block(int(blockIdx.x), NVB, remap, bh, vb);
  const int h = bh % H, hk = h / (H / a.Hk);
  const int lane = threadIdx.x & 63, li = lane & 15, g = lane >> 4;
  const SsmUnit sp = ssm_unit<C>(a, bh / H, h, lane);
  if (sp.seq < 0 || (LOCAL && sp.last)) return;
  const int64_t srow = state_row(a.slots, sp.seq, a.P);
  const int nc = int((sp.len + C - 1) / C), v0 = vb * BV;
  int role = wave_id();
  if (LOCAL && role >= S::kO) role = role == S::kO ? S::kGate : S::kDma;
  auto valid_of = [&](int n) { return int(sp.len - int64_t(n) * C < C ? sp.len - int64_t(n) * C : C); };
  auto tok_of = [&](int n) { return sp.bos + int64_t(n) * C; };
  // Barriers: one before chunk 0's operands are read, one before every chunk n
  // (its operands are in registers, chunk n + 1 is in the ring and its gates and
  // chunk n's S are in the LDS, chunk n - 1's P too), one before the last P V.
  auto sync = [&]() {
    wait_lgkm0();
    barrier_nowait();
  };

  // The longest path first: S, then on every SIMD the longest of the other roles
  // (wavefronts go round the four SIMDs in order).  us of 4 x 4096 tokens, 16 heads, d
  // 128 / of 16 packed prompts: 112 / 130 with this order, 118 / 135 with none, 121 / 137 where
  // P's first rows are left out.
  if (role < S::kO) __builtin_amdgcn_s_setprio(2);
  else if (role == S::kP || role == S::kGate || role == S::kP3 || role == S::kO + 3) __builtin_amdgcn_s_setprio(1);

  if (role == S::kDma) {
    // ---------------------------------------------------------------- DMA
    using U = const uint16_t*;
    const U q = static_cast<U>(a.q) + hk * DK, k = static_cast<U>(a.k) + hk * DK, v = static_cast<U>(a.v) + int64_t(h) * DV + v0;
    typename S::TQ tq, tk;
    typename S::TV tv;
    tq.init(a.q_row, lane, 0);
    tk.init(a.k_row, lane, 0);
    tv.init(a.v_row, lane, 0);
    auto issue = [&](int m) {
      const int64_t t = tok_of(m);
      const U qs = (U)uniform_ptr(q + t * a.q_row), ks = (U)uniform_ptr(k + t * a.k_row), vs = (U)uniform_ptr(v + t * a.v_row);
      const int valid = valid_of(m);
      const uint32_t addr = lds_addr_of(ring + (m % 3) * S::SLOT);
      auto body = [&](auto ragged) {
        constexpr bool R = decltype(ragged)::value;
#pragma unroll
        for (int j = 0; j < S::PV; ++j) tv.template issue<R>(j, addr + 2 * S::VOFF, vs, valid);
#pragma unroll
        for (int j = 0; j < S::PQ; ++j) tk.template issue<R>(j, addr + 2 * S::KOFF, ks, valid);
        if constexpr (!LOCAL) {
#pragma unroll
          for (int j = 0; j < S::PQ; ++j) tq.template issue<R>(j, addr + 2 * S::QOFF, qs, valid);
        }
      };
      if (valid == C) body(std::false_type{});
      else body(std::true_type{});
    };
    constexpr int COUNT = LOCAL ? S::COUNT - S::PQ : S::COUNT;
    static_assert(COUNT < 64, "one chunk's transfers fit the vmcnt counter");
    auto wait_for = [&](bool more) {  // all but the transfers issued last, where there are such
      if (more) wait_vmcnt<COUNT>();
      else wait_vmcnt<0>();
    };
    if (nc > 0) issue(0);
    if (nc > 1) issue(1);
    wait_for(nc > 1);
    barrier_nowait();  // chunk 0
    if (nc > 2) issue(2);
    wait_for(nc > 2);
    for (int n = 0; n < nc; ++n) {
      barrier_nowait();  // chunk n + 1 is there; chunk n's slot is free
      if (n + 3 < nc) issue(n + 3);
      wait_for(n + 3 < nc);
    }
    barrier_nowait();
  } else if (role == S::kGate) {
    // --------------------------------------------------------------- gates
    const auto* dt = static_cast<const uint16_t*>(a.dt) + h;
    const float rate = a.a[h], bias = a.bias != nullptr ? a.bias[h] : 0.0f;
    auto load = [&](int n) {
      if (n >= nc) return 0.0f;
      return lane < valid_of(n) ? to_f32(dt[(tok_of(n) + lane) * a.dt_row]) : 0.0f;
    };
    float now = load(0), next = load(1), then = load(2);
    auto put = [&](int n) {
      put_chunk_gates(gates[n % 3], now + bias, rate, n < nc && lane < valid_of(n), lane);
      now = next;
      next = then;
      then = load(n + 3);
    };
    put(0);
    sync();
    put(1);
    for (int n = 0; n < nc; ++n) {
      sync();
      put(n + 2);
    }
    sync();
  } else if (role < S::kO) {
    // ------------------------------------------------------------------- S
    constexpr int ND = NDT / 2;  // half of the key dims
    const int c = role & 1, d0 = ND * (role >> 1);
    const int col = v0 + value_phys(c, li);
    f32x4 St[ND];  // St[d][qq] = S[key_phys(16 (d0 + d) + 4 g + qq)][col]
    auto at = [&](int d, int qq) { return int64_t(key_phys(16 * (d0 + d) + 4 * g + qq)) * DV; };
    auto put_state = [&](float* dst) {
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int qq = 0; qq < 4; ++qq) dst[at(d, qq)] = St[d][qq];
    };
    const float* s0 = a.s0 == nullptr || srow < 0 ? nullptr : a.s0 + (srow * H + h) * DK * DV;
    s0 = sp.start(LOCAL, s0, a.seg_s, int64_t(DK) * DV);
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int qq = 0; qq < 4; ++qq) St[d][qq] = s0 != nullptr ? s0[at(d, qq) + col] : 0.0f;
    if constexpr (LOCAL) {
      if (sp.before == 0) put_state(a.seg_s + sp.end * DK * DV + col);
    } else {
      for (int64_t slot = sp.first + H; slot < sp.slot; slot += H) {  // the segments before, in order
        const float e = a.seg_e[slot];
        const float* src = a.seg_s + slot * DK * DV + col;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
          for (int qq = 0; qq < 4; ++qq) St[d][qq] = fmaf(e, St[d][qq], src[at(d, qq)]);
      }
    }
    float decay = 1.0f;  // of all chunks
    auto publish = [&](int buf) {
#pragma unroll
      for (int d = 0; d < ND; d += 2) bS[buf][c][(d0 + d) / 2][lane] = acc_frag<uint16_t>(St[d], St[d + 1]).v;
    };
    Frag<uint16_t> KT[2][ND], V[2], W[2][3];
    auto load = [&](int n) {
      const uint16_t* cur = ring + (n % 3) * S::SLOT;
#pragma unroll
      for (int ku = 0; ku < 2; ++ku) {
        V[ku] = value_frag<BV>(cur + S::VOFF, c, ku, lane);
      }
#pragma unroll
      for (int ku = 0; ku < 2; ++ku)
#pragma unroll
        for (int d = 0; d < ND; ++d) KT[ku][d] = wide_frag_tr<DK>(cur + S::KOFF, d0 + d, ku, lane);
    };
    auto weigh = [&](int n) {  // diag(w) V of chunk n in three parts
#pragma unroll
      for (int ku = 0; ku < 2; ++ku) {
        f32x4 x[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const f32x4 w = *reinterpret_cast<const f32x4*>(gates[n % 3].w + 32 * ku + 16 * e + 4 * g);
#pragma unroll
          for (int qq = 0; qq < 4; ++qq) x[e][qq] = w[qq] * static_cast<float>(V[ku].v[4 * e + qq]);
        }
        split3_frag(x[0], x[1], W[ku]);
      }
    };
    sync();
    load(0);
    if constexpr (!LOCAL) publish(0);
    weigh(0);
    for (int n = 0; n < nc; ++n) {
      sync();
      const float all = gates[n % 3].e[63];
      if constexpr (LOCAL) decay *= all;
#pragma unroll
      for (int d = 0; d < ND; ++d) St[d] = all * St[d];
#pragma unroll
      for (int ku = 0; ku < 2; ++ku)
#pragma unroll
        for (int part = 2; part >= 0; --part)
#pragma unroll
          for (int d = 0; d < ND; ++d) mma(St[d], KT[ku][d], W[ku][part]);
      load(n + 1);  // past the last chunk: stale values that nothing uses
      if constexpr (!LOCAL) publish((n + 1) & 1);
      weigh(n + 1);
    }
    sync();
    float* sf = LOCAL ? a.seg_s + sp.slot * DK * DV + col
                      : a.sfin == nullptr || srow < 0 || !sp.last ? nullptr : a.sfin + (srow * H + h) * DK * DV + col;
    if (sf != nullptr) put_state(sf);
    if (LOCAL && vb == 0 && threadIdx.x == 0) a.seg_e[sp.slot] = decay;
  } else if (role >= S::kP) {
    // ------------------------------------------------------------------- P
    auto p_role = [&](auto r0c, auto r1c) {
      constexpr int R0 = decltype(r0c)::value, R1 = decltype(r1c)::value;  // row tiles R0 .. R1 - 1, column tiles up to each
      constexpr int AHEAD = NKU / 2;  // k-units taken a chunk ahead; the others' registers are the budget's
      Frag<uint16_t> Q[R1 - R0][AHEAD], K[R1][AHEAD];
      auto load = [&](int n, int k0) {
        const uint16_t* cur = ring + (n % 3) * S::SLOT;
#pragma unroll
        for (int ku = 0; ku < AHEAD; ++ku) {
#pragma unroll
          for (int r = R0; r < R1; ++r) Q[r - R0][ku] = wide_frag<DK>(cur + S::QOFF, 16 * r + li, k0 + ku, g);
#pragma unroll
          for (int c = 0; c < R1; ++c) K[c][ku] = wide_frag<DK>(cur + S::KOFF, 16 * c + li, k0 + ku, g);
        }
      };
      f32x4 P[R1 - R0][R1];  // P[r - R0][c][qq] = row 16 r + li, column 16 c + 4 g + qq
      auto multiply = [&]() {
#pragma unroll
        for (int ku = 0; ku < AHEAD; ++ku)
#pragma unroll
          for (int c = 0; c < R1; ++c)
#pragma unroll
            for (int r = R0; r < R1; ++r)
              if (c <= r) mma(P[r - R0][c], K[c][ku], Q[r - R0][ku]);
      };
      sync();
      load(0, 0);
      for (int n = 0; n < nc; ++n) {
#pragma unroll
        for (int r = R0; r < R1; ++r)
#pragma unroll
          for (int c = 0; c < R1; ++c) P[r - R0][c] = zero4();
        multiply();
        load(n, AHEAD);
        sync();
        const ChunkGates& gt = gates[n % 3];
        multiply();
        load(n + 1, 0);
#pragma unroll
        for (int c = 0; c < R1; ++c) {
          const f32x4 ch = *reinterpret_cast<const f32x4*>(gt.hi + 16 * c + 4 * g);
          const f32x4 cl = *reinterpret_cast<const f32x4*>(gt.lo + 16 * c + 4 * g);
          const f32x4 D = *reinterpret_cast<const f32x4*>(gt.D + 16 * c + 4 * g);
#pragma unroll
          for (int r = R0; r < R1; ++r) {
            if (c > r) continue;
            const float hi = gt.hi[16 * r + li], lo = gt.lo[16 * r + li];
#pragma unroll
            for (int qq = 0; qq < 4; ++qq) {
              const float f = __builtin_amdgcn_exp2f((hi - ch[qq]) + (lo - cl[qq])) * D[qq];
              P[r - R0][c][qq] = (c < r || 4 * g + qq <= li) ? P[r - R0][c][qq] * f : 0.0f;
            }
          }
        }
#pragma unroll
        for (int r = R0; r < R1; ++r)
#pragma unroll
          for (int ku = 0; 2 * ku <= r; ++ku)
            bP[n & 1][pf_index(r, ku)][lane] =
                acc_frag<uint16_t>(P[r - R0][2 * ku], 2 * ku + 1 < R1 ? P[r - R0][2 * ku + 1 < R1 ? 2 * ku + 1 : 0] : zero4()).v;
      }
      sync();
    };
    using std::integral_constant;
    if (role == S::kP3) p_role(integral_constant<int, 3>{}, integral_constant<int, 4>{});
    else if (role == S::kP2) p_role(integral_constant<int, 2>{}, integral_constant<int, 3>{});
    else p_role(integral_constant<int, 0>{}, integral_constant<int, 2>{});
  } else {
    // ------------------------------------------------------------------- O
    auto o_role = [&](auto rowc) {
      constexpr int R = decltype(rowc)::value, KO = R / 2 + 1;  // row tile; k-units of its rows of P
      const int t = 16 * R + li;                                // this lane's token
      const float skip = a.d != nullptr ? a.d[h] : 0.0f;
      f32x4 Z[2];                             // o of the chunk before without P V: Z[c][qq], column value_phys(c, 4 g + qq)
      Frag<uint16_t> Q[NKU], V[2][KO], U[2][KO];  // V of this chunk, U of the one before
      bf16x8 own;                             // this token's v, columns 8 g ..
      uint16_t* o = static_cast<uint16_t*>(a.o) + int64_t(h) * DV + v0 + 8 * g;
      auto load = [&](int n) {
        const uint16_t* cur = ring + (n % 3) * S::SLOT;
#pragma unroll
        for (int ku = 0; ku < NKU; ++ku) Q[ku] = wide_frag<DK>(cur + S::QOFF, t, ku, g);
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int ku = 0; ku < KO; ++ku) V[c][ku] = value_frag<BV>(cur + S::VOFF, c, ku, lane);
        own = *reinterpret_cast<const bf16x8*>(cur + S::VOFF + swzw_off<BV>(t, 8 * g));
      };
      auto finish = [&](int n) {  // of chunk n, whose P is in the LDS
        Frag<uint16_t> p[KO];
#pragma unroll
        for (int ku = 0; ku < KO; ++ku) p[ku].v = bP[n & 1][pf_index(R, ku)][lane];
        bf16x8 ov;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
          for (int ku = 0; ku < KO; ++ku) mma(Z[c], U[c][ku], p[ku]);
#pragma unroll
          for (int qq = 0; qq < 4; ++qq) ov[4 * c + qq] = static_cast<__bf16>(Z[c][qq]);
        }
        if (t < valid_of(n)) *reinterpret_cast<bf16x8*>(o + (tok_of(n) + t) * a.o_row) = ov;
      };
      sync();
      load(0);
      for (int n = 0; n < nc; ++n) {
        sync();
        if (n > 0) finish(n - 1);
        Frag<uint16_t> Sf[2][NKU];
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int ku = 0; ku < NKU; ++ku) Sf[c][ku].v = bS[n & 1][c][ku][lane];
        const float e = gates[n % 3].e[t];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          Z[c] = zero4();
#pragma unroll
          for (int ku = 0; ku < NKU; ++ku) mma(Z[c], Sf[c][ku], Q[ku]);
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {  // diag(e) Q S + d V
#pragma unroll
          for (int qq = 0; qq < 4; ++qq) Z[c][qq] = fmaf(skip, static_cast<float>(own[4 * c + qq]), e * Z[c][qq]);
#pragma unroll
          for (int ku = 0; ku < KO; ++ku) U[c][ku] = V[c][ku];
        }
        load(n + 1);
      }
      sync();
      if (nc > 0) finish(nc - 1);
    };
    using std::integral_constant;
    switch (role - S::kO) {
      case 0: o_role(integral_constant<int, 0>{}); break;
      case 1: o_role(integral_constant<int, 1>{}); break;
      case 2: o_role(integral_constant<int, 2>{}); break;
      default: o_role(integral_constant<int, 3>{}); break;
    }
  }
}

}  // namespace efla
