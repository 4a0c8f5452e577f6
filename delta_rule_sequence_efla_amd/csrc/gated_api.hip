// gated_api.hip -- the C entry points of the gated delta rule and of the plan
// of a packed batch (include/efla.h): validation, workspace sizing, launches on
// the caller's stream.  Nothing here allocates device memory or synchronizes.
#include "checks.h"
#include "launchers.h"

namespace {

// Shapes of a gated call over `units` sequences of `L` tokens.
efla_status check_gated_shape(int B, int H, int Hk, int64_t L, int d_k, int d_v, int chunk, efla_dtype dt,
                              efla_rule rule) {
  if (!valid_rule(rule) || Hk < 1) return EFLA_ERR_INVALID_ARG;
  const efla_status st = check_chunk_shape(B, H, L, d_k, d_v, chunk, dt);
  if (st != EFLA_OK) return st;
  return H % Hk == 0 ? EFLA_OK : EFLA_ERR_INVALID_ARG;
}

// Which forward kernels run over `seqs` sequences of at most L tokens: the
// chunked matrix-core passes for bf16 at their shapes (whatever chunk the caller
// names: it does not change the result), else the fp32 recurrence.  The latter
// also where it is the faster of the two, short sequences and few workgroups:
// one launch against two, but a longer chain.  Measured (bf16, us, chunks /
// recurrence; workgroups = seqs H d_v / 16):
//   d 64,  32 .. 256 workgroups: L 48 13.0 / 7.9, 128 14.3 / 12.5, 160 15.2 / 14.7, 192 15.3 / 16.5
//   d 64,        512:            L 16 13.6 / 7.2, 48 14.0 / 12.8, 64 14.3 / 15.7
//   d 128, 64 .. 256:            L 48 14.0 / 9.3, 96 15.8 / 13.4, 128 16.0 / 16.3
//   d 128,       512:            L 16 14.0 / 10.4, 32 14.3 / 14.3, 48 14.8 / 18.8
//   d 128,      1024:            L 8 19.1 / 15.6, 16 19.2 / 19.2, 32 19.6 / 27.4
// Packed batches give T for L: the lengths are on the device, and T is the only
// bound on the longest of them, which sets the recurrence's time.  Measured
// (sequences x tokens, same units):
//   d 64, 8 heads:   16 x 128 16.8 / 26.6, 300 and 15 x 1 19.3 / 35.1, 600, 2, 3, 4 24.0 / 38.5
//                    but 64 x 8 29.5 / 18.7, 200 x 1 73.6 / 44.3, 256 x 4 91.9 / 61.0
//   d 128, 16 heads: 4 x 100 17.9 / 32.2, 64 x 8 88.9 / 106, 200 x 1 260 / 289, 600, 2, 3, 4 30.1 / 93.6
// so batches of many short requests at d 64 are where it takes the slower one.
bool gated_chunked(int64_t seqs, int H, int64_t L, int d_k, int d_v, efla_dtype dt) {
  if (dt != EFLA_BF16 || !efla::gated_chunk_supported(d_k, d_v)) return false;
  const int64_t wgs = seqs * H * (d_v / 16);
  if (wgs <= 256) return L > (d_k == 64 ? 176 : 112);
  return L > 48 || wgs > 4096 || L * wgs * d_k > 2000000;
}

// Whether the forward's largest launch over these sequences has fewer threads than
// the runtime takes (seqs > 0; L = 0 launches the recurrence, which copies states).
bool gated_fwd_fits(int64_t seqs, int H, int64_t L, bool packed, int d_k, int d_v, efla_dtype dt) {
  return (L > 0 && gated_chunked(seqs, H, L, d_k, d_v, dt) ? efla::gated_chunk_threads(seqs, H, L, packed, d_k, d_v)
                                                           : efla::gated_recurrent_threads(seqs, H, L, packed, d_k, d_v)) <=
         efla::kMaxLaunchThreads;
}

// Shapes of a gated call over N sequences packed into T tokens: what bounds it is
// the workgroups of the recurrence and the chunk slots of the whole batch (gated_fwd.hip:
// T / 64 + N a head), not N sequences of T tokens each, and not the chunk named.
efla_status check_gated_packed(int N, int H, int Hk, int64_t T, int d_k, int d_v, int chunk, efla_dtype dt,
                               efla_rule rule) {
  if (!valid_rule(rule) || !valid_dtype(dt) || N < 0 || T < 0 || T > INT32_MAX || H < 1 || Hk < 1)
    return EFLA_ERR_INVALID_ARG;
  if (!valid_dim(d_k) || !valid_dim(d_v) || !valid_chunk(chunk)) return EFLA_ERR_UNSUPPORTED;
  if (int64_t(N) * H * (d_v / 16) > kMaxGrid || int64_t(H) * (T / 64 + N) > kMaxGrid) return EFLA_ERR_UNSUPPORTED;
  if (N > 0 && !gated_fwd_fits(N, H, T, true, d_k, d_v, dt)) return EFLA_ERR_UNSUPPORTED;
  return H % Hk == 0 ? EFLA_OK : EFLA_ERR_INVALID_ARG;
}

template <typename F>
efla_status by_type(efla_dtype dt, F&& f) {
  return from_hip(dt == EFLA_BF16 ? f(uint16_t{}) : f(float{}));
}

efla_status gated_forward(const efla::GatedFwd& a, int chunk, efla_dtype dt, void* workspace, hipStream_t s) {
  if (a.L > 0 && gated_chunked(a.cu == nullptr ? a.B : a.N, a.H, a.L, a.DK, a.DV, dt)) return from_hip(efla::launch_gated_chunk(a, workspace, s));
  return by_type(dt, [&](auto t) { return efla::launch_gated_recurrent<decltype(t)>(a, nullptr, chunk, s); });
}

}  // namespace

extern "C" {

size_t efla_gated_chunk_fwd_workspace_size(int B, int H, int Hk, int64_t L, int d_k, int d_v, int chunk,
                                           efla_dtype dtype) {
  if (check_gated_shape(B, H, Hk, L, d_k, d_v, chunk, dtype, EFLA_RULE_EXACT) != EFLA_OK || L == 0) return 0;
  if (!gated_fwd_fits(B, H, L, false, d_k, d_v, dtype)) return 0;
  return gated_chunked(B, H, L, d_k, d_v, dtype) ? efla::gated_fwd_layout(B, 0, H, L, false).total : 0;
}

efla_status efla_gated_chunk_fwd(const void* q, const void* k, const void* v, const void* beta, const float* g,
                                 const float* s0, void* o, float* s_final, int B, int H, int Hk, int64_t L, int d_k,
                                 int d_v, int chunk, efla_dtype dtype, efla_rule rule, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  const efla_status st = check_gated_shape(B, H, Hk, L, d_k, d_v, chunk, dtype, rule);
  if (st != EFLA_OK) return st;
  if (!gated_fwd_fits(B, H, L, false, d_k, d_v, dtype)) return EFLA_ERR_UNSUPPORTED;
  if (L > 0) {
    if (q == nullptr || k == nullptr || v == nullptr || beta == nullptr || g == nullptr || o == nullptr)
      return EFLA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o)) return EFLA_ERR_INVALID_ARG;
  }
  const size_t need = efla_gated_chunk_fwd_workspace_size(B, H, Hk, L, d_k, d_v, chunk, dtype);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return EFLA_ERR_WORKSPACE;
  if (need > 0 && !aligned16(workspace)) return EFLA_ERR_INVALID_ARG;
  if (L == 0 && s_final == nullptr) return EFLA_OK;
  const efla::GatedFwd a{q,       k,       v,       beta, g, s0, o,  s_final, nullptr,   nullptr,
                         nullptr, B,       0,       B,    H, Hk, d_k, d_v,     int(rule), L};
  return gated_forward(a, chunk, dtype, workspace, static_cast<hipStream_t>(stream));
}

size_t efla_gated_chunk_fwd_varlen_workspace_size(int N, int H, int Hk, int64_t T, int d_k, int d_v, int chunk,
                                                  efla_dtype dtype) {
  if (check_gated_packed(N, H, Hk, T, d_k, d_v, chunk, dtype, EFLA_RULE_EXACT) != EFLA_OK || N == 0 || T == 0) return 0;
  return gated_chunked(N, H, T, d_k, d_v, dtype) ? efla::gated_fwd_layout(0, N, H, T, true).total : 0;
}

efla_status efla_gated_chunk_fwd_varlen(const void* q, const void* k, const void* v, const void* beta, const float* g,
                                        const int32_t* cu_seqlens, const int32_t* slots, const int32_t* order, int N,
                                        int P, const float* s0, void* o, float* s_final, int H, int Hk, int64_t T,
                                        int d_k, int d_v, int chunk, efla_dtype dtype, efla_rule rule,
                                        void* workspace, size_t workspace_bytes, void* stream) {
  if (P < 0) return EFLA_ERR_INVALID_ARG;
  const efla_status st = check_gated_packed(N, H, Hk, T, d_k, d_v, chunk, dtype, rule);
  if (st != EFLA_OK) return st;
  if (slots == nullptr && P < N) return EFLA_ERR_INVALID_ARG;
  if (N == 0) return EFLA_OK;
  if (cu_seqlens == nullptr) return EFLA_ERR_INVALID_ARG;
  if (T > 0) {
    if (q == nullptr || k == nullptr || v == nullptr || beta == nullptr || g == nullptr || o == nullptr)
      return EFLA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o)) return EFLA_ERR_INVALID_ARG;
  }
  const size_t need = efla_gated_chunk_fwd_varlen_workspace_size(N, H, Hk, T, d_k, d_v, chunk, dtype);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return EFLA_ERR_WORKSPACE;
  if (need > 0 && !aligned16(workspace)) return EFLA_ERR_INVALID_ARG;
  if (T == 0 && s_final == nullptr) return EFLA_OK;
  const efla::GatedFwd a{q,     k, v, beta, g, s0, o,   s_final, cu_seqlens, slots,
                         order, 0, N, P,    H, Hk, d_k, d_v,     int(rule),  T};
  return gated_forward(a, chunk, dtype, workspace, static_cast<hipStream_t>(stream));
}

size_t efla_gated_chunk_bwd_workspace_size(int B, int H, int Hk, int64_t L, int d_k, int d_v, int chunk,
                                           efla_dtype dtype) {
  if (check_gated_shape(B, H, Hk, L, d_k, d_v, chunk, dtype, EFLA_RULE_EXACT) != EFLA_OK || L == 0) return 0;
  if (efla::gated_bwd_threads(B, H, Hk, L, d_k, d_v, elem_bytes(dtype)) > efla::kMaxLaunchThreads) return 0;
  return efla::gated_bwd_workspace(B, H, Hk, L, d_k, d_v, elem_bytes(dtype));
}

efla_status efla_gated_chunk_bwd(const void* q, const void* k, const void* v, const void* beta, const float* g,
                                 const float* s0, const void* d_o, const float* ds_final, void* dq, void* dk, void* dv,
                                 void* dbeta, void* dg, float* ds0, int B, int H, int Hk, int64_t L, int d_k, int d_v,
                                 int chunk, efla_dtype dtype, efla_rule rule, void* workspace, size_t workspace_bytes,
                                 void* stream) {
  return efla_gated_chunk_bwd_typed(q, k, v, beta, g, s0, d_o, ds_final, dq, dk, dv, dbeta, dg, ds0, B, H, Hk, L, d_k,
                                    d_v, chunk, dtype, dtype, rule, workspace, workspace_bytes, stream);
}

efla_status efla_gated_chunk_bwd_typed(const void* q, const void* k, const void* v, const void* beta, const float* g,
                                       const float* s0, const void* d_o, const float* ds_final, void* dq, void* dk,
                                       void* dv, void* dbeta, void* dg, float* ds0, int B, int H, int Hk, int64_t L,
                                       int d_k, int d_v, int chunk, efla_dtype dtype, efla_dtype dg_dtype,
                                       efla_rule rule, void* workspace, size_t workspace_bytes, void* stream) {
  const efla_status st = check_gated_shape(B, H, Hk, L, d_k, d_v, chunk, dtype, rule);
  if (st != EFLA_OK) return st;
  if (dg_dtype != dtype && dg_dtype != EFLA_F32) return EFLA_ERR_INVALID_ARG;
  if (efla::gated_bwd_threads(B, H, Hk, L, d_k, d_v, elem_bytes(dtype)) > efla::kMaxLaunchThreads)
    return EFLA_ERR_UNSUPPORTED;
  if (L == 0 && ds0 == nullptr) return EFLA_OK;
  if (L > 0) {
    if (q == nullptr || k == nullptr || v == nullptr || beta == nullptr || g == nullptr || d_o == nullptr ||
        dq == nullptr || dk == nullptr || dv == nullptr || dbeta == nullptr || dg == nullptr)
      return EFLA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(d_o) || !aligned16(dq) || !aligned16(dk) ||
        !aligned16(dv))
      return EFLA_ERR_INVALID_ARG;
    const size_t need = efla_gated_chunk_bwd_workspace_size(B, H, Hk, L, d_k, d_v, chunk, dtype);
    if (workspace == nullptr || workspace_bytes < need) return EFLA_ERR_WORKSPACE;
    if (!aligned16(workspace)) return EFLA_ERR_INVALID_ARG;
  }
  const efla::GatedBwd b{q, k, v, beta, d_o, g, s0, ds_final, dq, dk, dv, dbeta, dg, ds0, B, H, Hk, d_k, d_v,
                         int(rule), L, dg_dtype == EFLA_F32 ? 1 : 0};
  return by_type(dtype, [&](auto t) {
    return efla::launch_gated_bwd<decltype(t)>(b, workspace, static_cast<hipStream_t>(stream));
  });
}

efla_status efla_gated_step(const void* q, const void* k, const void* v, const void* beta, const float* g,
                            float* state, const int32_t* slots, void* o, int N, int P, int H, int Hk, int d_k, int d_v,
                            efla_dtype dtype, efla_rule rule, void* stream) {
  if (!valid_rule(rule) || !valid_dtype(dtype) || N < 0 || P < 0 || H < 1 || Hk < 1 || H % Hk != 0)
    return EFLA_ERR_INVALID_ARG;
  if (!valid_dim(d_k) || !valid_dim(d_v) || int64_t(N) * H * (d_v / 16) > kMaxGrid ||
      efla::gated_step_threads(N, H, d_v) > efla::kMaxLaunchThreads)
    return EFLA_ERR_UNSUPPORTED;
  if (slots == nullptr && P < N) return EFLA_ERR_INVALID_ARG;
  if (N == 0 || P == 0) return EFLA_OK;
  if (q == nullptr || k == nullptr || v == nullptr || beta == nullptr || g == nullptr || state == nullptr ||
      o == nullptr)
    return EFLA_ERR_INVALID_ARG;
  if (!aligned16(state)) return EFLA_ERR_INVALID_ARG;
  const efla::GatedStep a{q, k, v, beta, g, state, slots, o, N, P, H, Hk, d_k, d_v, int(rule)};
  return by_type(dtype,
                 [&](auto t) { return efla::launch_gated_step<decltype(t)>(a, static_cast<hipStream_t>(stream)); });
}

efla_status efla_pack_plan(const int32_t* lengths, const int32_t* starts, int N, int64_t T, int chunk,
                           int32_t* cu_seqlens, int32_t* order, int32_t* token_seq, int32_t* token_pos, void* stream) {
  if (N < 0 || T < 0 || T > INT32_MAX || cu_seqlens == nullptr || (N > 0 && lengths == nullptr))
    return EFLA_ERR_INVALID_ARG;
  if (!valid_chunk(chunk)) return EFLA_ERR_UNSUPPORTED;
  return from_hip(efla::launch_plan(lengths, starts, N, int(T), chunk, cu_seqlens, order, token_seq, token_pos,
                                    static_cast<hipStream_t>(stream)));
}

}  // extern "C"
