// ssm_api.hip -- the C entry points of the short causal convolution, of the
// selective state space scan and of the moves of state-pool rows
// (include/efla.h): validation, workspace sizing, launches on the caller's
// stream.  Nothing here allocates device memory or synchronizes.
#include <initializer_list>

#include "checks.h"
#include "launchers.h"

namespace {

constexpr int64_t kMaxRow = int64_t(1) << 24;  // elements from one token's row to the next

bool aligned_to(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

bool all_aligned_to(std::initializer_list<const void*> ptrs, size_t n) {
  for (const void* p : ptrs)
    if (!aligned_to(p, n)) return false;
  return true;
}

template <typename F>
efla_status by_type(efla_dtype dt, F&& f) {
  return from_hip(dt == EFLA_BF16 ? f(uint16_t{}) : f(float{}));
}

bool all_given(std::initializer_list<const void*> ptrs) {
  for (const void* p : ptrs)
    if (p == nullptr) return false;
  return true;
}

// ---------------------------------------------------------------- convolution
efla_status check_conv(int64_t N, int64_t L, int D, int W, int silu, efla_dtype dt, std::initializer_list<int64_t> rows) {
  if (N < 0 || L < 0 || D < 1 || !valid_dtype(dt) || (silu != 0 && silu != 1)) return EFLA_ERR_INVALID_ARG;
  if (W < 2 || W > 4 || D >= kMaxRow) return EFLA_ERR_UNSUPPORTED;
  for (int64_t r : rows) {
    if (r < D) return EFLA_ERR_INVALID_ARG;
    if (r >= kMaxRow) return EFLA_ERR_UNSUPPORTED;
  }
  return EFLA_OK;
}

bool conv_aligned(efla_dtype dt, std::initializer_list<const void*> ptrs) { return all_aligned_to(ptrs, elem_bytes(dt)); }

bool conv_fits(int64_t seqs, int64_t L, int64_t N, int D) {
  return L <= kMaxGrid && seqs * D <= kMaxGrid && N * int64_t(D) <= (int64_t(1) << 40) &&
         efla::conv_threads(seqs, L, N, D) <= efla::kMaxLaunchThreads;
}

// Whether an output written row by row, width bytes every out_row, shares a byte with
// rows of an input that other wavefronts still read.  Rows of one length may lie side
// by side in a wider tensor's; of two lengths only disjoint stretches are told apart,
// and the rest is the caller's to keep.
bool rows_meet(const void* out, int64_t out_row, const void* in, int64_t in_row, int64_t rows, int64_t width) {
  if (out == nullptr || in == nullptr || rows == 0) return false;
  const auto x = reinterpret_cast<uintptr_t>(out), y = reinterpret_cast<uintptr_t>(in);
  if (y < x ? x - y >= uint64_t((rows - 1) * in_row + width) : y - x >= uint64_t((rows - 1) * out_row + width)) return false;
  if (rows == 1) return true;
  if (out_row != in_row) return false;
  const int64_t by = int64_t(y < x ? x - y : y - x) % out_row;  // of one row of the later from the one before it
  return by < width || out_row - by < width;
}

bool conv_meet(efla_dtype dt, const void* out, int64_t out_row, const void* in, int64_t in_row, int64_t rows, int64_t D) {
  const auto e = int64_t(elem_bytes(dt));
  return rows_meet(out, out_row * e, in, in_row * e, rows, D * e);
}

// ---------------------------------------------------------------- scan
// Shapes of a scan over `seqs` sequences (dense: of L tokens each; packed: L in all).
efla_status check_ssm(int64_t seqs, int H, int Hk, int64_t L, int d_k, int d_v, efla_dtype dt) {
  if (seqs < 0 || H < 1 || Hk < 1 || L < 0 || !valid_dtype(dt) || H % Hk != 0) return EFLA_ERR_INVALID_ARG;
  if (!valid_dim(d_k) || !valid_dim(d_v)) return EFLA_ERR_UNSUPPORTED;
  if (int64_t(H) * d_v >= kMaxRow || int64_t(Hk) * d_k >= kMaxRow || L > kMaxGrid || seqs * H > kMaxGrid)
    return EFLA_ERR_UNSUPPORTED;
  return EFLA_OK;
}

struct Rows {
  int64_t row, width;
  bool wide;  // moved in 16-byte pieces
};
efla_status check_rows(efla_dtype dt, std::initializer_list<Rows> rows) {
  for (const Rows& r : rows) {
    if (r.row < r.width || (r.wide && r.row * int64_t(elem_bytes(dt)) % 16 != 0)) return EFLA_ERR_INVALID_ARG;
    if (r.row >= kMaxRow) return EFLA_ERR_UNSUPPORTED;
  }
  return EFLA_OK;
}

bool all_aligned16(std::initializer_list<const void*> ptrs) { return all_aligned_to(ptrs, 16); }
bool ssm_aligned(efla_dtype dt, std::initializer_list<const void*> elems, std::initializer_list<const void*> floats) {
  return all_aligned_to(elems, elem_bytes(dt)) && all_aligned_to(floats, sizeof(float));
}

bool ssm_chunked(int d_k, int d_v, efla_dtype dt) { return dt == EFLA_BF16 && efla::ssm_chunk_supported(d_k, d_v); }

// How the forward cuts its sequences: where sequences, heads and value blocks leave
// most compute units without work, long ones are cut into segments of whole chunks.  A
// first launch brings each segment's end state (from zero, the first's from s0) and its
// decay, the second folds those before it into each segment's own first state and runs
// all side by side.
// Measured (us, whole / cut into segments for 256 workgroups):
//   bf16, workgroups 4-16:  1 x 3500 4 heads d 64 53 / 19, 1 x 800 16.2 / 12.4, packed 2 in 12000 tokens 133 / 37
//   bf16, 64, 16 heads d 128: 1 x 2048 44 / 32, 1 x 512 15.4 / 16.1;  128: 2 x 4096 83 / 90;  1024: packed 16 in 16384 130 / 181
//   float32, 32-64:  2 x 777 8 heads d 64 52 / 35, 1 x 1200 4 heads d 128 110 / 57;  512: packed 4 in 3000 167 / 192
struct Segments {
  int64_t seg = 0, slots = 0;  // tokens a segment (0: not cut), segments a head
};
Segments ssm_segments(int64_t seqs, bool packed, int H, int64_t L, int d_k, int d_v, efla_dtype dt) {
  const bool chunked = ssm_chunked(d_k, d_v, dt);
  const int64_t chunk = chunked ? 64 : 32, wgs = seqs * H * (d_v / (chunked ? 32 : 16));
  if (wgs <= 0 || wgs > 64) return {};
  // segments of the longest sequence there may be: a packed batch may be one sequence and empty ones
  const int64_t chunks = (L + chunk - 1) / chunk, want = 256 / (packed ? wgs / seqs : wgs);
  const int64_t even = (chunks + want - 1) / want, per = even < 2 ? 2 : even;  // chunks a segment
  if (chunks < 2 * per + 6) return {};
  Segments r;
  r.seg = per * chunk;
  r.slots = packed ? L / r.seg + seqs : seqs * ((L + r.seg - 1) / r.seg);
  return r;
}

size_t ssm_fwd_workspace(const Segments& g, int H, int d_k, int d_v) {
  return al256(size_t(g.slots) * H * d_k * d_v * sizeof(float)) + al256(size_t(g.slots) * H * sizeof(float));
}

// Whether the forward's launches over these sequences have fewer threads than the
// runtime takes.
bool ssm_fwd_fits(int64_t seqs, bool packed, int H, int64_t L, int d_k, int d_v, efla_dtype dt) {
  const Segments g = ssm_segments(seqs, packed, H, L, d_k, d_v, dt);
  const int64_t units = g.seg > 0 ? g.slots : seqs;
  return (ssm_chunked(d_k, d_v, dt) ? efla::ssm_chunk_threads(units, H, d_v) : efla::ssm_f32_threads(units, H, d_v)) <=
         efla::kMaxLaunchThreads;
}

efla_status ssm_forward(efla::SsmFwd a, efla_dtype dt, void* workspace, hipStream_t s) {
  const Segments g = ssm_segments(a.N, a.cu != nullptr, a.H, a.L, a.DK, a.DV, dt);
  auto launch = [&](bool local) {
    if (ssm_chunked(a.DK, a.DV, dt)) return from_hip(efla::launch_ssm_chunk(a, local, s));
    return by_type(dt, [&](auto t) { return efla::launch_ssm_f32<decltype(t)>(a, local, s); });
  };
  if (g.seg > 0) {
    a.seg = g.seg;
    a.seg_slots = g.slots;
    a.seg_s = static_cast<float*>(workspace);
    a.seg_e = a.seg_s + al256(size_t(g.slots) * a.H * a.DK * a.DV * sizeof(float)) / sizeof(float);
    const efla_status st = launch(true);
    if (st != EFLA_OK) return st;
  }
  return launch(false);
}

bool ssm_bwd_chunked(int64_t L, int d_k, int d_v, efla_dtype dt) { return L > 0 && ssm_chunked(d_k, d_v, dt); }

bool ssm_bwd_fits(int B, int H, int64_t L, int d_k, int d_v, efla_dtype dt) {
  if (int64_t(B) * H * ((L + 31) / 32) > kMaxGrid) return false;
  return (ssm_bwd_chunked(L, d_k, d_v, dt) ? efla::ssm_bwd_chunk_threads(B, H, L, d_v)
                                           : efla::ssm_bwd_f32_threads(B, H, L, d_v)) <= efla::kMaxLaunchThreads;
}

}  // namespace

extern "C" {

efla_status efla_conv_fwd(const void* x, int64_t x_row, const void* w, const void* bias, const void* s0, void* y,
                          int64_t y_row, void* s_final, int B, int64_t L, int D, int W, int silu, efla_dtype dtype,
                          void* stream) {
  const efla_status st = check_conv(B, L, D, W, silu, dtype, {x_row, y_row});
  if (st != EFLA_OK) return st;
  if (B < 1) return EFLA_ERR_INVALID_ARG;
  if (!conv_fits(B, L, B, D)) return EFLA_ERR_UNSUPPORTED;
  if (L > 0 && !all_given({x, w, y})) return EFLA_ERR_INVALID_ARG;
  if (!conv_aligned(dtype, {x, w, bias, s0, y, s_final})) return EFLA_ERR_INVALID_ARG;
  if (conv_meet(dtype, y, y_row, x, x_row, B * L, D)) return EFLA_ERR_INVALID_ARG;
  if (L == 0 && s_final == nullptr) return EFLA_OK;
  const efla::ConvFwd a{x, w, bias, s0, y, s_final, nullptr, nullptr, x_row, y_row, B, B, D, W, silu, L};
  return by_type(dtype, [&](auto t) { return efla::launch_conv_fwd<decltype(t)>(a, static_cast<hipStream_t>(stream)); });
}

efla_status efla_conv_fwd_varlen(const void* x, int64_t x_row, const void* w, const void* bias,
                                 const int32_t* cu_seqlens, const int32_t* slots, int N, int P, const void* s0, void* y,
                                 int64_t y_row, void* s_final, int64_t T, int D, int W, int silu, efla_dtype dtype,
                                 void* stream) {
  const efla_status st = check_conv(N, T, D, W, silu, dtype, {x_row, y_row});
  if (st != EFLA_OK) return st;
  if (P < 0 || T > INT32_MAX || (slots == nullptr && P < N)) return EFLA_ERR_INVALID_ARG;
  if (!conv_fits(1, T, N, D)) return EFLA_ERR_UNSUPPORTED;
  if (N == 0) return EFLA_OK;
  if (cu_seqlens == nullptr || (T > 0 && !all_given({x, w, y}))) return EFLA_ERR_INVALID_ARG;
  if (!conv_aligned(dtype, {x, w, bias, s0, y, s_final})) return EFLA_ERR_INVALID_ARG;
  if (conv_meet(dtype, y, y_row, x, x_row, T, D)) return EFLA_ERR_INVALID_ARG;
  if (T == 0 && s_final == nullptr) return EFLA_OK;
  const efla::ConvFwd a{x, w, bias, s0, y, s_final, cu_seqlens, slots, x_row, y_row, N, P, D, W, silu, T};
  return by_type(dtype, [&](auto t) { return efla::launch_conv_fwd<decltype(t)>(a, static_cast<hipStream_t>(stream)); });
}

efla_status efla_conv_step(const void* x, int64_t x_row, const void* w, const void* bias, void* state,
                           const int32_t* slots, void* y, int64_t y_row, int N, int P, int D, int W, int silu,
                           efla_dtype dtype, void* stream) {
  const efla_status st = check_conv(N, 1, D, W, silu, dtype, {x_row, y_row});
  if (st != EFLA_OK) return st;
  if (P < 0 || (slots == nullptr && P < N)) return EFLA_ERR_INVALID_ARG;
  if (!conv_fits(1, 1, N, D)) return EFLA_ERR_UNSUPPORTED;
  if (N == 0 || P == 0) return EFLA_OK;
  if (!all_given({x, w, state, y}) || !conv_aligned(dtype, {x, w, bias, state, y})) return EFLA_ERR_INVALID_ARG;
  const efla::ConvStep a{x, w, bias, state, y, slots, x_row, y_row, N, P, D, W, silu};
  return by_type(dtype, [&](auto t) { return efla::launch_conv_step<decltype(t)>(a, static_cast<hipStream_t>(stream)); });
}

size_t efla_conv_bwd_workspace_size(int B, int64_t L, int D, int W) {
  if (B < 1 || check_conv(B, L, D, W, 0, EFLA_F32, {}) != EFLA_OK || !conv_fits(B, L, B, D) || L == 0) return 0;
  return efla::conv_bwd_workspace(B, L, D, W);
}

efla_status efla_conv_bwd(const void* x, int64_t x_row, const void* w, const void* bias, const void* s0, const void* dy,
                          int64_t dy_row, const void* ds_final, void* dx, int64_t dx_row, float* dw, float* dbias,
                          void* ds0, int B, int64_t L, int D, int W, int silu, efla_dtype dtype, void* workspace,
                          size_t workspace_bytes, void* stream) {
  const efla_status st = check_conv(B, L, D, W, silu, dtype, {x_row, dy_row, dx_row});
  if (st != EFLA_OK) return st;
  if (B < 1) return EFLA_ERR_INVALID_ARG;
  if (!conv_fits(B, L, B, D)) return EFLA_ERR_UNSUPPORTED;
  if (L == 0 && ds0 != nullptr && efla::conv_copy_threads(B, D, W) > efla::kMaxLaunchThreads) return EFLA_ERR_UNSUPPORTED;
  if (dw == nullptr || (L > 0 && !all_given({x, w, dy, dx}))) return EFLA_ERR_INVALID_ARG;
  if (!conv_aligned(dtype, {x, w, bias, s0, dy, ds_final, dx, ds0}) || !aligned_to(dw, 4) || !aligned_to(dbias, 4))
    return EFLA_ERR_INVALID_ARG;
  const size_t need = efla_conv_bwd_workspace_size(B, L, D, W);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return EFLA_ERR_WORKSPACE;
  if (need > 0 && !aligned16(workspace)) return EFLA_ERR_INVALID_ARG;
  const int64_t states = int64_t(W - 1) * D;
  if (conv_meet(dtype, dx, dx_row, x, x_row, B * L, D) || conv_meet(dtype, dx, dx_row, dy, dy_row, B * L, D) ||
      (L > 0 && (conv_meet(dtype, ds0, states, ds_final, states, B, states) || conv_meet(dtype, ds0, states, s0, states, B, states))))
    return EFLA_ERR_INVALID_ARG;
  const efla::ConvBwd a{x, w, bias, s0, dy, ds_final, dx, ds0, dw, dbias, x_row, dy_row, dx_row, B, D, W, silu, L};
  return by_type(dtype, [&](auto t) {
    return efla::launch_conv_bwd<decltype(t)>(a, static_cast<float*>(workspace), static_cast<hipStream_t>(stream));
  });
}

size_t efla_ssm_fwd_workspace_size(int B, int H, int Hk, int64_t L, int d_k, int d_v, efla_dtype dtype) {
  if (B < 1 || check_ssm(B, H, Hk, L, d_k, d_v, dtype) != EFLA_OK) return 0;
  return ssm_fwd_workspace(ssm_segments(B, false, H, L, d_k, d_v, dtype), H, d_k, d_v);
}

efla_status efla_ssm_fwd(const void* q, int64_t q_row, const void* k, int64_t k_row, const void* v, int64_t v_row,
                         const void* dt, int64_t dt_row, const float* a, const float* d, const float* dt_bias,
                         const float* s0, void* o, int64_t o_row, float* s_final, int B, int H, int Hk, int64_t L,
                         int d_k, int d_v, efla_dtype dtype, void* workspace, size_t workspace_bytes, void* stream) {
  efla_status st = check_ssm(B, H, Hk, L, d_k, d_v, dtype);
  if (st != EFLA_OK) return st;
  if (B < 1) return EFLA_ERR_INVALID_ARG;
  const int64_t kw = int64_t(Hk) * d_k, vw = int64_t(H) * d_v;
  st = check_rows(dtype, {{q_row, kw, true}, {k_row, kw, true}, {v_row, vw, true}, {dt_row, H, false}, {o_row, vw, true}});
  if (st != EFLA_OK) return st;
  if (!ssm_fwd_fits(B, false, H, L, d_k, d_v, dtype)) return EFLA_ERR_UNSUPPORTED;
  if (a == nullptr || (L > 0 && !all_given({q, k, v, dt, o}))) return EFLA_ERR_INVALID_ARG;
  if (!all_aligned16({q, k, v, o, s0, s_final}) || !ssm_aligned(dtype, {dt}, {a, d, dt_bias})) return EFLA_ERR_INVALID_ARG;
  const size_t need = efla_ssm_fwd_workspace_size(B, H, Hk, L, d_k, d_v, dtype);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return EFLA_ERR_WORKSPACE;
  if (need > 0 && !aligned16(workspace)) return EFLA_ERR_INVALID_ARG;
  if (L == 0 && s_final == nullptr) return EFLA_OK;
  const efla::SsmFwd x{q,     k,     v,     dt,     a,     d, dt_bias, s0, o,  s_final, nullptr, nullptr, nullptr,
                       q_row, k_row, v_row, dt_row, o_row, B, B,       H,  Hk, d_k,     d_v,     L};
  return ssm_forward(x, dtype, workspace, static_cast<hipStream_t>(stream));
}

size_t efla_ssm_fwd_varlen_workspace_size(int N, int H, int Hk, int64_t T, int d_k, int d_v, efla_dtype dtype) {
  if (check_ssm(N, H, Hk, T, d_k, d_v, dtype) != EFLA_OK) return 0;
  return ssm_fwd_workspace(ssm_segments(N, true, H, T, d_k, d_v, dtype), H, d_k, d_v);
}

efla_status efla_ssm_fwd_varlen(const void* q, int64_t q_row, const void* k, int64_t k_row, const void* v, int64_t v_row,
                                const void* dt, int64_t dt_row, const float* a, const float* d, const float* dt_bias,
                                const int32_t* cu_seqlens, const int32_t* slots, const int32_t* order, int N, int P,
                                const float* s0, void* o, int64_t o_row, float* s_final, int H, int Hk, int64_t T,
                                int d_k, int d_v, efla_dtype dtype, void* workspace, size_t workspace_bytes,
                                void* stream) {
  efla_status st = check_ssm(N, H, Hk, T, d_k, d_v, dtype);
  if (st != EFLA_OK) return st;
  if (P < 0 || T > INT32_MAX || (slots == nullptr && P < N)) return EFLA_ERR_INVALID_ARG;
  const int64_t kw = int64_t(Hk) * d_k, vw = int64_t(H) * d_v;
  st = check_rows(dtype, {{q_row, kw, true}, {k_row, kw, true}, {v_row, vw, true}, {dt_row, H, false}, {o_row, vw, true}});
  if (st != EFLA_OK) return st;
  if (!ssm_fwd_fits(N, true, H, T, d_k, d_v, dtype)) return EFLA_ERR_UNSUPPORTED;
  if (N == 0) return EFLA_OK;
  if (a == nullptr || cu_seqlens == nullptr || (T > 0 && !all_given({q, k, v, dt, o}))) return EFLA_ERR_INVALID_ARG;
  if (!all_aligned16({q, k, v, o, s0, s_final}) || !ssm_aligned(dtype, {dt}, {a, d, dt_bias})) return EFLA_ERR_INVALID_ARG;
  const size_t need = efla_ssm_fwd_varlen_workspace_size(N, H, Hk, T, d_k, d_v, dtype);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return EFLA_ERR_WORKSPACE;
  if (need > 0 && !aligned16(workspace)) return EFLA_ERR_INVALID_ARG;
  if (T == 0 && s_final == nullptr) return EFLA_OK;
  const efla::SsmFwd x{q,     k,     v,     dt,     a,     d, dt_bias, s0, o,  s_final, cu_seqlens, slots, order,
                       q_row, k_row, v_row, dt_row, o_row, N, P,       H,  Hk, d_k,     d_v,        T};
  return ssm_forward(x, dtype, workspace, static_cast<hipStream_t>(stream));
}

efla_status efla_ssm_step(const void* q, int64_t q_row, const void* k, int64_t k_row, const void* v, int64_t v_row,
                          const void* dt, int64_t dt_row, const float* a, const float* d, const float* dt_bias,
                          float* state, const int32_t* slots, void* o, int64_t o_row, int N, int P, int H, int Hk,
                          int d_k, int d_v, efla_dtype dtype, void* stream) {
  efla_status st = check_ssm(N, H, Hk, 1, d_k, d_v, dtype);
  if (st != EFLA_OK) return st;
  if (P < 0 || (slots == nullptr && P < N)) return EFLA_ERR_INVALID_ARG;
  const int64_t kw = int64_t(Hk) * d_k, vw = int64_t(H) * d_v;
  st = check_rows(dtype, {{q_row, kw, false}, {k_row, kw, false}, {v_row, vw, false}, {dt_row, H, false}, {o_row, vw, false}});
  if (st != EFLA_OK) return st;
  if (efla::ssm_step_threads(N, H, d_v) > efla::kMaxLaunchThreads) return EFLA_ERR_UNSUPPORTED;
  if (N == 0 || P == 0) return EFLA_OK;
  if (!all_given({q, k, v, dt, a, state, o}) || !aligned16(state)) return EFLA_ERR_INVALID_ARG;
  if (!ssm_aligned(dtype, {q, k, v, dt, o}, {a, d, dt_bias})) return EFLA_ERR_INVALID_ARG;
  const efla::SsmStep x{q, k, v, dt, a, d, dt_bias, state, slots, o, q_row, k_row, v_row, dt_row, o_row, N, P, H, Hk, d_k, d_v};
  return by_type(dtype, [&](auto t) { return efla::launch_ssm_step<decltype(t)>(x, static_cast<hipStream_t>(stream)); });
}

size_t efla_ssm_bwd_workspace_size(int B, int H, int Hk, int64_t L, int d_k, int d_v, efla_dtype dtype) {
  if (B < 1 || check_ssm(B, H, Hk, L, d_k, d_v, dtype) != EFLA_OK || L == 0 || !ssm_bwd_fits(B, H, L, d_k, d_v, dtype)) return 0;
  return ssm_bwd_chunked(L, d_k, d_v, dtype) ? efla::ssm_bwd_chunk_workspace(B, H, L, d_k, d_v)
                                             : efla::ssm_bwd_f32_workspace(B, H, L, d_k, d_v);
}

efla_status efla_ssm_bwd(const void* q, int64_t q_row, const void* k, int64_t k_row, const void* v, int64_t v_row,
                         const void* dt, int64_t dt_row, const float* a, const float* d, const float* dt_bias,
                         const float* s0, const void* d_o, int64_t do_row, const float* ds_final, void* dq,
                         int64_t dq_row, void* dk, int64_t dk_row, void* dv, int64_t dv_row, void* ddt, int64_t ddt_row,
                         float* da, float* dd, float* dbias, float* ds0, int B, int H, int Hk, int64_t L, int d_k,
                         int d_v, efla_dtype dtype, void* workspace, size_t workspace_bytes, void* stream) {
  efla_status st = check_ssm(B, H, Hk, L, d_k, d_v, dtype);
  if (st != EFLA_OK) return st;
  if (B < 1) return EFLA_ERR_INVALID_ARG;
  const int64_t kw = int64_t(Hk) * d_k, vw = int64_t(H) * d_v;
  st = check_rows(dtype, {{q_row, kw, true}, {k_row, kw, true}, {v_row, vw, true}, {dt_row, H, false}, {do_row, vw, true},
                          {dq_row, kw, true}, {dk_row, kw, true}, {dv_row, vw, true}, {ddt_row, H, false}});
  if (st != EFLA_OK) return st;
  if (!ssm_bwd_fits(B, H, L, d_k, d_v, dtype)) return EFLA_ERR_UNSUPPORTED;
  if (a == nullptr || (L > 0 && !all_given({q, k, v, dt, d_o, dq, dk, dv, ddt}))) return EFLA_ERR_INVALID_ARG;
  if (!all_aligned16({q, k, v, d_o, dq, dk, dv, s0, ds_final, ds0}) ||
      !ssm_aligned(dtype, {dt, ddt}, {a, d, dt_bias, da, dd, dbias}))
    return EFLA_ERR_INVALID_ARG;
  const size_t need = efla_ssm_bwd_workspace_size(B, H, Hk, L, d_k, d_v, dtype);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return EFLA_ERR_WORKSPACE;
  if (need > 0 && !aligned16(workspace)) return EFLA_ERR_INVALID_ARG;
  const efla::SsmBwd x{q,     k,     v,      dt,     d_o,    a,      d,      dt_bias, s0,      ds_final, dq, dk, dv, ddt, da,
                       dd,    dbias, ds0,    q_row,  k_row,  v_row,  dt_row, do_row,  dq_row,  dk_row,   dv_row, ddt_row,
                       B,     H,     Hk,     d_k,    d_v,    L};
  if (ssm_bwd_chunked(L, d_k, d_v, dtype)) return from_hip(efla::launch_ssm_bwd_chunk(x, workspace, static_cast<hipStream_t>(stream)));
  return by_type(dtype, [&](auto t) {
    return efla::launch_ssm_bwd_f32<decltype(t)>(x, workspace, static_cast<hipStream_t>(stream));
  });
}

}  // extern "C"

namespace {

efla_status check_pools(void* const* pools, const size_t* row_bytes, int count, int N, int P) {
  if (count < 0 || N < 0 || P < 0 || (count > 0 && (pools == nullptr || row_bytes == nullptr))) return EFLA_ERR_INVALID_ARG;
  for (int i = 0; i < count; ++i) {
    if (pools[i] == nullptr || row_bytes[i] == 0 || row_bytes[i] % 2 != 0 || !aligned_to(pools[i], 2))
      return EFLA_ERR_INVALID_ARG;
    if (row_bytes[i] > (size_t(1) << 40)) return EFLA_ERR_UNSUPPORTED;
  }
  for (int i = 0; i < count; i += efla::kPoolsPerLaunch) {
    int64_t pieces = 0;
    for (int j = i; j < count && j < i + efla::kPoolsPerLaunch; ++j) pieces += efla::pool_pieces(row_bytes[j]);
    if (pieces > kMaxGrid || pieces * N * efla::kThreads > efla::kMaxLaunchThreads) return EFLA_ERR_UNSUPPORTED;
  }
  return EFLA_OK;
}

efla_status copy_rows(void* const* pools, const size_t* row_bytes, int count, const int32_t* src, const int32_t* dst, int N,
                      int P, bool share, hipStream_t s) {
  for (int i = 0; i < count; i += efla::kPoolsPerLaunch) {
    efla::PoolSet set{};
    set.count = count - i < efla::kPoolsPerLaunch ? count - i : efla::kPoolsPerLaunch;
    for (int j = 0; j < set.count; ++j) {
      set.base[j] = pools[i + j];
      set.bytes[j] = row_bytes[i + j];
      set.first[j + 1] = set.first[j] + uint32_t(efla::pool_pieces(row_bytes[i + j]));
    }
    const efla_status st = from_hip(efla::launch_pool_copy(set, src, dst, N, P, share, s));
    if (st != EFLA_OK) return st;
  }
  return EFLA_OK;
}

}  // namespace

extern "C" {

efla_status efla_pool_copy(void* const* pools, const size_t* row_bytes, int count, const int32_t* src, const int32_t* dst,
                           int N, int P, void* stream) {
  const efla_status st = check_pools(pools, row_bytes, count, N, P);
  if (st != EFLA_OK) return st;
  if (N == 0 || P == 0 || count == 0) return EFLA_OK;
  if (!all_given({src, dst})) return EFLA_ERR_INVALID_ARG;
  return copy_rows(pools, row_bytes, count, src, dst, N, P, true, static_cast<hipStream_t>(stream));
}

size_t efla_pool_compact_workspace_size(int N) { return N > 0 ? 8 * size_t(N) : 0; }

efla_status efla_pool_compact(void* const* pools, const size_t* row_bytes, int count, const int32_t* slots, int N, int P,
                              int32_t* new_slots, int32_t* live, void* workspace, size_t workspace_bytes, void* stream) {
  const efla_status st = check_pools(pools, row_bytes, count, N, P);
  if (st != EFLA_OK) return st;
  if (P > efla::kMaxCompactRows) return EFLA_ERR_UNSUPPORTED;
  if (live == nullptr || (N > 0 && !all_given({slots, new_slots}))) return EFLA_ERR_INVALID_ARG;
  const size_t need = efla_pool_compact_workspace_size(N);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return EFLA_ERR_WORKSPACE;
  if (need > 0 && !aligned16(workspace)) return EFLA_ERR_INVALID_ARG;
  auto* src = static_cast<int32_t*>(workspace);
  int32_t* dst = src + N;
  const auto s = static_cast<hipStream_t>(stream);
  const efla_status plan = from_hip(efla::launch_pool_plan(slots, N, P, new_slots, live, src, dst, s));
  if (plan != EFLA_OK || N == 0 || P == 0) return plan;
  return copy_rows(pools, row_bytes, count, src, dst, N, P, false, s);
}

}  // extern "C"
