// conv.hip -- the short causal convolution of a layer's projections: depthwise
// over the last W = 2, 3 or 4 tokens, with bias and SiLU, its gradient, and its
// form for one token a request.
//
//     u_t = bias + sum_{i < W} w_i x_{t-W+1+i},   y_t = u_t / (1 + e^{-u_t})
//
// per channel; the W - 1 inputs before the first token are the state.  All
// arithmetic is float32.  Every form reads each input and writes each output
// about once and is bound by that.
//
// A wavefront owns 64 vectors of channels (16 bytes a lane; one element a lane
// where the rows do not allow it) and a run of tokens, over which it slides the
// last W inputs in registers.
#include <type_traits>

#include "gated.h"
#include "launchers.h"

namespace efla {

template <typename T, int V>
struct alignas(V * sizeof(T) < 16 ? V * sizeof(T) : 16) ConvVec {
  T e[V];
};

// 1 / (1 + e^{-u}): e^{-u} overflows to infinity, whose reciprocal is zero.
__device__ __forceinline__ float sigmoid(float u) { return __builtin_amdgcn_rcpf(1.0f + __expf(-u)); }

template <typename T, int V, int W>
struct ConvTaps {
  float w[W][V], bias[V];
  // Channels ch .. ch + V - 1 of w [D, W] and bias [D].
  __device__ __forceinline__ void load(const T* __restrict__ wt, const T* __restrict__ bs, int64_t ch) {
    const ConvVec<T, V>* src = reinterpret_cast<const ConvVec<T, V>*>(wt + ch * W);
    T flat[W * V];
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const ConvVec<T, V> x = src[i];
#pragma unroll
      for (int e = 0; e < V; ++e) flat[i * V + e] = x.e[e];
    }
#pragma unroll
    for (int e = 0; e < V; ++e)
#pragma unroll
      for (int i = 0; i < W; ++i) w[i][e] = to_f32(flat[e * W + i]);
    ConvVec<T, V> b;
    if (bs != nullptr) b = *reinterpret_cast<const ConvVec<T, V>*>(bs + ch);
#pragma unroll
    for (int e = 0; e < V; ++e) bias[e] = bs != nullptr ? to_f32(b.e[e]) : 0.0f;
  }
  // u of a window of W inputs, oldest first.
  __device__ __forceinline__ float dot(const float (&x)[W][V], int e) const {
    float u = bias[e];
#pragma unroll
    for (int i = 0; i < W; ++i) u = fmaf(w[i][e], x[i][e], u);
    return u;
  }
};

template <typename T, int V, int W>
__device__ __forceinline__ void conv_push(float (&x)[W][V], const ConvVec<T, V>& in) {
#pragma unroll
  for (int i = 0; i + 1 < W; ++i)
#pragma unroll
    for (int e = 0; e < V; ++e) x[i][e] = x[i + 1][e];
#pragma unroll
  for (int e = 0; e < V; ++e) x[W - 1][e] = to_f32(in.e[e]);
}

template <typename T, int V, int W>
__device__ __forceinline__ ConvVec<T, V> conv_out(const ConvTaps<T, V, W>& taps, const float (&x)[W][V], int silu) {
  ConvVec<T, V> y;
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const float u = taps.dot(x, e);
    y.e[e] = from_f32<T>(silu ? u * sigmoid(u) : u);
  }
  return y;
}

template <typename T, int V>
__device__ __forceinline__ ConvVec<T, V> conv_zero() {
  ConvVec<T, V> z;
#pragma unroll
  for (int e = 0; e < V; ++e) z.e[e] = T(0);
  return z;
}

// The last sequence that starts at or before row t (offsets clamped into [0, T]),
// by all lanes: a step of the search tests 64 sequences.
__device__ __forceinline__ int conv_seq_of(const int32_t* __restrict__ cu, int N, int64_t T, int64_t t, int lane) {
  int lo = 0, left = N;
  while (left > 1) {
    const int step = (left + kWave - 1) / kWave;
    const int64_t u = int64_t(lane) * step;
    const bool before = u < left && clamp_offset(cu[lo + u], 0, T) <= t;
    const int cnt = __popcll(__ballot(before));
    const int at = cnt > 1 ? (cnt - 1) * step : 0;
    lo += at;
    left = left - at < step ? left - at : step;
  }
  return __builtin_amdgcn_readfirstlane(lo);
}

constexpr int kConvGroup = 4;  // rows asked for at once

// Forward.  The first W - 1 tokens of a sequence and its final state belong to
// one wavefront a sequence and channel block (the launch's first workgroups),
// which alone reads and writes states: so the final state may take the place of
// the initial one.  All other tokens see inputs only and are cut into runs of
// `run` rows wherever the sequences lie; a row that is not such a token is
// passed over.
template <typename T, int V, int W>
__global__ __launch_bounds__(kThreads) void conv_fwd_kernel(ConvFwd a, int blocks, int seq_wgs, int run) {
  const int lane = threadIdx.x & 63, w = wave_id();
  const bool packed = a.cu != nullptr;
  if (int(blockIdx.x) < seq_wgs) {
    const int64_t job = int64_t(blockIdx.x) * 4 + w;
    const int64_t seq = job / blocks;
    const int64_t ch = (job % blocks * kWave + lane) * V;
    if (seq >= a.N || ch >= a.D) return;
    int64_t bos = seq * a.L, len = a.L;
    if (packed) {
      bos = clamp_offset(a.cu[seq], 0, a.L);
      len = clamp_offset(a.cu[seq + 1], bos, a.L) - bos;
    }
    const int64_t row = state_row(a.slots, int(seq), a.P);
    const T* x = static_cast<const T*>(a.x) + bos * a.x_row + ch;
    ConvVec<T, V> st[W - 1];
#pragma unroll
    for (int i = 0; i < W - 1; ++i)
      st[i] = a.s0 != nullptr && row >= 0
                  ? *reinterpret_cast<const ConvVec<T, V>*>(static_cast<const T*>(a.s0) + (row * (W - 1) + i) * a.D + ch)
                  : conv_zero<T, V>();
    if (len > 0 && a.y != nullptr) {
      ConvTaps<T, V, W> taps;
      taps.load(static_cast<const T*>(a.w), static_cast<const T*>(a.bias), ch);
      float win[W][V] = {};
#pragma unroll
      for (int i = 0; i < W - 1; ++i) conv_push<T, V, W>(win, st[i]);
#pragma unroll
      for (int t = 0; t < W - 1; ++t)
        if (t < len) {
          conv_push<T, V, W>(win, *reinterpret_cast<const ConvVec<T, V>*>(x + t * a.x_row));
          *reinterpret_cast<ConvVec<T, V>*>(static_cast<T*>(a.y) + (bos + t) * a.y_row + ch) =
              conv_out<T, V, W>(taps, win, a.silu);
        }
    }
    if (a.sfin != nullptr && row >= 0) {
      ConvVec<T, V> end[W - 1];
#pragma unroll
      for (int i = 0; i < W - 1; ++i) {
        const int64_t t = len - (W - 1) + i;
        if (t >= 0) {
          end[i] = *reinterpret_cast<const ConvVec<T, V>*>(x + t * a.x_row);
        } else {
#pragma unroll
          for (int j = 0; j < W - 1; ++j)
            if (j == int(t) + W - 1) end[i] = st[j];
        }
      }
#pragma unroll
      for (int i = 0; i < W - 1; ++i)
        *reinterpret_cast<ConvVec<T, V>*>(static_cast<T*>(a.sfin) + (row * (W - 1) + i) * a.D + ch) = end[i];
    }
    return;
  }

  const uint32_t job = blockIdx.x - uint32_t(seq_wgs);
  const int64_t ch = (int64_t(job % uint32_t(blocks)) * kWave + lane) * V;
  const uint32_t tile = job / uint32_t(blocks);
  int64_t base = 0, t0 = 0;
  if (packed) {
    t0 = (int64_t(tile) * 4 + w) * run;
  } else {
    const uint32_t tiles = uint32_t((a.L + 4 * run - 1) / (4 * run));
    base = int64_t(tile / tiles) * a.L;
    t0 = (int64_t(tile % tiles) * 4 + w) * run;
  }
  if (t0 >= a.L) return;
  const int64_t t1 = t0 + run < a.L ? t0 + run : a.L;
  int64_t bos = 0, end = a.L;
  int seq = 0;
  auto enter = [&](int u) {
    seq = u;
    bos = clamp_offset(a.cu[u], 0, a.L);
    end = clamp_offset(a.cu[u + 1], bos, a.L);
  };
  if (packed) enter(conv_seq_of(a.cu, a.N, a.L, t0, lane));
  if (ch >= a.D) return;
  ConvTaps<T, V, W> taps;
  taps.load(static_cast<const T*>(a.w), static_cast<const T*>(a.bias), ch);
  const T* x = static_cast<const T*>(a.x) + base * a.x_row + ch;
  T* y = static_cast<T*>(a.y) + base * a.y_row + ch;
  auto row_of = [&](int64_t t) { return *reinterpret_cast<const ConvVec<T, V>*>(x + t * a.x_row); };
  float win[W][V] = {};
#pragma unroll
  for (int i = 0; i < W - 1; ++i) {
    const int64_t t = t0 - (W - 1) + i;
    conv_push<T, V, W>(win, row_of(t < 0 ? 0 : t));  // rows before a sequence's W - 1st feed no row that is stored
  }
  ConvVec<T, V> next[kConvGroup];  // the next rows, asked for a group ahead
  auto fetch = [&](int64_t t) {
#pragma unroll
    for (int i = 0; i < kConvGroup; ++i) next[i] = row_of(t + i < t1 ? t + i : t1 - 1);
  };
  fetch(t0);
  for (int64_t t = t0; t < t1; t += kConvGroup) {
    ConvVec<T, V> in[kConvGroup];
#pragma unroll
    for (int i = 0; i < kConvGroup; ++i) in[i] = next[i];
    if (t + kConvGroup < t1) fetch(t + kConvGroup);
#pragma unroll
    for (int i = 0; i < kConvGroup; ++i) {
      const int64_t at = t + i;
      conv_push<T, V, W>(win, in[i]);
      if (packed)
        while (at >= end && seq + 1 < a.N) enter(seq + 1);
      if (at < t1 && at >= bos + W - 1 && at < end)
        *reinterpret_cast<ConvVec<T, V>*>(y + at * a.y_row) = conv_out<T, V, W>(taps, win, a.silu);
    }
  }
}

// One token a request: the state's W - 1 inputs move up by one, in place.
template <typename T, int V, int W>
__global__ __launch_bounds__(kThreads) void conv_step_kernel(ConvStep a, int blocks) {
  const int64_t job = int64_t(blockIdx.x) * 4 + wave_id();
  const int64_t n = job / blocks;
  const int64_t ch = (job % blocks * kWave + (threadIdx.x & 63)) * V;
  if (n >= a.N || ch >= a.D) return;
  const int64_t row = state_row(a.slots, int(n), a.P);
  if (row < 0) return;
  T* st = static_cast<T*>(a.state) + row * (W - 1) * a.D + ch;
  ConvVec<T, V> in[W];
#pragma unroll
  for (int i = 0; i < W - 1; ++i) in[i] = *reinterpret_cast<const ConvVec<T, V>*>(st + int64_t(i) * a.D);
  in[W - 1] = *reinterpret_cast<const ConvVec<T, V>*>(static_cast<const T*>(a.x) + n * a.x_row + ch);
  ConvTaps<T, V, W> taps;
  taps.load(static_cast<const T*>(a.w), static_cast<const T*>(a.bias), ch);
  float win[W][V] = {};
#pragma unroll
  for (int i = 0; i < W; ++i) conv_push<T, V, W>(win, in[i]);
  *reinterpret_cast<ConvVec<T, V>*>(static_cast<T*>(a.y) + n * a.y_row + ch) = conv_out<T, V, W>(taps, win, a.silu);
#pragma unroll
  for (int i = 0; i < W - 1; ++i) *reinterpret_cast<ConvVec<T, V>*>(st + int64_t(i) * a.D) = in[i + 1];
}

// Gradient.  With du_t = dy_t silu'(u_t):
//     dx_s = sum_i w_i du_{s+W-1-i},   dw_i = sum_t x_{t-W+1+i} du_t,   dbias = sum_t du_t.
// A wavefront slides the windows of x and of du over its run of tokens and the
// W - 1 behind it (whose du it forms again), so dx_{t-W+1} leaves with du_t.
// The rows before the first token are the state: their dx is ds0.  dw and dbias
// are summed in registers over the run, over the workgroup's four runs through
// the LDS, and over the workgroups by conv_sum_kernel in a fixed order.
template <typename T, int V, int W>
__global__ __launch_bounds__(kThreads) void conv_bwd_kernel(ConvBwd a, int blocks, int run, float* __restrict__ part) {
  __shared__ float red[3][W + 1][V][kWave];
  const int lane = threadIdx.x & 63, w = wave_id();
  const uint32_t job = blockIdx.x;
  const int64_t ch = (int64_t(job % uint32_t(blocks)) * kWave + lane) * V;
  const uint32_t tile = job / uint32_t(blocks), tiles = uint32_t((a.L + 4 * run - 1) / (4 * run));
  const int64_t b = tile / tiles;
  const int64_t t0 = (int64_t(tile % tiles) * 4 + w) * run;
  const bool on = t0 < a.L && ch < a.D;
  float dw[W][V] = {}, db[V] = {};
  if (on) {
    const int64_t t1 = t0 + run < a.L ? t0 + run : a.L;  // this run: t0 .. t1 - 1
    ConvTaps<T, V, W> taps;
    taps.load(static_cast<const T*>(a.w), static_cast<const T*>(a.bias), ch);
    const T* x = static_cast<const T*>(a.x) + b * a.L * a.x_row + ch;
    const T* dy = static_cast<const T*>(a.dy) + b * a.L * a.dy_row + ch;
    T* dx = static_cast<T*>(a.dx) + b * a.L * a.dx_row + ch;
    const int64_t srow = b * (W - 1) * a.D + ch;
    float win[W][V] = {}, du[W][V] = {};
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
      const int64_t t = t0 - (W - 1) + i;
      ConvVec<T, V> in = conv_zero<T, V>();
      if (t >= 0) in = *reinterpret_cast<const ConvVec<T, V>*>(x + t * a.x_row);
      else if (a.s0 != nullptr)
        in = *reinterpret_cast<const ConvVec<T, V>*>(static_cast<const T*>(a.s0) + srow + (t + W - 1) * a.D);
      conv_push<T, V, W>(win, in);
    }
    constexpr int G = kConvGroup;
    ConvVec<T, V> xn[G], yn[G];  // the next rows, asked for a group ahead
    auto fetch = [&](int64_t t) {
#pragma unroll
      for (int i = 0; i < G; ++i) {
        const int64_t at = t + i < a.L ? t + i : a.L - 1;
        xn[i] = *reinterpret_cast<const ConvVec<T, V>*>(x + at * a.x_row);
        yn[i] = *reinterpret_cast<const ConvVec<T, V>*>(dy + at * a.dy_row);
      }
    };
    fetch(t0);
    for (int64_t t = t0; t < t1 + W - 1; t += G) {
      ConvVec<T, V> xi[G], yi[G];
#pragma unroll
      for (int i = 0; i < G; ++i) {
        xi[i] = xn[i];
        yi[i] = yn[i];
      }
      if (t + G < t1 + W - 1) fetch(t + G);
#pragma unroll
      for (int i = 0; i < G; ++i) {
        const int64_t at = t + i;
        if (at >= t1 + W - 1) break;
        conv_push<T, V, W>(win, xi[i]);
        const bool real = at < a.L, mine = at < t1;
        float next[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
          float d = real ? to_f32(yi[i].e[e]) : 0.0f;
          if (a.silu) {
            const float u = taps.dot(win, e), sg = sigmoid(u);
            // silu' = sg (1 + u (1 - sg)), where u (1 - sg) goes to zero for large u
            d = real ? d * sg * fmaf(u, 1.0f - sg, 1.0f) : 0.0f;
          }
          next[e] = d;
        }
#pragma unroll
        for (int j = 0; j + 1 < W; ++j)
#pragma unroll
          for (int e = 0; e < V; ++e) du[j][e] = du[j + 1][e];
#pragma unroll
        for (int e = 0; e < V; ++e) du[W - 1][e] = next[e];
        if (mine) {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            db[e] += next[e];
#pragma unroll
            for (int j = 0; j < W; ++j) dw[j][e] = fmaf(win[j][e], next[e], dw[j][e]);
          }
        }
        const int64_t s = at - (W - 1);  // this input's gradient is complete
        if (s >= t0 || (s < 0 && a.ds0 != nullptr)) {
          const int64_t fin = s - (a.L - (W - 1));  // its row of the final state
          ConvVec<T, V> add = conv_zero<T, V>(), out;
          if (a.dsf != nullptr && fin >= 0)
            add = *reinterpret_cast<const ConvVec<T, V>*>(static_cast<const T*>(a.dsf) + srow + fin * a.D);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            float d = to_f32(add.e[e]);
#pragma unroll
            for (int j = 0; j < W; ++j) d = fmaf(taps.w[j][e], du[W - 1 - j][e], d);
            out.e[e] = from_f32<T>(d);
          }
          T* dst = s >= 0 ? dx + s * a.dx_row : static_cast<T*>(a.ds0) + srow + (s + W - 1) * a.D;
          *reinterpret_cast<ConvVec<T, V>*>(dst) = out;
        }
      }
    }
  }
  if (w > 0) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      red[w - 1][W][e][lane] = db[e];
#pragma unroll
      for (int j = 0; j < W; ++j) red[w - 1][j][e][lane] = dw[j][e];
    }
  }
  __syncthreads();
  if (w == 0 && ch < a.D) {
    float* dst = part + int64_t(tile) * (W + 1) * a.D + ch;
#pragma unroll
    for (int j = 0; j <= W; ++j) {
      ConvVec<float, V> sum;
#pragma unroll
      for (int e = 0; e < V; ++e)
        sum.e[e] = (j < W ? dw[j < W ? j : 0][e] : db[e]) + red[0][j][e][lane] + red[1][j][e][lane] + red[2][j][e][lane];
#pragma unroll
      for (int e = 0; e < V; ++e) dst[int64_t(j) * a.D + e] = sum.e[e];
    }
  }
}

// dw [D, W] and dbias [D] from M partial rows of (W + 1) D sums each: 64 sums a
// workgroup, its 16 wavefronts a sixteenth of the rows each.
constexpr int kSumWaves = 16;
__global__ __launch_bounds__(kSumWaves * kWave) void conv_sum_kernel(const float* __restrict__ part, float* __restrict__ dw,
                                                                     float* __restrict__ db, int64_t M, int D, int W) {
  __shared__ float red[kSumWaves][kWave];
  const int lane = threadIdx.x & 63, w = wave_id();
  const int64_t col = int64_t(blockIdx.x) * kWave + lane, cols = int64_t(W + 1) * D;
  float sum = 0.0f;
  if (col < cols)
    for (int64_t m = w; m < M; m += kSumWaves) sum += part[m * cols + col];
  red[w][lane] = sum;
  __syncthreads();
  if (w > 0 || col >= cols) return;
#pragma unroll
  for (int i = 1; i < kSumWaves; ++i) sum += red[i][lane];
  const int64_t j = col / D, c = col % D;
  if (j < W) dw[c * W + j] = sum;
  else if (db != nullptr) db[c] = sum;
}

// A sequence of no tokens: the final state's gradient is the initial state's.
template <typename T>
__global__ __launch_bounds__(kThreads) void conv_copy_kernel(const T* __restrict__ src, T* __restrict__ dst, int64_t n) {
  const int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  if (i < n) dst[i] = src != nullptr ? src[i] : T(0);
}

// ---------------------------------------------------------------- launches
// 16-byte vectors where every row of every tensor starts on 16 bytes.
static bool conv_rows_aligned(std::initializer_list<const void*> ptrs, std::initializer_list<int64_t> strides, size_t esz) {
  for (const void* p : ptrs)
    if (reinterpret_cast<uintptr_t>(p) & 15) return false;
  for (int64_t s : strides)
    if (s * int64_t(esz) & 15) return false;
  return true;
}

template <typename F>
static hipError_t conv_by_width(int W, F&& f) {
  switch (W) {
    case 2: return f(std::integral_constant<int, 2>{});
    case 3: return f(std::integral_constant<int, 3>{});
    case 4: return f(std::integral_constant<int, 4>{});
  }
  return hipErrorInvalidValue;
}
template <typename T, typename F>
static hipError_t conv_by_vector(bool aligned, F&& f) {
  if (aligned) return f(std::integral_constant<int, 16 / sizeof(T)>{});
  return f(std::integral_constant<int, 1>{});
}

static int64_t conv_blocks(int D, int V) { return (int64_t(D) + kWave * V - 1) / (kWave * V); }

// Tokens a run of the forward pass: 8, whose windows overlap in the caches, and more only
// where the launch would have more threads than the runtime takes.  us with runs of 8 /
// 16 / 32 / 64, bf16, W = 4:
//   1 x 2048 tokens, 2048 channels  8.3 / 10.1 / 14.7 / 26    8 x 2048, 2048  26.0 / 29.4 / 25.1 / 27.8
//   4 x 4096, 6144  76 / 81 / 86 / 88                         8 x 4096, 6144  143 / 154 / 162 / 170
//   16 x 8192, 4096  369 / 393 / 407 / 413                    1 x 65536, 1024  48.8 / 53.0 / 49.0 / 47.8
// and float32:  4 x 4096, 6144  150 / 159 / 168 / 169         8 x 4096, 6144  288 / 305 / 326 / 329
static int64_t conv_fwd_wgs(int64_t seqs, int64_t L, int64_t N, int64_t blocks, int run) {
  return (N * blocks + 3) / 4 + seqs * ((L + 4 * run - 1) / (4 * run)) * blocks;
}
static int conv_fwd_run(int64_t seqs, int64_t L, int64_t N, int64_t blocks) {
  int run = 8;
  while (run < 64 && conv_fwd_wgs(seqs, L, N, blocks, run) * kThreads > kMaxLaunchThreads) run *= 2;
  return run;
}

template <typename T>
hipError_t launch_conv_fwd(const ConvFwd& a, hipStream_t s) {
  const bool aligned = conv_rows_aligned({a.x, a.w, a.bias, a.s0, a.y, a.sfin}, {a.D, a.x_row, a.y_row}, sizeof(T));
  return conv_by_width(a.W, [&](auto wc) {
    return conv_by_vector<T>(aligned, [&](auto vc) {
      constexpr int W = decltype(wc)::value, V = decltype(vc)::value;
      const int64_t blocks = conv_blocks(a.D, V), seqs = a.cu != nullptr ? 1 : a.N;
      const int run = conv_fwd_run(seqs, a.L, a.N, blocks);
      const int64_t seq_wgs = (a.N * blocks + 3) / 4;
      const int64_t wgs = a.y == nullptr ? seq_wgs : conv_fwd_wgs(seqs, a.L, a.N, blocks, run);
      if (wgs == 0) return hipSuccess;
      hipLaunchKernelGGL((conv_fwd_kernel<T, V, W>), dim3(unsigned(wgs)), dim3(kThreads), 0, s, a, int(blocks),
                         int(seq_wgs), run);
      return hipGetLastError();
    });
  });
}
template hipError_t launch_conv_fwd<float>(const ConvFwd&, hipStream_t);
template hipError_t launch_conv_fwd<uint16_t>(const ConvFwd&, hipStream_t);

template <typename T>
hipError_t launch_conv_step(const ConvStep& a, hipStream_t s) {
  const bool aligned = conv_rows_aligned({a.x, a.w, a.bias, a.state, a.y}, {a.D, a.x_row, a.y_row}, sizeof(T));
  return conv_by_width(a.W, [&](auto wc) {
    return conv_by_vector<T>(aligned, [&](auto vc) {
      constexpr int W = decltype(wc)::value, V = decltype(vc)::value;
      const int64_t blocks = conv_blocks(a.D, V), wgs = (a.N * blocks + 3) / 4;
      hipLaunchKernelGGL((conv_step_kernel<T, V, W>), dim3(unsigned(wgs)), dim3(kThreads), 0, s, a, int(blocks));
      return hipGetLastError();
    });
  });
}
template hipError_t launch_conv_step<float>(const ConvStep&, hipStream_t);
template hipError_t launch_conv_step<uint16_t>(const ConvStep&, hipStream_t);

// Tokens a run of the gradient, whose windows are longer and whose partial sums are one
// row a workgroup: as long as there are 2048 wavefronts (its registers leave two a SIMD),
// up to 64.  us with runs of 8 / 16 / 32 / 64, bf16, W = 4:
//   1 x 2048 tokens, 2048 channels  18 / 24 / 34 / 59         8 x 2048, 2048  76 / 69 / 50 / 62
//   1 x 4096, 6144  53 / 47 / 45 / 60 (takes 16)              4 x 4096, 6144  196 / 162 / 147 / 154 (64)
//   8 x 4096, 6144  378 / 308 / 277 / 272                     1 x 65536, 1024  166 / 126 / 106 / 100
// and float32:  8 x 2048, 2048  100 / 98 / 98 / 89 (32)       8 x 4096, 6144  502 / 489 / 498 / 507 (64)
// By one block count whatever the alignment, so that the workspace does not depend on it.
static int conv_bwd_run(int B, int64_t L, int D) {
  for (int run = 64; run > 8; run /= 2)
    if (B * ((L + run - 1) / run) * conv_blocks(D, 8) >= 2048) return run;
  return 8;
}
size_t conv_bwd_workspace(int B, int64_t L, int D, int W) {
  const int run = conv_bwd_run(B, L, D);
  return size_t(B) * size_t((L + 4 * run - 1) / (4 * run)) * size_t(W + 1) * size_t(D) * sizeof(float);
}
// Threads of the largest launch over these sizes (one element a lane).
int64_t conv_threads(int64_t seqs, int64_t L, int64_t N, int D) {
  const int64_t blocks = conv_blocks(D, 1);
  return conv_fwd_wgs(seqs, L, N, blocks, conv_fwd_run(seqs, L, N, blocks)) * kThreads;
}

int64_t conv_copy_threads(int64_t B, int D, int W) {
  return (B * (W - 1) * D + kThreads - 1) / kThreads * kThreads;
}

template <typename T>
hipError_t launch_conv_bwd(const ConvBwd& a, float* part, hipStream_t s) {
  if (a.L == 0) {
    if (a.ds0 != nullptr) {
      hipLaunchKernelGGL((conv_copy_kernel<T>), dim3(unsigned(conv_copy_threads(a.B, a.D, a.W) / kThreads)), dim3(kThreads), 0,
                         s, static_cast<const T*>(a.dsf), static_cast<T*>(a.ds0), int64_t(a.B) * (a.W - 1) * a.D);
    }
  } else {
    const bool aligned = conv_rows_aligned({a.x, a.w, a.bias, a.s0, a.dy, a.dsf, a.dx, a.ds0},
                                           {a.D, a.x_row, a.dy_row, a.dx_row}, sizeof(T));
    const hipError_t e = conv_by_width(a.W, [&](auto wc) {
      return conv_by_vector<T>(aligned, [&](auto vc) {
        constexpr int W = decltype(wc)::value, V = decltype(vc)::value;
        const int run = conv_bwd_run(a.B, a.L, a.D);
        const int64_t blocks = conv_blocks(a.D, V), wgs = int64_t(a.B) * ((a.L + 4 * run - 1) / (4 * run)) * blocks;
        hipLaunchKernelGGL((conv_bwd_kernel<T, V, W>), dim3(unsigned(wgs)), dim3(kThreads), 0, s, a, int(blocks), run, part);
        return hipGetLastError();
      });
    });
    if (e != hipSuccess) return e;
  }
  const int run = conv_bwd_run(a.B, a.L, a.D);
  const int64_t M = a.L == 0 ? 0 : int64_t(a.B) * ((a.L + 4 * run - 1) / (4 * run));
  const int64_t cols = int64_t(a.W + 1) * a.D;
  hipLaunchKernelGGL(conv_sum_kernel, dim3(unsigned((cols + kWave - 1) / kWave)), dim3(kSumWaves * kWave), 0, s, part,
                     a.dw, a.db, M, a.D, a.W);
  return hipGetLastError();
}
template hipError_t launch_conv_bwd<float>(const ConvBwd&, float*, hipStream_t);
template hipError_t launch_conv_bwd<uint16_t>(const ConvBwd&, float*, hipStream_t);

}  // namespace efla
