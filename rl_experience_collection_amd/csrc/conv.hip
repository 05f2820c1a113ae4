// Short causal convolution over a rollout: forward, gradient, single step
// (include/block.h).
//
// A thread takes 16 bytes of an episode's channels and a chunk of steps. It
// keeps the last W - 1 inputs in registers, so that an input is read once, and
// reads those before its chunk again; four steps' loads are in flight while
// the four before are worked on.  A done clears the window, which is all that
// keeps episodes apart.
//
// The gradient runs in the same direction: step t adds to the gradients of the
// inputs t - W + 1 .. t, which wait in W registers until no later step adds
// to them (W - 1 steps past the chunk's end are formed again for that).
// Weights' gradients are summed by threads over their steps, by a workgroup in
// LDS, and over workgroups by column sums.
#include <algorithm>

#include "block.hpp"
#include "elem.hpp"

namespace rl {

namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 4;  // steps loaded at a time

struct ConvRun {
  conv_grad_args g;  // forward: g.f alone
  int32_t packs;     // of a row
  int32_t across;    // of those, a workgroup's
  int32_t rows;      // (chunk, n) pairs of a workgroup
  int32_t chunk, chunks;
  int64_t items;     // chunks * N
  float* params;     // gradient: [workgroups][D (W + 1)]
};

constexpr float kLog2e = 1.44269504f;
__device__ __forceinline__ float sigmoid_of(float v) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-v * kLog2e));
}

// Which rows and channels a thread has.
struct ConvLane {
  int32_t n, d0, fresh, t0, t1, row, pack;
  bool active;
  __device__ __forceinline__ ConvLane(const ConvRun& q, int V) {
    row = threadIdx.x / q.across;
    pack = blockIdx.y * q.across + threadIdx.x % q.across;
    const int64_t item = (int64_t)blockIdx.x * q.rows + row;
    active = row < q.rows && item < q.items && pack < q.packs;
    const int32_t N = q.g.f.rows;
    n = active ? (int32_t)(item % N) : 0;
    const int32_t c = active ? (int32_t)(item / N) : 0;
    d0 = min(pack * V, q.g.f.width - V);
    fresh = pack * V - d0;  // elements before it are the pack's before
    t0 = c * q.chunk;
    t1 = min(t0 + q.chunk, q.g.f.steps);
  }
};

// Whether a done lies between step t - 1 and t.
__device__ __forceinline__ bool cut_before(const conv_args& a, int32_t n, int32_t t) {
  return a.dones && t > 0 && t <= a.steps && a.dones[(int64_t)(t - 1) * a.rows + n] != 0;
}

// The inputs before step t0 (age 1 first) and how many belong to its episode.
template <class T, int V, int W>
__device__ __forceinline__ int32_t open_window(const conv_args& a, const ConvLane& k,
                                               float (&win)[W][V]) {
  using raw = typename T::raw;
  int32_t age = 0;
  bool same = true;
#pragma unroll
  for (int i = 1; i < W; ++i) {
    const int32_t t = k.t0 - i;
    same = same && !cut_before(a, k.n, t + 1);
#pragma unroll
    for (int v = 0; v < V; ++v) win[i][v] = 0.0f;
    if (!same) continue;
    age = i;
    if (t >= 0)
      widen_pack<T, V>(
          load_pack<T, V>(static_cast<const raw*>(a.x) + t * a.x_step + k.n * a.x_row + k.d0), win[i]);
    else if (a.state)
      widen_pack<T, V>(load_pack<T, V>(static_cast<const raw*>(a.state) +
                                       ((int64_t)k.n * (W - 1) + (W - 1 + t)) * a.width + k.d0),
                       win[i]);
  }
  return age;
}

template <int V, int W>
__device__ __forceinline__ void load_weights(const conv_args& a, int32_t d0, float (&w)[W][V],
                                             float (&bias)[V]) {
#pragma unroll
  for (int v = 0; v < V; ++v) {
    bias[v] = a.bias ? a.bias[d0 + v] : 0.0f;
#pragma unroll
    for (int i = 0; i < W; ++i) w[i][v] = a.weight[(int64_t)(d0 + v) * W + (W - 1 - i)];  // by age
  }
}

template <class T, int V, int W>
__global__ void __launch_bounds__(kThreads) conv_forward_kernel(const ConvRun q) {
  using raw = typename T::raw;
  const conv_args& a = q.g.f;
  const ConvLane k(q, V);
  if (!k.active) return;
  float w[W][V], bias[V], win[W][V];
  load_weights<V, W>(a, k.d0, w, bias);
  open_window<T, V, W>(a, k, win);
  const raw* px = static_cast<const raw*>(a.x) + k.n * a.x_row + k.d0;
  raw* py = static_cast<raw*>(a.y) + k.n * a.y_row + k.d0;
  const bool silu = a.activation == BLOCK_SILU;
  const int32_t last = k.t1 - 1;

  Pack<T, V> next[kAhead];
  bool next_cut[kAhead];
  const auto fetch = [&](int32_t t) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      next[i] = load_pack<T, V>(px + min(t + i, last) * a.x_step);
      next_cut[i] = cut_before(a, k.n, min(t + i, last));
    }
  };
  fetch(k.t0);
  for (int32_t t = k.t0; t < k.t1; t += kAhead) {
    Pack<T, V> x[kAhead];
    bool cut[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      x[i] = next[i];
      cut[i] = next_cut[i];
    }
    fetch(t + kAhead);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (t + i >= k.t1) break;
      if (cut[i]) {
#pragma unroll
        for (int j = 1; j < W; ++j)
#pragma unroll
          for (int v = 0; v < V; ++v) win[j][v] = 0.0f;
      }
      widen_pack<T, V>(x[i], win[0]);
      float y[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float p = bias[v];
#pragma unroll
        for (int j = W - 1; j >= 0; --j) p = __builtin_fmaf(w[j][v], win[j][v], p);
        y[v] = silu ? p * sigmoid_of(p) : p;
      }
      store_pack<T, V>(py + (t + i) * a.y_step, narrow_pack<T, V>(y));
#pragma unroll
      for (int j = W - 1; j > 0; --j)
#pragma unroll
        for (int v = 0; v < V; ++v) win[j][v] = win[j - 1][v];
    }
  }
  if (k.t1 == a.steps && a.new_state) {
    const bool ended = cut_before(a, k.n, a.steps);
#pragma unroll
    for (int j = 1; j < W; ++j) {
      if (ended) {
#pragma unroll
        for (int v = 0; v < V; ++v) win[j][v] = 0.0f;
      }
      store_pack<T, V>(
          static_cast<raw*>(a.new_state) + ((int64_t)k.n * (W - 1) + (W - 1 - j)) * a.width + k.d0,
          narrow_pack<T, V>(win[j]));
    }
  }
}

template <class T, int V, int W>
__global__ void __launch_bounds__(kThreads) conv_backward_kernel(const ConvRun q) {
  using raw = typename T::raw;
  const conv_grad_args& g = q.g;
  const conv_args& a = g.f;
  const ConvLane k(q, V);
  float dw[W][V], db[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    db[v] = 0.0f;
#pragma unroll
    for (int j = 0; j < W; ++j) dw[j][v] = 0.0f;
  }
  if (k.active) {
    float w[W][V], bias[V], win[W][V], acc[W][V];
    load_weights<V, W>(a, k.d0, w, bias);
    int32_t age = open_window<T, V, W>(a, k, win);
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
      for (int v = 0; v < V; ++v) acc[j][v] = 0.0f;
    const raw* px = static_cast<const raw*>(a.x) + k.n * a.x_row + k.d0;
    const raw* pd = static_cast<const raw*>(g.dy) + k.n * g.dy_row + k.d0;
    const bool silu = a.activation == BLOCK_SILU;
    const int32_t end = min(k.t1 + W - 1, a.steps);

    // The gradient of the input of step e, if it is this chunk's.
    const auto emit = [&](int32_t e, const float(&v)[V]) {
      if (e >= k.t0 && e < k.t1)
        store_pack<T, V>(static_cast<raw*>(g.dx) + e * g.dx_step + k.n * g.dx_row + k.d0,
                         narrow_pack<T, V>(v));
      else if (e < 0 && k.t0 == 0 && g.dstate)
        store_pack<T, V>(static_cast<raw*>(g.dstate) + ((int64_t)k.n * (W - 1) + (W - 1 + e)) * a.width + k.d0,
                         narrow_pack<T, V>(v));
    };
    Pack<T, V> next_x[kAhead], next_d[kAhead];
    bool next_cut[kAhead];
    const auto fetch = [&](int32_t t) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int32_t at = min(t + i, end - 1);
        next_x[i] = load_pack<T, V>(px + at * a.x_step);
        next_d[i] = load_pack<T, V>(pd + at * g.dy_step);
        next_cut[i] = cut_before(a, k.n, at);
      }
    };
    fetch(k.t0);
    for (int32_t t = k.t0; t < end; t += kAhead) {
      Pack<T, V> x[kAhead], d[kAhead];
      bool cut[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        x[i] = next_x[i];
        d[i] = next_d[i];
        cut[i] = next_cut[i];
      }
      fetch(t + kAhead);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (t + i >= end) break;
        if (t + i > k.t0) age = min(age + 1, W - 1);
        if (cut[i]) {
          age = 0;
#pragma unroll
          for (int j = 1; j < W; ++j)
#pragma unroll
            for (int v = 0; v < V; ++v) win[j][v] = 0.0f;
        }
        widen_pack<T, V>(x[i], win[0]);
        float dp[V];
        widen_pack<T, V>(d[i], dp);
        if (silu) {
#pragma unroll
          for (int v = 0; v < V; ++v) {
            float p = bias[v];
#pragma unroll
            for (int j = W - 1; j >= 0; --j) p = __builtin_fmaf(w[j][v], win[j][v], p);
            const float s = sigmoid_of(p);
            dp[v] *= s * __builtin_fmaf(p, 1.0f - s, 1.0f);
          }
        }
        if (t + i < k.t1) {
#pragma unroll
          for (int v = 0; v < V; ++v) {
            db[v] += dp[v];
#pragma unroll
            for (int j = 0; j < W; ++j) dw[j][v] = __builtin_fmaf(dp[v], win[j][v], dw[j][v]);
          }
        }
#pragma unroll
        for (int j = 0; j < W; ++j) {
          if (j > age) continue;  // an input of another episode
#pragma unroll
          for (int v = 0; v < V; ++v) acc[j][v] = __builtin_fmaf(w[j][v], dp[v], acc[j][v]);
        }
        emit(t + i - (W - 1), acc[W - 1]);
#pragma unroll
        for (int j = W - 1; j > 0; --j)
#pragma unroll
          for (int v = 0; v < V; ++v) {
            win[j][v] = win[j - 1][v];
            acc[j][v] = acc[j - 1][v];
          }
#pragma unroll
        for (int v = 0; v < V; ++v) acc[0][v] = 0.0f;
      }
    }
    if (end == a.steps) {
      // The last inputs wait for no step; new_state sends them theirs.  (acc[j]
      // is now that of step L - j.)
      age = cut_before(a, k.n, a.steps) ? 0 : min(age + 1, W - 1);
#pragma unroll
      for (int j = W - 1; j > 0; --j) {
        if (g.dnew_state && j <= age) {
          float ds[V];
          widen_pack<T, V>(load_pack<T, V>(static_cast<const raw*>(g.dnew_state) +
                                           ((int64_t)k.n * (W - 1) + (W - 1 - j)) * a.width + k.d0),
                           ds);
#pragma unroll
          for (int v = 0; v < V; ++v) acc[j][v] += ds[v];
        }
        emit(a.steps - j, acc[j]);
      }
    }
  }
  // the workgroup's sums over its rows, one tap at a time (the bias last)
  __shared__ float s_sum[kThreads][V];
  const int32_t columns = q.across * V;
#pragma unroll
  for (int j = 0; j <= W; ++j) {
    __syncthreads();
#pragma unroll
    for (int v = 0; v < V; ++v) s_sum[threadIdx.x][v] = j < W ? dw[j < W ? j : 0][v] : db[v];
    __syncthreads();
    for (int32_t c = threadIdx.x; c < columns; c += kThreads) {
      const int32_t pack = blockIdx.y * q.across + c / V;
      if (pack >= q.packs) continue;
      const int32_t d0 = min(pack * V, a.width - V);
      if (c % V < pack * V - d0) continue;  // (counted in the pack before)
      float sum = 0.0f;
      for (int32_t r = 0; r < q.rows; ++r) sum += s_sum[r * q.across + c / V][c % V];
      const int64_t d = d0 + c % V;
      q.params[(int64_t)blockIdx.x * a.width * (W + 1) + (j < W ? d * W + (W - 1 - j) : (int64_t)a.width * W + d)] =
          sum;
    }
  }
}

struct StepRun {
  int32_t N, D, packs;
  const void *x, *state;
  const float *weight, *bias;
  const uint8_t* resets;
  void *y, *new_state;
  int64_t x_row, y_row;
  bool silu;
};

// One step.  No two threads share an element, so that the window may move on
// in place: a row's last elements are taken one by one.
template <class T, int V, int W>
__global__ void __launch_bounds__(kThreads) conv_step_kernel(const StepRun q) {
  using raw = typename T::raw;
  const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t n = id / q.packs;
  if (n >= q.N) return;
  const int32_t d0 = (int32_t)(id % q.packs) * V;
  const bool reset = q.resets && q.resets[n] != 0;
  const raw* px = static_cast<const raw*>(q.x) + n * q.x_row + d0;
  const raw* ps = static_cast<const raw*>(q.state) + n * (W - 1) * q.D + d0;
  raw* pn = static_cast<raw*>(q.new_state) + n * (W - 1) * q.D + d0;
  raw* py = static_cast<raw*>(q.y) + n * q.y_row + d0;
  const auto one = [&](auto width, int32_t at) {
    constexpr int E = decltype(width)::value;
    Pack<T, E> win[W], out;
#pragma unroll
    for (int j = 0; j < W; ++j) {  // oldest first
      win[j] = load_pack<T, E>(j < W - 1 ? ps + (int64_t)j * q.D + at : px + at);
      if (j < W - 1 && reset) {
#pragma unroll
        for (int v = 0; v < E; ++v) win[j].v[v] = 0;
      }
    }
#pragma unroll
    for (int v = 0; v < E; ++v) {
      float p = q.bias ? q.bias[d0 + at + v] : 0.0f;
#pragma unroll
      for (int j = 0; j < W; ++j)
        p = __builtin_fmaf(q.weight[(int64_t)(d0 + at + v) * W + j], T::widen(win[j].v[v]), p);
      out.v[v] = T::narrow(q.silu ? p * sigmoid_of(p) : p);
    }
    store_pack<T, E>(py + at, out);
#pragma unroll
    for (int j = 1; j < W; ++j) store_pack<T, E>(pn + (int64_t)(j - 1) * q.D + at, win[j]);
  };
  if (d0 + V <= q.D) {
    one(std::integral_constant<int, V>(), 0);
  } else {
    for (int32_t at = 0; d0 + at < q.D; ++at) one(std::integral_constant<int, 1>(), at);
  }
}

template <class T>
constexpr int wide() {
  return 16 / T::kBytes;
}

// Chunks are made until threads enough for every place are there (2048 a
// compute unit; the gradient holds more registers and takes half), of 16 steps
// at least, since a chunk reads W - 1 steps twice.
ConvRun plan(int32_t L, int32_t N, int32_t D, int32_t V, bool grad) {
  ConvRun q;
  q.packs = (D + V - 1) / V;
  q.across = std::min(q.packs, kThreads);
  q.rows = kThreads / q.across;
  const int64_t columns = (int64_t)N * q.packs;
  const int64_t wanted = ((grad ? 262144 : 524288) + columns - 1) / columns;
  const int64_t most = std::max(1, L / 16);
  const int32_t chunks = (int32_t)std::min(wanted, most);
  q.chunk = (L + chunks - 1) / chunks;
  q.chunks = (L + q.chunk - 1) / q.chunk;
  q.items = (int64_t)q.chunks * N;
  q.params = nullptr;
  return q;
}
int32_t pack_of(int32_t D, int32_t dtype) {
  const int32_t v = dtype == POLICY_F32 ? 4 : 8;
  return D >= v ? v : 1;
}
dim3 grid_of(const ConvRun& q) {
  return dim3((uint32_t)((q.items + q.rows - 1) / q.rows), (uint32_t)((q.packs + q.across - 1) / q.across));
}

template <class T, int V, int W, bool GRAD>
void launch(const ConvRun& q, hipStream_t stream) {
  if constexpr (GRAD)
    conv_backward_kernel<T, V, W><<<grid_of(q), kThreads, 0, stream>>>(q);
  else
    conv_forward_kernel<T, V, W><<<grid_of(q), kThreads, 0, stream>>>(q);
}
template <class T, int V, bool GRAD>
void launch_taps(const ConvRun& q, hipStream_t stream) {
  switch (q.g.f.taps) {
    case 1: return launch<T, V, 1, GRAD>(q, stream);
    case 2: return launch<T, V, 2, GRAD>(q, stream);
    case 3: return launch<T, V, 3, GRAD>(q, stream);
    case 4: return launch<T, V, 4, GRAD>(q, stream);
    case 5: return launch<T, V, 5, GRAD>(q, stream);
    case 6: return launch<T, V, 6, GRAD>(q, stream);
    case 7: return launch<T, V, 7, GRAD>(q, stream);
    default: return launch<T, V, 8, GRAD>(q, stream);
  }
}
template <bool GRAD>
void launch_any(const ConvRun& q, hipStream_t stream) {
  const int32_t dt = q.g.f.dtype;
  const bool packed = pack_of(q.g.f.width, dt) > 1;
  if (dt == POLICY_F32)
    packed ? launch_taps<F32, wide<F32>(), GRAD>(q, stream) : launch_taps<F32, 1, GRAD>(q, stream);
  else if (dt == POLICY_BF16)
    packed ? launch_taps<BF16, wide<BF16>(), GRAD>(q, stream) : launch_taps<BF16, 1, GRAD>(q, stream);
  else
    packed ? launch_taps<F16, wide<F16>(), GRAD>(q, stream) : launch_taps<F16, 1, GRAD>(q, stream);
}

template <class T, int V>
void launch_step(const StepRun& q, int32_t W, hipStream_t stream) {
  const dim3 grid((uint32_t)(((int64_t)q.N * q.packs + kThreads - 1) / kThreads));
  switch (W) {
    case 1: conv_step_kernel<T, V, 1><<<grid, kThreads, 0, stream>>>(q); return;
    case 2: conv_step_kernel<T, V, 2><<<grid, kThreads, 0, stream>>>(q); return;
    case 3: conv_step_kernel<T, V, 3><<<grid, kThreads, 0, stream>>>(q); return;
    case 4: conv_step_kernel<T, V, 4><<<grid, kThreads, 0, stream>>>(q); return;
    case 5: conv_step_kernel<T, V, 5><<<grid, kThreads, 0, stream>>>(q); return;
    case 6: conv_step_kernel<T, V, 6><<<grid, kThreads, 0, stream>>>(q); return;
    case 7: conv_step_kernel<T, V, 7><<<grid, kThreads, 0, stream>>>(q); return;
    default: conv_step_kernel<T, V, 8><<<grid, kThreads, 0, stream>>>(q); return;
  }
}

int64_t element_bytes(int32_t dtype) { return dtype == POLICY_F32 ? 4 : 2; }
int64_t up(int64_t bytes) { return (bytes + 255) / 256 * 256; }

}  // namespace

hipError_t conv_forward_launch(const conv_args& a, hipStream_t stream) {
  if (a.steps == 0)
    return a.new_state ? copy_or_clear_launch(a.state, a.new_state,
                                              (int64_t)a.rows * (a.taps - 1) * a.width * element_bytes(a.dtype),
                                              stream)
                       : hipSuccess;
  ConvRun q = plan(a.steps, a.rows, a.width, pack_of(a.width, a.dtype), false);
  q.g = {};
  q.g.f = a;
  launch_any<false>(q, stream);
  return hipGetLastError();
}

int64_t conv_workspace_bytes(int32_t L, int32_t N, int32_t D, int32_t W, int32_t dtype) {
  if (L == 0 || N == 0 || D == 0) return 0;
  const ConvRun q = plan(L, N, D, pack_of(D, dtype), true);
  const int64_t groups = grid_of(q).x;
  return up(groups * D * (W + 1) * 4) + up(sums_floats(groups, D * (W + 1)) * 4);
}

hipError_t conv_backward_launch(const conv_grad_args& g, hipStream_t stream) {
  const conv_args& a = g.f;
  const int64_t D = a.width, W = a.taps;
  if (a.steps == 0 || a.rows == 0) {
    hipError_t e = copy_or_clear_launch(nullptr, g.dweight, D * W * 4, stream);
    if (e == hipSuccess && g.dbias) e = copy_or_clear_launch(nullptr, g.dbias, D * 4, stream);
    if (e == hipSuccess && g.dstate)
      e = copy_or_clear_launch(g.dnew_state, g.dstate, a.rows * (W - 1) * D * element_bytes(a.dtype), stream);
    return e;
  }
  ConvRun q = plan(a.steps, a.rows, a.width, pack_of(a.width, a.dtype), true);
  q.g = g;
  q.params = static_cast<float*>(g.workspace);
  launch_any<true>(q, stream);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t groups = grid_of(q).x;
  const int32_t dw = (int32_t)(D * W), d = (int32_t)D;
  const SumsOut out = {{g.dweight, g.dbias, nullptr}, {dw, dw + d, dw + d}};
  return sums_launch(q.params, groups, dw + d,
                     reinterpret_cast<float*>(static_cast<char*>(g.workspace) + up(groups * (dw + d) * 4)), out,
                     stream);
}

hipError_t conv_step_launch(int32_t N, int32_t D, int32_t W, int32_t dtype, int32_t activation,
                            const void* x, int64_t x_row, const float* weight, const float* bias,
                            const void* state, const uint8_t* resets, void* y, int64_t y_row,
                            void* new_state, hipStream_t stream) {
  const int32_t V = dtype == POLICY_F32 ? 2 : 4;
  const StepRun q = {N, D, (D + V - 1) / V, x, state, weight, bias, resets, y, new_state, x_row, y_row,
                     activation == BLOCK_SILU};
  if (dtype == POLICY_F32)
    launch_step<F32, 2>(q, W, stream);
  else if (dtype == POLICY_BF16)
    launch_step<BF16, 4>(q, W, stream);
  else
    launch_step<F16, 4>(q, W, stream);
  return hipGetLastError();
}

}  // namespace rl
