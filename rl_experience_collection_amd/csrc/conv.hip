// Short causal convolution over a rollout: forward, gradient, single step
// (include/block.h).
//
// A thread takes some of an episode's channels and a chunk of steps. It keeps
// the last W - 1 inputs in registers, so that an input is read once, and reads
// those before its chunk again.  Steps go in groups of W (or 4), the next
// group's loads in flight while one is worked on; within a group the window is
// a ring whose places are known when the kernel is compiled, so that nothing
// moves.  A done clears the window, which is all that keeps episodes apart.
//
// The gradient runs in the same direction: step t adds to the gradients of the
// inputs t - W + 1 .. t, which wait in W registers until no later step adds
// to them (W - 1 steps past the chunk's end are formed again for that).
// Weights' gradients are summed by threads over their steps, by a workgroup in
// LDS, and over workgroups by column sums.
//
// HBM bounds both: 500 x 8192 x 64 bf16 with 4 taps takes 184 us forward (5.7
// TB/s) and 315 us backward (5.0 TB/s).  A step is a launch of 3.4 us.
#include <algorithm>

#include "block.hpp"
#include "buffer.hpp"
#include "elem.hpp"

namespace rl {

namespace {

constexpr int kThreads = 256;
// Steps of a group: a multiple of the W places of a ring.
constexpr int group_of(int W) { return W <= 2 ? 4 : W; }

struct ConvRun {
  conv_grad_args g;  // forward: g.f alone
  int32_t packs;     // of a row
  int32_t across;    // of those, a workgroup's
  int32_t rows;      // (chunk, n) pairs of a workgroup
  int32_t chunk, chunks;
  int64_t items;     // chunks * N
  uint32_t groups;   // workgroups that share a run of packs; the next run's follow them
  float* params;     // gradient: [workgroups][D (W + 1)]
};

constexpr float kLog2e = 1.44269504f;
__device__ __forceinline__ float sigmoid_of(float v) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-v * kLog2e));
}

// Which rows and channels a thread has.  (One number for all workgroups: a wide
// row has more runs of packs than a grid's second dimension holds.)
struct ConvLane {
  int32_t n, d0, fresh, t0, t1, row, pack, first;  // first: the workgroup's first pack
  uint32_t group;
  bool active;
  __device__ __forceinline__ ConvLane(const ConvRun& q, int V) {
    group = blockIdx.x % q.groups;
    first = (int32_t)(blockIdx.x / q.groups) * q.across;
    row = threadIdx.x / q.across;
    pack = first + threadIdx.x % q.across;
    const int64_t item = (int64_t)group * q.rows + row;
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

// The inputs before step t0, age j at place W - j, and how many belong to its
// episode.
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
    for (int v = 0; v < V; ++v) win[W - i][v] = 0.0f;
    if (!same) continue;
    age = i;
    if (t >= 0)
      widen_pack<T, V>(
          load_pack<T, V>(static_cast<const raw*>(a.x) + t * a.x_step + k.n * a.x_row + k.d0), win[W - i]);
    else if (a.state)
      widen_pack<T, V>(load_pack<T, V>(static_cast<const raw*>(a.state) +
                                       ((int64_t)k.n * (W - 1) + (W - 1 + t)) * a.width + k.d0),
                       win[W - i]);
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

// A row of one of the arrays as a thread walks along it.
template <class T, int V>
struct Walk {
  char* p;
  int64_t step;
  __device__ __forceinline__ Walk(const void* base, int64_t step_, int64_t row, const ConvLane& k, int32_t t)
      : p(const_cast<char*>(static_cast<const char*>(base)) + (t * step_ + k.n * row + k.d0) * T::kBytes),
        step(step_ * T::kBytes) {}
  // The next A of the `left` steps that remain; those past the end repeat the
  // last one.  (No branch: a wait would stand where its ways meet.)
  template <int A>
  __device__ __forceinline__ void load(int32_t left, Pack<T, V> (&x)[A]) {
#pragma unroll
    for (int i = 0; i < A; ++i) {
      x[i] = load_pack<T, V>(reinterpret_cast<const typename T::raw*>(p));
      p += i + 1 < left ? step : 0;
    }
  }
  __device__ __forceinline__ void store(const float (&f)[V]) {
    store_pack<T, V>(reinterpret_cast<typename T::raw*>(p), narrow_pack<T, V>(f));
    p += step;
  }
};

// The dones before a thread's steps, as loaded.
struct WalkDones {
  const uint8_t* p;
  int64_t step;
  bool any;
  __device__ __forceinline__ WalkDones(const conv_args& a, const ConvLane& k)
      : p(a.dones ? a.dones + (int64_t)max(k.t0 - 1, 0) * a.rows + k.n : reinterpret_cast<const uint8_t*>(a.weight)),
        step(a.dones ? a.rows : 0),
        any(a.dones != nullptr) {}
  template <int A>
  __device__ __forceinline__ void load(int32_t t, int32_t left, uint8_t (&x)[A]) {
#pragma unroll
    for (int i = 0; i < A; ++i) {
      x[i] = *p;
      p += t + i > 0 && i + 1 < left ? step : 0;  // (step 0 has none before it)
    }
  }
  __device__ __forceinline__ bool cuts(uint8_t x, int32_t t) const { return any && t > 0 && x != 0; }
};

// Clears the window but for the step at place `now`.
template <int V, int W>
__device__ __forceinline__ void forget(float (&win)[W][V], int now) {
#pragma unroll
  for (int j = 0; j < W; ++j) {
    if (j == now) continue;
#pragma unroll
    for (int v = 0; v < V; ++v) win[j][v] = 0.0f;
  }
}
// The input of age j (the steps since it) of group step i lies at this place.
template <int W>
constexpr int place(int i, int j) {
  return ((i - j) % W + W) % W;
}

template <class T, int V, int W>
__global__ void __launch_bounds__(kThreads) conv_forward_kernel(const ConvRun q) {
  using raw = typename T::raw;
  constexpr int A = group_of(W);
  const conv_args& a = q.g.f;
  const ConvLane k(q, V);
  if (!k.active) return;
  float w[W][V], bias[V], win[W][V];
  load_weights<V, W>(a, k.d0, w, bias);
  open_window<T, V, W>(a, k, win);
  Walk<T, V> x(a.x, a.x_step, a.x_row, k, k.t0), y(a.y, a.y_step, a.y_row, k, k.t0);
  const bool silu = a.activation == BLOCK_SILU;

  Pack<T, V> next[A];
  uint8_t next_dones[A];
  WalkDones dones(a, k);
  x.load(k.t1 - k.t0, next);
  dones.load(k.t0, k.t1 - k.t0, next_dones);
  no_stores(a.y, A);
  int32_t t = k.t0;
  const auto group = [&](auto whole) {
    Pack<T, V> now[A];
    bool cut[A];
#pragma unroll
    for (int i = 0; i < A; ++i) {
      now[i] = next[i];
      cut[i] = dones.cuts(next_dones[i], t + i);
    }
    x.load(k.t1 - t - A, next);
    dones.load(t + A, k.t1 - t - A, next_dones);
#pragma unroll
    for (int i = 0; i < A; ++i) {
      if (!decltype(whole)::value && t + i >= k.t1) continue;
      if (cut[i]) forget<V, W>(win, place<W>(i, 0));
      widen_pack<T, V>(now[i], win[place<W>(i, 0)]);
      float out[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float p = bias[v];
#pragma unroll
        for (int j = W - 1; j >= 0; --j) p = __builtin_fmaf(w[j][v], win[place<W>(i, j)][v], p);
        out[v] = silu ? p * sigmoid_of(p) : p;
      }
      y.store(out);
    }
    t += A;
  };
  while (t + A <= k.t1) group(std::true_type());
  const int32_t rest = k.t1 - t;
  if (rest > 0) group(std::false_type());
  if (k.t1 == a.steps && a.new_state) {
    const bool ended = cut_before(a, k.n, a.steps);
#pragma unroll
    for (int j = 1; j < W; ++j) {
      // (age j of the step after the last: the last group may have ended early)
      float left[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        left[v] = 0.0f;
#pragma unroll
        for (int r = 0; r < W; ++r)
          if (rest % W == r) left[v] = win[place<W>(r, j)][v];
        if (ended) left[v] = 0.0f;
      }
      store_pack<T, V>(
          static_cast<raw*>(a.new_state) + ((int64_t)k.n * (W - 1) + (W - 1 - j)) * a.width + k.d0,
          narrow_pack<T, V>(left));
    }
  }
}

template <class T, int V, int W>
__global__ void __launch_bounds__(kThreads) conv_backward_kernel(const ConvRun q) {
  using raw = typename T::raw;
  constexpr int A = group_of(W);
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
    // acc: the gradients of the last W inputs, as far as they are known, in the
    // places of the inputs
    float w[W][V], bias[V], win[W][V], acc[W][V];
    load_weights<V, W>(a, k.d0, w, bias);
    int32_t age = open_window<T, V, W>(a, k, win);
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
      for (int v = 0; v < V; ++v) acc[j][v] = 0.0f;
    const int32_t end = min(k.t1 + W - 1, a.steps);
    Walk<T, V> x(a.x, a.x_step, a.x_row, k, k.t0), dy(g.dy, g.dy_step, g.dy_row, k, k.t0),
        dx(g.dx, g.dx_step, g.dx_row, k, k.t0);
    const bool silu = a.activation == BLOCK_SILU;

    // The gradient of the input of step e, where it is this chunk's.
    const auto emit = [&](int32_t e, const float(&f)[V]) {
      if (e >= k.t0 && e < k.t1)
        dx.store(f);
      else if (e < 0 && k.t0 == 0 && g.dstate)
        store_pack<T, V>(static_cast<raw*>(g.dstate) + ((int64_t)k.n * (W - 1) + (W - 1 + e)) * a.width + k.d0,
                         narrow_pack<T, V>(f));
    };
    Pack<T, V> next_x[A], next_d[A];
    uint8_t next_dones[A];
    WalkDones dones(a, k);
    x.load(end - k.t0, next_x);
    dy.load(end - k.t0, next_d);
    dones.load(k.t0, end - k.t0, next_dones);
    int32_t t = k.t0;
    // `inside`: all steps lie in the chunk, and so do the inputs whose
    // gradients they complete.
    const auto group = [&](auto inside) {
      constexpr bool kInside = decltype(inside)::value;
      Pack<T, V> now_x[A], now_d[A];
      bool cut[A];
#pragma unroll
      for (int i = 0; i < A; ++i) {
        now_x[i] = next_x[i];
        now_d[i] = next_d[i];
        cut[i] = dones.cuts(next_dones[i], t + i);
      }
      x.load(end - t - A, next_x);
      dy.load(end - t - A, next_d);
      dones.load(t + A, end - t - A, next_dones);
#pragma unroll
      for (int i = 0; i < A; ++i) {
        if (!kInside && t + i >= end) continue;
        if (kInside || t + i > k.t0) age = min(age + 1, W - 1);
        if (cut[i]) {
          age = 0;
          forget<V, W>(win, place<W>(i, 0));
        }
        widen_pack<T, V>(now_x[i], win[place<W>(i, 0)]);
        float dp[V];
        widen_pack<T, V>(now_d[i], dp);
        if (silu) {
#pragma unroll
          for (int v = 0; v < V; ++v) {
            float p = bias[v];
#pragma unroll
            for (int j = W - 1; j >= 0; --j) p = __builtin_fmaf(w[j][v], win[place<W>(i, j)][v], p);
            const float s = sigmoid_of(p);
            dp[v] *= s * __builtin_fmaf(p, 1.0f - s, 1.0f);
          }
        }
        if (kInside || t + i < k.t1) {
#pragma unroll
          for (int v = 0; v < V; ++v) {
            db[v] += dp[v];
#pragma unroll
            for (int j = 0; j < W; ++j) dw[j][v] = __builtin_fmaf(dp[v], win[place<W>(i, j)][v], dw[j][v]);
          }
        }
        if (age == W - 1) {
#pragma unroll
          for (int j = 1; j < W; ++j)
#pragma unroll
            for (int v = 0; v < V; ++v)
              acc[place<W>(i, j)][v] = __builtin_fmaf(w[j][v], dp[v], acc[place<W>(i, j)][v]);
        } else {  // inputs of another episode take nothing
#pragma unroll
          for (int j = 1; j < W; ++j)
#pragma unroll
            for (int v = 0; v < V; ++v)
              acc[place<W>(i, j)][v] =
                  j <= age ? __builtin_fmaf(w[j][v], dp[v], acc[place<W>(i, j)][v]) : acc[place<W>(i, j)][v];
        }
#pragma unroll
        for (int v = 0; v < V; ++v) acc[place<W>(i, 0)][v] = w[0][v] * dp[v];
        if (kInside)
          dx.store(acc[place<W>(i, W - 1)]);
        else
          emit(t + i - (W - 1), acc[place<W>(i, W - 1)]);
      }
      t += A;
    };
    // (the first group completes inputs from before the chunk)
    group(std::false_type());
    no_stores(g.dx, A);
    while (t + A <= k.t1) group(std::true_type());
    while (t < end) group(std::false_type());
    if (end == a.steps) {
      // The last inputs wait for no step; new_state sends them theirs.
      age = cut_before(a, k.n, a.steps) ? 0 : min(age + 1, W - 1);
      const int32_t rest = (end - k.t0) % W;
#pragma unroll
      for (int j = W - 1; j > 0; --j) {
        // (age j of step L)
        float last[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          last[v] = 0.0f;
#pragma unroll
          for (int r = 0; r < W; ++r)
            if (rest == r) last[v] = acc[place<W>(r, j)][v];
        }
        if (g.dnew_state && j <= age) {
          float ds[V];
          widen_pack<T, V>(load_pack<T, V>(static_cast<const raw*>(g.dnew_state) +
                                           ((int64_t)k.n * (W - 1) + (W - 1 - j)) * a.width + k.d0),
                           ds);
#pragma unroll
          for (int v = 0; v < V; ++v) last[v] += ds[v];
        }
        emit(a.steps - j, last);
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
      const int32_t pack = k.first + c / V;
      if (pack >= q.packs) continue;
      const int32_t d0 = min(pack * V, a.width - V);
      if (c % V < pack * V - d0) continue;  // (counted in the pack before)
      float sum = 0.0f;
      for (int32_t r = 0; r < q.rows; ++r) sum += s_sum[r * q.across + c / V][c % V];
      const int64_t d = d0 + c % V;
      q.params[(int64_t)k.group * a.width * (W + 1) + (j < W ? d * W + (W - 1 - j) : (int64_t)a.width * W + d)] =
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
  const uint32_t id = blockIdx.x * kThreads + threadIdx.x;  // (below 2^29)
  const int64_t n = id / (uint32_t)q.packs;
  if (n >= q.N) return;
  const int32_t d0 = (int32_t)(id % (uint32_t)q.packs) * V;
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
  q.groups = (uint32_t)((q.items + q.rows - 1) / q.rows);
  q.params = nullptr;
  return q;
}
// Elements of a thread: 16 bytes going forward (8 from five taps on), 4
// elements of any type backward (2), where a thread holds four rows of W values
// for each.
constexpr int pack_for(int bytes, int W, bool grad) {
  return grad ? (W <= 4 ? 4 : 2) : (W <= 4 ? 16 : 8) / bytes;
}
int32_t pack_of(int32_t D, int32_t W, int32_t dtype, bool grad) {
  const int32_t v = pack_for(dtype == POLICY_F32 ? 4 : 2, W, grad);
  return D >= v ? v : 1;
}
// (below 2^23: what N * D < 2^28 leaves, workgroups half full)
dim3 grid_of(const ConvRun& q) { return dim3(q.groups * (uint32_t)((q.packs + q.across - 1) / q.across)); }

template <class T, int W, bool GRAD>
void launch(const ConvRun& q, hipStream_t stream) {
  constexpr int V = pack_for(T::kBytes, W, GRAD);
  const dim3 grid = grid_of(q);
  if constexpr (GRAD) {
    if (q.g.f.width >= V)
      conv_backward_kernel<T, V, W><<<grid, kThreads, 0, stream>>>(q);
    else
      conv_backward_kernel<T, 1, W><<<grid, kThreads, 0, stream>>>(q);
  } else {
    if (q.g.f.width >= V)
      conv_forward_kernel<T, V, W><<<grid, kThreads, 0, stream>>>(q);
    else
      conv_forward_kernel<T, 1, W><<<grid, kThreads, 0, stream>>>(q);
  }
}
template <class T, bool GRAD>
void launch_taps(const ConvRun& q, hipStream_t stream) {
  switch (q.g.f.taps) {
    case 1: return launch<T, 1, GRAD>(q, stream);
    case 2: return launch<T, 2, GRAD>(q, stream);
    case 3: return launch<T, 3, GRAD>(q, stream);
    case 4: return launch<T, 4, GRAD>(q, stream);
    case 5: return launch<T, 5, GRAD>(q, stream);
    case 6: return launch<T, 6, GRAD>(q, stream);
    case 7: return launch<T, 7, GRAD>(q, stream);
    default: return launch<T, 8, GRAD>(q, stream);
  }
}
template <bool GRAD>
void launch_any(const ConvRun& q, hipStream_t stream) {
  if (q.g.f.dtype == POLICY_F32)
    launch_taps<F32, GRAD>(q, stream);
  else if (q.g.f.dtype == POLICY_BF16)
    launch_taps<BF16, GRAD>(q, stream);
  else
    launch_taps<F16, GRAD>(q, stream);
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
  ConvRun q = plan(a.steps, a.rows, a.width, pack_of(a.width, a.taps, a.dtype, false), false);
  q.g = {};
  q.g.f = a;
  launch_any<false>(q, stream);
  return hipGetLastError();
}

int64_t conv_workspace_bytes(int32_t L, int32_t N, int32_t D, int32_t W, int32_t dtype) {
  if (L == 0 || N == 0 || D == 0) return 0;
  const ConvRun q = plan(L, N, D, pack_of(D, W, dtype, true), true);
  const int64_t groups = q.groups;
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
  ConvRun q = plan(a.steps, a.rows, a.width, pack_of(a.width, a.taps, a.dtype, true), true);
  q.g = g;
  q.params = static_cast<float*>(g.workspace);
  launch_any<true>(q, stream);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t groups = q.groups;
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
