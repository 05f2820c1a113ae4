// The norms after and before a block, with its gate, dropout, scales and
// residual between them, and their gradient (include/block.h).
//
// A row lies in the registers of a group of threads (8 to 1024, 8 elements
// each), so that it is read once for both norms; the next row's loads
// are in flight meanwhile.  Sums over a row meet by lane exchanges, beyond a
// wave in LDS.  The gradient forms the row again from the forward call's
// inputs and the two stored factors (8 bytes a row), rather than from a
// stream that was rounded when it was stored, and a thread sums the weights'
// gradients of its own columns over all rows that it takes.
//
// HBM bounds them: 1,024,000 x 128 bf16 with gate and dropout takes 262 us
// forward (5.0 TB/s) and 430 us backward (4.9 TB/s).  Where they fit the caches,
// latency: 4099 x 5001 fp16 takes 32 and 71 us.
#include <algorithm>

#include "block.hpp"
#include "buffer.hpp"
#include "elem.hpp"
#include "philox.hpp"

namespace rl {

namespace {

constexpr float kLog2e = 1.44269504f;

struct NormRun {
  norm_grad_args g;  // forward: g.f alone
  DropRule rule;
  void *stream, *normed;  // forward
  float* stats;
  int64_t stream_row, normed_row;
  float inv_width;
  bool past;      // outputs are stored past the caches
  float* params;  // gradient: [workgroups][2 or 3][D]
  void *dresidual, *dbranch, *dgate;  // gradient: the outputs, or a row for all of what is not wanted
  int64_t dresidual_row, dbranch_row, dgate_row;
};

enum GateKind { kNoGate, kRowGate, kChannelGate };

// ------------------------------------------------------------ sums of a row
template <int CTRL>
__device__ __forceinline__ float lane_dpp(float x) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xF, 0xF, true));
}
// Over 8, 16 or 64 lanes; every lane gets it.
template <int N>
__device__ __forceinline__ float lanes_sum(float x) {
  x += lane_dpp<0xB1>(x);   // quad_perm 1, 0, 3, 2
  x += lane_dpp<0x4E>(x);   // quad_perm 2, 3, 0, 1
  x += lane_dpp<0x141>(x);  // row_half_mirror
  if constexpr (N >= 16) x += lane_dpp<0x140>(x);  // row_mirror
  if constexpr (N == 64) {
    const int lane = threadIdx.x & 63;
    x += lane_xor16f(x, lane);
    x += lane_xor32f(x, lane);
  }
  return x;
}

// TPR up to 64: that many threads a row, 256 a workgroup.  Above: a workgroup a
// row, of as many waves as the row needs, at most TPR threads.
constexpr int threads_of(int TPR) { return TPR > 256 ? TPR : 256; }
template <int TPR>
__device__ __forceinline__ uint32_t row_threads() {
  return TPR <= 64 ? TPR : blockDim.x;
}
template <int TPR>
__device__ __forceinline__ uint32_t row_thread() {
  return TPR <= 64 ? threadIdx.x % TPR : threadIdx.x;
}

// Sums over the threads of a row.  The two halves of the LDS array are used in
// turn: a wave that writes one again has passed the barrier of the other, which
// no wave reaches before it has read the first.
template <int TPR>
struct RowSum {
  int turn = 0;
  __device__ __forceinline__ float operator()(float x, float (&s)[2][16]) {
    if constexpr (TPR <= 64) {
      return lanes_sum<TPR>(x);
    } else {
      x = lanes_sum<64>(x);
      if ((threadIdx.x & 63) == 0) s[turn][threadIdx.x >> 6] = x;
      __syncthreads();
      const uint32_t wave = threadIdx.x & 15;
      x = lanes_sum<16>(wave < blockDim.x / 64 ? s[turn][wave] : 0.0f);
      turn ^= 1;
      return x;
    }
  }
};

// ---------------------------------------------------------- a thread's share
// Packs of V elements: start, and how many of its first elements belong to the
// pack before (a row's last pack is moved back into the row).
template <class T, int V, int TPR, int K>
struct Share {
  int32_t at[K], fresh[K];
  bool whole;
  __device__ __forceinline__ explicit Share(int32_t D) {
    whole = true;
#pragma unroll
    for (int i = 0; i < K; ++i) {
      const int32_t e = ((int32_t)row_thread<TPR>() + row_threads<TPR>() * i) * V;
      at[i] = min(e, D - V);
      fresh[i] = e - at[i];
      whole = whole && fresh[i] == 0;
    }
    whole = __ballot(!whole) == 0;
  }
  using Row = Pack<T, V>[K];
  __device__ __forceinline__ void load(const void* p, int64_t row, int64_t r, Row& x) const {
#pragma unroll
    for (int i = 0; i < K; ++i)
      x[i] = load_pack<T, V>(static_cast<const typename T::raw*>(p) + r * row + at[i]);
  }
  // (Threads past a row's end, and rows past the last one, write what the last
  // pack or row holds once more: a branch would hide a store from the count of
  // those that a wait for later loads may leave under way.)
  template <bool PAST>
  __device__ __forceinline__ void store(void* p, int64_t row, int64_t r, const float (&f)[K][V]) const {
#pragma unroll
    for (int i = 0; i < K; ++i)
      store_pack<T, V>(static_cast<typename T::raw*>(p) + r * row + at[i], narrow_pack<T, V>(f[i]), PAST);
  }
  // The compiler keeps `from` and `to` apart: loads into the one may start while
  // the other is in use, and nothing has to be moved when they have arrived.
  static __device__ __forceinline__ void take(const Row& from, Row& to) {
#pragma unroll
    for (int i = 0; i < K; ++i) {
      if constexpr (V * T::kBytes == 16) {
        const quad_value x = __builtin_bit_cast(quad_value, from[i]);
        quad_value y;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t word;
          asm volatile("v_mov_b32 %0, %1" : "=v"(word) : "v"(x[w]));
          y[w] = word;
        }
        to[i] = __builtin_bit_cast(Pack<T, V>, y);
      } else {
        to[i] = from[i];
      }
    }
  }
  __device__ __forceinline__ void weights(const float* w, float (&f)[K][V]) const {
#pragma unroll
    for (int i = 0; i < K; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v) f[i][v] = w ? w[at[i] + v] : 1.0f;
  }
  // The sum of the products, each element once.  (Only waves that have a row's
  // last pack have anything to leave out.)
  __device__ __forceinline__ float dot(const float (&a)[K][V], const float (&b)[K][V]) const {
    float sum = 0.0f;
    if (whole) {
#pragma unroll
      for (int i = 0; i < K; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) sum = __builtin_fmaf(a[i][v], b[i][v], sum);
    } else {
#pragma unroll
      for (int i = 0; i < K; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) sum = v >= fresh[i] ? __builtin_fmaf(a[i][v], b[i][v], sum) : sum;
    }
    return sum;
  }
};

// Which of the V elements from i are kept: bit j for element i + j.  (A pack of
// four uses half of its draw, one that starts inside eight elements draws twice.)
template <int V>
__device__ __forceinline__ uint32_t kept_bits(const DropRule& rule, uint64_t seed, uint64_t i) {
  const uint32_t off = (uint32_t)i & 7;
  const uint4 d = drop_draws(rule, seed, i >> 3);
  uint32_t bits = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) bits |= (draw_of(d, j) >= rule.drop ? 1u : 0u) << j;
  if (off + V > 8) {
    const uint4 n = drop_draws(rule, seed, (i >> 3) + 1);
#pragma unroll
    for (int j = 0; j < 8; ++j) bits |= (draw_of(n, j) >= rule.drop ? 1u : 0u) << (8 + j);
  }
  return bits >> off;
}

// act(g) and its slope
__device__ __forceinline__ void activate(int32_t kind, float g, float& act, float& slope) {
  if (kind == BLOCK_NONE) {
    act = g;
    slope = 1.0f;
    return;
  }
  const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-g * kLog2e));
  if (kind == BLOCK_SIGMOID) {
    act = s;
    slope = s * (1.0f - s);
  } else {
    act = g * s;
    slope = s * __builtin_fmaf(g, 1.0f - s, 1.0f);
  }
}

// Waves a SIMD: 6, so that two rows of up to 768 threads share a compute unit,
// where that leaves enough registers (none are spilled).  With gate and dropout
// 419 MB a tensor of bf16 take 502 us at width 5001 so, 591 where the compiler is
// not told, but 555 and 531 at 600; other widths and gates are within 3%.
template <class T>
constexpr int forward_waves(int TPR, int gate) {
  return TPR > 64 && !(T::kBytes == 4 && gate == kRowGate) ? 6 : 1;
}

template <class T, int V, int TPR, int K, int GATE, bool PAST>
__global__ void __launch_bounds__(threads_of(TPR), forward_waves<T>(TPR, GATE)) norm_forward_kernel(const NormRun q) {
  const norm_args& a = q.g.f;
  constexpr int kRows = TPR <= 64 ? 256 / TPR : 1;
  __shared__ float s_sum[2][16];
  const Share<T, V, TPR, K> own(a.width);
  RowSum<TPR> row_sum;
  const bool branch = a.branch != nullptr, drops = q.rule.drop != 0;
  const uint64_t seed = q.rule.seed_at ? *q.rule.seed_at : q.rule.seed;
  float w[K][V], bw[K][V], gc[K][V];
  own.weights(a.weight, w);
  own.weights(a.branch_weight, bw);
  if (GATE == kChannelGate) {
    own.weights(static_cast<const float*>(a.gate), gc);
#pragma unroll
    for (int i = 0; i < K; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float slope;
        activate(a.activation, gc[i][v], gc[i][v], slope);
      }
  }
  typename Share<T, V, TPR, K>::Row res, br, ga;
#pragma unroll
  for (int i = 0; i < K; ++i) br[i] = Pack<T, V>{};
  const int64_t step = (int64_t)gridDim.x * kRows;
  // (all of a workgroup's threads go round as often: they meet in row_sum)
  int64_t next = (int64_t)blockIdx.x * kRows + (TPR <= 64 ? threadIdx.x / TPR : 0);
  const auto fetch = [&]() {
    next = next < a.rows ? next : a.rows - 1;
    own.load(a.residual, a.residual_row, next, res);
    if (branch) own.load(a.branch, a.branch_row, next, br);
    if (GATE == kRowGate) own.load(a.gate, a.gate_row, next, ga);
  };
  fetch();
  no_stores(q.stream, 2 * K);
  for (int64_t first = (int64_t)blockIdx.x * kRows; first < a.rows; first += step) {
    const int64_t r = next;
    typename Share<T, V, TPR, K>::Row xr, xb, xg;
    own.take(res, xr);
    own.take(br, xb);
    if (GATE == kRowGate) own.take(ga, xg);
    next += step;
    fetch();
    float s[K][V], b[K][V], g[K][V];
#pragma unroll
    for (int i = 0; i < K; ++i) {
      widen_pack<T, V>(xr[i], s[i]);
      widen_pack<T, V>(xb[i], b[i]);
      if (GATE == kRowGate) widen_pack<T, V>(xg[i], g[i]);
    }
    float inv_b = 1.0f;
    if (branch && a.branch_norm)
      inv_b = __builtin_amdgcn_rsqf(__builtin_fmaf(row_sum(own.dot(b, b), s_sum), q.inv_width, a.eps));
#pragma unroll
    for (int i = 0; i < K; ++i) {
      uint32_t kept = ~0u;
      if (branch && drops) kept = kept_bits<V>(q.rule, seed, (uint64_t)(r * a.width + own.at[i]));
#pragma unroll
      for (int v = 0; v < V; ++v) {
        s[i][v] *= a.residual_scale;
        if (!branch) continue;
        float z = b[i][v] * inv_b * bw[i][v];
        if (GATE == kChannelGate) z *= gc[i][v];
        if (GATE == kRowGate) {
          float act, slope;
          activate(a.activation, g[i][v], act, slope);
          z *= act;
        }
        if (drops) z = (kept >> v) & 1u ? z * q.rule.scale : 0.0f;
        s[i][v] = __builtin_fmaf(a.branch_scale, z, s[i][v]);
      }
    }
    const float inv = __builtin_amdgcn_rsqf(__builtin_fmaf(row_sum(own.dot(s, s), s_sum), q.inv_width, a.eps));
    if (q.stats && row_thread<TPR>() == 0) {
      q.stats[2 * r] = inv_b;
      q.stats[2 * r + 1] = inv;
    }
    own.template store<PAST>(q.stream, q.stream_row, r, s);
#pragma unroll
    for (int i = 0; i < K; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v) s[i][v] *= inv * w[i][v];
    own.template store<PAST>(q.normed, q.normed_row, r, s);
  }
}

// What a thread needs of its own columns at every row, in LDS: the registers
// that it would take are worth more to the rows in flight (1,024,000 x 128
// bf16 took 443 us so, 459 with weights in registers).
template <int K, int V, int THREADS>
struct OwnColumns {
  static constexpr int kQuads = K * V / 4;
  float4 v[kQuads > 0 ? kQuads : 1][THREADS];
  __device__ __forceinline__ void put(const float (&f)[K][V]) {
    if constexpr (V == 1) {
      v[0][threadIdx.x].x = f[0][0];
    } else {
#pragma unroll
      for (int i = 0; i < K; ++i)
#pragma unroll
        for (int q = 0; q < V / 4; ++q)
          v[i * (V / 4) + q][threadIdx.x] = make_float4(f[i][4 * q], f[i][4 * q + 1], f[i][4 * q + 2], f[i][4 * q + 3]);
    }
  }
  __device__ __forceinline__ void get(int i, float (&f)[V]) const {
    if constexpr (V == 1) {
      f[0] = v[0][threadIdx.x].x;
    } else {
#pragma unroll
      for (int q = 0; q < V / 4; ++q) {
        const float4 x = v[i * (V / 4) + q][threadIdx.x];
        f[4 * q] = x.x;
        f[4 * q + 1] = x.y;
        f[4 * q + 2] = x.z;
        f[4 * q + 3] = x.w;
      }
    }
  }
};

template <class T, int V, int TPR, int K, int GATE, bool PAST>
__global__ void __launch_bounds__(threads_of(TPR)) norm_backward_kernel(const NormRun q) {
  const norm_grad_args& p = q.g;
  const norm_args& a = p.f;
  constexpr int kThreads = threads_of(TPR), kRows = TPR <= 64 ? 256 / TPR : 1;
  __shared__ float s_sum[2][16];
  __shared__ OwnColumns<K, V, kThreads> s_w, s_bw;
  __shared__ OwnColumns<GATE == kChannelGate ? K : 1, GATE == kChannelGate ? V : 1, GATE == kChannelGate ? kThreads : 1> s_act;
  const Share<T, V, TPR, K> own(a.width);
  RowSum<TPR> row_sum;
  const bool branch = a.branch != nullptr, drops = q.rule.drop != 0;
  const uint64_t seed = q.rule.seed_at ? *q.rule.seed_at : q.rule.seed;
  float dw[K][V], dbw[K][V], dgc[K][V];
  own.weights(a.weight, dw);
  s_w.put(dw);
  own.weights(a.branch_weight, dw);
  s_bw.put(dw);
  if constexpr (GATE == kChannelGate) {
    own.weights(static_cast<const float*>(a.gate), dw);
#pragma unroll
    for (int i = 0; i < K; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float slope;
        activate(a.activation, dw[i][v], dw[i][v], slope);
      }
    s_act.put(dw);
  }
#pragma unroll
  for (int i = 0; i < K; ++i)
#pragma unroll
    for (int v = 0; v < V; ++v) dw[i][v] = dbw[i][v] = dgc[i][v] = 0.0f;
  typename Share<T, V, TPR, K>::Row res, br, ga, ds, dn;
#pragma unroll
  for (int i = 0; i < K; ++i) br[i] = ds[i] = dn[i] = Pack<T, V>{};  // those that are not given
  float inv_b_next = 1.0f, inv_next = 1.0f;
  const int64_t step = (int64_t)gridDim.x * kRows;
  int64_t wanted = (int64_t)blockIdx.x * kRows + (TPR <= 64 ? threadIdx.x / TPR : 0);
  const auto fetch = [&]() {
    const int64_t at = wanted < a.rows ? wanted : a.rows - 1;
    own.load(a.residual, a.residual_row, at, res);
    if (branch) own.load(a.branch, a.branch_row, at, br);
    if (GATE == kRowGate) own.load(a.gate, a.gate_row, at, ga);
    if (p.dstream) own.load(p.dstream, p.dstream_row, at, ds);
    if (p.dnormed) own.load(p.dnormed, p.dnormed_row, at, dn);
    inv_b_next = p.stats[2 * at];
    inv_next = p.stats[2 * at + 1];
  };
  fetch();
  no_stores(q.dresidual, K * (GATE == kRowGate ? 3 : 2));
  for (int64_t first = (int64_t)blockIdx.x * kRows; first < a.rows; first += step) {
    // (a row past the end repeats the last one and counts in no sum)
    const bool mine = kRows == 1 || wanted < a.rows;
    const int64_t r = mine ? wanted : a.rows - 1;
    float inv_b, inv;
    asm volatile("v_mov_b32 %0, %1" : "=v"(inv_b) : "v"(inv_b_next));
    asm volatile("v_mov_b32 %0, %1" : "=v"(inv) : "v"(inv_next));
    // s: the normed stream; u: the normed branch; g: the gate; d: dstream; e: dnormed weight
    float s[K][V], u[K][V], g[K][V], d[K][V], e[K][V];
    uint32_t kept[K];
    typename Share<T, V, TPR, K>::Row xr, xb, xg, xs, xn;
    own.take(res, xr);
    own.take(br, xb);
    if (GATE == kRowGate) own.take(ga, xg);
    own.take(ds, xs);
    own.take(dn, xn);
    wanted += step;
    fetch();
#pragma unroll
    for (int i = 0; i < K; ++i) {
      widen_pack<T, V>(xr[i], s[i]);
      widen_pack<T, V>(xb[i], u[i]);
      widen_pack<T, V>(xs[i], d[i]);
      widen_pack<T, V>(xn[i], e[i]);
      if (GATE == kRowGate) widen_pack<T, V>(xg[i], g[i]);
    }
#pragma unroll
    for (int i = 0; i < K; ++i) {
      float w[V], bw[V], act[V];
      s_w.get(i, w);
      s_bw.get(i, bw);
      if constexpr (GATE == kChannelGate) s_act.get(i, act);
      kept[i] = ~0u;
      if (branch && drops) kept[i] = kept_bits<V>(q.rule, seed, (uint64_t)(r * a.width + own.at[i]));
#pragma unroll
      for (int v = 0; v < V; ++v) {
        s[i][v] *= a.residual_scale;
        if (branch) {
          u[i][v] *= inv_b;
          float z = u[i][v] * bw[v], slope;
          if (GATE == kRowGate) activate(a.activation, g[i][v], act[v], slope);
          if (GATE != kNoGate) z *= act[v];
          if (drops) z = (kept[i] >> v) & 1u ? z * q.rule.scale : 0.0f;
          s[i][v] = __builtin_fmaf(a.branch_scale, z, s[i][v]);
        }
        s[i][v] *= inv;
      }
      if (mine) {
#pragma unroll
        for (int v = 0; v < V; ++v) dw[i][v] = __builtin_fmaf(e[i][v], s[i][v], dw[i][v]);
      }
#pragma unroll
      for (int v = 0; v < V; ++v) e[i][v] *= w[v];
    }
    float mean = 0.0f;
    if (p.dnormed) {
      mean = row_sum(own.dot(e, s), s_sum) * q.inv_width;
#pragma unroll
      for (int i = 0; i < K; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) d[i][v] = __builtin_fmaf(inv, __builtin_fmaf(-s[i][v], mean, e[i][v]), d[i][v]);
    }
#pragma unroll
    for (int i = 0; i < K; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v) s[i][v] = a.residual_scale * d[i][v];
    own.template store<PAST>(q.dresidual, q.dresidual_row, r, s);
    if (!branch) {
      no_stores(q.dresidual, K * (GATE == kRowGate ? 2 : 1));
      continue;
    }
    // (the empty statements keep the compiler from holding across the sum what
    // LDS or two transcendental operations give again)
    asm volatile("" ::: "memory");
#pragma unroll
    for (int i = 0; i < K; ++i) {
      float bw[V], act[V];
      s_bw.get(i, bw);
      if constexpr (GATE == kChannelGate) s_act.get(i, act);
#pragma unroll
      for (int v = 0; v < V; ++v) d[i][v] *= a.branch_scale;
      if (drops) {
        // What a dropped place holds does not matter: its factors become 0 with
        // its gradient.  (The normed branch is a factor of the whole row.)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const bool keep = (kept[i] >> v) & 1u;
          d[i][v] = keep ? d[i][v] * q.rule.scale : 0.0f;
          bw[v] = keep ? bw[v] : 0.0f;
          if (GATE == kRowGate) g[i][v] = keep ? g[i][v] : 0.0f;
          if (GATE == kChannelGate) act[v] = keep ? act[v] : 0.0f;
        }
        if (GATE != kNoGate && !a.branch_norm) {
#pragma unroll
          for (int v = 0; v < V; ++v) u[i][v] = (kept[i] >> v) & 1u ? u[i][v] : 0.0f;
        }
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float dz = d[i][v], dact = dz * (u[i][v] * bw[v]);
        float slope;
        if (GATE == kRowGate) {
          asm("" : "+v"(g[i][v]));
          activate(a.activation, g[i][v], act[v], slope);
          g[i][v] = dact * slope;
        }
        if (GATE == kChannelGate) d[i][v] = dact;
        e[i][v] = GATE == kNoGate ? dz : dz * act[v];
      }
      if (mine) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          if (GATE == kChannelGate) dgc[i][v] += d[i][v];
          dbw[i][v] = __builtin_fmaf(e[i][v], u[i][v], dbw[i][v]);
        }
      }
#pragma unroll
      for (int v = 0; v < V; ++v) e[i][v] *= bw[v];
    }
    if (GATE == kRowGate) own.template store<PAST>(q.dgate, q.dgate_row, r, g);
    if (a.branch_norm) {
      mean = row_sum(own.dot(e, u), s_sum) * q.inv_width;
#pragma unroll
      for (int i = 0; i < K; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) e[i][v] = inv_b * __builtin_fmaf(-u[i][v], mean, e[i][v]);
    }
    own.template store<PAST>(q.dbranch, q.dbranch_row, r, e);
  }
  if constexpr (GATE == kChannelGate) {
    // the activation's slope is the same for every row
    float gate[K][V];
    own.weights(static_cast<const float*>(a.gate), gate);
#pragma unroll
    for (int i = 0; i < K; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float act, slope;
        activate(a.activation, gate[i][v], act, slope);
        // (of a channel that was dropped in every row the slope does not matter either)
        dgc[i][v] = drops && dgc[i][v] == 0.0f ? 0.0f : dgc[i][v] * slope;
      }
  }
  // the workgroup's sums over its rows, pack by pack
  __shared__ float s_part[kRows > 1 ? kThreads : 1][V];
  const auto put = [&](int which, const float(&f)[K][V]) {
#pragma unroll
    for (int i = 0; i < K; ++i) {
      float* out = q.params + ((int64_t)blockIdx.x * (GATE == kChannelGate ? 3 : 2) + which) * a.width;
      if constexpr (kRows == 1) {
#pragma unroll
        for (int v = 0; v < V; ++v)
          if (v >= own.fresh[i]) out[own.at[i] + v] = f[i][v];
      } else {
        __syncthreads();
#pragma unroll
        for (int v = 0; v < V; ++v) s_part[threadIdx.x][v] = f[i][v];
        __syncthreads();
        for (int32_t c = threadIdx.x; c < TPR * V; c += kThreads) {
          const int32_t start = (c / V + TPR * i) * V, at = min(start, a.width - V);
          if (c % V < start - at) continue;
          float sum = 0.0f;
          for (int32_t row = 0; row < kRows; ++row) sum += s_part[row * TPR + c / V][c % V];
          out[at + c % V] = sum;
        }
      }
    }
  };
  put(0, dw);
  put(1, dbw);
  if (GATE == kChannelGate) put(2, dgc);
}

// Threads of a row, of 8 elements each: 8, 16 or 64, then as many waves as it
// needs.  (Those past its end go over its last pack again: of 64, 32 at width
// 256, and 47 at 129.)
int32_t threads_for(int32_t D) {
  return D <= 64 ? 8 : D <= 128 ? 16 : D <= 512 ? 64 : (D + 511) / 512 * 64;
}
// Waves of a compute unit: 20 going forward, 16 where there is no branch, whose
// work would hide the loads of more (419 MB a tensor of bf16: 299 us at width 600
// so, 332 with 20; 233 either way at 8000), 12 backward.
constexpr int32_t kGradWaves = 12;
int32_t waves_of(const norm_args& a, bool grad) { return grad ? kGradWaves : a.branch ? 20 : 16; }
// Workgroups: what is resident on 256 compute units, so that a workgroup reads
// its weights and writes their gradients once for many rows.
uint32_t groups_of(int64_t R, int32_t D, int32_t waves) {
  const int32_t threads = threads_for(D), rows = threads <= 64 ? 256 / threads : 1;
  const int64_t most = 256 * std::max(1, waves * 64 / (threads <= 64 ? 256 : threads));
  return (uint32_t)std::min((R + rows - 1) / rows, most);
}

template <class T, int V, int TPR, int K, int GATE, bool GRAD>
void launch(const NormRun& q, hipStream_t stream) {
  const int32_t D = q.g.f.width;
  const dim3 grid(groups_of(q.g.f.rows, D, waves_of(q.g.f, GRAD))), threads(TPR <= 64 ? 256 : threads_for(D));
  if constexpr (GRAD)
    q.past ? norm_backward_kernel<T, V, TPR, K, GATE, true><<<grid, threads, 0, stream>>>(q)
           : norm_backward_kernel<T, V, TPR, K, GATE, false><<<grid, threads, 0, stream>>>(q);
  else
    q.past ? norm_forward_kernel<T, V, TPR, K, GATE, true><<<grid, threads, 0, stream>>>(q)
           : norm_forward_kernel<T, V, TPR, K, GATE, false><<<grid, threads, 0, stream>>>(q);
}
// (768 threads may hold 168 registers each, 1024 hold 128.)
template <class T, int GATE, bool GRAD>
void launch_shape(const NormRun& q, hipStream_t stream) {
  constexpr int V = 16 / T::kBytes, K = 8 / V;
  const int32_t threads = threads_for(q.g.f.width);
  if (q.g.f.width < V) return launch<T, 1, 8, 1, GATE, GRAD>(q, stream);
  if (threads == 8) return launch<T, V, 8, K, GATE, GRAD>(q, stream);
  if (threads == 16) return launch<T, V, 16, K, GATE, GRAD>(q, stream);
  if (threads == 64) return launch<T, V, 64, K, GATE, GRAD>(q, stream);
  if (threads <= 256) return launch<T, V, 256, K, GATE, GRAD>(q, stream);
  if (threads <= 768) return launch<T, V, 768, K, GATE, GRAD>(q, stream);
  return launch<T, V, 1024, K, GATE, GRAD>(q, stream);
}
template <class T, bool GRAD>
void launch_gate(const NormRun& q, hipStream_t stream) {
  const norm_args& a = q.g.f;
  if (!a.gate || !a.branch) return launch_shape<T, kNoGate, GRAD>(q, stream);
  if (a.gate_row) return launch_shape<T, kRowGate, GRAD>(q, stream);
  return launch_shape<T, kChannelGate, GRAD>(q, stream);
}
template <bool GRAD>
void launch_any(const NormRun& q, hipStream_t stream) {
  if (q.g.f.dtype == POLICY_F32)
    launch_gate<F32, GRAD>(q, stream);
  else if (q.g.f.dtype == POLICY_BF16)
    launch_gate<BF16, GRAD>(q, stream);
  else
    launch_gate<F16, GRAD>(q, stream);
}

int64_t up(int64_t bytes) { return (bytes + 255) / 256 * 256; }

// Whether outputs go past the caches: large ones (kPastBytes), but for rows of less
// than 1 KB that are no whole lines of 128 bytes, whose lines two workgroups fill.
// Forward of 419 MB a tensor, past and through: bf16 of width 200, no branch 319 and
// 286 us, with one 431 and 391; fp32 of 100, 403 and 351; bf16 of 600, 432 and 437.
bool stored_past(int64_t R, int64_t row_bytes) {
  return R * row_bytes > kPastBytes && (row_bytes % 128 == 0 || row_bytes >= 1024);
}

NormRun run_of(const norm_args& a) {
  NormRun q = {};
  q.g.f = a;
  q.rule = drop_rule(a.drop, a.seed, a.seed_at, a.offset);
  q.inv_width = (float)(1.0 / a.width);
  q.past = stored_past(a.rows, (int64_t)a.width * (a.dtype == POLICY_F32 ? 4 : 2));
  return q;
}

}  // namespace

hipError_t norm_forward_launch(const norm_args& a, void* stream_out, int64_t stream_row,
                               void* normed, int64_t normed_row, float* stats, hipStream_t stream) {
  NormRun q = run_of(a);
  q.stream = stream_out;
  q.stream_row = stream_row;
  q.normed = normed;
  q.normed_row = normed_row;
  q.stats = stats;
  launch_any<false>(q, stream);
  return hipGetLastError();
}

int64_t norm_workspace_bytes(int64_t R, int32_t D, int32_t dtype) {
  if (R == 0) return 0;
  const int64_t groups = groups_of(R, D, kGradWaves);
  return up(groups * 3 * D * 4) + up(sums_floats(groups, 3 * D) * 4) + up(D * 4);
}

hipError_t norm_backward_launch(const norm_grad_args& g, hipStream_t stream) {
  const norm_args& a = g.f;
  const int64_t D = a.width;
  const bool channel = a.gate && a.gate_row == 0;
  if (a.rows == 0) {
    hipError_t e = hipSuccess;
    if (g.dweight) e = copy_or_clear_launch(nullptr, g.dweight, D * 4, stream);
    if (e == hipSuccess && g.dbranch_weight) e = copy_or_clear_launch(nullptr, g.dbranch_weight, D * 4, stream);
    if (e == hipSuccess && channel && g.dgate) e = copy_or_clear_launch(nullptr, g.dgate, D * 4, stream);
    return e;
  }
  NormRun q = run_of(a);
  q.g = g;
  q.params = static_cast<float*>(g.workspace);
  // (the workspace ends with a row of D values)
  char* nowhere = static_cast<char*>(g.workspace) + norm_workspace_bytes(a.rows, a.width, a.dtype) - up(D * 4);
  const auto put = [&](void* wanted, void*& p, int64_t& row) {
    p = wanted ? wanted : nowhere;
    row = wanted ? D : 0;
  };
  put(g.dresidual, q.dresidual, q.dresidual_row);
  put(g.dbranch, q.dbranch, q.dbranch_row);
  put(channel ? nullptr : g.dgate, q.dgate, q.dgate_row);
  launch_any<true>(q, stream);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !(g.dweight || g.dbranch_weight || (channel && g.dgate))) return e;
  const int64_t groups = groups_of(a.rows, a.width, kGradWaves);
  const int32_t d = a.width, columns = (channel ? 3 : 2) * d;
  const SumsOut out = {{g.dweight, g.dbranch_weight, channel ? static_cast<float*>(g.dgate) : nullptr},
                       {d, 2 * d, columns}};
  return sums_launch(q.params, groups, columns,
                     reinterpret_cast<float*>(static_cast<char*>(g.workspace) + up(groups * columns * 4)), out,
                     stream);
}

}  // namespace rl
