// Gated linear recurrence over time-major rollouts (include/policy.h):
//   h_t = a_t m_t h_{t-1} + b_t,
// and its gradient, the same kind of recurrence run backwards:
//   G_t = a_t m_t (dh_t + G_{t+1}).
//
// A run of steps maps the state that enters it to the one that leaves it by
// an affine map (A, B): h -> A h + B.  A run that holds a done forgets what
// entered it; its A is stored as -0.0, a value no run without a done stores,
// so that the map then selects B instead of multiplying a possibly infinite
// or NaN state by zero.
//
// A workgroup of 8 waves owns a column of 64 lanes x V channels and walks
// time in tiles of 8 slots, one slot of S steps per wave.  A wave loads its
// slot into registers, folds it into its map, and leaves the map in LDS;
// after one barrier every wave folds the maps before its own onto the
// tile's carry, replays its slot from registers and stores it.  So each
// element is read and written once.  Where the columns are too few to fill
// the chip, time is also cut into chunks: a first launch writes every
// chunk's map to the workspace, and the main launch starts each chunk from
// the fold of the maps before it.  That reads x and gate twice.  The order
// of every fold depends on the sizes alone: results are deterministic.
#include "elem.hpp"
#include "policy.hpp"

namespace rl {

namespace {

constexpr int kWaves = 8;
constexpr int kSlot = 8;                  // steps per wave and tile
constexpr int kTile = kWaves * kSlot;     // steps per tile
constexpr float kReset = -0.0f;

struct Map {
  float a, b;
};

__device__ __forceinline__ bool is_reset(float a) { return __float_as_uint(a) == 0x80000000u; }
// A product of slopes in its stored form: +0 for either zero, -0 after a done.
__device__ __forceinline__ float stored_slope(float a, bool reset) {
  return reset ? kReset : a + 0.0f;
}
__device__ __forceinline__ float apply(Map m, float h) {
  return is_reset(m.a) ? m.b : __builtin_fmaf(m.a, h, m.b);
}
// first, then second
__device__ __forceinline__ Map chain(Map first, Map second) {
  Map r;
  r.a = stored_slope(first.a * second.a, is_reset(first.a) || is_reset(second.a));
  r.b = apply(second, first.b);
  return r;
}

// sigmoid(g) and sigmoid(-g), each to within a few fp32 roundings: with
// E = exp(-|g|) they are 1 / (1 + E) and E / (1 + E), so neither is formed
// by a difference.  E is 2^(hi + lo), hi + lo the product |g| log2(e) in two
// parts.
__device__ __forceinline__ void sigmoids(float g, float& a, float& keep) {
  float m = __builtin_fabsf(g);
  m = m > 200.0f ? 200.0f : m;  // (a NaN passes)
  const float hi = m * -1.44269502f;
  const float lo = __builtin_fmaf(m, -1.44269502f, -hi) + m * -1.92596300e-8f;
  float E = __builtin_amdgcn_exp2f(hi);
  E = __builtin_fmaf(E * lo, 0.693147182f, E);
  const float r = __builtin_amdgcn_rcpf(1.0f + E);
  const float s = E * r;
  a = g >= 0.0f ? r : s;
  keep = g >= 0.0f ? s : r;
}

struct RecurArgs {
  int32_t L, N, D;
  int32_t units;     // N * (D / V): lanes with work
  int32_t per_row;   // D / V
  int32_t chunk;     // steps per chunk (a multiple of kTile)
  int32_t chunks;
  int64_t x_step, x_row, g_step, g_row, h_step, h_row;
  int64_t dh_step, dh_row, dx_step, dx_row, dg_step, dg_row;
  const void *x, *gate, *h, *dh;
  const float *start;  // h0 / dh_last
  const float *h0;     // backward
  const uint8_t* dones;
  void *out, *dx, *dg;
  float* last;         // h_last / dh0
  Map* maps;           // [chunks][units][V]
};

// The carry into chunk `q` of a column: the maps of chunks [lo, hi) folded
// onto `c`, in the order lo, lo+1, ... (forward) or hi-1, hi-2, ...
// (backward).  Each wave folds a run of chunks; the runs are joined in LDS.
template <int V, bool BACK>
__device__ __forceinline__ void fold_chunks(const RecurArgs& p, int lo, int hi, int32_t u, int w,
                                            int lane, Map (&s)[kWaves][64][V], float (&c)[V]) {
  const int count = hi - lo;
  const int per = (count + kWaves - 1) / kWaves;
  Map m[V];
#pragma unroll
  for (int v = 0; v < V; ++v) m[v] = Map{1.0f, 0.0f};
  const int first = w * per, last = min(count, first + per);
#pragma unroll 4
  for (int j = first; j < last; ++j) {
    const int q = BACK ? hi - 1 - j : lo + j;
    const Map* e = p.maps + ((int64_t)q * p.units + u) * V;
#pragma unroll
    for (int v = 0; v < V; ++v) m[v] = chain(m[v], e[v]);
  }
#pragma unroll
  for (int v = 0; v < V; ++v) s[w][lane][v] = m[v];
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kWaves; ++j)
#pragma unroll
    for (int v = 0; v < V; ++v) c[v] = apply(s[j][lane][v], c[v]);
}

// MAPS: only the chunks' maps are formed (the first launch of a cut scan).
template <class T, int V, bool SIG, bool MAPS>
__global__ __launch_bounds__(64 * kWaves) void recur_forward_kernel(const RecurArgs p) {
  using raw = typename T::raw;
  __shared__ Map s_map[2][kWaves][64][V];
  const int lane = (int)threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int q = (int)blockIdx.y;
  const int32_t u0 = (int32_t)blockIdx.x * 64 + lane;
  const bool active = u0 < p.units;
  const int32_t u = active ? u0 : p.units - 1;  // idle lanes read a valid element
  const int32_t n = u / p.per_row;
  const int32_t d = (u - n * p.per_row) * V;
  const raw* x = static_cast<const raw*>(p.x) + n * p.x_row + d;
  const raw* gate = static_cast<const raw*>(p.gate) + n * p.g_row + d;
  raw* out = static_cast<raw*>(p.out) + n * p.h_row + d;
  const int64_t cell = (int64_t)n * p.D + d;
  const int32_t tb = q * p.chunk, te = min(p.L, tb + p.chunk);

  float c[V];  // state entering the tile (MAPS: the map's b so far, ca its slope)
  float ca[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    c[v] = 0.0f;
    ca[v] = 1.0f;
  }
  if (!MAPS) {
    if (p.start)
#pragma unroll
      for (int v = 0; v < V; ++v) c[v] = p.start[cell + v];
    if (q > 0) {
      fold_chunks<V, false>(p, 0, q, u, w, lane, s_map[1], c);
    }
  }

  int buf = 0;
  for (int32_t t0 = tb; t0 < te; t0 += kTile, buf ^= 1) {
    const int32_t ts = t0 + w * kSlot;
    Pack<T, V> xr[kSlot], gr[kSlot];
    uint32_t done = 0;
#pragma unroll
    for (int i = 0; i < kSlot; ++i) {
      const int32_t t = min(ts + i, te - 1);  // steps past the end: loaded, not used
      xr[i] = load_pack<T, V>(x + t * p.x_step);
      gr[i] = load_pack<T, V>(gate + t * p.g_step);
    }
    if (p.dones) {
      uint8_t db[kSlot];
#pragma unroll
      for (int i = 0; i < kSlot; ++i) {
        const int32_t t = max(min(ts + i, te - 1), 1);
        db[i] = p.dones[(int64_t)(t - 1) * p.N + n];
      }
#pragma unroll
      for (int i = 0; i < kSlot; ++i) done |= (ts + i > 0 && db[i] ? 1u : 0u) << i;
    }
    float a[kSlot][V], b[kSlot][V];
    Map m[V];
#pragma unroll
    for (int v = 0; v < V; ++v) m[v] = Map{1.0f, 0.0f};
    uint32_t forgets = 0;
#pragma unroll
    for (int i = 0; i < kSlot; ++i) {
      float xf[V], gf[V];
      widen_pack<T, V>(xr[i], xf);
      widen_pack<T, V>(gr[i], gf);
      const bool in = ts + i < te;
      const bool cut = (done >> i) & 1u;
      forgets |= in && cut;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (SIG) {
          float keep;
          sigmoids(gf[v], a[i][v], keep);
          b[i][v] = keep * xf[v];
        } else {
          a[i][v] = gf[v];
          b[i][v] = xf[v];
        }
        const float nb = cut ? b[i][v] : __builtin_fmaf(a[i][v], m[v].b, b[i][v]);
        m[v].b = in ? nb : m[v].b;
        m[v].a = in ? m[v].a * a[i][v] : m[v].a;
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      m[v].a = stored_slope(m[v].a, forgets != 0);
      s_map[buf][w][lane][v] = m[v];
    }
    __syncthreads();
    if (MAPS) {
#pragma unroll
      for (int j = 0; j < kWaves; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const Map r = chain(Map{ca[v], c[v]}, s_map[buf][j][lane][v]);
          ca[v] = r.a;
          c[v] = r.b;
        }
      continue;
    }
    float h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = 0.0f;
#pragma unroll
    for (int j = 0; j < kWaves; ++j) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (j == w) h[v] = c[v];
        c[v] = apply(s_map[buf][j][lane][v], c[v]);
      }
    }
#pragma unroll
    for (int i = 0; i < kSlot; ++i) {
      if (ts + i >= te) break;
      const bool cut = (done >> i) & 1u;
#pragma unroll
      for (int v = 0; v < V; ++v)
        h[v] = cut ? b[i][v] : __builtin_fmaf(a[i][v], h[v], b[i][v]);
      if (active) store_pack<T, V>(out + (ts + i) * p.h_step, narrow_pack<T, V>(h));
      if (ts + i == p.L - 1 && p.last && active) {
        const bool end = p.dones && p.dones[(int64_t)(p.L - 1) * p.N + n];
#pragma unroll
        for (int v = 0; v < V; ++v) p.last[cell + v] = end ? 0.0f : h[v];
      }
    }
  }
  if (MAPS && active && w == 0) {
    Map* e = p.maps + ((int64_t)q * p.units + u) * V;
#pragma unroll
    for (int v = 0; v < V; ++v) e[v] = Map{ca[v], c[v]};
  }
}

template <class T, int V, bool SIG, bool MAPS>
__global__ __launch_bounds__(64 * kWaves) void recur_backward_kernel(const RecurArgs p) {
  using raw = typename T::raw;
  __shared__ Map s_map[2][kWaves][64][V];
  const int lane = (int)threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int q = (int)blockIdx.y + (MAPS ? 1 : 0);  // the first chunk's map is not needed
  const int32_t u0 = (int32_t)blockIdx.x * 64 + lane;
  const bool active = u0 < p.units;
  const int32_t u = active ? u0 : p.units - 1;
  const int32_t n = u / p.per_row;
  const int32_t d = (u - n * p.per_row) * V;
  const raw* x = static_cast<const raw*>(p.x) + n * p.x_row + d;
  const raw* gate = static_cast<const raw*>(p.gate) + n * p.g_row + d;
  const raw* hs = static_cast<const raw*>(p.h) + n * p.h_row + d;
  const raw* dh = static_cast<const raw*>(p.dh) + n * p.dh_row + d;
  raw* dx = static_cast<raw*>(p.dx) + n * p.dx_row + d;
  raw* dg = static_cast<raw*>(p.dg) + n * p.dg_row + d;
  const int64_t cell = (int64_t)n * p.D + d;
  const int32_t tb = q * p.chunk, te = min(p.L, tb + p.chunk);

  float c[V], ca[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    c[v] = 0.0f;
    ca[v] = 1.0f;
  }
  if (!MAPS) {
    if (p.start && !(p.dones && p.dones[(int64_t)(p.L - 1) * p.N + n]))
#pragma unroll
      for (int v = 0; v < V; ++v) c[v] = p.start[cell + v];
    if (q < p.chunks - 1) {
      fold_chunks<V, true>(p, q + 1, p.chunks, u, w, lane, s_map[1], c);
    }
  }

  int buf = 0;
  for (int32_t t1 = te; t1 > tb; t1 -= kTile, buf ^= 1) {
    const int32_t top = t1 - 1 - w * kSlot;  // this wave's latest step
    Pack<T, V> gr[kSlot], dr[kSlot], xr[MAPS ? 1 : kSlot], hr[MAPS ? 1 : kSlot];
    uint32_t done = 0;
#pragma unroll
    for (int i = 0; i < kSlot; ++i) {
      const int32_t t = max(top - i, tb);
      gr[i] = load_pack<T, V>(gate + t * p.g_step);
      dr[i] = load_pack<T, V>(dh + t * p.dh_step);
      if (!MAPS) {
        if (SIG) xr[i] = load_pack<T, V>(x + t * p.x_step);
        hr[i] = load_pack<T, V>(hs + max(t - 1, 0) * p.h_step);
      }
    }
    if (p.dones) {
      uint8_t db[kSlot];
#pragma unroll
      for (int i = 0; i < kSlot; ++i)
        db[i] = p.dones[(int64_t)(max(max(top - i, tb), 1) - 1) * p.N + n];
#pragma unroll
      for (int i = 0; i < kSlot; ++i) done |= (top - i > 0 && db[i] ? 1u : 0u) << i;
    }
    float a[kSlot][V], k[kSlot][V];
    Map m[V];
#pragma unroll
    for (int v = 0; v < V; ++v) m[v] = Map{1.0f, 0.0f};
    uint32_t forgets = 0;
#pragma unroll
    for (int i = 0; i < kSlot; ++i) {
      float gf[V], df[V];
      widen_pack<T, V>(gr[i], gf);
      widen_pack<T, V>(dr[i], df);
      const bool in = top - i >= tb;
      const bool cut = (done >> i) & 1u;
      forgets |= in && cut;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (SIG)
          sigmoids(gf[v], a[i][v], k[i][v]);
        else
          a[i][v] = gf[v];
        const float nb = cut ? 0.0f : a[i][v] * (df[v] + m[v].b);
        m[v].b = in ? nb : m[v].b;
        m[v].a = in ? m[v].a * a[i][v] : m[v].a;
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      m[v].a = stored_slope(m[v].a, forgets != 0);
      s_map[buf][w][lane][v] = m[v];
    }
    __syncthreads();
    if (MAPS) {
#pragma unroll
      for (int j = 0; j < kWaves; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const Map r = chain(Map{ca[v], c[v]}, s_map[buf][j][lane][v]);
          ca[v] = r.a;
          c[v] = r.b;
        }
      continue;
    }
    float G[V];
#pragma unroll
    for (int v = 0; v < V; ++v) G[v] = 0.0f;
#pragma unroll
    for (int j = 0; j < kWaves; ++j) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (j == w) G[v] = c[v];
        c[v] = apply(s_map[buf][j][lane][v], c[v]);
      }
    }
#pragma unroll
    for (int i = 0; i < kSlot; ++i) {
      const int32_t t = top - i;
      if (t < tb) break;
      const bool cut = (done >> i) & 1u;
      float df[V], hf[V], xf[V], ox[V], og[V];
      widen_pack<T, V>(dr[i], df);
      widen_pack<T, V>(hr[MAPS ? 0 : i], hf);
      if (SIG) widen_pack<T, V>(xr[MAPS ? 0 : i], xf);
      if (t == 0) {
#pragma unroll
        for (int v = 0; v < V; ++v) hf[v] = p.h0 ? p.h0[cell + v] : 0.0f;
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float del = df[v] + G[v];
        const float prev = cut ? 0.0f : hf[v];
        if (SIG) {
          ox[v] = k[i][v] * del;
          og[v] = a[i][v] * ox[v] * (prev - xf[v]);
        } else {
          ox[v] = del;
          og[v] = cut ? 0.0f : del * prev;
        }
        G[v] = cut ? 0.0f : a[i][v] * del;
      }
      if (active) {
        store_pack<T, V>(dx + t * p.dx_step, narrow_pack<T, V>(ox));
        store_pack<T, V>(dg + t * p.dg_step, narrow_pack<T, V>(og));
        if (t == 0 && p.last) {
#pragma unroll
          for (int v = 0; v < V; ++v) p.last[cell + v] = G[v];
        }
      }
    }
  }
  if (MAPS && active && w == 0) {
    Map* e = p.maps + ((int64_t)q * p.units + u) * V;
#pragma unroll
    for (int v = 0; v < V; ++v) e[v] = Map{ca[v], c[v]};
  }
}

template <class T, int V>
__global__ __launch_bounds__(256) void recur_step_kernel(
    int32_t units, int32_t per_row, int32_t D, bool sig, const void* x_, int64_t x_row,
    const void* gate_, int64_t g_row, const float* state, const uint8_t* resets, void* h_,
    int64_t h_row, float* new_state) {
  using raw = typename T::raw;
  const int32_t u = (int32_t)(blockIdx.x * 256 + threadIdx.x);
  if (u >= units) return;
  const int32_t n = u / per_row;
  const int32_t d = (u - n * per_row) * V;
  const int64_t cell = (int64_t)n * D + d;
  float xf[V], gf[V], s[V];
  widen_pack<T, V>(load_pack<T, V>(static_cast<const raw*>(x_) + n * x_row + d), xf);
  widen_pack<T, V>(load_pack<T, V>(static_cast<const raw*>(gate_) + n * g_row + d), gf);
#pragma unroll
  for (int v = 0; v < V; ++v) s[v] = state[cell + v];
  const bool cut = resets && resets[n];
  float o[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float a = gf[v], b = xf[v];
    if (sig) {
      float keep;
      sigmoids(gf[v], a, keep);
      b = keep * xf[v];
    }
    o[v] = cut ? b : __builtin_fmaf(a, s[v], b);
    new_state[cell + v] = o[v];
  }
  store_pack<T, V>(static_cast<raw*>(h_) + n * h_row + d, narrow_pack<T, V>(o));
}

__global__ __launch_bounds__(256) void copy_or_zero_kernel(const float* from, float* to, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
    to[i] = from ? from[i] : 0.0f;
}

hipError_t copy_state(const float* from, float* to, int64_t n, hipStream_t stream) {
  if (!to || n == 0) return hipSuccess;
  const int64_t blocks = (n + 255) / 256;
  hipLaunchKernelGGL(copy_or_zero_kernel, dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(256),
                     0, stream, from, to, n);
  return hipGetLastError();
}

// Workgroups a launch should have before time is cut into chunks.
constexpr int64_t kWantGroups = 512;

// Chunks of time: one where the columns alone give the chip enough
// workgroups, else enough for kWantGroups, each of at least four tiles.
void cut(int32_t L, int64_t units, int32_t* chunk, int32_t* chunks) {
  const int64_t columns = units > 0 ? (units + 63) / 64 : 1;
  int64_t k = (kWantGroups + columns - 1) / columns;
  const int64_t most = L / (4 * kTile);
  if (k > most) k = most;
  if (columns >= kWantGroups / 2 || k <= 1) {
    *chunk = L;
    *chunks = 1;
    return;
  }
  int64_t steps = (L + k - 1) / k;
  steps = (steps + kTile - 1) / kTile * kTile;
  *chunk = (int32_t)steps;
  *chunks = (int32_t)((L + steps - 1) / steps);
}

bool strides_even(int64_t a, int64_t b) { return ((a | b) & 1) == 0; }

template <class T, int V, bool SIG, bool BACK>
hipError_t launch(RecurArgs p, hipStream_t stream) {
  p.per_row = p.D / V;
  p.units = p.N * p.per_row;
  cut(p.L, p.units, &p.chunk, &p.chunks);
  const unsigned columns = (unsigned)((p.units + 63) / 64);
  if (p.chunks > 1) {
    const dim3 grid(columns, (unsigned)(p.chunks - 1));
    if (BACK)
      hipLaunchKernelGGL((recur_backward_kernel<T, V, SIG, true>), grid, dim3(64 * kWaves), 0,
                         stream, p);
    else
      hipLaunchKernelGGL((recur_forward_kernel<T, V, SIG, true>), grid, dim3(64 * kWaves), 0,
                         stream, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const dim3 grid(columns, (unsigned)p.chunks);
  if (BACK)
    hipLaunchKernelGGL((recur_backward_kernel<T, V, SIG, false>), grid, dim3(64 * kWaves), 0,
                       stream, p);
  else
    hipLaunchKernelGGL((recur_forward_kernel<T, V, SIG, false>), grid, dim3(64 * kWaves), 0,
                       stream, p);
  return hipGetLastError();
}

template <class T, bool BACK>
hipError_t pick(const RecurArgs& p, bool sig, bool pairs, hipStream_t stream) {
  if (pairs)
    return sig ? launch<T, 2, true, BACK>(p, stream) : launch<T, 2, false, BACK>(p, stream);
  return sig ? launch<T, 1, true, BACK>(p, stream) : launch<T, 1, false, BACK>(p, stream);
}

template <bool BACK>
hipError_t pick_type(const RecurArgs& p, int32_t dtype, bool sig, bool pairs, hipStream_t stream) {
  switch (dtype) {
    case POLICY_F32: return pick<F32, BACK>(p, sig, pairs, stream);
    case POLICY_BF16: return pick<BF16, BACK>(p, sig, pairs, stream);
    default: return pick<F16, BACK>(p, sig, pairs, stream);
  }
}

}  // namespace

int64_t recur_workspace_bytes(int32_t L, int32_t N, int32_t D, int32_t dtype) {
  (void)dtype;
  int64_t most = 0;
  for (int v = 1; v <= 2; ++v) {
    if (D % v) continue;
    int32_t chunk, chunks;
    cut(L, (int64_t)N * (D / v), &chunk, &chunks);
    const int64_t bytes = chunks > 1 ? (int64_t)chunks * N * D * (int64_t)sizeof(Map) : 0;
    if (bytes > most) most = bytes;
  }
  return most;
}

hipError_t recur_forward_launch(const recur_args& a, hipStream_t stream) {
  const int64_t cells = (int64_t)a.rows * a.width;
  if (cells == 0) return hipSuccess;
  if (a.steps == 0) return copy_state(a.h0, a.h_last, cells, stream);
  RecurArgs p{};
  p.L = a.steps;
  p.N = a.rows;
  p.D = a.width;
  p.x_step = a.x_step;
  p.x_row = a.x_row;
  p.g_step = a.gate_step;
  p.g_row = a.gate_row;
  p.h_step = a.h_step;
  p.h_row = a.h_row;
  p.x = a.x;
  p.gate = a.gate;
  p.start = a.h0;
  p.dones = a.dones;
  p.out = a.h;
  p.last = a.h_last;
  p.maps = static_cast<Map*>(a.workspace);
  const size_t two = a.dtype == POLICY_F32 ? 8 : 4;
  const bool pairs = a.width % 2 == 0 && strides_even(a.x_step, a.x_row) &&
                     strides_even(a.gate_step, a.gate_row) && strides_even(a.h_step, a.h_row) &&
                     aligned_to(a.x, two) && aligned_to(a.gate, two) && aligned_to(a.h, two);
  return pick_type<false>(p, a.dtype, a.form == RECUR_SIGMOID, pairs, stream);
}

hipError_t recur_backward_launch(const recur_grad_args& a, hipStream_t stream) {
  const int64_t cells = (int64_t)a.rows * a.width;
  if (cells == 0) return hipSuccess;
  if (a.steps == 0) return copy_state(a.dh_last, a.dh0, cells, stream);
  RecurArgs p{};
  p.L = a.steps;
  p.N = a.rows;
  p.D = a.width;
  p.x_step = a.x_step;
  p.x_row = a.x_row;
  p.g_step = a.gate_step;
  p.g_row = a.gate_row;
  p.h_step = a.h_step;
  p.h_row = a.h_row;
  p.dh_step = a.dh_step;
  p.dh_row = a.dh_row;
  p.dx_step = a.dx_step;
  p.dx_row = a.dx_row;
  p.dg_step = a.dgate_step;
  p.dg_row = a.dgate_row;
  p.x = a.x;
  p.gate = a.gate;
  p.h = a.h;
  p.dh = a.dh;
  p.start = a.dh_last;
  p.h0 = a.h0;
  p.dones = a.dones;
  p.dx = a.dx;
  p.dg = a.dgate;
  p.last = a.dh0;
  p.maps = static_cast<Map*>(a.workspace);
  const bool sig = a.form == RECUR_SIGMOID;
  const size_t two = a.dtype == POLICY_F32 ? 8 : 4;
  const bool pairs =
      a.width % 2 == 0 && (!sig || (strides_even(a.x_step, a.x_row) && aligned_to(a.x, two))) &&
      strides_even(a.gate_step, a.gate_row) && strides_even(a.h_step, a.h_row) &&
      strides_even(a.dh_step, a.dh_row) && strides_even(a.dx_step, a.dx_row) &&
      strides_even(a.dgate_step, a.dgate_row) && aligned_to(a.gate, two) && aligned_to(a.h, two) &&
      aligned_to(a.dh, two) && aligned_to(a.dx, two) && aligned_to(a.dgate, two);
  return pick_type<true>(p, a.dtype, sig, pairs, stream);
}

hipError_t recur_step_launch(int32_t N, int32_t D, int32_t dtype, int32_t form, const void* x,
                             int64_t x_row, const void* gate, int64_t gate_row, const float* state,
                             const uint8_t* resets, void* h, int64_t h_row, float* new_state,
                             hipStream_t stream) {
  if ((int64_t)N * D == 0) return hipSuccess;
  const size_t two = dtype == POLICY_F32 ? 8 : 4;
  const bool pairs = D % 2 == 0 && ((x_row | gate_row | h_row) & 1) == 0 && aligned_to(x, two) &&
                     aligned_to(gate, two) && aligned_to(h, two);
  const int32_t per_row = pairs ? D / 2 : D, units = N * per_row;
  const dim3 grid((unsigned)(((int64_t)units + 255) / 256));
  const bool sig = form == RECUR_SIGMOID;
#define RL_STEP(T, V)                                                                            \
  hipLaunchKernelGGL((recur_step_kernel<T, V>), grid, dim3(256), 0, stream, units, per_row, D,   \
                     sig, x, x_row, gate, gate_row, state, resets, h, h_row, new_state)
  if (dtype == POLICY_F32) {
    if (pairs) RL_STEP(F32, 2); else RL_STEP(F32, 1);
  } else if (dtype == POLICY_BF16) {
    if (pairs) RL_STEP(BF16, 2); else RL_STEP(BF16, 1);
  } else {
    if (pairs) RL_STEP(F16, 2); else RL_STEP(F16, 1);
  }
#undef RL_STEP
  return hipGetLastError();
}

}  // namespace rl
