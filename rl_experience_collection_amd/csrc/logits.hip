// Penalties, bias and mask on logits, and their gradient (include/policy.h).
//
// A workgroup owns a tile: whole rows where a row is short, a run of one
// row's columns where it is long.  It counts the history's tokens that fall
// into the tile in LDS (integer adds, so their order does not matter), then
// passes over the tile once.  The gradient needs a logit only where a count
// is not zero (its sign picks the factor) and loads just those.
#include <initializer_list>

#include "elem.hpp"
#include "policy.hpp"

namespace rl {

namespace {

constexpr int kThreads = 256;
constexpr int kTile = 4096;     // elements of a tile, at most
constexpr int kTileRows = 256;  // rows of a tile, at most
constexpr int kShortRow = 2048; // rows up to this long are tiled whole
constexpr float kBanned = -__builtin_inff();

struct LogitsArgs {
  logits_args a;
  const void* dout;   // gradient
  void* out;          // out or dlogits
  int64_t dout_row, out_row;
  int32_t tile_rows, tile_cols;  // rows of a tile (1 for long rows), columns of a tile
  int32_t spread;                // lanes that share a row's history (a power of two)
  uint32_t magic;                // for a quotient by vocab (short rows)
  bool penalties;
};

struct RowTerms {
  float rho, alpha, beta;
  int64_t mask;  // offset of the row's mask, or -1
};

__device__ __forceinline__ RowTerms row_terms(const logits_args& a, int64_t r) {
  RowTerms t;
  t.rho = a.repetition_rows ? a.repetition_rows[r] : a.repetition;
  t.alpha = a.presence_rows ? a.presence_rows[r] : a.presence;
  t.beta = a.frequency_rows ? a.frequency_rows[r] : a.frequency;
  t.mask = -1;
  if (a.mask_kind != LOGITS_MASK_NONE) {
    const int64_t m = a.mask_rows ? (int64_t)a.mask_rows[r] : (a.mask_count == 1 ? 0 : r);
    if (m >= 0 && m < a.mask_count) t.mask = m * a.mask_row;
  }
  return t;
}

__device__ __forceinline__ bool allowed(const logits_args& a, int64_t at, int32_t v) {
  if (at < 0) return true;
  if (a.mask_kind == LOGITS_MASK_BYTES) return static_cast<const uint8_t*>(a.mask)[at + v] != 0;
  return (static_cast<const uint32_t*>(a.mask)[at + (v >> 5)] >> (v & 31)) & 1u;
}

__device__ __forceinline__ uint32_t quotient(uint32_t n, uint32_t d, uint32_t magic) {
  return d == 1 ? n : __umulhi(n, magic);
}

// FLAT: tiles of whole rows whose elements lie one after another, addressed
// as one run.  Otherwise a tile is a run of columns of one row.
template <class T, int V, bool GRAD, bool FLAT>
__global__ __launch_bounds__(kThreads) void logits_kernel(LogitsArgs p) {
  using raw = typename T::raw;
  __shared__ uint32_t s_count[kTile];
  __shared__ RowTerms s_row[FLAT ? kTileRows : 1];
  const logits_args& a = p.a;
  const int tid = threadIdx.x;
  const int32_t vocab = a.vocab;
  const int64_t tiles = FLAT ? (a.rows + p.tile_rows - 1) / p.tile_rows : a.rows;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int64_t r0 = FLAT ? tile * p.tile_rows : tile;
    const int32_t rows = FLAT ? (int32_t)min((int64_t)p.tile_rows, a.rows - r0) : 1;
    const int32_t c0 = FLAT ? 0 : (int32_t)blockIdx.y * p.tile_cols;
    const int32_t cols = FLAT ? vocab : min(p.tile_cols, vocab - c0);
    const int32_t n = FLAT ? rows * vocab : cols;
    __syncthreads();  // the previous tile's counts are read
    for (int32_t r = tid; r < rows; r += kThreads) s_row[r] = row_terms(a, r0 + r);
    if (p.penalties) {
      for (int32_t e = tid; e < n; e += kThreads) s_count[e] = 0;
      __syncthreads();
      const int lane = tid & (p.spread - 1), step = kThreads / p.spread;
      for (int32_t r = tid / p.spread; r < rows; r += step) {
        const int32_t* h = a.history + (r0 + r) * a.history_row;
        const int32_t len = a.history_len ? min(max(a.history_len[r0 + r], 0), a.history_width)
                                          : a.history_width;
        for (int32_t i = lane; i < len; i += p.spread) {
          const int32_t v = h[i];
          if (v >= c0 && v - c0 < cols) atomicAdd(&s_count[r * vocab + v - c0], 1u);
        }
      }
    }
    __syncthreads();
    const raw* in = static_cast<const raw*>(GRAD ? p.dout : a.logits) +
                    r0 * (GRAD ? p.dout_row : a.logits_row) + c0;
    const raw* z0 = static_cast<const raw*>(a.logits) + r0 * a.logits_row + c0;
    raw* out = static_cast<raw*>(p.out) + r0 * p.out_row + c0;
    for (int32_t e = tid * V; e < n; e += kThreads * V) {
      float f[V];
      widen_pack<T, V>(load_pack<T, V>(in + e), f);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int32_t r = FLAT ? (int32_t)quotient((uint32_t)(e + i), (uint32_t)vocab, p.magic) : 0;
        const int32_t v = FLAT ? e + i - r * vocab : c0 + e + i;
        const RowTerms& t = s_row[r];
        const uint32_t count = p.penalties ? s_count[e + i] : 0u;
        if (GRAD) {
          if (count) {
            const float z = T::widen(z0[e + i]);
            f[i] = z > 0.0f ? f[i] / t.rho : f[i] * t.rho;
          }
          if (!allowed(a, t.mask, v)) f[i] = 0.0f;
        } else {
          if (count) {
            f[i] = f[i] > 0.0f ? f[i] / t.rho : f[i] * t.rho;
            f[i] -= t.alpha;
            f[i] -= t.beta * (float)count;
          }
          if (a.bias) f[i] += a.bias[(r0 + r) * a.bias_row + v];
          if (!allowed(a, t.mask, v)) f[i] = kBanned;
        }
      }
      store_pack<T, V>(out + e, narrow_pack<T, V>(f));
    }
  }
}

// dbias: a workgroup sums one run of rows for 64 columns, its four waves
// taking every fourth row; the runs' sums are joined in order afterwards.
constexpr int kBiasRuns = 256;

template <class T>
__global__ __launch_bounds__(kThreads) void bias_run_kernel(LogitsArgs p, float* partial,
                                                            int64_t run_rows) {
  using raw = typename T::raw;
  __shared__ float s_sum[4][64];
  const logits_args& a = p.a;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t v = (int64_t)blockIdx.x * 64 + lane;
  const int64_t lo = blockIdx.y * run_rows, hi = min(a.rows, lo + run_rows);
  float sum = 0.0f;
  if (v < a.vocab) {
    const raw* g = static_cast<const raw*>(p.dout) + v;
    for (int64_t r = lo + w; r < hi; r += 4) {
      const RowTerms t = row_terms(a, r);
      if (allowed(a, t.mask, (int32_t)v)) sum += T::widen(g[r * p.dout_row]);
    }
  }
  s_sum[w][lane] = sum;
  __syncthreads();
  if (w == 0 && v < a.vocab)
    partial[blockIdx.y * (int64_t)a.vocab + v] =
        (s_sum[0][lane] + s_sum[1][lane]) + (s_sum[2][lane] + s_sum[3][lane]);
}

__global__ __launch_bounds__(kThreads) void bias_join_kernel(const float* partial, int32_t runs,
                                                             int32_t vocab, float* dbias) {
  const int64_t v = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (v >= vocab) return;
  float sum = 0.0f;
  for (int32_t k = 0; k < runs; ++k) sum += partial[(int64_t)k * vocab + v];
  dbias[v] = sum;
}

__global__ __launch_bounds__(kThreads) void clear_kernel(float* p, int64_t n) {
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i < n) p[i] = 0.0f;
}

int64_t bias_runs(int64_t rows) { return rows < 4 * kBiasRuns ? (rows + 3) / 4 : kBiasRuns; }

bool neutral(const logits_args& a) {
  return !a.history || a.history_width == 0 ||
         (!a.repetition_rows && !a.presence_rows && !a.frequency_rows && a.repetition == 1.0f &&
          a.presence == 0.0f && a.frequency == 0.0f);
}

template <class T, int V, bool GRAD>
hipError_t launch_tiles(LogitsArgs p, bool flat, hipStream_t stream) {
  const int64_t most = (int64_t)1 << 22;  // larger grids loop
  if (flat) {
    const int64_t tiles = (p.a.rows + p.tile_rows - 1) / p.tile_rows;
    hipLaunchKernelGGL((logits_kernel<T, V, GRAD, true>),
                       dim3((unsigned)(tiles < most ? tiles : most)), dim3(kThreads), 0, stream, p);
  } else {
    const unsigned runs = (unsigned)((p.a.vocab + p.tile_cols - 1) / p.tile_cols);
    const int64_t cap = 1 << 16;
    hipLaunchKernelGGL((logits_kernel<T, V, GRAD, false>),
                       dim3((unsigned)(p.a.rows < cap ? p.a.rows : cap), runs), dim3(kThreads), 0,
                       stream, p);
  }
  return hipGetLastError();
}

template <class T, bool GRAD>
hipError_t tiles(LogitsArgs p, hipStream_t stream) {
  const logits_args& a = p.a;
  const int64_t V = a.vocab;
  const bool dense = p.out_row == V && (GRAD ? p.dout_row == V : true) &&
                     (a.logits_row == V || (GRAD && !p.penalties));
  const bool flat = V <= kShortRow && dense;
  constexpr int kPack = 16 / T::kBytes;
  if (flat) {
    // a multiple of a pack's elements, so that tiles start on packs
    int64_t rows = kTile / V;
    if (rows > kTileRows) rows = kTileRows;
    if (rows > kPack) rows = rows / kPack * kPack;
    p.tile_rows = (int32_t)rows;
    p.magic = (uint32_t)((1ull << 32) / V + 1);
  } else {
    p.tile_rows = 1;
    p.tile_cols = kTile;
  }
  int pack = kPack;
  auto fits = [&](int v) {
    const size_t bytes = (size_t)v * T::kBytes;
    const bool tail = flat ? (p.tile_rows * V) % v == 0 && (a.rows * V) % v == 0
                           : V % v == 0 && p.out_row % v == 0 &&
                                 (GRAD ? p.dout_row : a.logits_row) % v == 0;
    return tail && aligned_to(GRAD ? p.dout : a.logits, bytes) && aligned_to(p.out, bytes);
  };
  while (pack > 1 && !fits(pack)) pack /= 2;
  p.spread = 1;
  while (p.spread < 64 && p.spread < a.history_width) p.spread *= 2;
  if (!flat) p.spread = kThreads;
  switch (pack) {
    case 8: return launch_tiles<T, (T::kBytes == 2 ? 8 : 4), GRAD>(p, flat, stream);
    case 4: return launch_tiles<T, 4, GRAD>(p, flat, stream);
    case 2: return launch_tiles<T, 2, GRAD>(p, flat, stream);
    default: return launch_tiles<T, 1, GRAD>(p, flat, stream);
  }
}

template <bool GRAD>
hipError_t any_type(const LogitsArgs& p, hipStream_t stream) {
  switch (p.a.dtype) {
    case POLICY_F32: return tiles<F32, GRAD>(p, stream);
    case POLICY_BF16: return tiles<BF16, GRAD>(p, stream);
    default: return tiles<F16, GRAD>(p, stream);
  }
}

}  // namespace

hipError_t logits_forward_launch(const logits_args& a, void* out, int64_t out_row,
                                 hipStream_t stream) {
  if (a.rows == 0 || a.vocab == 0) return hipSuccess;
  LogitsArgs p{};
  p.a = a;
  p.out = out;
  p.out_row = out_row;
  p.penalties = !neutral(a);
  return any_type<false>(p, stream);
}

bool logits_gradient_reads_logits(const logits_args& a) {
  return a.history && a.history_width > 0 && (a.repetition_rows || a.repetition != 1.0f);
}

int64_t logits_workspace_bytes(int64_t rows, int32_t vocab) {
  return bias_runs(rows) * (int64_t)vocab * 4;
}

hipError_t logits_backward_launch(const logits_args& a, const void* dout, int64_t dout_row,
                                  void* dlogits, int64_t dlogits_row, float* dbias,
                                  void* workspace, hipStream_t stream) {
  if (a.vocab == 0) return hipSuccess;
  LogitsArgs p{};
  p.a = a;
  p.dout = dout;
  p.dout_row = dout_row;
  p.out = dlogits;
  p.out_row = dlogits_row;
  p.penalties = logits_gradient_reads_logits(a);
  hipError_t e = hipSuccess;
  if (dbias) {
    // before dlogits, which may replace dout
    if (a.rows == 0) {
      hipLaunchKernelGGL(clear_kernel, dim3((unsigned)(((int64_t)a.vocab + 255) / 256)),
                         dim3(kThreads), 0, stream, dbias, (int64_t)a.vocab);
      return hipGetLastError();
    }
    const int64_t runs = bias_runs(a.rows), run_rows = (a.rows + runs - 1) / runs;
    float* partial = static_cast<float*>(workspace);
    const dim3 grid((unsigned)(((int64_t)a.vocab + 63) / 64), (unsigned)runs);
    switch (a.dtype) {
      case POLICY_F32:
        hipLaunchKernelGGL(bias_run_kernel<F32>, grid, dim3(kThreads), 0, stream, p, partial, run_rows);
        break;
      case POLICY_BF16:
        hipLaunchKernelGGL(bias_run_kernel<BF16>, grid, dim3(kThreads), 0, stream, p, partial, run_rows);
        break;
      default:
        hipLaunchKernelGGL(bias_run_kernel<F16>, grid, dim3(kThreads), 0, stream, p, partial, run_rows);
    }
    if ((e = hipGetLastError()) != hipSuccess) return e;
    hipLaunchKernelGGL(bias_join_kernel, dim3((unsigned)(((int64_t)a.vocab + 255) / 256)),
                       dim3(kThreads), 0, stream, partial, (int32_t)runs, a.vocab, dbias);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (a.rows == 0 || !dlogits) return hipSuccess;
  return any_type<true>(p, stream);
}

}  // namespace rl
