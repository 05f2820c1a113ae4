// Scaled embedding lookup and its gradient (include/policy.h).
//
// The lookup is a copy of rows: a workgroup owns a run of output rows whose
// elements its threads walk in order, one pack per access.
//
// The gradient sums the rows of dout that share an index.  The positions are
// sorted by index, stably, by a radix sort of digits of at most 9 bits; an
// index outside the vocabulary sorts behind it.  The sorted list is cut into
// pieces of equal length, and a thread owns one pack of columns of one
// piece: it walks the piece in order, adds in fp32 and, at each change of
// index, writes the finished row.  A row that crosses the border of pieces
// leaves a partial sum in each of them, and a last kernel over the
// vocabulary joins those in order and clears the rows no index names.  So
// dout is read once, whatever the skew of the indices, and every sum has a
// fixed order.
#include <initializer_list>

#include "elem.hpp"
#include "policy.hpp"

namespace rl {

namespace {

constexpr int kThreads = 256;

// --------------------------------------------------------------- the lookup
// Quotient of n by d for n * d < 2^32 (magic = floor(2^32 / d) + 1, d > 1).
__device__ __forceinline__ uint32_t quotient(uint32_t n, uint32_t d, uint32_t magic) {
  return d == 1 ? n : __umulhi(n, magic);
}
uint32_t magic_of(uint32_t d) { return (uint32_t)((1ull << 32) / d + 1); }

constexpr int kPacks = 8;  // packs per thread of the lookup

__device__ __forceinline__ int64_t index_at(const void* p, bool wide, int64_t i) {
  return wide ? static_cast<const int64_t*>(p)[i] : static_cast<const int32_t*>(p)[i];
}

template <class T, int V>
__global__ __launch_bounds__(kThreads) void embed_forward_kernel(EmbedForward a, int32_t per_row,
                                                                 int32_t rows, uint32_t magic) {
  using raw = typename T::raw;
  const raw* weight = static_cast<const raw*>(a.weight);
  raw* out = static_cast<raw*>(a.out);
  const bool wide = a.index_bytes == 8;
  for (int64_t r0 = (int64_t)blockIdx.x * rows; r0 < a.count; r0 += (int64_t)gridDim.x * rows) {
    const int32_t here = (int32_t)min((int64_t)rows, a.count - r0);
    const int32_t c0 = (int32_t)blockIdx.y * (kThreads * kPacks);  // packs of a long row
    const int32_t packs = rows == 1 ? min(per_row - c0, kThreads * kPacks) : here * per_row;
#pragma unroll
    for (int k = 0; k < kPacks; ++k) {
      const int32_t e = k * kThreads + (int32_t)threadIdx.x;
      if (e >= packs) break;
      const int32_t r = rows == 1 ? 0 : (int32_t)quotient((uint32_t)e, (uint32_t)per_row, magic);
      const int32_t c = (rows == 1 ? c0 + e : e - r * per_row) * V;
      const int64_t v = index_at(a.index, wide, r0 + r);
      float f[V];
      if (v >= 0 && v < a.vocab) {
        widen_pack<T, V>(load_pack<T, V>(weight + v * a.weight_row + c), f);
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] *= a.scale;
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = 0.0f;
      }
      store_pack<T, V>(out + (r0 + r) * a.out_row + c, narrow_pack<T, V>(f));
    }
  }
}

// ------------------------------------------------------------- sorted order
constexpr int kMaxDigits = 512;
constexpr int kSortWaves = 4;

struct SortPlan {
  int32_t passes, bits;     // digits of `bits` bits
  int32_t blocks, keys;     // workgroups of a pass, keys of each
};
SortPlan sort_plan(int64_t vocab, int64_t count) {
  int32_t need = 1;
  while (need < 31 && ((int64_t)1 << need) <= vocab) ++need;  // the key `vocab` has to fit
  SortPlan s;
  s.passes = (need + 8) / 9;
  s.bits = (need + s.passes - 1) / s.passes;
  // whole rounds of 64 keys per wave, at most 512 workgroups
  const int64_t round = 64 * kSortWaves;
  int64_t keys = (count + 511) / 512;
  if (keys < 2048) keys = 2048;
  s.keys = (int32_t)((keys + round - 1) / round * round);
  s.blocks = (int32_t)((count + s.keys - 1) / s.keys);
  return s;
}

struct SortPass {
  const void* index;        // first pass: the caller's indices
  int32_t index_bytes;
  const uint32_t *keys_in, *pos_in;
  uint32_t *keys_out, *pos_out;
  uint32_t* hist;           // [digits][blocks]
  int64_t vocab;
  uint32_t count;
  int32_t shift, bits, keys, blocks;
};

__device__ __forceinline__ uint32_t sort_key(const SortPass& p, uint32_t i) {
  if (p.keys_in) return p.keys_in[i];
  const int64_t v = index_at(p.index, p.index_bytes == 8, i);
  return v >= 0 && v < p.vocab ? (uint32_t)v : (uint32_t)p.vocab;
}

__global__ __launch_bounds__(64 * kSortWaves) void sort_count_kernel(SortPass p) {
  __shared__ uint32_t s_count[kMaxDigits];
  const int digits = 1 << p.bits;
  for (int d = threadIdx.x; d < digits; d += blockDim.x) s_count[d] = 0;
  __syncthreads();
  const uint32_t lo = blockIdx.x * (uint32_t)p.keys;
  const uint32_t hi = min(p.count, lo + (uint32_t)p.keys);
  for (uint32_t i = lo + threadIdx.x; i < hi; i += blockDim.x)
    atomicAdd(&s_count[(sort_key(p, i) >> p.shift) & (digits - 1)], 1u);
  __syncthreads();
  for (int d = threadIdx.x; d < digits; d += blockDim.x)
    p.hist[(int64_t)d * p.blocks + blockIdx.x] = s_count[d];
}

// Exclusive prefix sums of hist, in place, by one workgroup.
__global__ __launch_bounds__(1024) void sort_scan_kernel(uint32_t* hist, int32_t n) {
  __shared__ uint32_t s_wave[16];
  const int t = threadIdx.x, lane = t & 63, w = t >> 6;
  const int32_t per = (n + 1023) / 1024;
  const int32_t lo = min(n, t * per), hi = min(n, lo + per);
  uint32_t run = 0;
  for (int32_t i = lo; i < hi; ++i) run += hist[i];
  uint32_t incl = run;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t y = __shfl_up(incl, d, 64);
    if (lane >= d) incl += y;
  }
  if (lane == 63) s_wave[w] = incl;
  __syncthreads();
  uint32_t off = incl - run;
  for (int j = 0; j < w; ++j) off += s_wave[j];
  for (int32_t i = lo; i < hi; ++i) {
    const uint32_t x = hist[i];
    hist[i] = off;
    off += x;
  }
}

// Each wave owns a contiguous run of the workgroup's keys and walks it 64 at a
// time; lanes with the same digit find each other by one ballot per bit, so
// a key's place is its digit's cursor plus the matching lanes before it.
__global__ __launch_bounds__(64 * kSortWaves) void sort_place_kernel(SortPass p) {
  __shared__ uint32_t s_cursor[kSortWaves][kMaxDigits];
  const int digits = 1 << p.bits;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  for (int d = threadIdx.x; d < kSortWaves * kMaxDigits; d += blockDim.x) (&s_cursor[0][0])[d] = 0;
  __syncthreads();
  const uint32_t per = (uint32_t)p.keys / kSortWaves;
  const uint32_t lo = min(p.count, blockIdx.x * (uint32_t)p.keys + w * per);
  const uint32_t hi = min(p.count, lo + per);
  for (uint32_t i = lo + lane; i < hi; i += 64)
    atomicAdd(&s_cursor[w][(sort_key(p, i) >> p.shift) & (digits - 1)], 1u);
  __syncthreads();
  for (int d = threadIdx.x; d < digits; d += blockDim.x) {
    uint32_t off = p.hist[(int64_t)d * p.blocks + blockIdx.x];
    for (int j = 0; j < kSortWaves; ++j) {
      const uint32_t c = s_cursor[j][d];
      s_cursor[j][d] = off;
      off += c;
    }
  }
  __syncthreads();
  for (uint32_t i0 = lo; i0 < hi; i0 += 64) {
    const uint32_t i = i0 + lane;
    const bool in = i < hi;
    const uint32_t key = in ? sort_key(p, i) : 0u;
    const uint32_t digit = (key >> p.shift) & (digits - 1);
    uint64_t same = __ballot(in);
    for (int b = 0; b < p.bits; ++b) {
      const uint64_t ones = __ballot(in && ((digit >> b) & 1u));
      same &= ((digit >> b) & 1u) ? ones : ~ones;
    }
    const int before = __popcll(same & ((1ull << lane) - 1));
    uint32_t place = 0;
    if (in) place = s_cursor[w][digit] + before;
    __builtin_amdgcn_wave_barrier();
    if (in && before == 0) s_cursor[w][digit] += __popcll(same);
    __builtin_amdgcn_wave_barrier();
    if (in) {
      p.keys_out[place] = key;
      p.pos_out[place] = p.pos_in ? p.pos_in[i] : i;
    }
  }
}

// starts[v] = the first place of the sorted keys that holds v or more.
__global__ __launch_bounds__(kThreads) void row_starts_kernel(const uint32_t* keys, uint32_t count,
                                                              uint32_t vocab, uint32_t* starts) {
  const uint32_t v = blockIdx.x * kThreads + threadIdx.x;
  if (v > vocab) return;
  uint32_t lo = 0, hi = count;
  while (lo < hi) {
    const uint32_t mid = lo + (hi - lo) / 2;
    if (keys[mid] < v)
      lo = mid + 1;
    else
      hi = mid;
  }
  starts[v] = lo;
}

// ----------------------------------------------------------------- the sums
constexpr int kAhead = 8;  // rows of dout in flight per thread

struct SumArgs {
  const void* dout;
  const uint32_t *keys, *pos;
  const uint32_t* starts;
  void* dweight;
  float* partial;  // [pieces][2][width]: a row begun earlier, a row begun here
  int64_t dout_row, dweight_row;
  uint32_t count, vocab;
  int32_t width, per_row, piece, pieces;
  float scale;
};

template <class T, int V>
__device__ __forceinline__ void sum_piece(const SumArgs& a, int64_t g) {
  using raw = typename T::raw;
  const int64_t piece = g / a.per_row;
  if (piece >= a.pieces) return;
  const int32_t col = (int32_t)(g - piece * a.per_row) * V;
  const raw* dout = static_cast<const raw*>(a.dout) + col;
  raw* dw = static_cast<raw*>(a.dweight) + col;
  const uint32_t lo = (uint32_t)piece * (uint32_t)a.piece;
  // the keys behind the vocabulary (no index) are last: stop before them
  const uint32_t end = a.starts[a.vocab];
  const uint32_t hi = min(end, lo + (uint32_t)a.piece);
  if (lo >= hi) return;
  float* partial = a.partial + piece * 2 * (int64_t)a.width + col;
  uint32_t key = a.keys[lo];
  bool earlier = lo > 0 && a.keys[lo - 1] == key;
  float acc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.0f;
  auto finish = [&](bool later) {
    if (earlier || later) {
      float* to = partial + (earlier ? 0 : a.width);
#pragma unroll
      for (int i = 0; i < V; ++i) to[i] = acc[i];
    } else {
      float f[V];
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = acc[i] * a.scale;
      store_pack<T, V>(dw + (int64_t)key * a.dweight_row, narrow_pack<T, V>(f));
    }
  };
  for (uint32_t i = lo; i < hi; i += kAhead) {
    uint32_t k[kAhead];
    Pack<T, V> d[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const uint32_t q = min(i + j, hi - 1);
      k[j] = a.keys[q];
      d[j] = load_pack<T, V>(dout + (int64_t)a.pos[q] * a.dout_row);
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (i + j >= hi) break;
      if (k[j] != key) {
        finish(false);
        key = k[j];
        earlier = false;
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] = 0.0f;
      }
      float f[V];
      widen_pack<T, V>(d[j], f);
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e] += f[e];
    }
  }
  finish(hi < end && a.keys[hi] == key);
}

template <class T, int V>
__global__ __launch_bounds__(kThreads) void embed_sum_kernel(SumArgs a) {
  const int64_t all = (int64_t)a.pieces * a.per_row;
  for (int64_t g = (int64_t)blockIdx.x * kThreads + threadIdx.x; g < all;
       g += (int64_t)gridDim.x * kThreads)
    sum_piece<T, V>(a, g);
}

// One thread per pack of a row: clears a row without an index, joins the
// partial sums of one that crosses pieces.
template <class T, int V>
__device__ __forceinline__ void join_row(const SumArgs& a, int64_t g) {
  using raw = typename T::raw;
  const int64_t v = g / a.per_row;
  const int32_t col = (int32_t)(g - v * a.per_row) * V;
  const uint32_t lo = a.starts[v], hi = a.starts[v + 1];
  float acc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.0f;
  if (lo < hi) {
    const uint32_t first = lo / (uint32_t)a.piece, last = (hi - 1) / (uint32_t)a.piece;
    if (first == last) return;  // written by its piece
    const float* p = a.partial + (int64_t)first * 2 * a.width + col;
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = p[a.width + i];
#pragma unroll 8
    for (uint32_t q = first + 1; q <= last; ++q) {
      p += 2 * (int64_t)a.width;
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] += p[i];
    }
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] *= a.scale;
  }
  store_pack<T, V>(static_cast<raw*>(a.dweight) + v * a.dweight_row + col, narrow_pack<T, V>(acc));
}

template <class T, int V>
__global__ __launch_bounds__(kThreads) void embed_join_kernel(SumArgs a) {
  const int64_t all = (int64_t)a.vocab * a.per_row;
  for (int64_t g = (int64_t)blockIdx.x * kThreads + threadIdx.x; g < all;
       g += (int64_t)gridDim.x * kThreads)
    join_row<T, V>(a, g);
}

// Entries of the sorted list per piece.
int32_t piece_length(int64_t count) {
  int64_t piece = count / 4096;
  piece = (piece + 31) / 32 * 32;
  return (int32_t)(piece < 32 ? 32 : piece);
}

size_t round_up(size_t n) { return (n + 255) / 256 * 256; }

struct EmbedScratch {
  uint32_t *keys[2], *pos[2], *hist, *starts;
  float* partial;
  size_t bytes;
};
EmbedScratch scratch_of(char* base, int64_t vocab, int32_t width, int64_t count) {
  const SortPlan plan = sort_plan(vocab, count);
  const int32_t piece = piece_length(count);
  const int64_t pieces = (count + piece - 1) / piece;
  EmbedScratch s;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char* p = base + at;
    at += round_up(bytes);
    return p;
  };
  for (int i = 0; i < 2; ++i) {
    s.keys[i] = reinterpret_cast<uint32_t*>(take((size_t)count * 4));
    s.pos[i] = reinterpret_cast<uint32_t*>(take((size_t)count * 4));
  }
  s.hist = reinterpret_cast<uint32_t*>(take(((size_t)plan.blocks << plan.bits) * 4));
  s.starts = reinterpret_cast<uint32_t*>(take(((size_t)vocab + 1) * 4));
  s.partial = reinterpret_cast<float*>(take((size_t)pieces * 2 * width * 4));
  s.bytes = at;
  return s;
}

// Largest pack (up to 16 bytes) that divides the width, the row strides and
// the addresses.
template <class T>
int pack_of(int32_t width, std::initializer_list<int64_t> strides,
            std::initializer_list<const void*> pointers) {
  for (int v = 16 / T::kBytes; v > 1; v /= 2) {
    bool ok = width % v == 0;
    for (int64_t s : strides) ok = ok && s % v == 0;
    for (const void* p : pointers) ok = ok && aligned_to(p, (size_t)v * T::kBytes);
    if (ok) return v;
  }
  return 1;
}

// Workgroups of a launch: its threads are counted in 32 bits, so a larger
// grid loops.
unsigned capped(int64_t blocks) { return (unsigned)(blocks < (1 << 22) ? blocks : 1 << 22); }

template <class T, int V>
hipError_t forward(const EmbedForward& a, hipStream_t stream) {
  const int32_t per_row = a.width / V;
  const int32_t most = kThreads * kPacks;
  const int32_t rows = per_row >= most ? 1 : most / per_row;
  const int64_t blocks = (a.count + rows - 1) / rows;
  const unsigned cols = rows == 1 ? (unsigned)((per_row + most - 1) / most) : 1u;
  hipLaunchKernelGGL((embed_forward_kernel<T, V>), dim3(capped(blocks), cols), dim3(kThreads), 0,
                     stream, a, per_row, rows, magic_of((uint32_t)per_row));
  return hipGetLastError();
}

template <class T, int V>
hipError_t sums(SumArgs s, hipStream_t stream) {
  s.per_row = s.width / V;
  if (s.count > 0) {
    const int64_t threads = (int64_t)s.pieces * s.per_row;
    hipLaunchKernelGGL((embed_sum_kernel<T, V>), dim3(capped((threads + kThreads - 1) / kThreads)),
                       dim3(kThreads), 0, stream, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const int64_t threads = (int64_t)s.vocab * s.per_row;
  hipLaunchKernelGGL((embed_join_kernel<T, V>), dim3(capped((threads + kThreads - 1) / kThreads)),
                     dim3(kThreads), 0, stream, s);
  return hipGetLastError();
}

// Calls F<T, V> for the dtype and the pack size.
#define RL_PACKS(T, pack, F, ...)                       \
  switch (pack) {                                       \
    case 8: return F<T, (T::kBytes == 2 ? 8 : 4)>(__VA_ARGS__); \
    case 4: return F<T, 4>(__VA_ARGS__);                \
    case 2: return F<T, 2>(__VA_ARGS__);                \
    default: return F<T, 1>(__VA_ARGS__);               \
  }

template <class T>
hipError_t forward_any(const EmbedForward& a, hipStream_t stream) {
  RL_PACKS(T, pack_of<T>(a.width, {a.weight_row, a.out_row}, {a.weight, a.out}), forward, a, stream)
}
template <class T>
hipError_t sums_any(const SumArgs& s, hipStream_t stream) {
  RL_PACKS(T, pack_of<T>(s.width, {s.dout_row, s.dweight_row}, {s.dout, s.dweight}), sums, s, stream)
}

}  // namespace

hipError_t embed_forward_launch(const EmbedForward& a, hipStream_t stream) {
  if (a.count == 0 || a.width == 0) return hipSuccess;
  switch (a.dtype) {
    case POLICY_F32: return forward_any<F32>(a, stream);
    case POLICY_BF16: return forward_any<BF16>(a, stream);
    default: return forward_any<F16>(a, stream);
  }
}

int64_t embed_workspace_bytes(int64_t vocab, int32_t width, int64_t count) {
  return (int64_t)scratch_of(nullptr, vocab, width, count).bytes;
}

hipError_t embed_backward_launch(const EmbedBackward& a, hipStream_t stream) {
  if (a.vocab == 0 || a.width == 0) return hipSuccess;
  const SortPlan plan = sort_plan(a.vocab, a.count);
  const EmbedScratch sc = scratch_of(static_cast<char*>(a.workspace), a.vocab, a.width, a.count);
  hipError_t e;
  int at = 0;
  if (a.count > 0) {
    for (int pass = 0; pass < plan.passes; ++pass) {
      SortPass p{};
      p.index = a.index;
      p.index_bytes = a.index_bytes;
      p.keys_in = pass ? sc.keys[at] : nullptr;
      p.pos_in = pass ? sc.pos[at] : nullptr;
      at ^= 1;
      p.keys_out = sc.keys[at];
      p.pos_out = sc.pos[at];
      p.hist = sc.hist;
      p.vocab = a.vocab;
      p.count = (uint32_t)a.count;
      p.shift = pass * plan.bits;
      p.bits = plan.bits;
      p.keys = plan.keys;
      p.blocks = plan.blocks;
      const dim3 grid((unsigned)plan.blocks), threads(64 * kSortWaves);
      hipLaunchKernelGGL(sort_count_kernel, grid, threads, 0, stream, p);
      if ((e = hipGetLastError()) != hipSuccess) return e;
      hipLaunchKernelGGL(sort_scan_kernel, dim3(1), dim3(1024), 0, stream, sc.hist,
                         plan.blocks << plan.bits);
      if ((e = hipGetLastError()) != hipSuccess) return e;
      hipLaunchKernelGGL(sort_place_kernel, grid, threads, 0, stream, p);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
  }
  hipLaunchKernelGGL(row_starts_kernel, dim3((unsigned)(a.vocab / kThreads + 1)), dim3(kThreads), 0,
                     stream, sc.keys[at], (uint32_t)a.count, (uint32_t)a.vocab, sc.starts);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  SumArgs s{};
  s.dout = a.dout;
  s.keys = sc.keys[at];
  s.pos = sc.pos[at];
  s.starts = sc.starts;
  s.dweight = a.dweight;
  s.partial = sc.partial;
  s.dout_row = a.dout_row;
  s.dweight_row = a.dweight_row;
  s.count = (uint32_t)a.count;
  s.vocab = (uint32_t)a.vocab;
  s.width = a.width;
  s.piece = piece_length(a.count);
  s.pieces = (int32_t)((a.count + s.piece - 1) / s.piece);
  s.scale = a.scale;
  switch (a.dtype) {
    case POLICY_F32: return sums_any<F32>(s, stream);
    case POLICY_BF16: return sums_any<BF16>(s, stream);
    default: return sums_any<F16>(s, stream);
  }
}

}  // namespace rl
