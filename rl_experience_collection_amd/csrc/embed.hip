// Scaled embedding lookup and its gradient (include/policy.h).
//
// The lookup copies rows: a workgroup owns a run of output rows, a thread
// fixed 16-byte packs of the run, whose indices, then rows, are all loaded
// before the first is used.  A width that is no multiple of a pack ends in a
// pack moved back to the row's end: it repeats elements of the one before
// with the same values.  (The same goes for the gradient below.)
//
// The gradient sums the rows of dout that share an index.  Few indices (1024 at
// most) take one launch: every workgroup owns a few rows of the vocabulary and
// reads all indices.  More are sorted: a stable radix sort of the positions by
// index with digits of at most 9 bits, two launches a digit (counts, then
// places; each workgroup of the second sums the counts before its own).  An
// index outside the vocabulary sorts behind it.  The sorted list is cut into
// pieces of equal length; a thread owns one pack of columns of one piece,
// walks the piece in order, adds in fp32 and at each change of index writes
// the finished row.  A row that crosses the border of pieces leaves a partial
// sum in each of them, and a last launch over the vocabulary joins those in
// order and clears the rows no index names.  So dout is read once, whatever
// the skew of the indices, and every sum has a fixed order.
#include <initializer_list>

#include "elem.hpp"
#include "policy.hpp"

namespace rl {

namespace {

constexpr int kThreads = 256;

// Orders a wave's accesses to LDS: what its lanes read before is read before
// any of them writes after.  The LDS takes a wave's accesses in order, so this
// costs nothing; it holds the compiler to that order.
__device__ __forceinline__ void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}
// Quotient of n by d for n * d < 2^32 (magic = floor(2^32 / d) + 1, d > 1).
__device__ __forceinline__ uint32_t quotient(uint32_t n, uint32_t d, uint32_t magic) {
  return d == 1 ? n : __umulhi(n, magic);
}
uint32_t magic_of(uint32_t d) { return (uint32_t)((1ull << 32) / d + 1); }

// An index as loaded: its low and high words (of a 4-byte index the word
// twice), so that no conversion waits for the load.
struct RawIndex {
  int32_t lo, hi;
};
__device__ __forceinline__ RawIndex raw_index(const void* p, int32_t bytes, int64_t i) {
  const int32_t* w = static_cast<const int32_t*>(p);
  const int32_t two = bytes >> 3;
  return RawIndex{w[i << two], w[(i << two) + two]};
}
// Whether it names a row of the vocabulary (below 2^31 - 1 rows).
__device__ __forceinline__ bool names_row(RawIndex x, int32_t bytes, int64_t vocab) {
  return x.lo >= 0 && x.lo < vocab && (bytes == 4 || x.hi == 0);
}
// The row, or `vocab` where there is none.
__device__ __forceinline__ uint32_t key_at(const void* p, int32_t bytes, int64_t vocab, int64_t i) {
  const RawIndex x = raw_index(p, bytes, i);
  return names_row(x, bytes, vocab) ? (uint32_t)x.lo : (uint32_t)vocab;
}

// --------------------------------------------------------------- the lookup
// Bound by memory: 65,536 of 131,072 rows of 1024 bf16 in 41 us (203 MB, 4.9
// TB/s), 262,147 of 50,021 rows of 500 fp16 in 71 us (277 MB written as the
// lines of rows of 1000 bytes, 109 MB read).
constexpr int kPacks = 4;  // packs per thread

template <class T, int V>
__global__ __launch_bounds__(kThreads) void embed_forward_kernel(EmbedForward a, int32_t per_row,
                                                                 int32_t rows, uint32_t magic,
                                                                 bool past) {
  using raw = typename T::raw;
  const raw* weight = static_cast<const raw*>(a.weight);
  raw* out = static_cast<raw*>(a.out);
  const int32_t c0 = (int32_t)blockIdx.y * (kThreads * kPacks);  // packs of a long row
  for (int64_t r0 = (int64_t)blockIdx.x * rows; r0 < a.count; r0 += (int64_t)gridDim.x * rows) {
    const int32_t here = (int32_t)min((int64_t)rows, a.count - r0);
    const int32_t packs = rows == 1 ? min(per_row - c0, kThreads * kPacks) : here * per_row;
    RawIndex v[kPacks];
    int32_t r[kPacks], c[kPacks];
#pragma unroll
    for (int k = 0; k < kPacks; ++k) {
      const int32_t e = min(k * kThreads + (int32_t)threadIdx.x, packs - 1);
      r[k] = rows == 1 ? 0 : (int32_t)quotient((uint32_t)e, (uint32_t)per_row, magic);
      c[k] = min((rows == 1 ? c0 + e : e - r[k] * per_row) * V, a.width - V);
      v[k] = raw_index(a.index, a.index_bytes, r0 + r[k]);
    }
    Pack<T, V> x[kPacks];
#pragma unroll
    for (int k = 0; k < kPacks; ++k) {
      const bool named = names_row(v[k], a.index_bytes, a.vocab);
      x[k] = load_pack<T, V>(weight + (int64_t)(named ? v[k].lo : 0) * a.weight_row + c[k]);
    }
#pragma unroll
    for (int k = 0; k < kPacks; ++k) {
      if (k * kThreads + (int32_t)threadIdx.x >= packs) break;
      const bool named = names_row(v[k], a.index_bytes, a.vocab);
      float f[V];
      widen_pack<T, V>(x[k], f);
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = named ? f[i] * a.scale : 0.0f;
      store_pack<T, V>(out + (r0 + r[k]) * a.out_row + c[k], narrow_pack<T, V>(f), past);
    }
  }
}

// A vocabulary without rows: every index is outside it.
template <class T>
__global__ __launch_bounds__(kThreads) void embed_zero_kernel(EmbedForward a) {
  using raw = typename T::raw;
  const int64_t all = a.count * a.width;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < all;
       i += (int64_t)gridDim.x * kThreads)
    static_cast<raw*>(a.out)[i / a.width * a.out_row + i % a.width] = raw{};
}

// ------------------------------------------------------------- sorted order
constexpr int kMaxDigits = 512;
constexpr int kSortWaves = 4;
constexpr int kSortBlocks = 128;  // at most
constexpr uint32_t kNoRow = 0xffffffffu;

struct SortPlan {
  int32_t passes, bits;  // digits of `bits` bits
  int32_t blocks, keys;  // workgroups of a pass, keys of each
};
SortPlan sort_plan(int64_t vocab, int64_t count) {
  int32_t need = 1;
  while (need < 31 && ((int64_t)1 << need) <= vocab) ++need;  // the key `vocab` has to fit
  SortPlan s;
  s.passes = (need + 8) / 9;
  s.bits = (need + s.passes - 1) / s.passes;
  // whole rounds of 64 keys per wave
  const int64_t round = 64 * kSortWaves;
  int64_t keys = (count + kSortBlocks - 1) / kSortBlocks;
  if (keys < 4 * round) keys = 4 * round;
  s.keys = (int32_t)((keys + round - 1) / round * round);
  s.blocks = (int32_t)((count + s.keys - 1) / s.keys);
  return s;
}

struct SortPass {
  const void* index;  // first pass: the caller's indices
  int32_t index_bytes;
  const uint32_t *keys_in, *pos_in;
  uint32_t *keys_out, *pos_out;
  uint32_t* hist;       // [blocks][digits]
  uint32_t* row_first;  // first pass: [vocab], set to kNoRow
  int64_t vocab;
  uint32_t count;
  int32_t shift, bits, keys, blocks;
};

__device__ __forceinline__ uint32_t sort_key(const SortPass& p, uint32_t i) {
  return p.keys_in ? p.keys_in[i] : key_at(p.index, p.index_bytes, p.vocab, i);
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
  if (p.row_first) {
    for (int64_t v = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; v < p.vocab;
         v += (int64_t)gridDim.x * blockDim.x)
      p.row_first[v] = kNoRow;
  }
  __syncthreads();
  for (int d = threadIdx.x; d < digits; d += blockDim.x)
    p.hist[(int64_t)blockIdx.x * digits + d] = s_count[d];
}

// Each wave owns a contiguous run of the workgroup's keys and walks it 64 at a
// time; lanes with the same digit find each other by one ballot per bit, so
// a key's place is its digit's cursor plus the matching lanes before it.
__global__ __launch_bounds__(64 * kSortWaves) void sort_place_kernel(SortPass p) {
  __shared__ uint32_t s_cursor[kSortWaves][kMaxDigits];
  __shared__ uint32_t s_wave[kSortWaves];
  const int digits = 1 << p.bits;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  for (int d = tid; d < kSortWaves * kMaxDigits; d += blockDim.x) (&s_cursor[0][0])[d] = 0;
  __syncthreads();
  const uint32_t per = (uint32_t)p.keys / kSortWaves;
  const uint32_t lo = min(p.count, blockIdx.x * (uint32_t)p.keys + w * per);
  const uint32_t hi = min(p.count, lo + per);
  for (uint32_t i = lo + lane; i < hi; i += 64)
    atomicAdd(&s_cursor[w][(sort_key(p, i) >> p.shift) & (digits - 1)], 1u);
  // digits 2 tid and 2 tid + 1: the keys of all workgroups, and of those before
  uint32_t all[2] = {0, 0}, before[2] = {0, 0};
  if (2 * tid < digits) {
    const uint2* h = reinterpret_cast<const uint2*>(p.hist) + tid;
    constexpr int kRows = 16;  // loads in flight
    for (int b0 = 0; b0 < p.blocks; b0 += kRows) {
      uint2 c[kRows];
#pragma unroll
      for (int j = 0; j < kRows; ++j) c[j] = h[(int64_t)min(b0 + j, p.blocks - 1) * (digits / 2)];
#pragma unroll
      for (int j = 0; j < kRows; ++j) {
        const bool in = b0 + j < p.blocks, earlier = b0 + j < (int)blockIdx.x;
        all[0] += in ? c[j].x : 0u;
        all[1] += in ? c[j].y : 0u;
        before[0] += earlier ? c[j].x : 0u;
        before[1] += earlier ? c[j].y : 0u;
      }
    }
  }
  const uint32_t mine = all[0] + all[1];
  uint32_t incl = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t y = __shfl_up(incl, d, 64);
    if (lane >= d) incl += y;
  }
  if (lane == 63) s_wave[w] = incl;
  __syncthreads();
  uint32_t base = incl - mine;
  for (int j = 0; j < w; ++j) base += s_wave[j];
  if (2 * tid < digits) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      uint32_t off = base + before[k];
      for (int j = 0; j < kSortWaves; ++j) {
        const uint32_t c = s_cursor[j][2 * tid + k];
        s_cursor[j][2 * tid + k] = off;
        off += c;
      }
      base += all[k];
    }
  }
  __syncthreads();
  constexpr int kAhead = 4;
  for (uint32_t i0 = lo; i0 < hi; i0 += 64 * kAhead) {
    uint32_t key[kAhead], pos[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const uint32_t i = min(i0 + 64 * j + lane, hi - 1);
      key[j] = sort_key(p, i);
      pos[j] = p.pos_in ? p.pos_in[i] : i;
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const bool in = i0 + 64 * j + lane < hi;
      const uint32_t digit = (key[j] >> p.shift) & (digits - 1);
      uint64_t same = __ballot(in);
      for (int b = 0; b < p.bits; ++b) {
        const uint64_t ones = __ballot((digit >> b) & 1u);
        same &= ((digit >> b) & 1u) ? ones : ~ones;
      }
      const int earlier = __popcll(same & ((1ull << lane) - 1));
      // every lane of a digit reads its cursor before the first of them moves
      // it, and that before the next round reads it
      const uint32_t place = s_cursor[w][digit] + earlier;
      wave_order();
      if (in && earlier == 0) s_cursor[w][digit] = place + __popcll(same);
      wave_order();
      if (in) {
        p.keys_out[place] = key[j];
        p.pos_out[place] = pos[j];
      }
    }
  }
}

// ----------------------------------------------------------------- the sums
constexpr int kAhead = 8;  // rows of dout in flight per thread

struct SumArgs {
  const void* dout;
  uint32_t *row_first, *row_end;  // [vocab]: a row's places in the sorted list
  void* dweight;
  float* partial;  // [pieces][2][width]: a row begun earlier, a row begun here
  int64_t dout_row, dweight_row;
  uint32_t count, vocab;
  int32_t width, per_row, piece, pieces;
  float scale;
  bool past;
};

// The piece `piece` of the columns `col`; `names`: this thread records the
// rows' places.
template <class T, int V>
__device__ __forceinline__ void sum_piece(const SumArgs& a, const uint32_t* __restrict__ keys,
                                          const uint32_t* __restrict__ pos, uint32_t piece, int32_t col,
                                          bool names) {
  using raw = typename T::raw;
  const raw* dout = static_cast<const raw*>(a.dout) + col;
  raw* dw = static_cast<raw*>(a.dweight) + col;
  const uint32_t lo = piece * (uint32_t)a.piece;
  const uint32_t hi = min(a.count, lo + (uint32_t)a.piece);
  float* partial = a.partial + (int64_t)piece * 2 * a.width + col;
  uint32_t key = keys[lo];
  bool earlier = lo > 0 && keys[lo - 1] == key;
  float acc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.0f;
  if (names && !earlier && key < a.vocab) a.row_first[key] = lo;
  auto finish = [&](uint32_t end, bool later) {
    if (key >= a.vocab) return;  // no index: behind the vocabulary
    if (names && !later) a.row_end[key] = end;
    if (earlier || later) {
      float* to = partial + (earlier ? 0 : a.width);
#pragma unroll
      for (int i = 0; i < V; ++i) to[i] = acc[i];
    } else {
      float f[V];
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = acc[i] * a.scale;
      store_pack<T, V>(dw + (int64_t)key * a.dweight_row, narrow_pack<T, V>(f), a.past);
    }
  };
  uint32_t next_key[kAhead], next_at[kAhead];
  auto look = [&](uint32_t i) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const uint32_t q = min(i + j, hi - 1);
      next_key[j] = keys[q];
      next_at[j] = pos[q];
    }
  };
  look(lo);
  for (uint32_t i = lo; i < hi && key < a.vocab; i += kAhead) {
    uint32_t k[kAhead];
    Pack<T, V> d[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      k[j] = next_key[j];
      d[j] = load_pack<T, V>(dout + (int64_t)next_at[j] * a.dout_row);
    }
    look(i + kAhead);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (i + j >= hi) break;
      if (k[j] != key) {
        finish(i + j, false);
        key = k[j];
        earlier = false;
        if (names && key < a.vocab) a.row_first[key] = i + j;
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] = 0.0f;
      }
      float f[V];
      widen_pack<T, V>(d[j], f);
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e] += f[e];
    }
  }
  finish(hi, hi < a.count && keys[hi] == key);
}

// WAVE: a wave owns 64 packs of one piece, so that keys and positions are
// the same in all its lanes and come through the scalar cache.
template <class T, int V, bool WAVE>
__global__ __launch_bounds__(kThreads) void embed_sum_kernel(SumArgs a,
                                                             const uint32_t* __restrict__ keys,
                                                             const uint32_t* __restrict__ pos) {
  if (WAVE) {
    const int32_t blocks = (a.per_row + 63) / 64;
    const int64_t all = (int64_t)a.pieces * blocks;
    for (int64_t g = (int64_t)blockIdx.x * (kThreads / 64) +
                     __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
         g < all; g += (int64_t)gridDim.x * (kThreads / 64)) {
      const int64_t piece = g / blocks;
      const int32_t c = (int32_t)(g - piece * blocks) * 64 + (threadIdx.x & 63);
      if (c < a.per_row) sum_piece<T, V>(a, keys, pos, (uint32_t)piece, min(c * V, a.width - V), c == 0);
    }
  } else {
    const int64_t all = (int64_t)a.pieces * a.per_row;
    for (int64_t g = (int64_t)blockIdx.x * kThreads + threadIdx.x; g < all;
         g += (int64_t)gridDim.x * kThreads) {
      const int64_t piece = g / a.per_row;
      const int32_t c = (int32_t)(g - piece * a.per_row);
      sum_piece<T, V>(a, keys, pos, (uint32_t)piece, min(c * V, a.width - V), c == 0);
    }
  }
}

// Clears the rows without an index and joins the partial sums of those that
// cross pieces.  SPLIT threads share a pack of a row: each adds a run of its
// partial sums, and the runs are added in order.  One where the vocabulary
// alone fills the chip, else 8: a small vocabulary has many sums a row (the
// gradient of 64,000 rows into 45 x 128 fp32 takes 23.6 us so, 27.6 with one;
// that of 262,144 into 8192 x 256 86 us with one, 96 with 8).
template <class T, int V, int SPLIT>
__global__ __launch_bounds__(kThreads) void embed_join_kernel(SumArgs a) {
  using raw = typename T::raw;
  constexpr int kHere = kThreads / SPLIT;
  __shared__ float s_sum[SPLIT > 1 ? SPLIT : 1][SPLIT > 1 ? kHere : 1][V];
  const int part = SPLIT > 1 ? (int)threadIdx.x / kHere : 0;
  const int here = (int)threadIdx.x % kHere;
  const int64_t all = (int64_t)a.vocab * a.per_row;
  for (int64_t g0 = (int64_t)blockIdx.x * kHere; g0 < all; g0 += (int64_t)gridDim.x * kHere) {
    const int64_t g = min(g0 + here, all - 1);
    const int64_t v = g / a.per_row;
    const int32_t col = min((int32_t)(g - v * a.per_row) * V, a.width - V);
    const uint32_t lo = a.row_first[v];
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.0f;
    bool write = true;
    if (lo != kNoRow) {
      const uint32_t first = lo / (uint32_t)a.piece, last = (a.row_end[v] - 1) / (uint32_t)a.piece;
      write = first != last;  // else its piece has written it
      // partial sum 0 is the one begun in its own piece
      const uint32_t sums = write ? last - first + 1 : 0;
      const uint32_t per = (sums + SPLIT - 1) / SPLIT;
      const uint32_t from = min(sums, part * per), to = min(sums, from + per);
      const float* p = a.partial + (int64_t)first * 2 * a.width + col;
#pragma unroll 8
      for (uint32_t q = from; q < to; ++q) {
        const float* x = p + (int64_t)q * 2 * a.width + (q == 0 ? a.width : 0);
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] += x[i];
      }
    }
    if (SPLIT > 1) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < V; ++i) s_sum[part][here][i] = acc[i];
      __syncthreads();
      if (part > 0) continue;
      for (int j = 1; j < SPLIT; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] += s_sum[j][here][i];
    }
    if (!write || g0 + here >= all) continue;
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] *= a.scale;
    store_pack<T, V>(static_cast<raw*>(a.dweight) + v * a.dweight_row + col, narrow_pack<T, V>(acc),
                     a.past);
  }
}

// ------------------------------------------------------------- few indices
// Indices, at most.  1000 spread over a vocabulary of 45 x 128 fp32 take 5.8 us
// in this one launch, 15.8 sorted (50,021 x 500 bf16: 28 and 40); 1000 times
// the same index 28 and 17.5.  2000 take as long either way at 50,021 x 500.
constexpr int kFewMost = 1024;
constexpr int kFewRows = 32;    // rows of the vocabulary per workgroup, at most
constexpr int kFewParts = 8;    // threads that share a pack of a row
constexpr int kFewPacks = kThreads / kFewParts;  // packs of a row per workgroup

// One row per workgroup, as long as the grid stays small.
int32_t few_rows(int64_t vocab, int64_t chunks) {
  const int64_t rows = (vocab * chunks) >> 13;
  return (int32_t)(rows < 1 ? 1 : rows < kFewRows ? rows : kFewRows);
}

// The places of the indices among this workgroup's rows are listed in LDS, by
// row and in order.  The rows that have none are cleared.  Of the others one
// after another is summed: each part takes a run of its places, and the parts
// are added in order, so that one index repeated is not one thread's work.
template <class T, int V>
__global__ __launch_bounds__(kThreads) void embed_few_kernel(EmbedBackward a, int32_t per_row,
                                                             int32_t block_rows, bool past) {
  using raw = typename T::raw;
  __shared__ uint32_t s_list[kFewMost];    // row << 16 | position, in order of position
  __shared__ uint16_t s_place[kFewMost];   // positions by row
  __shared__ uint32_t s_wave[kThreads / 64];
  __shared__ uint32_t s_end[kFewRows];     // counts of the rows, then ends of their places
  __shared__ float s_sum[kFewParts][kFewPacks][V];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int part = tid / kFewPacks, here = tid % kFewPacks;
  const int32_t count = (int32_t)a.count;
  const int64_t chunks = (per_row + kFewPacks - 1) / kFewPacks;
  const int64_t blocks = (a.vocab + block_rows - 1) / block_rows * chunks;
  for (int64_t block = blockIdx.x; block < blocks; block += gridDim.x) {
    const int64_t v0 = block / chunks * block_rows;
    const int32_t rows = (int32_t)min((int64_t)block_rows, a.vocab - v0);
    const int32_t c0 = (int32_t)(block % chunks) * kFewPacks;
    const int32_t packs = min(per_row - c0, kFewPacks);
    if (tid < kFewRows) s_end[tid] = 0u;
    __syncthreads();
    int32_t n = 0;
    for (int32_t i0 = 0; i0 < count; i0 += kThreads) {
      const int32_t i = i0 + tid;
      const int64_t v = (int64_t)key_at(a.index, a.index_bytes, a.vocab, min(i, count - 1)) - v0;
      const bool mine = i < count && v >= 0 && v < rows;
      const uint64_t m = __ballot(mine);
      __syncthreads();
      if (lane == 0) s_wave[w] = (uint32_t)__popcll(m);
      __syncthreads();
      int32_t at = n + __popcll(m & ((1ull << lane) - 1));
      for (int j = 0; j < kThreads / 64; ++j) {
        if (j < w) at += s_wave[j];
        n += s_wave[j];
      }
      if (mine) {
        s_list[at] = (uint32_t)v << 16 | (uint32_t)i;
        atomicAdd(&s_end[v], 1u);
      }
    }
    __syncthreads();
    if (n > 0 && w == 0) {
      // ends of the rows' places; then, 64 entries at a time, each to its row's
      // next place (s_end counts up from the row's first)
      const uint32_t mine = lane < kFewRows ? s_end[lane] : 0u;
      uint32_t end = mine;
#pragma unroll
      for (int d = 1; d < kFewRows; d <<= 1) {
        const uint32_t y = __shfl_up(end, d, 64);
        if (lane >= d) end += y;
      }
      if (lane < kFewRows) s_end[lane] = end - mine;
      wave_order();
      for (int32_t i0 = 0; i0 < n; i0 += 64) {
        const bool in = i0 + lane < n;
        const uint32_t e = s_list[min(i0 + lane, n - 1)], row = e >> 16;
        uint64_t same = __ballot(in);
#pragma unroll
        for (int b = 1; b < kFewRows; b <<= 1) {
          const uint64_t ones = __ballot((row & b) != 0);
          same &= row & b ? ones : ~ones;
        }
        const int earlier = __popcll(same & ((1ull << lane) - 1));
        // every lane of a row reads its cursor before the first of them moves
        // it, and that before the next round reads it
        const uint32_t place = s_end[row] + earlier;
        wave_order();
        if (in && earlier == 0) s_end[row] = place + __popcll(same);
        wave_order();
        if (in) s_place[place] = (uint16_t)e;
      }
    }
    __syncthreads();
    auto first_of = [&](int32_t r) { return r ? (int32_t)s_end[r - 1] : 0; };
    for (int32_t g = tid; g < rows * packs; g += kThreads) {
      const int32_t r = g / packs;
      if (first_of(r) != (int32_t)s_end[r]) continue;
      const int32_t col = min((c0 + g - r * packs) * V, a.width - V);
      const float zero[V] = {};
      store_pack<T, V>(static_cast<raw*>(a.dweight) + (v0 + r) * a.dweight_row + col,
                       narrow_pack<T, V>(zero), past);
    }
    const int32_t col = min((c0 + min(here, packs - 1)) * V, a.width - V);
    const raw* dout = static_cast<const raw*>(a.dout) + col;
    for (int32_t r = 0; r < rows && n > 0; ++r) {
      const int32_t lo = first_of(r), hi = (int32_t)s_end[r];
      if (lo == hi) continue;  // (the same for all threads)
      const int32_t per = (hi - lo + kFewParts - 1) / kFewParts;
      const int32_t from = min(hi, lo + part * per), to = min(hi, from + per);
      float acc[V];
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] = 0.0f;
      for (int32_t j0 = from; j0 < to; j0 += kAhead) {
        Pack<T, V> d[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
          d[j] = load_pack<T, V>(dout + (int64_t)s_place[min(j0 + j, to - 1)] * a.dout_row);
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          if (j0 + j >= to) break;
          float f[V];
          widen_pack<T, V>(d[j], f);
#pragma unroll
          for (int i = 0; i < V; ++i) acc[i] += f[i];
        }
      }
#pragma unroll
      for (int i = 0; i < V; ++i) s_sum[part][here][i] = acc[i];
      __syncthreads();
      if (part == 0 && here < packs) {
        for (int j = 1; j < kFewParts; ++j)
#pragma unroll
          for (int i = 0; i < V; ++i) acc[i] += s_sum[j][here][i];
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] *= a.scale;
        store_pack<T, V>(static_cast<raw*>(a.dweight) + (v0 + r) * a.dweight_row + col,
                         narrow_pack<T, V>(acc), past);
      }
      __syncthreads();
    }
    __syncthreads();
  }
}

// Entries of the sorted list per piece: about 2^17 threads in all, but pieces
// long enough that partial sums stay a small part of the traffic.  (2^16 and
// 2^18 threads: within 3% at every size tried, 45 x 32 to 131,072 x 1024.)
int32_t piece_length(int64_t count, int64_t per_row) {
  int64_t piece = (count * per_row) >> 17;
  piece = (piece + 15) / 16 * 16;
  if (piece < 16) piece = 16;
  return (int32_t)(piece < 1024 ? piece : 1024);
}

size_t round_up(size_t n) { return (n + 255) / 256 * 256; }

struct EmbedScratch {
  uint32_t *keys[2], *pos[2], *hist, *row_first, *row_end;
  float* partial;
  size_t bytes;
};
EmbedScratch scratch_of(char* base, int64_t vocab, int32_t width, int64_t count, int64_t per_row) {
  const SortPlan plan = sort_plan(vocab, count);
  const int32_t piece = piece_length(count, per_row);
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
  s.row_first = reinterpret_cast<uint32_t*>(take((size_t)vocab * 4));
  s.row_end = reinterpret_cast<uint32_t*>(take((size_t)vocab * 4));
  s.partial = reinterpret_cast<float*>(take((size_t)pieces * 2 * width * 4));
  s.bytes = at;
  return s;
}

// The largest pack, up to 16 bytes, that a row holds.
int pack_of(int32_t dtype, int32_t width) {
  int v = dtype == POLICY_F32 ? 4 : 8;
  while (v > width) v /= 2;
  return v;
}

// Workgroups of a launch: its threads are counted in 32 bits, so a larger
// grid loops.
unsigned capped(int64_t blocks) { return (unsigned)(blocks < (1 << 22) ? blocks : 1 << 22); }

template <class T, int V>
hipError_t forward(const EmbedForward& a, hipStream_t stream) {
  if (a.vocab == 0) {
    hipLaunchKernelGGL(embed_zero_kernel<T>, dim3(capped((a.count * a.width + kThreads - 1) / kThreads)),
                       dim3(kThreads), 0, stream, a);
    return hipGetLastError();
  }
  const int32_t per_row = (a.width + V - 1) / V;
  const int32_t most = kThreads * kPacks;
  const int32_t rows = per_row >= most ? 1 : most / per_row;
  const int64_t blocks = (a.count + rows - 1) / rows;
  const unsigned cols = rows == 1 ? (unsigned)((per_row + most - 1) / most) : 1u;
  const bool past = a.count * a.width * T::kBytes > kPastBytes;
  hipLaunchKernelGGL((embed_forward_kernel<T, V>), dim3(capped(blocks), cols), dim3(kThreads), 0,
                     stream, a, per_row, rows, magic_of((uint32_t)per_row), past);
  return hipGetLastError();
}

template <class T, int V>
hipError_t backward(const EmbedBackward& a, hipStream_t stream) {
  const int32_t per_row = (a.width + V - 1) / V;
  const bool past = a.vocab * a.width * T::kBytes > kPastBytes;
  if (a.count <= kFewMost) {
    const int64_t chunks = (per_row + kFewPacks - 1) / kFewPacks;
    const int32_t rows = few_rows(a.vocab, chunks);
    hipLaunchKernelGGL((embed_few_kernel<T, V>), dim3(capped((a.vocab + rows - 1) / rows * chunks)),
                       dim3(kThreads), 0, stream, a, per_row, rows, past);
    return hipGetLastError();
  }
  const SortPlan plan = sort_plan(a.vocab, a.count);
  const EmbedScratch sc =
      scratch_of(static_cast<char*>(a.workspace), a.vocab, a.width, a.count, per_row);
  hipError_t e;
  int at = 0;
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
    p.row_first = pass ? nullptr : sc.row_first;
    p.vocab = a.vocab;
    p.count = (uint32_t)a.count;
    p.shift = pass * plan.bits;
    p.bits = plan.bits;
    p.keys = plan.keys;
    p.blocks = plan.blocks;
    const dim3 grid((unsigned)plan.blocks), threads(64 * kSortWaves);
    hipLaunchKernelGGL(sort_count_kernel, grid, threads, 0, stream, p);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    hipLaunchKernelGGL(sort_place_kernel, grid, threads, 0, stream, p);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  SumArgs s{};
  s.dout = a.dout;
  const uint32_t *keys = sc.keys[at], *pos = sc.pos[at];
  s.row_first = sc.row_first;
  s.row_end = sc.row_end;
  s.dweight = a.dweight;
  s.partial = sc.partial;
  s.dout_row = a.dout_row;
  s.dweight_row = a.dweight_row;
  s.count = (uint32_t)a.count;
  s.vocab = (uint32_t)a.vocab;
  s.width = a.width;
  s.per_row = per_row;
  s.piece = piece_length(a.count, per_row);
  s.pieces = (int32_t)((a.count + s.piece - 1) / s.piece);
  s.scale = a.scale;
  s.past = past;
  // at least half the lanes of a wave have a pack of their own (262,144 rows of
  // 1024 bf16 into 512: 143 us so, 148 otherwise; 64,000 of 32 fp32 into 45:
  // 21.9 and 20.6)
  if (per_row > 32) {
    const int64_t waves = (int64_t)s.pieces * ((per_row + 63) / 64);
    hipLaunchKernelGGL((embed_sum_kernel<T, V, true>), dim3(capped((waves + 3) / 4)), dim3(kThreads), 0,
                       stream, s, keys, pos);
  } else {
    const int64_t threads = (int64_t)s.pieces * per_row;
    hipLaunchKernelGGL((embed_sum_kernel<T, V, false>),
                       dim3(capped((threads + kThreads - 1) / kThreads)), dim3(kThreads), 0, stream, s,
                       keys, pos);
  }
  if ((e = hipGetLastError()) != hipSuccess) return e;
  const int64_t packs = a.vocab * per_row;
  if (packs <= 65536)
    hipLaunchKernelGGL((embed_join_kernel<T, V, 8>), dim3((unsigned)((packs + kThreads / 8 - 1) / (kThreads / 8))),
                       dim3(kThreads), 0, stream, s);
  else
    hipLaunchKernelGGL((embed_join_kernel<T, V, 1>), dim3(capped((packs + kThreads - 1) / kThreads)),
                       dim3(kThreads), 0, stream, s);
  return hipGetLastError();
}

// Calls F<T, V> for the dtype and the pack.
#define RL_PACKS(T, F, ...)                                     \
  switch (pack_of(a.dtype, a.width)) {                          \
    case 8: return F<T, (T::kBytes == 2 ? 8 : 4)>(__VA_ARGS__); \
    case 4: return F<T, 4>(__VA_ARGS__);                        \
    case 2: return F<T, 2>(__VA_ARGS__);                        \
    default: return F<T, 1>(__VA_ARGS__);                       \
  }

}  // namespace

hipError_t embed_forward_launch(const EmbedForward& a, hipStream_t stream) {
  if (a.count == 0 || a.width == 0) return hipSuccess;
  switch (a.dtype) {
    case POLICY_F32: RL_PACKS(F32, forward, a, stream)
    case POLICY_BF16: RL_PACKS(BF16, forward, a, stream)
    default: RL_PACKS(F16, forward, a, stream)
  }
}

int64_t embed_workspace_bytes(int32_t dtype, int64_t vocab, int32_t width, int64_t count) {
  if (vocab == 0 || width == 0 || count <= kFewMost) return 0;
  const int v = pack_of(dtype, width);
  return (int64_t)scratch_of(nullptr, vocab, width, count, (width + v - 1) / v).bytes;
}

hipError_t embed_backward_launch(const EmbedBackward& a, hipStream_t stream) {
  if (a.vocab == 0 || a.width == 0) return hipSuccess;
  switch (a.dtype) {
    case POLICY_F32: RL_PACKS(F32, backward, a, stream)
    case POLICY_BF16: RL_PACKS(BF16, backward, a, stream)
    default: RL_PACKS(F16, backward, a, stream)
  }
}

#undef RL_PACKS

}  // namespace rl
