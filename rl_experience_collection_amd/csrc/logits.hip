// Penalties, bias and mask on logits, and their gradient (include/policy.h).
//
// Two shapes.  Many short rows (a quarter of a run of columns at most) that lie
// one after another are taken several at a time: a tile is a run of whole rows
// addressed as one array.  Longer (or strided) rows are cut into runs of columns,
// one row at a time.  In both a thread owns fixed 16-byte packs of the tile, loads them
// first, and while they are on their way the workgroup counts the history's
// tokens that fall into the tile in LDS (integer adds: their order does not
// matter).  In the first shape rows and packs do not line up, and most packs
// hold a counted token: the tile's values are staged in LDS, the history
// entry that counts a token first replaces the token's value there, and the
// mask becomes one bit per element of the tile, so that the last pass over
// the packs has no branch per element.
//
// The gradient needs a logit only where a token occurred (its sign picks the
// factor).  Short rows load all of them, as nearly every line holds one; in
// long ones the history's entries load theirs and leave the sign beside the
// mark.
// dbias is summed by the pass that forms dlogits: a thread's packs cover the
// same columns in every tile, so it adds up its own columns in registers
// over all tiles it takes, and one more kernel joins the workgroups' sums in
// a fixed order.
#include "elem.hpp"
#include "policy.hpp"

namespace rl {

namespace {

constexpr int kThreads = 256;
constexpr int kTile = 2048;      // elements of a tile of whole rows, at most
constexpr int kTileRows = 128;   // its rows, at most
constexpr int kRunPacks = 2;     // packs per thread of a run of columns
// Workgroups of a launch over tiles: what is resident at once on 256 compute
// units.  The kernel is held to 128 registers a thread (4 waves a SIMD): a
// 4,096,000 x 45 training pass takes 880 us so, 960 with the 150 that the
// compiler takes by itself and 978 at 96, where it spills.
constexpr int kTileWaves = 4;
constexpr int kTileGroups = 256 * kTileWaves;
// (96 registers: a 4096 x 32,003 training pass takes 304 us so and with 128, 359
// with 80, where it spills; 64 x 128,001 forward 13.0, 13.0 and 16.0)
constexpr int kRunWaves = 5;
// Workgroups of a launch over runs, about: four times what is resident, so that
// a bias is loaded once for many rows.  4096 x 32,003 bf16 forward takes 110 us
// so, 124 with a workgroup a row; 32,768 x 4000 98 and 123.
constexpr int kRunGroups = 5120;
constexpr int kBiasGroups = 1024;  // about, of runs in all, with dbias
constexpr float kBanned = -__builtin_inff();

struct LogitsArgs {
  logits_args a;
  const void* dout;  // gradient
  void* out;         // out or dlogits
  float* partial;    // gradient: [groups][vocab] sums of dbias, or NULL
  int64_t dout_row, out_row;
  int32_t tile_rows;     // rows of a tile
  uint32_t magic_vocab;  // for a quotient by vocab
  uint32_t magic_words;  // for one by the words of a row of bits
  uint32_t magic_width;  // for one by history_width
  bool penalties;        // the history matters
  bool past;             // the output is stored past the caches
};

__device__ __forceinline__ uint32_t quotient(uint32_t n, uint32_t d, uint32_t magic) {
  return d == 1 ? n : __umulhi(n, magic);
}

// Offset of a row's mask, or -1 where everything is allowed.
__device__ __forceinline__ int64_t mask_offset(const logits_args& a, int64_t r) {
  if (a.mask_kind == LOGITS_MASK_NONE) return -1;
  const int64_t m = a.mask_rows ? (int64_t)a.mask_rows[r] : (a.mask_count == 1 ? 0 : r);
  return m >= 0 && m < a.mask_count ? m * a.mask_row : -1;
}
// z / rho from 1 / rho (itself rounded to nearest): one Newton correction of
// the quotient.  Where that says nothing (an infinite z, a rho so far from 1
// that terms_of left no reciprocal) the division itself.
__device__ __forceinline__ float divide(float z, float rho, float inv) {
  const float q = z * inv;
  const float c = __builtin_fmaf(__builtin_fmaf(-q, rho, z), inv, q);
  return __builtin_fabsf(q) < __builtin_inff() ? c : z / rho;
}

struct Terms {
  float rho, inv, alpha, beta;
};
__device__ __forceinline__ Terms terms_of(float rho, float alpha, float beta) {
  const bool plain = rho > 0x1p-100f && rho < 0x1p100f;
  return Terms{rho, plain ? 1.0f / rho : __builtin_nanf(""), alpha, beta};
}
__device__ __forceinline__ float penalise(float z, const Terms& t, uint32_t count) {
  z = z > 0.0f ? divide(z, t.rho, t.inv) : z * t.rho;
  z -= t.alpha;
  return z - t.beta * (float)count;
}

// The first `n` of a pack's elements.
template <class T, int V>
__device__ __forceinline__ void store_some(typename T::raw* p, const Pack<T, V>& x, int n, bool past) {
  if (n >= V) {
    store_pack<T, V>(p, x, past);
    return;
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (i < n) p[i] = x.v[i];
}

// N 32-bit words from LDS, four at a time where N allows.
template <int N>
__device__ __forceinline__ void read_words(const uint32_t* p, uint32_t (&w)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const uint4 q = *reinterpret_cast<const uint4*>(p + i);
      w[i] = q.x;
      w[i + 1] = q.y;
      w[i + 2] = q.z;
      w[i + 3] = q.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = p[i];
  }
}
template <int N>
__device__ __forceinline__ void write_words(uint32_t* p, const uint32_t (&w)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4)
      *reinterpret_cast<uint4*>(p + i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = w[i];
  }
}

// The new value of a tile's cell whose token occurred: its logit penalised, or
// its gradient scaled.
template <bool GRAD>
__device__ __forceinline__ float replaced(const uint32_t* val, const uint32_t* count,
                                          const uint32_t* pos, const Terms& t, int32_t c) {
  const float f = __uint_as_float(val[c]);
  if (GRAD) return (pos[c >> 5] >> (c & 31)) & 1u ? divide(f, t.rho, t.inv) : f * t.rho;
  return penalise(f, t, (count[c >> 1] >> ((c & 1) << 4)) & 0xffffu);
}

// The mask of the V columns from c0 + e, as loaded: a byte of bits, or V bytes
// (moved back like load_inside).
template <int V, int MASK>
__device__ __forceinline__ uint64_t load_mask(const logits_args& a, int64_t at, int32_t c0, int32_t e,
                                              int32_t n) {
  const uint8_t* m = static_cast<const uint8_t*>(a.mask);
  if constexpr (MASK == LOGITS_MASK_BITS) {
    return m[at * 4 + ((c0 + min(e, n - 1)) >> 3)];
  } else if constexpr (V == 8) {
    typedef uint64_t eight __attribute__((aligned(1)));
    return *reinterpret_cast<const eight*>(m + at + c0 + min(e, n - V));
  } else if constexpr (V == 4) {
    typedef uint32_t four __attribute__((aligned(1)));
    return *reinterpret_cast<const four*>(m + at + c0 + min(e, n - V));
  } else {
    return m[at + c0 + min(e, n - V)];
  }
}
// Bit i: column c0 + e + i is allowed.
template <int V, int MASK>
__device__ __forceinline__ uint32_t mask_bits(uint64_t raw, int32_t c0, int32_t e, int32_t n) {
  if constexpr (MASK == LOGITS_MASK_BITS) {
    return (uint32_t)raw >> ((c0 + e) & 7);
  } else {
    const int32_t back = e - (n - V);
    if (back > 0) raw >>= 8 * back;
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) bits |= ((raw >> (8 * i)) & 0xffu ? 1u : 0u) << i;
    return bits;
  }
}

// ------------------------------------------------------- tiles of whole rows
constexpr int kAhead = 4;  // history entries a thread loads before it uses the first

// How a tile takes its mask: bits and bytes become bits of the tile in LDS; a
// byte per logit, one after another like them, is read like them.
enum MaskMode { kNoMask, kBitMask, kByteMask, kFlatMask };

// What a workgroup needs of a tile, loaded while the one before is worked on.
template <class T, int V, bool GRAD, int MODE>
struct RowsTile {
  static constexpr int kPacks = kTile / (kThreads * V);
  Pack<T, V> x[kPacks], z[GRAD ? kPacks : 1];
  int32_t token[kAhead];
  int32_t len;
  float rho, alpha, beta;
  uint32_t word;  // a mask of bits: this thread's word of the tile's masks,
  bool named;     // if it has one
  uint64_t mask[MODE == kFlatMask ? kPacks : 1];  // the packs' bytes of the mask
};

// A mask of bits gives every thread at most one word of a tile's masks (128
// rows of at most 32 logits, or 2048 / vocab rows of more): word j of row r.
struct MaskWord {
  int32_t r, j;
};
__device__ __forceinline__ MaskWord mask_word(const LogitsArgs& p) {
  const uint32_t W = (uint32_t)(p.a.vocab + 31) >> 5;
  const int32_t r = (int32_t)quotient(threadIdx.x, W, p.magic_words);
  return MaskWord{r, (int32_t)(threadIdx.x - r * W)};
}
// The mask row of that row; -1: everything is allowed.  Loaded two tiles
// ahead, as the word's address waits for it.
__device__ __forceinline__ int32_t mask_row_ahead(const LogitsArgs& p, int64_t r0, MaskWord m) {
  const logits_args& a = p.a;
  const int64_t r = min(r0 + m.r, a.rows - 1);
  // (one row per row of logits: mask_count, and so r, is below 2^31)
  return a.mask_rows ? a.mask_rows[r] : (a.mask_count == 1 ? 0 : (int32_t)r);
}

// Elements from a tile's first row to the array's end, as far as a pack reaches.
template <int V>
__device__ __forceinline__ int32_t tile_reach(const logits_args& a, int64_t r0) {
  return (int32_t)min((int64_t)(kTile + V), (a.rows - r0) * a.vocab);
}

// Every load before the first wait: no load behind a branch of its lanes.
template <class T, int V, bool GRAD, int MODE>
__device__ __forceinline__ void load_tile(const LogitsArgs& p, int64_t r0, MaskWord m, int32_t mrow,
                                          RowsTile<T, V, GRAD, MODE>& q) {
  using raw = typename T::raw;
  const logits_args& a = p.a;
  const int tid = threadIdx.x;
  const int32_t rows = (int32_t)min((int64_t)p.tile_rows, a.rows - r0);
  const int32_t reach = tile_reach<V>(a, r0);
  if (p.penalties) {
    const int64_t r = r0 + min(tid, rows - 1);
    q.len = a.history_len ? a.history_len[r] : a.history_width;
    q.rho = a.repetition_rows ? a.repetition_rows[r] : a.repetition;
    q.alpha = a.presence_rows ? a.presence_rows[r] : a.presence;
    q.beta = a.frequency_rows ? a.frequency_rows[r] : a.frequency;
    const int32_t* h = a.history + r0 * a.history_width;
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      q.token[j] = h[min(j * kThreads + tid, rows * a.history_width - 1)];
  }
  if (MODE == kBitMask) {
    q.named = m.r < rows && mrow >= 0 && mrow < a.mask_count;
    q.word = static_cast<const uint32_t*>(a.mask)[q.named ? (int64_t)mrow * a.mask_row + m.j : 0];
  }
  if (MODE == kFlatMask) {
#pragma unroll
    for (int k = 0; k < q.kPacks; ++k)
      q.mask[MODE == kFlatMask ? k : 0] = load_mask<V, LOGITS_MASK_BYTES>(a, r0 * a.vocab, 0, (k * kThreads + tid) * V, reach);
  }
  const raw* in = static_cast<const raw*>(GRAD ? p.dout : a.logits) + r0 * a.vocab;
#pragma unroll
  for (int k = 0; k < q.kPacks; ++k)
    q.x[k] = load_inside<T, V>(in, (k * kThreads + tid) * V, reach);
  if (GRAD && p.penalties) {
    const raw* z = static_cast<const raw*>(a.logits) + r0 * a.vocab;
#pragma unroll
    for (int k = 0; k < q.kPacks; ++k)
      q.z[GRAD ? k : 0] = load_inside<T, V>(z, (k * kThreads + tid) * V, reach);
  }
}

// 4,096,000 x 45 fp32 with a table of masks and a history of 20 in 419 us (1.9 GB
// at 4.5 TB/s), the gradient with dbias in 517 (2.6 GB at 5.0): bound by the four
// barriers of a tile at 4 workgroups a compute unit, and by memory.
template <class T, int V, bool GRAD, int MODE>
__global__ __launch_bounds__(kThreads, kTileWaves) void logits_rows_kernel(LogitsArgs p) {
  using raw = typename T::raw;
  constexpr int kPacks = kTile / (kThreads * V);
  __shared__ alignas(16) uint32_t s_val[kTile];  // the tile's values (fp32), penalised in place
  __shared__ alignas(16) uint32_t s_count[kTile / 2];  // two 16-bit counts a word
  __shared__ uint32_t s_ban[kTile / 32 + 1];     // a bit per element: not allowed
  __shared__ uint32_t s_pos[GRAD ? kTile / 32 : 1];  // a bit per element: its logit is above 0
  __shared__ Terms s_terms[kTileRows];
  __shared__ int32_t s_len[kTileRows];
  const logits_args& a = p.a;
  const int tid = threadIdx.x, lane = tid & 63;
  const int32_t vocab = a.vocab, width = a.history_width;
  constexpr bool masked = MODE == kBitMask || MODE == kByteMask;  // by bits in LDS
  const int64_t tiles = (a.rows + p.tile_rows - 1) / p.tile_rows;
  // per element of the thread's packs, whose columns are the same in every
  // tile: the running sums of dbias (gradient) or a bias that all rows share
  float col[kPacks][V];
#pragma unroll
  for (int k = 0; k < kPacks; ++k)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      col[k][i] = 0.0f;
      if (!GRAD && a.bias && a.bias_row == 0) {
        const uint32_t e = (uint32_t)((k * kThreads + tid) * V + i);
        col[k][i] = a.bias[e - quotient(e, (uint32_t)vocab, p.magic_vocab) * vocab];
      }
    }
  RowsTile<T, V, GRAD, MODE> next;
  MaskWord m{0, 0};
  if (MODE == kBitMask) m = mask_word(p);
  const int64_t first = (int64_t)blockIdx.x * p.tile_rows, step = (int64_t)gridDim.x * p.tile_rows;
  load_tile<T, V, GRAD, MODE>(p, first, m, MODE == kBitMask ? mask_row_ahead(p, first, m) : -1, next);
  int32_t mrow = MODE == kBitMask ? mask_row_ahead(p, first + step, m) : -1;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int64_t r0 = tile * p.tile_rows;
    const int32_t rows = (int32_t)min((int64_t)p.tile_rows, a.rows - r0);
    const int32_t n = rows * vocab;
    raw* out = static_cast<raw*>(p.out) + r0 * vocab;
    const int32_t* h = p.penalties ? a.history + r0 * width : nullptr;
    const int32_t entries = p.penalties ? rows * width : 0;
    const int32_t reach = tile_reach<V>(a, r0);
    RowsTile<T, V, GRAD, MODE> q = next;
    if (tile + gridDim.x < tiles) {
      load_tile<T, V, GRAD, MODE>(p, r0 + step, m, mrow, next);
      if (MODE == kBitMask) mrow = mask_row_ahead(p, r0 + 2 * step, m);
    }
    if (masked || p.penalties) {
      __syncthreads();  // the previous tile's words are read
      if (p.penalties) {
        if (tid < rows) {
          s_terms[tid] = terms_of(q.rho, q.alpha, q.beta);
          s_len[tid] = min(max(q.len, 0), width);
        }
        for (int i = tid * 4; i < kTile / 2; i += kThreads * 4)
          *reinterpret_cast<uint4*>(&s_count[i]) = make_uint4(0, 0, 0, 0);
        if (GRAD && tid < kTile / 32) s_pos[tid] = 0u;
      }
      if (masked && tid < kTile / 32 + 1) s_ban[tid] = 0u;
      __syncthreads();
      if (MODE == kBitMask) {
        // a row's words are shifted to the row's place among the tile's bits
        if (q.named) {
          const int32_t left = vocab - 32 * m.j;
          const uint32_t ban = ~q.word & (left < 32 ? (1u << left) - 1u : ~0u);
          const int32_t bit = m.r * vocab + 32 * m.j, sh = bit & 31;
          atomicOr(&s_ban[bit >> 5], ban << sh);
          if (sh) atomicOr(&s_ban[(bit >> 5) + 1], ban >> (32 - sh));
        }
      } else if (MODE == kByteMask) {
        for (int32_t e = tid; e < kTile; e += kThreads) {
          bool ban = false;
          if (e < n) {
            const int32_t r = (int32_t)quotient((uint32_t)e, (uint32_t)vocab, p.magic_vocab);
            const int64_t at = mask_offset(a, r0 + r);
            ban = at >= 0 && static_cast<const uint8_t*>(a.mask)[at + e - r * vocab] == 0;
          }
          const uint64_t bits = __ballot(ban);
          if (lane == 0) s_ban[e >> 5] = (uint32_t)bits;
          if (lane == 32) s_ban[e >> 5] = (uint32_t)(bits >> 32);
        }
      }
    }
    if (p.penalties) {
#pragma unroll
      for (int k = 0; k < kPacks; ++k) {
        const int32_t e = (k * kThreads + tid) * V;
        if (e >= n) continue;
        settle<T, V>(q.x[k], e, reach);
        uint32_t word[V];
#pragma unroll
        for (int i = 0; i < V; ++i) word[i] = __float_as_uint(T::widen(q.x[k].v[i]));
        write_words<V>(s_val + e, word);
        if (GRAD) {
          settle<T, V>(q.z[GRAD ? k : 0], e, reach);
          float g[V];
          widen_pack<T, V>(q.z[GRAD ? k : 0], g);
          uint32_t bits = 0;
#pragma unroll
          for (int i = 0; i < V; ++i) bits |= (g[i] > 0.0f ? 1u : 0u) << i;
          atomicOr(&s_pos[e >> 5], bits << (e & 31));
        }
      }
      // Count the tokens; the entry that counts a token first owns it and,
      // once all are counted, replaces the token's value.
      for (int32_t e0 = 0; e0 < entries; e0 += kAhead * kThreads) {
        if (e0 > 0) {
#pragma unroll
          for (int j = 0; j < kAhead; ++j)
            q.token[j] = h[min(e0 + j * kThreads + tid, entries - 1)];
        }
        // entries that do not count add 0, each thread's to a word of its own:
        // no branches, so the LDS works on all of them at once
        int32_t row[kAhead], cell[kAhead];
        uint32_t old[kAhead];
        bool owner[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          const int32_t e = min(e0 + j * kThreads + tid, entries - 1);
          row[j] = (int32_t)quotient((uint32_t)e, (uint32_t)width, p.magic_width);
          cell[j] = e - row[j] * width;
          old[j] = (uint32_t)s_len[row[j]];
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          owner[j] = e0 + j * kThreads + tid < entries && cell[j] < (int32_t)old[j] &&
                     q.token[j] >= 0 && q.token[j] < vocab;
          cell[j] = owner[j] ? row[j] * vocab + q.token[j] : 2 * tid;
          old[j] = atomicAdd(&s_count[cell[j] >> 1], owner[j] ? 1u << ((cell[j] & 1) << 4) : 0u);
        }
        if (entries <= kAhead * kThreads) {
#pragma unroll
          for (int j = 0; j < kAhead; ++j)
            owner[j] = owner[j] && ((old[j] >> ((cell[j] & 1) << 4)) & 0xffffu) == 0u;
          __syncthreads();
          float f[kAhead];
#pragma unroll
          for (int j = 0; j < kAhead; ++j)
            f[j] = replaced<GRAD>(s_val, s_count, s_pos, s_terms[row[j]], cell[j]);
#pragma unroll
          for (int j = 0; j < kAhead; ++j)
            if (owner[j]) s_val[cell[j]] = __float_as_uint(f[j]);
        }
      }
      if (entries > kAhead * kThreads) {
        // too many entries to keep their owners: every cell is looked at
        __syncthreads();
        for (int32_t c = tid; c < n; c += kThreads)
          if ((s_count[c >> 1] >> ((c & 1) << 4)) & 0xffffu) {
            const int32_t r = (int32_t)quotient((uint32_t)c, (uint32_t)vocab, p.magic_vocab);
            s_val[c] = __float_as_uint(replaced<GRAD>(s_val, s_count, s_pos, s_terms[r], c));
          }
      }
    }
    if (masked || p.penalties) __syncthreads();
#pragma unroll
    for (int k = 0; k < kPacks; ++k) {
      const int32_t e = (k * kThreads + tid) * V;
      if (e >= n) continue;
      float f[V];
      if (p.penalties) {
        uint32_t word[V];
        read_words<V>(s_val + e, word);
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = __uint_as_float(word[i]);
      } else {
        settle<T, V>(q.x[k], e, reach);
        widen_pack<T, V>(q.x[k], f);
      }
      uint32_t ban = masked ? s_ban[e >> 5] >> (e & 31) : 0u;
      if (MODE == kFlatMask) ban = ~mask_bits<V, LOGITS_MASK_BYTES>(q.mask[MODE == kFlatMask ? k : 0], 0, e, reach);
      if (!GRAD && a.bias && a.bias_row == 0) {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] += col[k][i];
      } else if (!GRAD && a.bias) {
        const int32_t r = (int32_t)quotient((uint32_t)e, (uint32_t)vocab, p.magic_vocab);
        int32_t v = e - r * vocab;
        const float* b = a.bias + (r0 + r) * a.bias_row;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          if (e + i < n) f[i] += b[v];
          if (++v == vocab) {
            v = 0;
            b += a.bias_row;
          }
        }
      }
      if (GRAD && p.partial) {
        float g[V];
        widen_pack<T, V>(q.x[k], g);
#pragma unroll
        for (int i = 0; i < V; ++i)
          col[k][i] += e + i < n && !((ban >> i) & 1u) ? g[i] : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = (ban >> i) & 1u ? (GRAD ? 0.0f : kBanned) : f[i];
      if (!GRAD || p.out) store_some<T, V>(out + e, narrow_pack<T, V>(f), n - e, p.past);
    }
  }
  if (GRAD && p.partial) {
    // this workgroup's sum of each column, row by row of its tile
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kPacks; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) s_val[(k * kThreads + tid) * V + i] = __float_as_uint(col[k][i]);
    __syncthreads();
    for (int32_t v = tid; v < vocab; v += kThreads) {
      float sum = 0.0f;
      for (int32_t r = 0; r < p.tile_rows; ++r) sum += __uint_as_float(s_val[r * vocab + v]);
      p.partial[(int64_t)blockIdx.x * vocab + v] = sum;
    }
  }
}

// ------------------------------------------------ runs of columns of one row
// 4096 x 32,003 bf16 with a mask of bits in 129 us (540 MB at 4.2 TB/s), the
// gradient with dbias in 169 (3.2): bound by memory, whose lines the rows of
// 64,006 bytes do not respect, and by the counting's barriers.  64 x 128,001 with
// a history of 2048 in 12.6: 2048 workgroups, of which 1280 are resident, so two
// rounds of loads and counting, each of which reads its row's whole history.
template <class T, int V, bool GRAD, int MASK>
__global__ __launch_bounds__(kThreads, kRunWaves) void logits_runs_kernel(LogitsArgs p) {
  using raw = typename T::raw;
  constexpr int kRun = kThreads * V * kRunPacks;
  __shared__ alignas(16) uint32_t s_count[kRun];
  const logits_args& a = p.a;
  const int tid = threadIdx.x;
  const int32_t c0 = (int32_t)blockIdx.x * kRun;
  const int32_t n = min(kRun, a.vocab - c0);
  // Columns a load may reach.  The last run may hold fewer than a pack: its
  // loads then begin before it, in the same row (vocab >= V).
  const int32_t rest = a.vocab - c0;
  // the running sums of dbias of the thread's columns
  float col[kRunPacks][V] = {};
  // their bias, as loaded; one that all rows share is loaded once
  constexpr int B = V < 4 ? V : 4;  // elements of an access
  Pack<F32, B> bias[GRAD ? 1 : kRunPacks][V / B];
  auto load_bias = [&](int64_t r) {
    const uint32_t* b = reinterpret_cast<const uint32_t*>(a.bias) + r * a.bias_row + c0;
#pragma unroll
    for (int k = 0; k < kRunPacks; ++k)
#pragma unroll
      for (int j = 0; j < V / B; ++j)
        bias[GRAD ? 0 : k][j] = load_inside<F32, B>(b, (k * kThreads + tid) * V + j * B, rest);
  };
  auto settle_bias = [&]() {
#pragma unroll
    for (int k = 0; k < kRunPacks; ++k)
#pragma unroll
      for (int j = 0; j < V / B; ++j)
        settle<F32, B>(bias[GRAD ? 0 : k][j], (k * kThreads + tid) * V + j * B, rest);
  };
  if (!GRAD && a.bias && !a.bias_row) {
    load_bias(0);
    settle_bias();
  }
  for (int64_t r = blockIdx.y; r < a.rows; r += gridDim.y) {
    const raw* in = GRAD ? static_cast<const raw*>(p.dout) + r * p.dout_row + c0
                         : static_cast<const raw*>(a.logits) + r * a.logits_row + c0;
    const raw* z0 = static_cast<const raw*>(a.logits) + r * a.logits_row + c0;
    raw* out = static_cast<raw*>(p.out) + r * p.out_row + c0;
    const int32_t* h = a.history + r * a.history_row;
    // Every load before the first wait.  Loads return in order, so what is
    // needed first is loaded first: the row's terms and history, then the
    // packs; the mask last, as its address may wait for the row's index.
    int32_t token[4], len = 0;
    float rho = 1.0f, alpha = 0.0f, beta = 0.0f;
    int64_t mrow = r;
    if (MASK != LOGITS_MASK_NONE && a.mask_rows) mrow = a.mask_rows[r];
    if (p.penalties) {
      len = a.history_len ? a.history_len[r] : a.history_width;
      rho = a.repetition_rows ? a.repetition_rows[r] : a.repetition;
      alpha = a.presence_rows ? a.presence_rows[r] : a.presence;
      beta = a.frequency_rows ? a.frequency_rows[r] : a.frequency;
#pragma unroll
      for (int j = 0; j < 4; ++j) token[j] = h[min(j * kThreads + tid, a.history_width - 1)];
    }
    Pack<T, V> x[kRunPacks];
#pragma unroll
    for (int k = 0; k < kRunPacks; ++k)
      x[k] = load_inside<T, V>(in, (k * kThreads + tid) * V, rest);
    if (!GRAD && a.bias && a.bias_row) load_bias(r);
    uint64_t mraw[kRunPacks] = {};
    bool free_row = true;  // everything is allowed
    if (MASK != LOGITS_MASK_NONE) {
      if (!a.mask_rows && a.mask_count == 1) mrow = 0;
      free_row = mrow < 0 || mrow >= a.mask_count;
#pragma unroll
      for (int k = 0; k < kRunPacks; ++k)
        mraw[k] = load_mask<V, MASK>(a, free_row ? 0 : mrow * a.mask_row, c0, (k * kThreads + tid) * V,
                                     rest);
    }
    len = min(max(len, 0), a.history_width);
    Terms t{};
    if (len) {
      t = terms_of(rho, alpha, beta);
      __syncthreads();  // the previous row's counts are read
#pragma unroll
      for (int k = 0; k < kRunPacks; ++k) {
        const uint32_t zero[V] = {};
        write_words<V>(&s_count[(k * kThreads + tid) * V], zero);
      }
      __syncthreads();
      for (int32_t i0 = tid; i0 < len; i0 += 4 * kThreads) {
        if (i0 != tid) {
#pragma unroll
          for (int j = 0; j < 4; ++j) token[j] = h[min(i0 + j * kThreads, len - 1)];
        }
        bool here[4];
        raw z[GRAD ? 4 : 1];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          here[j] = i0 + j * kThreads < len && token[j] >= c0 && token[j] - c0 < n;
          if (GRAD) z[GRAD ? j : 0] = here[j] ? z0[token[j] - c0] : raw{};
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (!here[j]) continue;
          if (GRAD)
            atomicOr(&s_count[token[j] - c0], T::widen(z[GRAD ? j : 0]) > 0.0f ? 3u : 1u);
          else
            atomicAdd(&s_count[token[j] - c0], 1u);
        }
      }
      __syncthreads();
    }
    if (!GRAD && a.bias && a.bias_row) settle_bias();
#pragma unroll
    for (int k = 0; k < kRunPacks; ++k) {
      const int32_t e = (k * kThreads + tid) * V;
      if (e >= n) continue;
      settle<T, V>(x[k], e, rest);
      const uint32_t ok = MASK == LOGITS_MASK_NONE || free_row ? ~0u
                                                               : mask_bits<V, MASK>(mraw[k], c0, e, rest);
      float f[V];
      widen_pack<T, V>(x[k], f);
      if (GRAD && p.partial) {
#pragma unroll
        for (int i = 0; i < V; ++i) col[k][i] += (ok >> i) & 1u ? f[i] : 0.0f;
      }
      if (len) {
        uint32_t c[V], any = 0u;
        read_words<V>(&s_count[e], c);
#pragma unroll
        for (int i = 0; i < V; ++i) any |= c[i];
        if (any) {
#pragma unroll
          for (int i = 0; i < V; ++i) {
            if (!c[i]) continue;
            if (GRAD) {
              f[i] = c[i] & 2u ? divide(f[i], t.rho, t.inv) : f[i] * t.rho;
            } else {
              f[i] = penalise(f[i], t, c[i]);
            }
          }
        }
      }
      if (!GRAD && a.bias) {
#pragma unroll
        for (int j = 0; j < V / B; ++j) {
          const Pack<F32, B>& b = bias[GRAD ? 0 : k][j];
#pragma unroll
          for (int i = 0; i < B; ++i) f[j * B + i] += F32::widen(b.v[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = (ok >> i) & 1u ? f[i] : (GRAD ? 0.0f : kBanned);
      if (!GRAD || p.out) store_some<T, V>(out + e, narrow_pack<T, V>(f), n - e, p.past);
    }
  }
  if (GRAD && p.partial) {
    float* to = p.partial + (int64_t)blockIdx.y * a.vocab + c0;
#pragma unroll
    for (int k = 0; k < kRunPacks; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int32_t e = (k * kThreads + tid) * V + i;
        if (e < n) to[e] = col[k][i];
      }
  }
}

// dbias[v] = the sum of the groups' sums of column v: 16 waves take every
// 16th group of 64 columns, then the waves' sums are added in order.
__global__ __launch_bounds__(1024) void bias_join_kernel(const float* partial, int32_t groups,
                                                         int32_t vocab, float* dbias) {
  __shared__ float s_sum[16][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t v = (int64_t)blockIdx.x * 64 + lane;
  float sum = 0.0f;
  if (v < vocab) {
#pragma unroll 8
    for (int32_t k = w; k < groups; k += 16) sum += partial[(int64_t)k * vocab + v];
  }
  s_sum[w][lane] = sum;
  __syncthreads();
  if (w == 0 && v < vocab) {
    for (int j = 1; j < 16; ++j) sum += s_sum[j][lane];
    dbias[v] = sum;
  }
}

// The longest rows taken several at a time, a quarter of a run of columns.
// 32,768 rows of bf16 with a history of 64 (forward, gradient): 63 and 78 us at
// 900 logits, as runs 67 and 88; at 1100 115 and 137, as runs 65 and 85.  fp32:
// 36 and 47 us at 500, as runs 44 and 66; at 700 62 and 90, as runs 45 and 82.
int32_t flat_most(int32_t dtype) { return dtype == POLICY_F32 ? 512 : 1024; }
// As many rows are taken one at a time whatever their length, which spreads
// them over more of the chip: 512 rows of 45 fp32 logits take 4.2 and 7.4 us so,
// 7.9 and 9.9 as tiles; 8192 take 14 and 21, 8.3 and 11 as tiles.
constexpr int64_t kFewRows = 512;

// Rows of a tile of whole rows.
int32_t tile_rows_of(int32_t vocab) {
  const int32_t rows = kTile / vocab;
  return rows < kTileRows ? rows : kTileRows;
}
// Workgroups along the rows: dbias is summed over as many partial sums.
int64_t flat_groups(int64_t rows, int32_t vocab) {
  const int64_t tiles = (rows + tile_rows_of(vocab) - 1) / tile_rows_of(vocab);
  return tiles < kTileGroups ? tiles : kTileGroups;
}
int64_t run_groups(int64_t rows, int32_t vocab, bool bias) {
  // with dbias few groups of many rows, as each adds a row of partial sums to
  // the traffic, but enough to fill the chip: the gradient of 4096 x 32,003 bf16
  // takes 151 us with 1024 groups in all, 166 with 2048, 169 with 768
  const int64_t runs = (vocab + 4095) / 4096;
  const int64_t most = ((bias ? kBiasGroups : kRunGroups) + runs - 1) / runs;
  return rows < most ? rows : most;
}

// The launch over whole rows: its workgroups.
template <class T, bool GRAD>
int64_t launch_rows(const LogitsArgs& p, hipStream_t stream) {
  constexpr int V = 16 / T::kBytes;
  const logits_args& a = p.a;
  const int64_t groups = flat_groups(a.rows, a.vocab);
  const bool flat_mask = a.mask_kind == LOGITS_MASK_BYTES && !a.mask_rows &&
                         a.mask_count == a.rows && a.mask_row == a.vocab;
  auto kernel = flat_mask                            ? logits_rows_kernel<T, V, GRAD, kFlatMask>
                : a.mask_kind == LOGITS_MASK_BITS  ? logits_rows_kernel<T, V, GRAD, kBitMask>
                : a.mask_kind == LOGITS_MASK_BYTES ? logits_rows_kernel<T, V, GRAD, kByteMask>
                                                   : logits_rows_kernel<T, V, GRAD, kNoMask>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)groups), dim3(kThreads), 0, stream, p);
  return groups;
}

// The launch over runs of columns: its workgroups along the rows.
template <class T, int V, bool GRAD>
int64_t launch_runs(const LogitsArgs& p, bool bias, hipStream_t stream) {
  constexpr int kRun = kThreads * V * kRunPacks;
  const logits_args& a = p.a;
  const int64_t groups = run_groups(a.rows, a.vocab, bias);
  const dim3 grid((unsigned)((a.vocab + kRun - 1) / kRun), (unsigned)groups);
  auto kernel = a.mask_kind == LOGITS_MASK_BITS    ? logits_runs_kernel<T, V, GRAD, LOGITS_MASK_BITS>
                : a.mask_kind == LOGITS_MASK_BYTES ? logits_runs_kernel<T, V, GRAD, LOGITS_MASK_BYTES>
                                                   : logits_runs_kernel<T, V, GRAD, LOGITS_MASK_NONE>;
  hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, stream, p);
  return groups;
}

template <class T, bool GRAD>
hipError_t shape(LogitsArgs p, float* dbias, hipStream_t stream) {
  const logits_args& a = p.a;
  const bool dense = (!p.out || p.out_row == a.vocab) && (!GRAD || p.dout_row == a.vocab) &&
                     (a.logits_row == a.vocab || (GRAD && !p.penalties));
  // the tile's quotients are exact, and its counts 16 bits, for histories that
  // are not very long
  const int64_t w = a.history_width;
  const bool countable = !p.penalties ||
                         (a.history_row == w && w < (1 << 16) &&
                          tile_rows_of(a.vocab < kTile ? a.vocab : kTile) * w * w < ((int64_t)1 << 32));
  const bool flat = a.vocab <= flat_most(a.dtype) && a.rows > kFewRows && dense && countable;
  if (flat) {
    p.tile_rows = tile_rows_of(a.vocab);
    p.magic_vocab = (uint32_t)((1ull << 32) / (uint32_t)a.vocab + 1);
    p.magic_words = (uint32_t)((1ull << 32) / (uint32_t)((a.vocab + 31) / 32) + 1);
    if (p.penalties) p.magic_width = (uint32_t)((1ull << 32) / (uint32_t)a.history_width + 1);
  }
  if (a.mask_count == 0) p.a.mask_kind = LOGITS_MASK_NONE;  // a table without rows bans nothing
  p.past = a.rows * a.vocab * T::kBytes > kPastBytes;
  // a pack has to fit into the row (whole rows are many, so it fits into those)
  constexpr int V = 16 / T::kBytes;
  const int64_t groups = flat           ? launch_rows<T, GRAD>(p, stream)
                         : a.vocab >= V ? launch_runs<T, V, GRAD>(p, dbias != nullptr, stream)
                                        : launch_runs<T, 1, GRAD>(p, dbias != nullptr, stream);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !dbias) return e;
  hipLaunchKernelGGL(bias_join_kernel, dim3((unsigned)(((int64_t)a.vocab + 63) / 64)), dim3(1024), 0,
                     stream, p.partial, (int32_t)groups, a.vocab, dbias);
  return hipGetLastError();
}

template <bool GRAD>
hipError_t any_type(const LogitsArgs& p, float* dbias, hipStream_t stream) {
  switch (p.a.dtype) {
    case POLICY_F32: return shape<F32, GRAD>(p, dbias, stream);
    case POLICY_BF16: return shape<BF16, GRAD>(p, dbias, stream);
    default: return shape<F16, GRAD>(p, dbias, stream);
  }
}

__global__ __launch_bounds__(kThreads) void clear_kernel(float* p, int32_t n) {
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i < n) p[i] = 0.0f;
}

}  // namespace

hipError_t logits_forward_launch(const logits_args& a, void* out, int64_t out_row,
                                 hipStream_t stream) {
  if (a.rows == 0 || a.vocab == 0) return hipSuccess;
  LogitsArgs p{};
  p.a = a;
  p.out = out;
  p.out_row = out_row;
  p.penalties = a.history && a.history_width > 0 &&
                (a.repetition_rows || a.presence_rows || a.frequency_rows || a.repetition != 1.0f ||
                 a.presence != 0.0f || a.frequency != 0.0f);
  return any_type<false>(p, nullptr, stream);
}

bool logits_gradient_reads_logits(const logits_args& a) {
  return a.history && a.history_width > 0 && (a.repetition_rows || a.repetition != 1.0f);
}

int64_t logits_workspace_bytes(int64_t rows, int32_t vocab) {
  if (rows == 0 || vocab == 0) return 0;
  int64_t groups = run_groups(rows, vocab, true);
  if (vocab <= flat_most(POLICY_BF16) && flat_groups(rows, vocab) > groups)
    groups = flat_groups(rows, vocab);
  return groups * vocab * 4;
}

hipError_t logits_backward_launch(const logits_args& a, const void* dout, int64_t dout_row,
                                  void* dlogits, int64_t dlogits_row, float* dbias,
                                  void* workspace, hipStream_t stream) {
  if (a.vocab == 0) return hipSuccess;
  if (a.rows == 0) {
    if (!dbias) return hipSuccess;
    hipLaunchKernelGGL(clear_kernel, dim3((unsigned)(((int64_t)a.vocab + 255) / 256)),
                       dim3(kThreads), 0, stream, dbias, a.vocab);
    return hipGetLastError();
  }
  if (!dbias && !dlogits) return hipSuccess;
  LogitsArgs p{};
  p.a = a;
  p.dout = dout;
  p.dout_row = dout_row;
  p.out = dlogits;
  p.out_row = dlogits_row;
  p.partial = dbias ? static_cast<float*>(workspace) : nullptr;
  // without dlogits the factor is not needed
  p.penalties = dlogits && logits_gradient_reads_logits(a);
  return any_type<true>(p, dbias, stream);
}

}  // namespace rl
