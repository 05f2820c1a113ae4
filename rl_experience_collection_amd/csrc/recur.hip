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
// A workgroup of W waves (8, or 16 where it is alone on its compute unit) owns
// a column of 64 lanes x V channels and takes time in tiles, one slot of S steps
// per wave.  A wave loads its slot into registers, folds it into its map, and leaves the map in LDS; after one
// barrier every wave folds the maps before its own onto the state that enters
// the tile, replays its slot from registers and stores it.  So each element is
// read and written once.
//
// Where the columns alone fill the chip a workgroup walks all tiles of its
// column.  Where they are few (CHAIN) every tile has a workgroup of its own,
// taken in order from a ticket, and the states pass between them: a tile
// publishes its map, waits until one of the 16 tiles before it has published
// a state (a map with a done is one) and all nearer ones their maps, folds
// these onto it, oldest first, and publishes the state that leaves it.
// Every published map is one 64-bit word, stored and polled by device-coherent
// relaxed atomics, so no fence is needed; a kernel marks the words as empty
// first.  Each wait is on workgroups with earlier tickets, which run already
// and wait on earlier ones only, so every wait ends; a wait that reached its
// bound all the same would leave NaN, never a wrong number.  A state is the
// same expression wherever the walk found its start: results do not depend on
// timing.
//
// Linear gates may be larger than 1, and their products leave fp32's range
// where the states do not.  A slot whose slope or b is no finite number for a
// channel has no map there; one whose slope is below 2^-126 (faint) has one only
// for states so small beside b that what the slope has lost is below b's
// rounding.  Without a map the slot's wave runs it step by step on the state that
// enters it, once the slots before have passed.  A chained tile publishes no map of such a channel, or a faint one, and a walk
// that cannot use it waits for the state that leaves the tile.  Other channels
// and episodes keep their results to the bit.  (Sigmoid gates are at most 1: no
// product grows again, and what a faint slope loses stays below 2^-126 of the
// state it multiplies.)
#include <type_traits>

#include "elem.hpp"
#include "policy.hpp"
#include "wait.hpp"

namespace rl {

namespace {

// Steps per wave and tile (a slot's values stay in registers).  A chained tile is
// as long as a workgroup's registers allow: each costs a walk, and the walks of
// a column follow each other.  Backward, lanes of two channels take 4 steps: 64 x
// 4096 x 128 fp32 159 us with sigmoid gates against 170 with 8 (with linear ones
// 136 and 133); lanes of one or four 8.  A gradient on kept states takes the
// steps between two of them.
constexpr int slot_steps(int v, bool back, bool chained, bool kept) {
  return chained ? (back ? 8 : 16) : back && v == 2 && !kept ? 4 : 8;
}
// Steps between two states that are kept for the gradient.  dgate's factor
// h_{t-1} - x_t of the sigmoid form is a difference of near numbers where the
// state follows its input; from an h of 16 bits it keeps few digits or none
// (inputs of a constant and 1% noise: dgate off by 16% in bf16).  So the forward
// pass keeps every eighth state in fp32, a quarter of what h takes, and the
// gradient runs from there through x and gate, which it has in registers, and
// reads no h: both passes of 500 x 8192 x 64 bf16 take 886 us, from h 941 (500 x
// 128 x 128 56 and 55, 500 x 1024 x 64 119 and 130).
constexpr int kKeep = 8;
template <class T, bool SIG>
constexpr bool kKeeps = SIG && T::kBytes == 2;
constexpr float kReset = -0.0f;

struct Map {
  float a, b;
};

__device__ __forceinline__ bool is_reset(float a) { return __float_as_uint(a) == 0x80000000u; }
// Below 2^-126 a product of slopes is faint: it has lost digits, if not all.
constexpr float kFaint = 0x1p-149f;
__device__ __forceinline__ bool is_faint(float a) {
  return (__float_as_uint(a) & 0x7fffffffu) - 1u < 0x007fffffu;
}
// A product of slopes in its stored form: -0 after a done; of linear gates +0
// for either zero; of sigmoid gates never zero, so that an infinite state
// stays infinite.
template <bool SIG>
__device__ __forceinline__ float stored_slope(float a, bool reset) {
  return reset ? kReset : SIG ? __builtin_elementwise_maximum(a, kFaint) : a + 0.0f;
}
// Not a finite number.
__device__ __forceinline__ bool is_wild(float a) { return !(__builtin_fabsf(a) < __builtin_inff()); }
__device__ __forceinline__ float apply(Map m, float h) {
  return is_reset(m.a) ? m.b : __builtin_fmaf(m.a, h, m.b);
}
// first, then second
template <bool SIG>
__device__ __forceinline__ Map chain(Map first, Map second) {
  Map r;
  r.a = stored_slope<SIG>(first.a * second.a, is_reset(first.a) || is_reset(second.a));
  r.b = apply(second, first.b);
  return r;
}
// A product of up to 16 linear slopes, its exponent apart: it loses nothing on
// its way out of fp32's range and back.  A faint slope counts as 2^-126, which
// it is below.
struct Product {
  float m = 1.0f;
  int32_t e = 0;
  bool faint = false;
  __device__ __forceinline__ void times(float s) {
    m *= __builtin_amdgcn_frexp_mantf(s);
    e += __builtin_amdgcn_frexp_expf(s);
  }
  __device__ __forceinline__ void times_stored(float s) {
    faint = faint || is_faint(s);
    times(is_faint(s) ? 0x1p-126f : s);
  }
  // 0 only for a slope of zero; no number where it is not known to be faint
  __device__ __forceinline__ float value() const {
    const float p = __builtin_amdgcn_ldexpf(m, e);
    const bool low = __builtin_fabsf(p) <= 0x1p-126f && m != 0.0f;
    return low ? kFaint : faint && m != 0.0f ? __builtin_nanf("") : p;
  }
};

// Whether the map says nothing of what becomes of h.
template <bool SIG>
__device__ __forceinline__ bool is_lost(Map m, float h) {
  return !SIG && (is_wild(m.a) ||
                  (is_faint(m.a) && __builtin_fabsf(h) > 0x1p99f * __builtin_fabsf(m.b)));
}

// sigmoid(g) and sigmoid(-g), each to within a few fp32 roundings: with
// E = exp(-g) they are 1 / (1 + E) and E / (1 + E), so neither is formed by a
// difference.  E is 2^hi (1 + lo ln 2) with hi the rounded product -g log2(e)
// and lo what the rounding took off; the product's constant itself is off by
// 1.3e-8 |g| relative to E.  A large g leaves E = 0.  A g below -126 ln 2 is
// held there, where the reciprocal is 2^-126, the smallest it forms; taking
// that off makes sigmoid(g) 0 beyond and changes no larger one by more.
__device__ __forceinline__ void sigmoids(float g, float& a, float& keep) {
  // (a NaN passes both)
  const float m = __builtin_elementwise_maximum(__builtin_elementwise_minimum(g, 200.0f), -87.3365402f);
  const float hi = m * -1.44269502f;
  const float lo = __builtin_fmaf(m, -1.44269502f, -hi);
  float E = __builtin_amdgcn_exp2f(hi);
  E = __builtin_fmaf(E * lo, 0.693147182f, E);
  a = __builtin_amdgcn_rcpf(1.0f + E);
  keep = E * a;
  a -= 0x1p-126f;
}

struct RecurArgs {
  int32_t L, N, D;
  int32_t units;     // N * ceil(D / V): lanes with work
  int32_t per_row;   // ceil(D / V)
  int32_t columns;
  uint32_t tiles;    // chained: tiles of all columns
  int64_t x_step, x_row, g_step, g_row, h_step, h_row;
  int64_t dh_step, dh_row, dx_step, dx_row, dg_step, dg_row;
  const void *x, *gate, *h, *dh;
  const float *start;  // h0 / dh_last
  const float *h0;     // backward
  const uint8_t* dones;
  void *out, *dx, *dg;
  float* last;         // h_last / dh0
  float* kept;         // [ceil(L / 8)][N][D] states, or NULL (forward)
  uint32_t* ticket;    // chained: the next tile
  uint64_t* words;     // chained: [tiles][units][V] published maps
};

// One of the strided arrays as a column sees it: the address of its first
// row (the same for the workgroup) and this lane's offset from there.  With
// 32-bit offsets an access needs no arithmetic per lane.
template <class T, int V, bool OFF32>
struct Lane {
  char* base;
  typename std::conditional<OFF32, uint32_t, int64_t>::type off;
  int64_t step;
  __device__ __forceinline__ Lane(const void* p, int64_t step_, int64_t row, int32_t n0, int32_t n,
                                  int32_t d)
      : base(const_cast<char*>(static_cast<const char*>(p)) + n0 * row * T::kBytes),
        off((((int64_t)(n - n0) * row) + d) * T::kBytes),
        step(step_ * T::kBytes) {}
  __device__ __forceinline__ Pack<T, V> load(int32_t t) const {
    if constexpr (OFF32)
      return load_pack_at<T, V>(base + t * step, off);
    else
      return load_pack<T, V>(reinterpret_cast<const typename T::raw*>(base + t * step + off));
  }
  __device__ __forceinline__ void store(int32_t t, const Pack<T, V>& x) const {
    if constexpr (OFF32)
      store_pack_at<T, V>(base + t * step, off, x);
    else
      store_pack<T, V>(reinterpret_cast<typename T::raw*>(base + t * step + off), x);
  }
};

constexpr int kWalk = 16;              // tiles looked back over at most
constexpr uint32_t kPolls = 1u << 24;  // of a wait, at most

// A published word is a map: its slope below, its b above.  A state is the
// map that forgets and gives the state.  A slope of these bits is one not yet
// published: published slopes that are no numbers all have the same bits,
// others.
constexpr uint32_t kNothing = 0xffffffffu;

__device__ __forceinline__ void put_map(uint64_t* p, Map m) {
  const float a = m.a == m.a ? m.a : __builtin_nanf("");
  __hip_atomic_store(p, (uint64_t)__float_as_uint(a) | (uint64_t)__float_as_uint(m.b) << 32,
                     __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ Map get_map(const uint64_t* p) {
  const uint64_t w = __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return Map{__uint_as_float((uint32_t)w), __uint_as_float((uint32_t)(w >> 32))};
}

// The next tile of a chained workgroup, in the order of the scan, and its
// column; false when all are taken.
struct Chained {
  int32_t order, column;
  __device__ __forceinline__ bool take(const RecurArgs& p) {
    __shared__ uint32_t s_ticket;
    if (threadIdx.x == 0)
      s_ticket = __hip_atomic_fetch_add(p.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();  // (and the tile before is done with its LDS)
    const uint32_t k = __builtin_amdgcn_readfirstlane(s_ticket);
    order = (int32_t)(k / (uint32_t)p.columns);
    column = (int32_t)(k % (uint32_t)p.columns);
    return k < p.tiles;
  }
};

// What a workgroup of a chained scan keeps in LDS besides its slots' maps.
template <int V>
struct ChainLds {
  Map before[kWalk][64][V];  // the maps of the tiles before
  float state[64][V];        // that enters this tile
  int32_t walk;              // tiles to look at; 0: the state is there
};

// The tiles before tile `o` that have to be looked at, as far as one of their
// words tells: polled by wave 0 until a state and all nearer maps are out.
// `sample` is that word of tile o; `left` the polls that remain.
__device__ __forceinline__ int32_t poll_chain(const uint64_t* sample, int64_t stride, int32_t o, int lane,
                                              uint32_t& left) {
  const uint64_t* at = sample - (int64_t)min(min(lane, kWalk - 1) + 1, o) * stride;
  for (;;) {
    const float a = get_map(at).a;
    const uint64_t out = __ballot(__float_as_uint(a) != kNothing), state = __ballot(is_reset(a));
    const int nearest = state ? __builtin_ctzll(state) : 64;
    // (lanes past the walk repeat its end)
    if (nearest < kWalk && (~out & ((2ull << nearest) - 1)) == 0) return nearest + 1;
    if (wait_over(false, left)) return kWalk;
    __builtin_amdgcn_s_sleep(1);
  }
}

// The state that enters tile `o` (in the order of the scan), for every wave:
// `c` is the state that enters the scan and becomes that.  Wave 0 learns whether
// it has to publish the state that leaves the tile itself, later, for some
// channel: one that the tile's map does not take there.  `odd`: a slot has no
// map, or a faint one.
template <bool SIG, int V, int W>
__device__ __forceinline__ bool enter_tile(const RecurArgs& p, int32_t o, int32_t u, bool active,
                                               int w, int lane, bool odd,
                                               const float (&sa)[W][64][V],
                                               const float (&sb)[W][64][V], ChainLds<V>& s,
                                               float (&c)[V]) {
  const int64_t stride = (int64_t)p.units * V;  // words of a tile
  uint64_t* mine = p.words + o * stride + (int64_t)u * V;
  Map t[V];
  bool none[V];  // no map
  if (w == 0) {
    // the tile's map
#pragma unroll
    for (int v = 0; v < V; ++v) {
      t[v] = Map{sa[0][lane][v], sb[0][lane][v]};
      none[v] = false;
    }
    if constexpr (SIG) {
#pragma unroll
      for (int j = 1; j < W; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) t[v] = chain<SIG>(t[v], Map{sa[j][lane][v], sb[j][lane][v]});
    } else {
      // (All later tiles wait for this: 4096 x 16 x 128 bf16 takes 22 us so, 21
      // with a plain product.)
      Product a[V];
      bool cut[V];
#pragma unroll
      for (int v = 0; v < V; ++v) cut[v] = is_reset(t[v].a);
      if (!odd) {
#pragma unroll
        for (int v = 0; v < V; ++v) a[v].times(t[v].a);
#pragma unroll
        for (int j = 1; j < W; ++j)
#pragma unroll
          for (int v = 0; v < V; ++v) {
            const Map m = Map{sa[j][lane][v], sb[j][lane][v]};
            cut[v] = cut[v] || is_reset(m.a);
            a[v].times(m.a);
            t[v].b = apply(m, t[v].b);
          }
      } else {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          none[v] = is_wild(t[v].a);
          a[v].times_stored(t[v].a);
        }
#pragma unroll 1
        for (int j = 1; j < W; ++j)
#pragma unroll
          for (int v = 0; v < V; ++v) {
            const Map m = Map{sa[j][lane][v], sb[j][lane][v]};
            // (a done forgets what went wrong before it)
            none[v] = !is_reset(m.a) && (none[v] || is_lost<SIG>(m, t[v].b));
            cut[v] = cut[v] || is_reset(m.a);
            a[v].times_stored(m.a);
            t[v].b = apply(m, t[v].b);
          }
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        t[v].a = stored_slope<SIG>(a[v].value(), cut[v]);
        none[v] = none[v] || (!cut[v] && (is_wild(t[v].a) || is_wild(t[v].b)));
      }
    }
    if (o > 0 && active) {
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (!none[v]) put_map(mine + v, t[v]);
    }
  }
  if (o > 0) {
    uint32_t left = kPolls;
    for (;;) {
      if (w == 0) {
        // the word of the column's first unit stands for all
        const int32_t u0 = __builtin_amdgcn_readfirstlane(u);
        const int32_t walk = poll_chain(p.words + o * stride + (int64_t)u0 * V, stride, o, lane, left);
        if (lane == 0) s.walk = walk;
      }
      __syncthreads();
      const int32_t walk = __builtin_amdgcn_readfirstlane(s.walk);
#pragma unroll
      for (int k = 0; k < kWalk / W; ++k) {
        const int back = w + k * W;  // tiles in between
        if (back >= walk) continue;
        const uint64_t* at = mine - (int64_t)min(back + 1, o) * stride;
#pragma unroll
        for (int v = 0; v < V; ++v) s.before[back][lane][v] = get_map(at + v);
      }
      __syncthreads();
      if (w == 0) {
        // from the oldest to the nearest: a state starts anew, a gap ends it
        bool ready = true;
        float x[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          x[v] = 0.0f;
          bool known = false;
          for (int k = walk - 1; k >= 0; --k) {
            const Map m = s.before[k][lane][v];
            known = is_reset(m.a) ||
                    (known && __float_as_uint(m.a) != kNothing && !is_lost<SIG>(m, x[v]));
            x[v] = apply(m, x[v]);
          }
          ready = ready && known;
        }
        const bool done = __all(ready || !active);
        if (wait_over(done, left)) {
#pragma unroll
          for (int v = 0; v < V; ++v) s.state[lane][v] = done ? x[v] : __builtin_nanf("");
          if (lane == 0) s.walk = 0;
        }
      }
      __syncthreads();
      if (__builtin_amdgcn_readfirstlane(s.walk) == 0) break;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) c[v] = s.state[lane][v];
  }
  bool held = false;
  if (w == 0) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (!none[v] && o > 0 && is_reset(t[v].a)) continue;  // its map was its state
      const bool later = none[v] || is_lost<SIG>(t[v], c[v]);
      held = held || later;
      if (active && !later) put_map(mine + v, Map{kReset, apply(t[v], c[v])});
    }
    held = !SIG && __ballot(held) != 0;
  }
  return held;
}

// The state that leaves tile `o`, where wave 0 has published no state yet.
template <int V>
__device__ __forceinline__ void put_held(const RecurArgs& p, int32_t o, int32_t u, bool active,
                                         const float (&c)[V]) {
  if (!active) return;
  uint64_t* mine = p.words + (o * (int64_t)p.units + u) * V;
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (!is_reset(get_map(mine + v).a)) put_map(mine + v, Map{kReset, c[v]});
}

// Joins the tile's slots: `c` is the state that enters the tile, and then the
// one that leaves it; `h` becomes the state that enters this wave's slot.  Bit
// j of `cuts`: slot j holds a done in some lane.  The choices are the same for
// the whole wave and stay branches (the empty statements keep them so): as
// selects they would cost as much as the sums.
template <int V, int W>
__device__ __forceinline__ void join_slots(const float (&sa)[W][64][V], const float (&sb)[W][64][V],
                                           uint32_t cuts, int w, int lane, float (&c)[V],
                                           float (&h)[V]) {
#pragma unroll
  for (int j = 0; j < W; ++j) {
    Map m[V];
#pragma unroll
    for (int v = 0; v < V; ++v) m[v] = Map{sa[j][lane][v], sb[j][lane][v]};
    if (j == w) {
      asm volatile("");
#pragma unroll
      for (int v = 0; v < V; ++v) h[v] = c[v];
    }
    if ((cuts >> j) & 1u) {
      asm volatile("");
#pragma unroll
      for (int v = 0; v < V; ++v) c[v] = apply(m[v], c[v]);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) c[v] = __builtin_fmaf(m[v].a, c[v], m[v].b);
    }
  }
}

// The same where some slot has no map for a channel, or a faint one.  A slot
// that needs it is run by its wave on the state that enters it, for those
// channels (run: h -> the state that leaves), and leaves the result in the place
// of the map's b.  All waves hold the same states and maps here, so they agree
// on which slots those are.
template <int V, int W, class Run>
__device__ __forceinline__ void join_odd(const float (&sa)[W][64][V], float (&sb)[W][64][V], int w,
                                         int lane, float (&c)[V], float (&h)[V], Run run) {
#pragma unroll 1
  for (int j = 0; j < W; ++j) {
    Map m[V];
    bool lost[V], any = false;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      m[v] = Map{sa[j][lane][v], sb[j][lane][v]};
      lost[v] = is_lost<false>(m[v], c[v]);
      any = any || lost[v];
    }
    if (j == w) {
#pragma unroll
      for (int v = 0; v < V; ++v) h[v] = c[v];
    }
    if (__ballot(any)) {
      __syncthreads();  // every wave has the slot's maps
      if (j == w) {
        float step[V];
#pragma unroll
        for (int v = 0; v < V; ++v) step[v] = c[v];
        run(step);
#pragma unroll
        for (int v = 0; v < V; ++v)
          if (lost[v]) sb[j][lane][v] = step[v];
      }
      __syncthreads();
#pragma unroll
      for (int v = 0; v < V; ++v) c[v] = lost[v] ? sb[j][lane][v] : apply(m[v], c[v]);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) c[v] = apply(m[v], c[v]);
    }
  }
}

// What a slot tells of itself besides its maps: a done in some lane; no map, or
// a faint one, of some channel.
constexpr uint32_t kCut = 1, kOdd = 2;

// The stored slope of a slot's steps from their product `a`.  `low`: the least
// magnitude on the way (linear gates); where it left the normal numbers the
// product is formed again.  A b that is no finite number leaves no map.
template <int S, int V, bool SIG>
__device__ __forceinline__ void settle_slopes(const float (&a)[S][V], const float (&low)[V], bool cut,
                                              Map (&m)[V]) {
  if constexpr (!SIG) {
    bool again = false;
#pragma unroll
    for (int v = 0; v < V; ++v) again = again || low[v] < 0x1p-126f;
    if (__ballot(again)) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        Product p;
#pragma unroll
        for (int i = 0; i < S; ++i) p.times(a[i][v]);
        if (low[v] < 0x1p-126f) m[v].a = p.value();
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (is_wild(m[v].b)) m[v].a = __builtin_nanf("");
  }
#pragma unroll
  for (int v = 0; v < V; ++v) m[v].a = stored_slope<SIG>(m[v].a, cut);
}
template <int V>
__device__ __forceinline__ bool is_odd(const Map (&m)[V]) {
  bool odd = false;
#pragma unroll
  for (int v = 0; v < V; ++v) odd = odd || is_wild(m[v].a) || is_faint(m[v].a);
  return odd;
}

// Where a workgroup and its lane stand.
struct Place {
  int lane, w;
  int32_t u, n0, n, d;
  bool active;
  int64_t cell;
  template <int V>
  static __device__ __forceinline__ Place of(const RecurArgs& p, int32_t column) {
    Place s;
    s.lane = (int)threadIdx.x & 63;
    s.w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int32_t first = column * 64;
    s.active = first + s.lane < p.units;
    s.u = s.active ? first + s.lane : p.units - 1;  // idle lanes read a valid element
    s.n0 = first / p.per_row;
    s.n = s.u / p.per_row;
    // a row's last unit is moved back to end with it: where D is no multiple
    // of V it repeats channels of the one before, with the same results
    s.d = min((s.u - s.n * p.per_row) * V, p.D - V);
    s.cell = (int64_t)s.n * p.D + s.d;
    return s;
  }
};

// The dones that cut this slot's steps, bit i for step t(i): the state that
// enters step t is cut where dones[t - 1] is set.
template <int S, bool BACK>
__device__ __forceinline__ uint32_t load_dones(const RecurArgs& p, int32_t n, int32_t from, int32_t tb,
                                               int32_t te) {
  uint8_t db[S];
#pragma unroll
  for (int i = 0; i < S; ++i) {
    const int32_t t = BACK ? from - i : from + i;
    const uint8_t* row = p.dones + (int64_t)(max(min(max(t, tb), te - 1), 1) - 1) * p.N;
    db[i] = *reinterpret_cast<uint8_t RL_GLOBAL*>(shared_address(row) + (uint32_t)n);
  }
  uint32_t done = 0;
#pragma unroll
  for (int i = 0; i < S; ++i) {
    const int32_t t = BACK ? from - i : from + i;
    done |= (t > 0 && t >= tb && t < te && db[i] ? 1u : 0u) << i;
  }
  return done;
}

// A slot's map, of steps a h + b.
template <int V, int S, bool SIG, bool CUT>
__device__ __forceinline__ void fold_forward(const float (&a)[S][V], const float (&b)[S][V],
                                             uint32_t done, Map (&m)[V]) {
  float low[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    m[v] = Map{a[0][v], b[0][v]};
    low[v] = __builtin_fabsf(a[0][v]);
  }
#pragma unroll
  for (int i = 1; i < S; ++i)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float nb = __builtin_fmaf(a[i][v], m[v].b, b[i][v]);
      m[v].b = CUT && ((done >> i) & 1u) ? b[i][v] : nb;
      m[v].a *= a[i][v];
      if (!SIG) low[v] = __builtin_fminf(low[v], __builtin_fabsf(m[v].a));
    }
  settle_slopes<S, V, SIG>(a, low, CUT && done != 0, m);
}

// Bound by memory where the columns fill the chip: 500 x 8192 x 64 bf16 in 318
// us (1.58 GB at 5.0 TB/s; 341 with the kept states, 1.71 GB); 500 x 128 x 128
// fp32, whose 256 columns give each compute unit one workgroup, in 26 (98 MB at
// 3.7 TB/s).  Chained, by the states' way from tile to tile: 65,537 x 2 x 1000
// fp16 in 262 us (786 MB at 3.0 TB/s).
template <class T, int V, bool SIG, bool CHAIN, bool OFF32, int W>
__global__ __launch_bounds__(64 * W) void recur_forward_kernel(const RecurArgs p) {
  constexpr bool KEEPS = kKeeps<T, SIG>;
  constexpr int S = slot_steps(V, false, CHAIN, KEEPS), kTile = S * W;
  static_assert(S % kKeep == 0, "a slot begins at a kept state");
  __shared__ typename std::conditional<CHAIN, ChainLds<V>, char>::type s_chain;
  constexpr int kBufs = CHAIN ? 1 : 2;
  __shared__ alignas(16) float s_a[kBufs][W][64][V], s_b[kBufs][W][64][V];
  __shared__ uint32_t s_note[kBufs][W];
  Chained tile{0, (int32_t)blockIdx.x};
  do {
    if (CHAIN && !tile.take(p)) break;
    const Place at = Place::of<V>(p, tile.column);
    const int lane = at.lane, w = at.w;
    const Lane<T, V, OFF32> x(p.x, p.x_step, p.x_row, at.n0, at.n, at.d);
    const Lane<T, V, OFF32> gate(p.gate, p.g_step, p.g_row, at.n0, at.n, at.d);
    const Lane<T, V, OFF32> out(p.out, p.h_step, p.h_row, at.n0, at.n, at.d);
    const int32_t tb = CHAIN ? tile.order * kTile : 0, te = CHAIN ? min(p.L, tb + kTile) : p.L;

    float c[V];  // the state that enters the tile
#pragma unroll
    for (int v = 0; v < V; ++v) c[v] = p.start ? p.start[at.cell + v] : 0.0f;

    int buf = 0;
    for (int32_t t0 = tb; t0 < te; t0 += kTile, buf = (buf + 1) % kBufs) {
      const int32_t ts = t0 + w * S;
      Pack<T, V> xr[S], gr[S];
#pragma unroll
      for (int i = 0; i < S; ++i) {
        const int32_t t = min(ts + i, te - 1);  // steps past the end: loaded, not used
        xr[i] = x.load(t);
        gr[i] = gate.load(t);
      }
      const uint32_t done = p.dones ? load_dones<S, false>(p, at.n, ts, tb, te) : 0u;
      float a[S][V], b[S][V];
#pragma unroll
      for (int i = 0; i < S; ++i) {
        float xf[V], gf[V];
        widen_pack<T, V>(xr[i], xf);
        widen_pack<T, V>(gr[i], gf);
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
        }
      }
      if (ts + S > te) {
        // steps past the end leave the state as it is
#pragma unroll
        for (int i = 0; i < S; ++i)
          if (ts + i >= te)
#pragma unroll
            for (int v = 0; v < V; ++v) {
              a[i][v] = 1.0f;
              b[i][v] = 0.0f;
            }
      }
      const bool cut = __ballot(done != 0) != 0;  // (of the wave)
      Map m[V];
      if (cut)
        fold_forward<V, S, SIG, true>(a, b, done, m);
      else
        fold_forward<V, S, SIG, false>(a, b, done, m);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        s_a[buf][w][lane][v] = m[v].a;
        s_b[buf][w][lane][v] = m[v].b;
      }
      uint32_t note = cut ? kCut : 0u;
      if constexpr (!SIG) {
        if (__ballot(is_odd<V>(m))) note |= kOdd;
      }
      if (lane == 0) s_note[buf][w] = note;
      __syncthreads();
      const uint32_t notes = s_note[buf][lane % W];
      const uint32_t cuts = (uint32_t)__ballot((notes & kCut) != 0);
      const bool odd = !SIG && __ballot((notes & kOdd) != 0) != 0;
      bool held = false;
      if constexpr (CHAIN)
        held = enter_tile<SIG, V, W>(p, tile.order, at.u, at.active, w, lane, odd, s_a[buf], s_b[buf],
                                     s_chain, c);
      float h[V];
      if (odd) {
        join_odd<V, W>(s_a[buf], s_b[buf], w, lane, c, h, [&](float (&s)[V]) {
#pragma unroll
          for (int i = 0; i < S; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v)
              s[v] = (done >> i) & 1u ? b[i][v] : __builtin_fmaf(a[i][v], s[v], b[i][v]);
        });
      } else {
        join_slots<V, W>(s_a[buf], s_b[buf], cuts, w, lane, c, h);
      }
      if constexpr (CHAIN && !SIG) {
        if (held) put_held<V>(p, tile.order, at.u, at.active, c);
      }
      auto replay = [&](auto cuts_here) {
#pragma unroll
        for (int i = 0; i < S; ++i) {
          if (ts + i >= te) break;
          if (KEEPS && i % kKeep == 0 && p.kept && at.active)
            store_pack<F32, V>(reinterpret_cast<uint32_t*>(p.kept) +
                                   (int64_t)((ts + i) / kKeep) * p.N * p.D + at.cell,
                               narrow_pack<F32, V>(h));
#pragma unroll
          for (int v = 0; v < V; ++v) {
            const float nh = __builtin_fmaf(a[i][v], h[v], b[i][v]);
            h[v] = cuts_here.value && ((done >> i) & 1u) ? b[i][v] : nh;
          }
          if (at.active && (!KEEPS || p.out)) out.store(ts + i, narrow_pack<T, V>(h));
        }
      };
      if (cut)
        replay(std::true_type{});
      else
        replay(std::false_type{});
      // h is the state of the slot's last step
      if (p.last && at.active && ts < p.L && ts + S >= p.L && te == p.L) {
        const bool end = p.dones && p.dones[(int64_t)(p.L - 1) * p.N + at.n];
#pragma unroll
        for (int v = 0; v < V; ++v) p.last[at.cell + v] = end ? 0.0f : h[v];
      }
    }
  } while (CHAIN);
}

// A slot's map backwards, of steps a (dh + G).
template <int V, int S, bool SIG, bool CUT>
__device__ __forceinline__ void fold_backward(const float (&a)[S][V], const float (&dh)[S][V],
                                              uint32_t done, Map (&m)[V]) {
  float low[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    m[v] = Map{1.0f, 0.0f};
    low[v] = 1.0f;
  }
#pragma unroll
  for (int i = 0; i < S; ++i)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float nb = a[i][v] * (dh[i][v] + m[v].b);
      m[v].b = CUT && ((done >> i) & 1u) ? 0.0f : nb;
      m[v].a *= a[i][v];
      if (!SIG) low[v] = __builtin_fminf(low[v], __builtin_fabsf(m[v].a));
    }
  settle_slopes<S, V, SIG>(a, low, CUT && done != 0, m);
}

// Bound like the forward pass: 500 x 8192 x 64 bf16 in 551 us (2.76 GB at 5.0
// TB/s), 500 x 128 x 128 fp32 with linear gates in 36 (164 MB at 4.5 TB/s).
template <class T, int V, bool SIG, bool CHAIN, bool OFF32, int W>
__global__ __launch_bounds__(64 * W) void recur_backward_kernel(const RecurArgs p) {
  constexpr bool KEEPS = kKeeps<T, SIG>;
  constexpr int S = slot_steps(V, true, CHAIN, KEEPS), kTile = S * W;
  static_assert(!KEEPS || S == kKeep, "a slot is the steps from a kept state to the next");
  __shared__ typename std::conditional<CHAIN, ChainLds<V>, char>::type s_chain;
  constexpr int kBufs = CHAIN ? 1 : 2;
  __shared__ alignas(16) float s_a[kBufs][W][64][V], s_b[kBufs][W][64][V];
  __shared__ uint32_t s_note[kBufs][W];
  Chained tile{0, (int32_t)blockIdx.x};
  do {
    if (CHAIN && !tile.take(p)) break;
    const Place at = Place::of<V>(p, tile.column);
    const int lane = at.lane, w = at.w;
    const Lane<T, V, OFF32> x(p.x, p.x_step, p.x_row, at.n0, at.n, at.d);
    const Lane<T, V, OFF32> gate(p.gate, p.g_step, p.g_row, at.n0, at.n, at.d);
    const Lane<T, V, OFF32> hs(p.h, p.h_step, p.h_row, at.n0, at.n, at.d);
    const Lane<T, V, OFF32> dh(p.dh, p.dh_step, p.dh_row, at.n0, at.n, at.d);
    const Lane<T, V, OFF32> dx(p.dx, p.dx_step, p.dx_row, at.n0, at.n, at.d);
    const Lane<T, V, OFF32> dg(p.dg, p.dg_step, p.dg_row, at.n0, at.n, at.d);
    // Chained tiles are counted from the end, the last of them in time whole;
    // with kept states tiles begin at a multiple of their length, the last of
    // them in time may be short.
    const int32_t whole = KEEPS ? (p.L + kTile - 1) / kTile * kTile : p.L;
    const int32_t tt = CHAIN ? whole - tile.order * kTile : whole, te = min(tt, p.L);
    const int32_t tb = CHAIN ? max(0, tt - kTile) : 0;

    float c[V];  // G of the step after the tile
    const bool end = p.dones && p.dones[(int64_t)(p.L - 1) * p.N + at.n];
#pragma unroll
    for (int v = 0; v < V; ++v) c[v] = p.start && !end ? p.start[at.cell + v] : 0.0f;

    int buf = 0;
    for (int32_t t1 = tt; t1 > tb; t1 -= kTile, buf = (buf + 1) % kBufs) {
      const int32_t top = t1 - 1 - w * S;  // this wave's latest step
      auto inside = [&](int32_t t) { return KEEPS ? min(t, te - 1) : max(t, tb); };
      Pack<T, V> gr[S], dr[S], xr[SIG ? S : 1], hr[KEEPS ? 1 : S];
      Pack<F32, V> kr;
#pragma unroll
      for (int i = 0; i < S; ++i) {
        const int32_t t = inside(top - i);
        gr[i] = gate.load(t);
        dr[i] = dh.load(t);
      }
      const uint32_t done = p.dones ? load_dones<S, true>(p, at.n, top, tb, te) : 0u;
#pragma unroll
      for (int i = 0; i < S; ++i) {
        const int32_t t = inside(top - i);
        if (SIG) xr[SIG ? i : 0] = x.load(t);
        if (!KEEPS) hr[KEEPS ? 0 : i] = hs.load(max(t - 1, 0));
      }
      if constexpr (KEEPS)
        kr = load_pack<F32, V>(reinterpret_cast<const uint32_t*>(p.kept) +
                               (int64_t)(inside(top - S + 1) / kKeep) * p.N * p.D + at.cell);
      float a[S][V], k[SIG ? S : 1][V], df[S][V];
#pragma unroll
      for (int i = 0; i < S; ++i) {
        float gf[V];
        widen_pack<T, V>(gr[i], gf);
        widen_pack<T, V>(dr[i], df[i]);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          if (SIG)
            sigmoids(gf[v], a[i][v], k[SIG ? i : 0][v]);
          else
            a[i][v] = gf[v];
        }
      }
      // the state that enters each step, less its input
      float q[KEEPS ? S : 1][V];
      if constexpr (KEEPS) {
        float s[V];
        widen_pack<F32, V>(kr, s);
#pragma unroll
        for (int i = S - 1; i >= 0; --i) {
          float xf[V];
          widen_pack<T, V>(xr[i], xf);
#pragma unroll
          for (int v = 0; v < V; ++v) {
            const bool drop = (done >> i) & 1u;
            const float b = k[i][v] * xf[v];
            q[i][v] = (drop ? 0.0f : s[v]) - xf[v];
            const float ns = __builtin_fmaf(a[i][v], s[v], b);
            s[v] = drop ? b : ns;
          }
        }
      }
      if (KEEPS ? top >= te : top - S + 1 < tb) {
        // steps outside the tile leave the carry as it is
#pragma unroll
        for (int i = 0; i < S; ++i)
          if (KEEPS ? top - i >= te : top - i < tb)
#pragma unroll
            for (int v = 0; v < V; ++v) {
              a[i][v] = 1.0f;
              df[i][v] = 0.0f;
            }
      }
      const bool cut = __ballot(done != 0) != 0;
      Map m[V];
      if (cut)
        fold_backward<V, S, SIG, true>(a, df, done, m);
      else
        fold_backward<V, S, SIG, false>(a, df, done, m);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        s_a[buf][w][lane][v] = m[v].a;
        s_b[buf][w][lane][v] = m[v].b;
      }
      uint32_t note = cut ? kCut : 0u;
      if constexpr (!SIG) {
        if (__ballot(is_odd<V>(m))) note |= kOdd;
      }
      if (lane == 0) s_note[buf][w] = note;
      __syncthreads();
      const uint32_t notes = s_note[buf][lane % W];
      const uint32_t cuts = (uint32_t)__ballot((notes & kCut) != 0);
      const bool odd = !SIG && __ballot((notes & kOdd) != 0) != 0;
      bool held = false;
      if constexpr (CHAIN)
        held = enter_tile<SIG, V, W>(p, tile.order, at.u, at.active, w, lane, odd, s_a[buf], s_b[buf],
                                     s_chain, c);
      float G[V];
      if (odd) {
        join_odd<V, W>(s_a[buf], s_b[buf], w, lane, c, G, [&](float (&s)[V]) {
#pragma unroll
          for (int i = 0; i < S; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v)
              s[v] = (done >> i) & 1u ? 0.0f : a[i][v] * (df[i][v] + s[v]);
        });
      } else {
        join_slots<V, W>(s_a[buf], s_b[buf], cuts, w, lane, c, G);
      }
      if constexpr (CHAIN && !SIG) {
        if (held) put_held<V>(p, tile.order, at.u, at.active, c);
      }
      auto replay = [&](auto cuts_here) {
#pragma unroll
        for (int i = 0; i < S; ++i) {
          const int32_t t = top - i;
          if (KEEPS ? t >= te : t < tb) {
            if (KEEPS) continue;
            break;
          }
          const bool drop = cuts_here.value && ((done >> i) & 1u);
          float hf[V], xf[V], ox[V], og[V];
          if (!KEEPS) widen_pack<T, V>(hr[KEEPS ? 0 : i], hf);
          if (SIG && !KEEPS) widen_pack<T, V>(xr[SIG ? i : 0], xf);
          if (!KEEPS && t == 0) {
#pragma unroll
            for (int v = 0; v < V; ++v) hf[v] = p.h0 ? p.h0[at.cell + v] : 0.0f;
          }
#pragma unroll
          for (int v = 0; v < V; ++v) {
            const float del = df[i][v] + G[v];
            const float prev = KEEPS || drop ? 0.0f : hf[v];
            if (SIG) {
              ox[v] = k[SIG ? i : 0][v] * del;
              og[v] = a[i][v] * ox[v] * (KEEPS ? q[KEEPS ? i : 0][v] : prev - xf[v]);
            } else {
              ox[v] = del;
              og[v] = drop ? 0.0f : del * prev;
            }
            G[v] = drop ? 0.0f : a[i][v] * del;
          }
          if (at.active) {
            dx.store(t, narrow_pack<T, V>(ox));
            dg.store(t, narrow_pack<T, V>(og));
          }
        }
      };
      if (cut)
        replay(std::true_type{});
      else
        replay(std::false_type{});
      // G is that of the slot's earliest step
      if (p.last && at.active && top >= 0 && top - S < 0 && tb == 0) {
#pragma unroll
        for (int v = 0; v < V; ++v) p.last[at.cell + v] = G[v];
      }
    }
  } while (CHAIN);
}

// Bound by its launch: 128 x 128 bf16 in 3.0 us, of 0.2 MB.
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

// Before a chained scan: the ticket at 0, every word empty.
__global__ __launch_bounds__(256) void empty_chain_kernel(uint32_t* ticket, uint64_t* words, int64_t n) {
  if (blockIdx.x == 0 && threadIdx.x == 0) *ticket = 0;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
    words[i] = kNothing;
}

// Columns that give the chip enough workgroups, each walking all of time: one
// for each compute unit.  Forward, 4096 steps of sigmoid gates, fp32: 128 columns
// take 164 us so, chained 103; 256 take 182, chained 210.
constexpr int64_t kWantColumns = 256;

// Waves of a workgroup that has a compute unit to itself.  (Lanes of 8 bytes
// have enough loads on their way from 8: 500 x 256 x 128 fp32 takes 35 + 77 us
// so, 37 + 82 from 16.  Lanes of 4: 8192 x 128 x 256 bf16 369 + 749 us from 8,
// 339 + 647 from 16; with more workgroups, 500 x 200 x 128 fp32, 30 + 67 and
// 38 + 69; within a tile of 8 waves, 30 x 128 x 128 fp32, 5.0 + 6.8 and 6.8 +
// 8.4.)
constexpr int kManyWaves = 16, kFewWaves = 8;

int64_t per_row_of(int32_t D, int v) { return (D + v - 1) / v; }

// Channels of a lane: as many as leave the launch enough columns.  4096 x 256 x
// 128 fp32 takes 282 + 571 us in lanes of two channels, 256 columns, and 310 +
// 633 us in lanes of one, 512.
int lane_channels(int32_t N, int32_t D, int32_t dtype) {
  for (int v = dtype == POLICY_F32 ? 2 : 4; v > 1; v /= 2)
    if (D >= v && (N * per_row_of(D, v) + 63) / 64 >= kWantColumns) return v;
  return D >= 2 && dtype != POLICY_F32 ? 2 : 1;
}

// Tiles of a chained scan, or 0 where the columns are enough, or one tile is
// the whole time.  400 x 4 x 128 fp32 forward: 12.6 us as two tiles, 16.2 in one
// workgroup's walk.
int32_t chained_tiles(int32_t L, int64_t units, bool back) {
  const int32_t tile = kManyWaves * slot_steps(1, back, true, false);
  const int64_t columns = (units + 63) / 64;
  return columns >= kWantColumns || L <= tile ? 0 : (L + tile - 1) / tile;
}
// Workspace: a ticket, then the words.
constexpr size_t kTicketBytes = 256;
int64_t chained_bytes(int32_t tiles, int64_t units, int v) {
  return tiles ? (int64_t)kTicketBytes + tiles * units * v * 8 : 0;
}

template <class T, int V, bool SIG, bool BACK, bool CHAIN, bool OFF32, int W>
hipError_t start(const RecurArgs& p, dim3 grid, hipStream_t stream) {
  if constexpr (BACK)
    hipLaunchKernelGGL((recur_backward_kernel<T, V, SIG, CHAIN, OFF32, W>), grid, dim3(64 * W), 0, stream, p);
  else
    hipLaunchKernelGGL((recur_forward_kernel<T, V, SIG, CHAIN, OFF32, W>), grid, dim3(64 * W), 0, stream, p);
  return hipGetLastError();
}

template <class T, int V, bool SIG, bool BACK, bool OFF32>
hipError_t launch(RecurArgs p, void* workspace, hipStream_t stream) {
  p.per_row = (int32_t)per_row_of(p.D, V);
  p.units = p.N * p.per_row;
  p.columns = (p.units + 63) / 64;
  const int32_t tiles = chained_tiles(p.L, p.units, BACK);
  if constexpr (V * T::kBytes <= 4) if (tiles) {  // (wider lanes only where columns are plenty)
    p.ticket = static_cast<uint32_t*>(workspace);
    p.words = reinterpret_cast<uint64_t*>(static_cast<char*>(workspace) + kTicketBytes);
    const int64_t words = tiles * (int64_t)p.units * V, blocks = (words + 255) / 256;
    hipLaunchKernelGGL(empty_chain_kernel, dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(256), 0,
                       stream, p.ticket, p.words, words);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    p.tiles = (uint32_t)tiles * (uint32_t)p.columns;
    const dim3 grid(p.tiles < (1u << 21) ? p.tiles : 1u << 21);
    return start<T, V, SIG, BACK, true, OFF32, kManyWaves>(p, grid, stream);
  }
  const dim3 grid((unsigned)p.columns);
  if constexpr (V * T::kBytes <= 4)
    if (p.columns <= kWantColumns && p.L > kFewWaves * slot_steps(V, BACK, false, kKeeps<T, SIG>))
      return start<T, V, SIG, BACK, false, OFF32, kManyWaves>(p, grid, stream);
  return start<T, V, SIG, BACK, false, OFF32, kFewWaves>(p, grid, stream);
}

template <class T, bool SIG, bool BACK>
hipError_t pick(const RecurArgs& p, int32_t dtype, void* ws, hipStream_t stream) {
  const int v = lane_channels(p.N, p.D, dtype);
  // a column's rows, seen from its first, within 32-bit offsets
  int64_t row = p.x_row;
  for (int64_t r : {p.g_row, p.h_row, p.dh_row, p.dx_row, p.dg_row}) row = r > row ? r : row;
  const int64_t rows = 64 / per_row_of(p.D, v) + 1;
  if (row > (((int64_t)1 << 31) / T::kBytes - p.D) / rows) {
    if (v == 1) return launch<T, 1, SIG, BACK, false>(p, ws, stream);
    return launch<T, 2, SIG, BACK, false>(p, ws, stream);
  }
  switch (v) {
    case 4: if constexpr (T::kBytes == 2) return launch<T, 4, SIG, BACK, true>(p, ws, stream);
    case 2: return launch<T, 2, SIG, BACK, true>(p, ws, stream);
    default: return launch<T, 1, SIG, BACK, true>(p, ws, stream);
  }
}

template <bool BACK>
hipError_t pick_type(const RecurArgs& p, int32_t dtype, bool sig, void* ws, hipStream_t stream) {
  switch (dtype) {
    case POLICY_F32:
      return sig ? pick<F32, true, BACK>(p, dtype, ws, stream)
                 : pick<F32, false, BACK>(p, dtype, ws, stream);
    case POLICY_BF16:
      return sig ? pick<BF16, true, BACK>(p, dtype, ws, stream)
                 : pick<BF16, false, BACK>(p, dtype, ws, stream);
    default:
      return sig ? pick<F16, true, BACK>(p, dtype, ws, stream)
                 : pick<F16, false, BACK>(p, dtype, ws, stream);
  }
}

}  // namespace

bool recur_keeps(int32_t dtype, int32_t form) {
  return dtype != POLICY_F32 && form == RECUR_SIGMOID;
}

int64_t recur_kept_floats(int32_t L, int32_t N, int32_t D) {
  return ((int64_t)L + kKeep - 1) / kKeep * N * D;
}

int64_t recur_chain_bytes(int32_t L, int32_t N, int32_t D) {
  int64_t most = 0;
  if ((int64_t)N * D == 0) return 0;
  for (int v = 1; v <= 4; v *= 2) {  // whichever the strides allow, in both directions
    if (D < v) continue;
    const int64_t units = N * per_row_of(D, v);
    for (const bool back : {false, true}) {
      const int64_t bytes = chained_bytes(chained_tiles(L, units, back), units, v);
      if (bytes > most) most = bytes;
    }
  }
  return most;
}

hipError_t recur_forward_launch(const recur_args& a, float* kept, hipStream_t stream) {
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
  p.kept = kept;
  p.last = a.h_last;
  return pick_type<false>(p, a.dtype, a.form == RECUR_SIGMOID, a.workspace, stream);
}

hipError_t recur_backward_launch(const recur_grad_args& a, const float* kept, hipStream_t stream) {
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
  p.kept = const_cast<float*>(kept);
  p.dh = a.dh;
  p.start = a.dh_last;
  p.h0 = a.h0;
  p.dones = a.dones;
  p.dx = a.dx;
  p.dg = a.dgate;
  p.last = a.dh0;
  return pick_type<true>(p, a.dtype, a.form == RECUR_SIGMOID, a.workspace, stream);
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
