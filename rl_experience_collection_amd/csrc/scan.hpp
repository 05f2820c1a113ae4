// The selective scan's wave (scan.hip, scan_grad.hip).
//
// A wave takes 64 channels of one episode and group, and 16 of the S states
// of each.  Lane l reads, converts and writes channel l of its steps; the
// states are spread the other way: lane 4 i + j holds states 4 j .. 4 j + 3
// of the four channels of its quad, channel 4 i + (r ^ j) in its place r.  By
// that order a channel's value comes to place r, and a sum over its states
// goes back from there, by the one exchange of lanes j ^ r (nothing has to be
// selected; places in one order for all lanes took 9 operations a sum, this
// 3).  The b and c of a step are four values a lane (one LDS read each, the
// same for all quads), and sums over channels (the gradients of b and c) run
// over a lane's own four channels for free before lanes have to meet.  With
// more than 16 states a workgroup's waves take 16 each of the same channels.
// States and channels that do not exist cost what others do: 1 state as much as
// 16, 17 as 32, 33 as 64, a group of 16 channels as one of 64.
//
// Steps go in units of eight.  Long scans of few columns are cut into chunks
// of units: one launch finds what each chunk makes of a state of zero and how
// far it decays what enters it (the sum of D_t is enough for that), the next
// runs the chunks from the states that these give.
#pragma once

#include "block.hpp"
#include "buffer.hpp"
#include "device.hpp"
#include "elem.hpp"

namespace rl {

constexpr int kUnit = 8;
constexpr int kBlock = 16;  // states of a wave
constexpr float kLog2e = 1.44269504f, kLn2 = 0.693147181f;

// Chunks of a scan and what they are made of.
struct ScanPlan {
  int32_t group_width;  // channels of a group
  int32_t blocks;       // waves across a group's channels
  int32_t units;        // ceil(L / 8)
  int32_t chunks, chunk_units;
  int32_t state_blocks;  // ceil(S / 16)
  int64_t columns;       // N * G * blocks: workgroups of a chunk
  bool joined;           // scan_join_launch() has joined the summaries
};

// Per chunk, for chunks > 1.
struct ScanSummary {
  float* state;  // [chunks][N][D][S]: what the chunk makes of a state of zero, or of what enters it
  float* total;  // [chunks][N][D]: the sum of D_t
  int32_t* cut;  // [chunks][N]: a done lies inside
};

ScanPlan scan_plan(int32_t L, int32_t N, int32_t D, int32_t S, int32_t G);
int64_t scan_summary_bytes(const ScanPlan& p, int32_t N, int32_t D, int32_t S);
ScanSummary scan_summary(const ScanPlan& p, int32_t N, int32_t D, int32_t S, void* workspace);
// Joins the summaries of all chunks but the last in the direction of the scan
// (1, from `state`, which may be NULL) or of its gradient (-1, from zero).
void scan_join_launch(const ScanPlan& p, const ScanSummary& sum, int32_t N, int32_t D, int32_t S,
                      const float* rate, const float* state, int32_t direction, hipStream_t stream);

// The value of lane j ^ R of this lane's quad.
template <int R>
__device__ __forceinline__ float quad_xor(float x) {
  constexpr int kPerm = (R ^ 0) | (R ^ 1) << 2 | (R ^ 2) << 4 | (R ^ 3) << 6;
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), kPerm, 0xF, 0xF, true));
}
// A channel's value in the places of its quad's lanes.
__device__ __forceinline__ void quad_give(float x, float (&v)[4]) {
  v[0] = x;
  v[1] = quad_xor<1>(x);
  v[2] = quad_xor<2>(x);
  v[3] = quad_xor<3>(x);
}
// The quad's sum for the lane's own channel.  (The empty statement keeps the
// additions here, where they take the exchanges as operands; moved to where
// the sum is used they would leave those, which cannot move, on their own.)
__device__ __forceinline__ float quad_sum(const float (&v)[4]) {
  float sum = ((v[0] + quad_xor<1>(v[1])) + quad_xor<2>(v[2])) + quad_xor<3>(v[3]);
  asm("" : "+v"(sum));
  return sum;
}

// softplus(v) and sigmoid(v) from E = exp(-|v|): log(1 + E) = 2 artanh(E / (2 + E)),
// whose argument is at most 1/3: seven terms leave 1.4e-8 of it.
__device__ __forceinline__ float softplus_of(float v, float& E) {
  E = __builtin_amdgcn_exp2f(-__builtin_fabsf(v) * kLog2e);
  const float z = E * __builtin_amdgcn_rcpf(2.0f + E);
  const float q = z * z;
  float s = __builtin_fmaf(q, 1.0f / 13, 1.0f / 11);
  s = __builtin_fmaf(q, s, 1.0f / 9);
  s = __builtin_fmaf(q, s, 1.0f / 7);
  s = __builtin_fmaf(q, s, 1.0f / 5);
  s = __builtin_fmaf(q, s, 1.0f / 3);
  s = __builtin_fmaf(q, s, 1.0f);
  return __builtin_fmaf(z + z, s, __builtin_fmaxf(v, 0.0f));
}
__device__ __forceinline__ float sigmoid_from(float v, float E) {
  const float r = __builtin_amdgcn_rcpf(1.0f + E);
  return v >= 0.0f ? r : E * r;
}
__device__ __forceinline__ float sigmoid_of(float v) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-v * kLog2e));
}

// LDS written by some lanes of a wave, read by others.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Where a wave stands.
struct ScanWave {
  int32_t lane, w;      // w: its 16 states
  int32_t chunk, n, g, block;
  int32_t j;            // the lane's states are s0 = 16 w + 4 j ...
  int32_t s0;
  int32_t channel;      // lane's own, within D (clamped into the group)
  int32_t first;        // of the lane's quad, unclamped, within the group
  bool mine;            // the lane's own channel exists
  __device__ __forceinline__ ScanWave(const ScanPlan& p, int32_t N, int32_t G, int32_t states) {
    lane = threadIdx.x & 63;
    w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    uint32_t id = blockIdx.x;
    block = id % p.blocks;
    id /= p.blocks;
    g = id % G;
    id /= G;
    n = id % N;
    chunk = id / N;
    j = lane & 3;
    s0 = w * kBlock + 4 * j;
    const int32_t local = block * 64 + lane;
    mine = local < p.group_width;
    channel = g * p.group_width + min(local, p.group_width - 1);
    first = block * 64 + (lane & ~3);
  }
  // The channel of place r, clamped into the group.
  __device__ __forceinline__ int32_t quad_channel(const ScanPlan& p, int r) const {
    return g * p.group_width + min(first + (r ^ j), p.group_width - 1);
  }
  __device__ __forceinline__ bool quad_has(const ScanPlan& p, int r) const {
    return first + (r ^ j) < p.group_width;
  }
};

// Rates and states of channels that the group does not have, which loads
// take from its last one, become 0: with an input of 0 (what a row's loads
// give past its end) and no bias their states stay 0 under a decay of 1, whatever
// the last channel's are, and add nothing to the sums over channels.
__device__ __forceinline__ void clear_missing(const ScanPlan& p, const ScanWave& k, float (&v)[4][4]) {
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const bool has = k.quad_has(p, r);
#pragma unroll
    for (int s = 0; s < 4; ++s) v[r][s] = has ? v[r][s] : 0.0f;
  }
}

// The four states from s0 of a row of S; those that do not exist are 0.
__device__ __forceinline__ void load_states(const float* row, int32_t s0, int32_t S, float (&h)[4]) {
  if (s0 + 4 <= S) {
    const Pack<F32, 4> x = load_pack<F32, 4>(reinterpret_cast<const uint32_t*>(row + s0));
    widen_pack<F32, 4>(x, h);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = s0 + i < S ? row[s0 + i] : 0.0f;
  }
}
__device__ __forceinline__ void store_states(float* row, int32_t s0, int32_t S, const float (&h)[4]) {
  if (s0 + 4 <= S) {
    store_pack<F32, 4>(reinterpret_cast<uint32_t*>(row + s0), narrow_pack<F32, 4>(h));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (s0 + i < S) row[s0 + i] = h[i];
  }
}

// The b and c of a unit on their way to LDS: lane l takes four values of step
// l / 8, of b where l % 8 < 4, else of c.  (As loaded: nothing that follows a
// load here may wait for it.)
template <class T>
struct UnitInputs {
  Pack<T, 4> x;
  __device__ __forceinline__ void load(const scan_args& a, const ScanWave& k, int32_t t0) {
    const int32_t t = min(t0 + (k.lane >> 3), a.steps - 1);
    const bool is_c = k.lane & 4;
    const int32_t s0 = k.s0;
    const typename T::raw* row = static_cast<const typename T::raw*>(is_c ? a.c : a.b) +
                                 t * (is_c ? a.c_step : a.b_step) + k.n * (is_c ? a.c_row : a.b_row) +
                                 k.g * (is_c ? a.c_group : a.b_group);
    if (a.states % 4 == 0) {
      x = load_pack<T, 4>(row + min(s0, a.states - 4));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) x.v[i] = row[min(s0 + i, a.states - 1)];
    }
  }
  __device__ __forceinline__ void put(float (&lds)[kUnit][32], const ScanWave& k, int32_t states) const {
    float v[4];
    widen_pack<T, 4>(x, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = k.s0 + i < states ? v[i] : 0.0f;
    *reinterpret_cast<float4*>(&lds[k.lane >> 3][4 * (k.lane & 7)]) = make_float4(v[0], v[1], v[2], v[3]);
  }
};

// p + n.  (The empty statement keeps the compiler from making one pointer
// of a loop's chain into one for each step, which no scalar registers are left for.)
template <class P>
__device__ __forceinline__ P walk(P p, int64_t n) {
  p += n;
  asm("" : "+s"(p));
  return p;
}

// A lane's own channel in one of the [L][N][D] arrays.
template <class T>
struct Column {
  char* row;  // the wave's channels at step 0
  int64_t step;
  uint32_t bytes, at;
  int32_t steps;
  __device__ __forceinline__ Column(const scan_args& a, const ScanPlan& p, const ScanWave& k, const void* base,
                                    int64_t step_, int64_t row_)
      : row(const_cast<char*>(static_cast<const char*>(base)) +
            (k.n * row_ + k.g * p.group_width + k.block * 64) * T::kBytes),
        step(step_ * T::kBytes),
        bytes((uint32_t)min(64, p.group_width - k.block * 64) * T::kBytes),
        at(k.lane * T::kBytes),
        steps(a.steps) {}
  __device__ __forceinline__ char* unit(int32_t t0) const { return row + t0 * step; }
  __device__ __forceinline__ void load(int32_t t0, typename T::raw (&x)[kUnit]) const {
    const char* p = unit(t0);
#pragma unroll
    for (int i = 0; i < kUnit; ++i, p += step) x[i] = row_load<T>(p, t0 + i < steps ? bytes : 0, at);
  }
  // The same from the unit's last step, at `p`, to its first; p is left at the
  // unit before, whose steps may not exist.
  __device__ __forceinline__ void load_back(const char*& p, int32_t t0, typename T::raw (&x)[kUnit]) const {
#pragma unroll
    for (int i = kUnit - 1; i >= 0; --i) {
      x[i] = row_load<T>(p, (uint32_t)(t0 + i) < (uint32_t)steps ? bytes : 0, at);
      p = walk(p, -step);
    }
  }
  // Step t = t0 + i of the unit at `p`.
  __device__ __forceinline__ void store(char* p, int i, int32_t t, float x) const {
    row_store<T>(p + i * step, t < steps ? bytes : 0, at, x);
  }
};

// The states that enter the units, as they lie in the lanes: [units][N][G][quads]
// [places][4 ceil(S / 4)], so that a quad's lanes write one run of 64 bytes.
// (In the order of the channels a store of a wave would touch four times as
// many lines.)
struct Kept {
  float* base;
  int64_t unit;  // floats of a unit
  uint32_t bytes, at, place;
  __device__ __forceinline__ Kept(const scan_args& a, const ScanPlan& p, const ScanWave& k) {
    const int32_t quads = (p.group_width + 3) / 4, wide = (a.states + 3) / 4 * 4;
    const int64_t row = (int64_t)quads * 4 * wide;
    unit = (int64_t)a.rows * a.groups * row;
    base = a.kept + ((int64_t)k.n * a.groups + k.g) * row + (int64_t)k.block * 64 * wide;
    bytes = (uint32_t)min(16, quads - k.block * 16) * 16 * wide;
    place = wide * 4;
    // (states past the last run: an offset past the end)
    at = k.s0 < wide ? ((k.lane >> 2) * 4 * wide + k.s0) * 4 : 1u << 31;
  }
  // Of the unit at `p`, which may not exist.
  __device__ __forceinline__ void load(const float* p, bool exists, float (&h)[4][4]) const {
    const auto rsrc = row_of(p, exists ? bytes : 0);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const words4 x = __builtin_amdgcn_raw_buffer_load_b128(rsrc, at + r * place, 0, 0);
#pragma unroll
      for (int s = 0; s < 4; ++s) h[r][s] = __uint_as_float(x[s]);
    }
  }
  __device__ __forceinline__ void store(int32_t u, const float (&h)[4][4]) const {
    const auto rsrc = row_of(base + u * unit, bytes);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      words4 x;
#pragma unroll
      for (int s = 0; s < 4; ++s) x[s] = __float_as_uint(h[r][s]);
      __builtin_amdgcn_raw_buffer_store_b128(x, rsrc, at + r * place, 0, 0);
    }
  }
};

// The dones of a unit: lane l has that of step t0 + l - 1, and bit l of cuts()
// says that one cuts the state that enters step t0 + l.
struct UnitDones {
  uint8_t done;
  __device__ __forceinline__ void load(const scan_args& a, const ScanWave& k, int32_t t0) {
    const int32_t first = max(t0 - 1, 0);  // (step -1 has none: an offset past the end)
    const uint8_t* p = a.dones + (int64_t)first * a.rows + k.n;
    const uint32_t rows = (uint32_t)min(a.steps - first, kUnit + 1);
    done = __builtin_amdgcn_raw_buffer_load_b8(row_of(p, a.dones ? rows * a.rows - k.n : 0),
                                               (uint32_t)(k.lane - (t0 == 0)) * a.rows, 0, 0);
  }
  __device__ __forceinline__ uint32_t cuts(const scan_args& a, const ScanWave& k, int32_t t0) const {
    const int32_t t = t0 + k.lane;
    return (uint32_t)__ballot(k.lane < kUnit && t < a.steps && done != 0);
  }
};

// h becomes what `count` chunks make of it one after another, from chunk
// `first` on in the given direction; four summaries are loaded at a time.
// Where they are joined, it is the last one's.
__device__ __forceinline__ void join_chunks(const ScanPlan& p, const ScanSummary& sum, const ScanWave& k,
                                            int32_t N, int32_t D, int32_t S, int32_t first, int32_t direction,
                                            int32_t count, const float (&rate)[4][4], float (&h)[4][4]) {
  if (p.joined) {
    if (count == 0) return;
    const int64_t chunk = first + direction * (count - 1);
#pragma unroll
    for (int r = 0; r < 4; ++r)
      load_states(sum.state + ((chunk * N + k.n) * D + k.quad_channel(p, r)) * S, k.s0, S, h[r]);
    return;
  }
  constexpr int kAt = 4;
  for (int32_t i0 = 0; i0 < count; i0 += kAt) {
    float own[kAt][4][4], total[kAt][4];
    int32_t cut[kAt];
#pragma unroll
    for (int m = 0; m < kAt; ++m) {
      const int64_t chunk = first + direction * min(i0 + m, count - 1);
      cut[m] = sum.cut[chunk * N + k.n];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int64_t c = (chunk * N + k.n) * D + k.quad_channel(p, r);
        load_states(sum.state + c * S, k.s0, S, own[m][r]);
        total[m][r] = sum.total[c];
      }
    }
#pragma unroll
    for (int m = 0; m < kAt; ++m) {
      if (i0 + m >= count) continue;
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          // (a state of 0 stays 0 under any decay)
          const float left =
              h[r][s] == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(total[m][r] * rate[r][s]) * h[r][s];
          h[r][s] = cut[m] != 0 ? own[m][r][s] : left + own[m][r][s];
        }
    }
  }
}

}  // namespace rl
