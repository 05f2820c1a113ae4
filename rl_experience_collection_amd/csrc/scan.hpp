// The selective scan's wave (scan.hip, scan_grad.hip).
//
// A wave takes 64 channels of one episode and group, and 16 of the S states
// of each.  Lane l reads, converts and writes channel l of its steps; the
// states are spread the other way: lane 4 i + j holds states 4 j .. 4 j + 3
// of the channels 4 i .. 4 i + 3 of its quad.  What a step needs of a channel
// comes by quad broadcasts, what the states sum up to goes back by a
// transposed sum over the quad, the b and c of a step are four values a lane
// (one LDS read each, the same for all quads), and sums over channels (the
// gradients of b and c) run over a lane's own four channels for free before
// lanes have to meet.  With more than 16 states a workgroup's waves take 16
// each of the same channels.
//
// Steps go in units of eight.  Long scans of few columns are cut into chunks
// of units: one launch finds what each chunk makes of a state of zero and how
// far it decays what enters it (the sum of D_t is enough for that), the next
// runs the chunks from the states that these give.
#pragma once

#include "block.hpp"
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
};

// Per chunk, for chunks > 1.
struct ScanSummary {
  float* state;  // [chunks][N][D][S]: what the chunk makes of a state of zero
  float* total;  // [chunks][N][D]: the sum of D_t
  int32_t* cut;  // [chunks][N]: a done lies inside
};

ScanPlan scan_plan(int32_t L, int32_t N, int32_t D, int32_t S, int32_t G, bool grad);
int64_t scan_summary_bytes(const ScanPlan& p, int32_t N, int32_t D, int32_t S);
ScanSummary scan_summary(const ScanPlan& p, int32_t N, int32_t D, int32_t S, void* workspace);

// The value lane 4 i + R of this lane's quad holds.
template <int R>
__device__ __forceinline__ float quad_get(float x) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), R * 0x55, 0xF, 0xF, true));
}
template <int CTRL>
__device__ __forceinline__ float from_lane(float x) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xF, 0xF, true));
}
// Lane j of a quad gets the quad's sum of v[j].
__device__ __forceinline__ float quad_turn(const float (&v)[4], int lane) {
  const bool odd = lane & 1, high = lane & 2;
  const float a = (odd ? v[1] : v[0]) + from_lane<0xB1>(odd ? v[0] : v[1]);
  const float b = (odd ? v[3] : v[2]) + from_lane<0xB1>(odd ? v[2] : v[3]);
  return (high ? b : a) + from_lane<0x4E>(high ? a : b);
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
  // Channel r of the lane's quad, clamped into the group.
  __device__ __forceinline__ int32_t quad_channel(const ScanPlan& p, int r) const {
    return g * p.group_width + min(first + r, p.group_width - 1);
  }
  __device__ __forceinline__ bool quad_has(const ScanPlan& p, int r) const {
    return first + r < p.group_width;
  }
};

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
// l / 8, of b where l % 8 < 4, else of c.
template <class T>
struct UnitInputs {
  float v[4];
  __device__ __forceinline__ void load(const scan_args& a, const ScanWave& k, int32_t t0) {
    const int32_t t = min(t0 + (k.lane >> 3), a.steps - 1);
    const bool is_c = k.lane & 4;
    const int32_t s0 = k.w * kBlock + 4 * (k.lane & 3);
    const typename T::raw* row = static_cast<const typename T::raw*>(is_c ? a.c : a.b) +
                                 t * (is_c ? a.c_step : a.b_step) + k.n * (is_c ? a.c_row : a.b_row) +
                                 k.g * (is_c ? a.c_group : a.b_group);
    if (s0 + 4 <= a.states) {
      widen_pack<T, 4>(load_pack<T, 4>(row + s0), v);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = s0 + i < a.states ? T::widen(row[s0 + i]) : 0.0f;
    }
  }
  __device__ __forceinline__ void put(float (&lds)[kUnit][32], int lane) const {
    *reinterpret_cast<float4*>(&lds[lane >> 3][4 * (lane & 7)]) = make_float4(v[0], v[1], v[2], v[3]);
  }
};

// Bit k: a done cuts the state that enters step t0 + k.
__device__ __forceinline__ uint32_t unit_cuts(const scan_args& a, const ScanWave& k, int32_t t0) {
  if (!a.dones) return 0;
  const int32_t t = t0 + k.lane - 1;
  const bool cut = k.lane < kUnit && t >= 0 && t < a.steps - 1 && a.dones[(int64_t)t * a.rows + k.n] != 0;
  return (uint32_t)__ballot(cut);
}

}  // namespace rl
