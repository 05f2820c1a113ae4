// Selective state space scan: forward and single step (include/block.h).
//
// Per state of a step the scan takes an exponent's product, an exp2 (a
// quarter-rate instruction), the input's product and two multiply-adds: eight
// issue slots, beside some sixty per channel and step for softplus, gate and
// conversions.  At 16 states that, not memory, bounds it: 500 x 2048 x 128 bf16
// with a gate takes 610 us (590 where no states are kept for the gradient, so
// their gigabyte costs little), 3.5 TB/s.  Four waves a SIMD in place of three,
// or exp2s in runs apart from the rest, gained nothing.
#include "scan.hpp"

namespace rl {

namespace {

struct ScanRun {
  scan_args a;
  ScanPlan p;
  ScanSummary sum;
};

// A chunk of the scan.  SUMMARY: from a state of zero, without outputs.
template <class T, int NB, bool GATED, bool SUMMARY>
__global__ void __launch_bounds__(64 * NB) scan_forward_kernel(const ScanRun q) {
  const scan_args& a = q.a;
  const ScanWave k(q.p, a.rows, a.groups, a.states);
  __shared__ float s_bc[NB][kUnit][32];
  __shared__ float s_part[NB > 1 && !SUMMARY ? 2 : 1][NB > 1 && !SUMMARY ? NB : 1][kUnit][64];
  const int32_t L = a.steps, S = a.states;
  const int32_t u0 = k.chunk * q.p.chunk_units, u1 = min(u0 + q.p.chunk_units, q.p.units);

  float rate[4][4], h[4][4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int32_t c = k.quad_channel(q.p, r);
    load_states(a.rate + (int64_t)c * S, k.s0, S, rate[r]);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      rate[r][s] *= kLog2e;
      h[r][s] = 0.0f;
    }
    if (!SUMMARY && a.state) load_states(a.state + ((int64_t)k.n * a.width + c) * S, k.s0, S, h[r]);
  }
  if constexpr (!SUMMARY) {
    join_chunks(q.p, q.sum, k, a.rows, a.width, S, 0, 1, k.chunk, rate, h);
    clear_missing(q.p, k, h);
  }
  clear_missing(q.p, k, rate);
  const float bias = a.delta_bias && k.mine ? a.delta_bias[k.channel] : 0.0f;
  const float skip = a.skip ? a.skip[k.channel] : 0.0f;
  float total = 0.0f;
  uint32_t any_cut = 0;

  const Column<T> cx(a, q.p, k, a.x, a.x_step, a.x_row), cd(a, q.p, k, a.delta, a.delta_step, a.delta_row),
      cz(a, q.p, k, a.gate, a.gate_step, a.gate_row), cy(a, q.p, k, a.y, a.y_step, a.y_row);
  const Kept kept(a, q.p, k);
  UnitInputs<T> in;
  UnitDones dones;
  typename T::raw rx[kUnit], rd[kUnit], rz[kUnit];
  const auto fetch = [&](int32_t u) {
    in.load(a, k, u * kUnit);
    cx.load(u * kUnit, rx);
    cd.load(u * kUnit, rd);
    if (GATED) cz.load(u * kUnit, rz);
    dones.load(a, k, u * kUnit);
  };
  fetch(u0);
  if constexpr (!SUMMARY) no_stores(a.y, kUnit / NB);
  for (int32_t u = u0; u < u1; ++u) {
    const int32_t t0 = u * kUnit;
    wave_sync();  // (the reads of the unit before)
    in.put(s_bc[k.w], k, S);
    wave_sync();
    float x[kUnit], dt[kUnit], du[kUnit], z[kUnit], y[kUnit];
#pragma unroll
    for (int i = 0; i < kUnit; ++i) {
      x[i] = T::widen(rx[i]);
      const float v = T::widen(rd[i]) + bias;
      float E;
      const float sp = softplus_of(v, E);
      dt[i] = a.softplus ? sp : v;
      du[i] = dt[i] * x[i];
      if (t0 + i >= L) dt[i] = du[i] = 0.0f;  // past the end: the state stays
      if (SUMMARY) total += dt[i];
      if (GATED) z[i] = T::widen(rz[i]);
    }
    const uint32_t cut = dones.cuts(a, k, t0);
    any_cut |= cut;
    if constexpr (!SUMMARY) {
      if (a.kept) kept.store(u, h);
    }
    fetch(min(u + 1, u1 - 1));
#pragma unroll
    for (int i = 0; i < kUnit; ++i) {
      if ((cut >> i) & 1u) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int s = 0; s < 4; ++s) h[r][s] = 0.0f;
      }
      const float4 b4 = *reinterpret_cast<const float4*>(&s_bc[k.w][i][4 * k.j]);
      const float b[4] = {b4.x, b4.y, b4.z, b4.w};
      float dts[4], dus[4];
      quad_give(dt[i], dts);
      quad_give(du[i], dus);
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int s = 0; s < 4; ++s)
          h[r][s] = __builtin_fmaf(__builtin_amdgcn_exp2f(dts[r] * rate[r][s]), h[r][s], dus[r] * b[s]);
      if constexpr (!SUMMARY) {
        const float4 c4 = *reinterpret_cast<const float4*>(&s_bc[k.w][i][16 + 4 * k.j]);
        const float c[4] = {c4.x, c4.y, c4.z, c4.w};
        float part[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          part[r] = c[0] * h[r][0];
#pragma unroll
          for (int s = 1; s < 4; ++s) part[r] = __builtin_fmaf(c[s], h[r][s], part[r]);
        }
        y[i] = quad_sum(part);
      }
    }
    if constexpr (!SUMMARY) {
      if constexpr (NB > 1) {
        float(&buf)[NB][kUnit][64] = s_part[u & 1];
#pragma unroll
        for (int i = 0; i < kUnit; ++i) buf[k.w][i][k.lane] = y[i];
        __syncthreads();  // (a wave that is a unit ahead writes the other half)
#pragma unroll
        for (int i = 0; i < kUnit; ++i) {
          if (i % NB != k.w) continue;
          y[i] = buf[0][i][k.lane];
#pragma unroll
          for (int v = 1; v < NB; ++v) y[i] += buf[v][i][k.lane];
        }
      }
      char* out = cy.unit(t0);
#pragma unroll
      for (int i = 0; i < kUnit; ++i) {
        if (NB > 1 && i % NB != k.w) continue;
        float v = __builtin_fmaf(skip, x[i], y[i]);
        if (GATED) v *= z[i] * sigmoid_of(z[i]);
        cy.store(out, i, t0 + i, v);
      }
    }
  }

  const int64_t row = (int64_t)k.n * a.width;
  if constexpr (SUMMARY) {
    const int64_t at = (int64_t)k.chunk * a.rows * a.width + row;
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (k.quad_has(q.p, r)) store_states(q.sum.state + (at + k.quad_channel(q.p, r)) * S, k.s0, S, h[r]);
    if (k.mine && k.w == 0) q.sum.total[at + k.channel] = total;
    if (k.block == 0 && k.g == 0 && threadIdx.x == 0)
      q.sum.cut[(int64_t)k.chunk * a.rows + k.n] = any_cut != 0;
  } else if (a.new_state && u1 == q.p.units) {
    const bool ended = a.dones && a.dones[(int64_t)(L - 1) * a.rows + k.n] != 0;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if (ended) {
#pragma unroll
        for (int s = 0; s < 4; ++s) h[r][s] = 0.0f;
      }
      if (k.quad_has(q.p, r))
        store_states(a.new_state + (row + k.quad_channel(q.p, r)) * S, k.s0, S, h[r]);
    }
  }
}

// One step: a lane takes four states of a channel, 2^`shift` lanes a channel.
// State in, state out, nothing else of size: what it costs is a launch and the
// way of one load after another, which is why there is one division and no
// branch before the loads are out.
template <class T>
__global__ void __launch_bounds__(256) scan_step_kernel(const scan_args a, int32_t shift) {
  using raw = typename T::raw;
  const uint32_t id = blockIdx.x * 256 + threadIdx.x;  // (below 2^31)
  const uint32_t column = id >> shift;
  if (column >= (uint32_t)(a.rows * a.width)) return;  // (all of a column's lanes together)
  const int32_t s0 = 4 * (int32_t)(id & ((1u << shift) - 1)), S = a.states;
  const int32_t n = (int32_t)(column / (uint32_t)a.width), d = (int32_t)column - n * a.width;
  const int32_t g = a.groups == 1 ? 0 : d / (a.width / a.groups);
  const raw* b = static_cast<const raw*>(a.b) + n * a.b_row + g * a.b_group;
  const raw* c = static_cast<const raw*>(a.c) + n * a.c_row + g * a.c_group;
  const float* state = a.state + (int64_t)column * S;
  const float* rates = a.rate + (int64_t)d * S;
  float h[4], rate[4];
  Pack<T, 4> bs, cs;
  if (S % 4 == 0) {
    // (lanes past the last state load it again and use nothing)
    const int32_t at = min(s0, S - 4);
    widen_pack<F32, 4>(load_pack<F32, 4>(reinterpret_cast<const uint32_t*>(state + at)), h);
    widen_pack<F32, 4>(load_pack<F32, 4>(reinterpret_cast<const uint32_t*>(rates + at)), rate);
    bs = load_pack<T, 4>(b + at);
    cs = load_pack<T, 4>(c + at);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int32_t at = min(s0 + i, S - 1);
      h[i] = state[at];
      rate[i] = rates[at];
      bs.v[i] = b[at];
      cs.v[i] = c[at];
    }
  }
  const raw xr = (static_cast<const raw*>(a.x) + n * a.x_row)[d];
  const raw dr = (static_cast<const raw*>(a.delta) + n * a.delta_row)[d];
  const raw zr = a.gate ? (static_cast<const raw*>(a.gate) + n * a.gate_row)[d] : raw(0);
  const float bias = a.delta_bias ? a.delta_bias[d] : 0.0f;
  const float skip = a.skip ? a.skip[d] : 0.0f;
  const bool cut = a.dones && a.dones[n] != 0;
  const float x = T::widen(xr), v = T::widen(dr) + bias;
  float E;
  const float sp = softplus_of(v, E);
  const float dt = a.softplus ? sp : v;
  float y = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float decay = __builtin_amdgcn_exp2f(dt * (rate[i] * kLog2e));
    h[i] = __builtin_fmaf(decay, cut ? 0.0f : h[i], (dt * x) * T::widen(bs.v[i]));
    y = s0 + i < S ? __builtin_fmaf(T::widen(cs.v[i]), h[i], y) : y;
  }
  if (s0 < S) store_states(a.new_state + (int64_t)column * S, s0, S, h);
  for (int32_t i = 1; i < 1 << shift; i <<= 1) y += __shfl_xor(y, i);
  if (s0 != 0) return;
  y = __builtin_fmaf(skip, x, y);
  if (a.gate) {
    const float z = T::widen(zr);
    y *= z * sigmoid_of(z);
  }
  (static_cast<raw*>(a.y) + n * a.y_row)[d] = T::narrow(y);
}

// A thread takes a state, and its summaries sixteen at a time.
__global__ void __launch_bounds__(256) scan_join_kernel(const ScanSummary sum, int32_t chunks, int64_t states,
                                                        int32_t D, int32_t S, const float* rates,
                                                        const float* state, int32_t direction) {
  constexpr int kAt = 16;
  const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (e >= states) return;
  const int64_t column = e / S, columns = states / S;  // column: n * D + d
  const int32_t n = (int32_t)(column / D), N = (int32_t)(columns / D);
  const float rate = rates[e % ((int64_t)D * S)] * kLog2e;
  const int32_t first = direction > 0 ? 0 : chunks - 1, count = chunks - 1;
  float h = state ? state[e] : 0.0f;
  for (int32_t i0 = 0; i0 < count; i0 += kAt) {
    float own[kAt], total[kAt];
    int32_t cut[kAt];
#pragma unroll
    for (int m = 0; m < kAt; ++m) {
      const int64_t chunk = first + direction * min(i0 + m, count - 1);
      own[m] = sum.state[chunk * states + e];
      total[m] = sum.total[chunk * columns + column];
      cut[m] = sum.cut[chunk * N + n];
    }
#pragma unroll
    for (int m = 0; m < kAt; ++m) {
      if (i0 + m >= count) continue;
      // (a state of 0 stays 0 under any decay)
      const float left = h == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(total[m] * rate) * h;
      h = cut[m] != 0 ? own[m] : left + own[m];
      sum.state[(int64_t)(first + direction * (i0 + m)) * states + e] = h;
    }
  }
}

template <class T, int NB>
void launch_forward(const ScanRun& q, hipStream_t stream) {
  const dim3 threads(64 * NB), groups((uint32_t)(q.p.columns * q.p.chunks));
  // (the last chunk's summary is read by none)
  if (q.p.chunks > 1)
    scan_forward_kernel<T, NB, false, true>
        <<<dim3((uint32_t)(q.p.columns * (q.p.chunks - 1))), threads, 0, stream>>>(q);
  if (q.p.joined)
    scan_join_launch(q.p, q.sum, q.a.rows, q.a.width, q.a.states, q.a.rate, q.a.state, 1, stream);
  if (q.a.gate)
    scan_forward_kernel<T, NB, true, false><<<groups, threads, 0, stream>>>(q);
  else
    scan_forward_kernel<T, NB, false, false><<<groups, threads, 0, stream>>>(q);
}

template <class T>
void launch_states(const ScanRun& q, hipStream_t stream) {
  if (q.p.state_blocks == 1) return launch_forward<T, 1>(q, stream);
  if (q.p.state_blocks == 2) return launch_forward<T, 2>(q, stream);
  return launch_forward<T, 4>(q, stream);
}

}  // namespace

// A chunk has four units at least, and chunks are made until two waves a SIMD
// have work (1024 SIMDs; 16,385 x 2 x 1000 fp16 took 332 us so, 340 and 378 with
// three and four), from columns of up to a quarter of that: 500 steps of 512
// waves, fp32 with a gate, take 143 us forward and 291 backward cut in four, 182
// and 525 whole.  Above, two chunks lose forward (768 waves: 222 us, 181 whole;
// 520: 178 and 183) what they would gain backward (477 and 521; 361 and 524).
// More than 16 summaries are joined once for all chunks (16,385 x 2 x 1000 in 64
// takes 301 us so and 319 where every chunk joins those before it; in 32 280 and
// 286; in 16 278 and 277, 8 chunks of 64 steps 84 and 77).
ScanPlan scan_plan(int32_t L, int32_t N, int32_t D, int32_t S, int32_t G) {
  ScanPlan p;
  p.group_width = D / G;
  p.blocks = cdiv(p.group_width, 64);
  p.units = cdiv(L, kUnit);
  p.state_blocks = S <= kBlock ? 1 : S <= 2 * kBlock ? 2 : 4;
  p.columns = (int64_t)N * G * p.blocks;
  const int64_t waves = p.columns * p.state_blocks;
  p.chunks = 1;
  p.chunk_units = p.units;
  if (waves <= 512) {
    const int64_t wanted = min((int64_t)64, 2048 / waves);
    p.chunk_units = max(4, cdiv(p.units, (int)wanted));
    p.chunks = cdiv(p.units, p.chunk_units);
  }
  if (p.chunks == 1) p.chunk_units = p.units;
  p.joined = p.chunks > 16;
  return p;
}

namespace {
int64_t up(int64_t bytes) { return (bytes + 255) / 256 * 256; }
}  // namespace

int64_t scan_summary_bytes(const ScanPlan& p, int32_t N, int32_t D, int32_t S) {
  if (p.chunks == 1) return 0;
  const int64_t nd = (int64_t)p.chunks * N * D;
  return up(nd * S * 4) + up(nd * 4) + up((int64_t)p.chunks * N * 4);
}
ScanSummary scan_summary(const ScanPlan& p, int32_t N, int32_t D, int32_t S, void* workspace) {
  const int64_t nd = (int64_t)p.chunks * N * D;
  char* w = static_cast<char*>(workspace);
  return ScanSummary{reinterpret_cast<float*>(w), reinterpret_cast<float*>(w + up(nd * S * 4)),
                     reinterpret_cast<int32_t*>(w + up(nd * S * 4) + up(nd * 4))};
}

int64_t scan_kept_floats(int32_t L, int32_t N, int32_t D, int32_t S, int32_t G) {
  const int64_t quads = (D / G + 3) / 4;
  return (int64_t)cdiv(L, kUnit) * N * G * quads * 4 * ((S + 3) / 4 * 4);
}

int64_t scan_workspace_bytes(int32_t L, int32_t N, int32_t D, int32_t S, int32_t G) {
  if (L == 0 || N == 0 || D == 0) return 0;
  return scan_summary_bytes(scan_plan(L, N, D, S, G), N, D, S);
}

void scan_join_launch(const ScanPlan& p, const ScanSummary& sum, int32_t N, int32_t D, int32_t S,
                      const float* rate, const float* state, int32_t direction, hipStream_t stream) {
  const int64_t states = (int64_t)N * D * S;
  scan_join_kernel<<<dim3((uint32_t)((states + 255) / 256)), 256, 0, stream>>>(sum, p.chunks, states, D, S, rate,
                                                                              state, direction);
}

hipError_t scan_forward_launch(const scan_args& a, hipStream_t stream) {
  const int64_t state_bytes = (int64_t)a.rows * a.width * a.states * 4;
  if (a.steps == 0)
    return a.new_state ? copy_or_clear_launch(a.state, a.new_state, state_bytes, stream) : hipSuccess;
  ScanRun q;
  q.a = a;
  q.p = scan_plan(a.steps, a.rows, a.width, a.states, a.groups);
  q.sum = scan_summary(q.p, a.rows, a.width, a.states, a.workspace);
  if (a.dtype == POLICY_F32)
    launch_states<F32>(q, stream);
  else if (a.dtype == POLICY_BF16)
    launch_states<BF16>(q, stream);
  else
    launch_states<F16>(q, stream);
  return hipGetLastError();
}

hipError_t scan_step_launch(const scan_args& a, hipStream_t stream) {
  int32_t shift = 0;
  while ((4 << shift) < a.states) ++shift;
  const int64_t threads = (int64_t)a.rows * a.width << shift;
  const dim3 grid((uint32_t)((threads + 255) / 256));
  if (a.dtype == POLICY_F32)
    scan_step_kernel<F32><<<grid, 256, 0, stream>>>(a, shift);
  else if (a.dtype == POLICY_BF16)
    scan_step_kernel<BF16><<<grid, 256, 0, stream>>>(a, shift);
  else
    scan_step_kernel<F16><<<grid, 256, 0, stream>>>(a, shift);
  return hipGetLastError();
}

}  // namespace rl
