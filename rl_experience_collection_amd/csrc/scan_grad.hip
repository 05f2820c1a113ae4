// Gradient of the selective state space scan (include/block.h).
//
// With v_t = c_t h_t + skip x_t, w_t = dL/dv_t (dy times the gate's silu) and
// d_t = dL/dh_t,
//   d_t = c_t w_t + a_{t+1} m_{t+1} d_{t+1},   a_t = exp(D_t rate),
//   db = sum over channels of d D x,  dc = sum over channels of w h,
//   q_t = a_t m_t h_{t-1} d_t,  drate = sum D q,
//   dD = x sum over s of b d + sum over s of rate q,  dx = D sum of b d + skip w.
// A wave runs its units from the last to the first.  Of a unit it takes the
// state that enters it from what the forward call kept, forms its eight states
// again, the first four to LDS and the others in registers, and goes back over
// them.  (Four in registers alone, formed twice, took half as many more states
// to form; eight in registers leave a SIMD one wave.)  Decays are formed twice:
// an exp2 costs less than the place to hold it.  Some 360 instructions a step at
// 16 states bound it: 500 x 2048 x 128 bf16 with a gate takes 1540 us, 2 TB/s.
// From 17 states on registers (with a gate) or, from 33, LDS leave a SIMD one wave.
#include "scan.hpp"

namespace rl {

namespace {

constexpr int kHeld = 4;  // steps whose states are held in registers, and as many in LDS

template <int CTRL>
__device__ __forceinline__ float from_lane(float x) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xF, 0xF, true));
}

struct GradRun {
  scan_grad_args g;
  int32_t pairs;  // of steps
  ScanPlan p;
  ScanSummary sum;
  float* shared;  // [blocks][pairs of steps][N][G][state blocks][2][32]: db and dc of the blocks, or NULL
  float* params;  // [chunks][N][D S + 2 D]: drate, dskip, ddelta_bias
};

__device__ __forceinline__ void read4(const float* p, float (&v)[4]) {
  const float4 x = *reinterpret_cast<const float4*>(p);
  v[0] = x.x;
  v[1] = x.y;
  v[2] = x.z;
  v[3] = x.w;
}

// Sums over the wave's quads of the four values of b's and c's gradients that
// every lane holds.  Halving the values at each meeting, lane l ends with one:
// of b where its bit 5 is 0, else of c, state 2 (bit 4) + (bit 3) of the four
// of lane l & 3, and a sum over bit 2 still to come.
__device__ __forceinline__ float meet(const float (&b)[4], const float (&c)[4], int lane) {
  float w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(b[i]), __float_as_uint(c[i]), false, false);
    w[i] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  float v[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(w[i]), __float_as_uint(w[i + 2]), false, false);
    v[i] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  const bool up = lane & 8;
  return (up ? v[1] : v[0]) + from_lane<0x128>(up ? v[0] : v[1]);  // row_ror:8
}
// The sum over bit 2 of two steps at once: of the first where bit 2 is 0.
__device__ __forceinline__ float meet_pair(float first, float second, int lane) {
  const bool up = lane & 4;
  const float other = up ? first : second;
  int x = __builtin_amdgcn_update_dpp(0, __float_as_int(other), 0x104, 0xF, 0x5, true);  // row_shl:4
  x = __builtin_amdgcn_update_dpp(x, __float_as_int(other), 0x114, 0xF, 0xA, false);     // row_shr:4
  return (up ? second : first) + __int_as_float(x);
}

template <class T, int NB, bool GATED, bool SUMMARY>
__global__ void __launch_bounds__(64 * NB, NB == 1 ? 2 : 1) scan_backward_kernel(const GradRun q) {
  const scan_grad_args& g = q.g;
  const scan_args& a = g.f;
  ScanWave k(q.p, a.rows, a.groups, a.states);
  if (SUMMARY) ++k.chunk;  // (the first chunk's is read by none)
  __shared__ float s_bc[NB][kUnit][32];
  __shared__ float4 s_held[SUMMARY ? 1 : NB][kHeld][4][64];  // the states of a unit's first steps
  __shared__ float s_slope[SUMMARY ? 1 : NB][kUnit][64];     // D's slopes
  // the waves' shares of y, p1 and p2
  __shared__ float s_sums[!SUMMARY && NB > 1 ? NB : 1][3][kUnit][64];
  const int32_t L = a.steps, S = a.states;
  const int32_t u0 = k.chunk * q.p.chunk_units, u1 = min(u0 + q.p.chunk_units, q.p.units);

  float rate[4][4], G[4][4], drate[4][4];
  const bool ended = a.dones && a.dones[(int64_t)(L - 1) * a.rows + k.n] != 0;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int32_t c = k.quad_channel(q.p, r);
    load_states(a.rate + (int64_t)c * S, k.s0, S, rate[r]);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      rate[r][s] *= kLog2e;
      G[r][s] = drate[r][s] = 0.0f;
    }
    // (the last chunk's summary starts from the gradient of new_state itself)
    if ((!SUMMARY || k.chunk == q.p.chunks - 1) && g.dnew_state && !ended)
      load_states(g.dnew_state + ((int64_t)k.n * a.width + c) * S, k.s0, S, G[r]);
  }
  if constexpr (!SUMMARY) {
    if (k.chunk < q.p.chunks - 1) {
      // (the last chunk's summary holds what dnew_state sends)
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int s = 0; s < 4; ++s) G[r][s] = 0.0f;
      join_chunks(q.p, q.sum, k, a.rows, a.width, S, q.p.chunks - 1, -1, q.p.chunks - 1 - k.chunk, rate, G);
    }
  }
  clear_missing(q.p, k, rate);
  clear_missing(q.p, k, G);
  const float bias = a.delta_bias && k.mine ? a.delta_bias[k.channel] : 0.0f;
  const float skip = a.skip ? a.skip[k.channel] : 0.0f;
  float total = 0.0f, dskip = 0.0f, dbias = 0.0f;
  uint32_t any_cut = 0;

  const Column<T> cx(a, q.p, k, a.x, a.x_step, a.x_row), cd(a, q.p, k, a.delta, a.delta_step, a.delta_row),
      cz(a, q.p, k, a.gate, a.gate_step, a.gate_row), cy(a, q.p, k, g.dy, g.dy_step, g.dy_row);
  const Column<T> gx(a, q.p, k, g.dx, g.dx_step, g.dx_row), gd(a, q.p, k, g.ddelta, g.ddelta_step, g.ddelta_row),
      gz(a, q.p, k, g.dgate, g.dgate_step, g.dgate_row);
  const Kept states(a, q.p, k);
  // Which of the sums over channels a lane ends with: of the even step of a
  // pair or the odd one, of b or c, of a state; and where it goes.
  const bool met_odd = k.lane & 4, met_c = k.lane & 32;
  const int met_place = 4 * k.j + 2 * ((k.lane >> 4) & 1) + ((k.lane >> 3) & 1);
  const int met_state = k.w * kBlock + met_place;
  const uint32_t met_at = (met_odd * 32 + met_c * 16 + met_place) * 4;
  using raw = typename T::raw;
  const int64_t own_step = met_c ? g.dc_step : g.db_step;
  raw* own = static_cast<raw*>(met_c ? g.dc : g.db) + k.n * (met_c ? g.dc_row : g.db_row) +
             k.g * (met_c ? g.dc_group : g.db_group) + met_state + (int64_t)(u1 * kUnit - 2 + met_odd) * own_step;
  // (the last pair of the last unit may lie behind the others: a row of no length)
  float* shared = q.shared + ((((int64_t)k.block * q.pairs + u1 * (kUnit / 2) - 1) * a.rows + k.n) * a.groups + k.g) *
                                 NB * 64 + k.w * 64;
  UnitInputs<T> in;
  UnitDones dones;
  raw rx[kUnit], rd[kUnit], rz[kUnit], ry[kUnit];
  float kept[4][4];
  // (pointers that walk with the steps: products of steps and strides would be
  // held in more scalar registers than there are)
  const char *px = cx.unit(u1 * kUnit - 1), *pd = cd.unit(u1 * kUnit - 1), *pz = cz.unit(u1 * kUnit - 1),
             *py = cy.unit(u1 * kUnit - 1);
  char *ox = gx.unit(u1 * kUnit - 1), *od = gd.unit(u1 * kUnit - 1), *oz = gz.unit(u1 * kUnit - 1);
  const float* ps = states.base + (int64_t)(u1 - 1) * states.unit;
  const auto fetch = [&](int32_t unit) {
    const int32_t u = max(unit, u0);
    in.load(a, k, u * kUnit);
    cd.load_back(pd, unit * kUnit, rd);
    cy.load_back(py, unit * kUnit, ry);
    if (GATED) cz.load_back(pz, unit * kUnit, rz);
    if constexpr (!SUMMARY) {
      cx.load_back(px, unit * kUnit, rx);
      states.load(ps, unit >= u0, kept);
      ps = walk(ps, -states.unit);
    }
    dones.load(a, k, u * kUnit);
  };
  fetch(u1 - 1);
  if constexpr (!SUMMARY) no_stores(g.dx, kHeld * (GATED ? 3 : 2));
  for (int32_t u = u1 - 1; u >= u0; --u) {
    const int32_t t0 = u * kUnit;
    wave_sync();
    in.put(s_bc[k.w], k, S);
    wave_sync();
    // dt: D; w: the gradient of v; f: dgate / v
    float x[kUnit], dt[kUnit], w[kUnit], f[kUnit];
#pragma unroll
    for (int i = 0; i < kUnit; ++i) {
      const float v = T::widen(rd[i]) + bias;
      float E;
      const float sp = softplus_of(v, E), sl = sigmoid_from(v, E);
      dt[i] = a.softplus ? sp : v;
      float slope = a.softplus ? sl : 1.0f;
      w[i] = T::widen(ry[i]);
      if (!SUMMARY) x[i] = T::widen(rx[i]);
      if (GATED) {
        const float z = T::widen(rz[i]);
        const float sz = sigmoid_of(z);
        f[i] = w[i] * sz * __builtin_fmaf(z, 1.0f - sz, 1.0f);
        w[i] *= z * sz;
      }
      // past the end, where w and x are 0, the gradient of the state passes through
      if (t0 + i >= L) dt[i] = slope = 0.0f;
      if (SUMMARY)
        total += dt[i];
      else
        s_slope[k.w][i][k.lane] = slope;  // (read again by this lane alone)
    }
    const uint32_t cut = dones.cuts(a, k, t0);
    any_cut |= cut;
    if (SUMMARY) fetch(u - 1);

    if constexpr (SUMMARY) {
#pragma unroll
      for (int i = kUnit - 1; i >= 0; --i) {
        float c[4], dts[4], ws[4];
        read4(&s_bc[k.w][i][16 + 4 * k.j], c);
        quad_give(dt[i], dts);
        quad_give(w[i], ws);
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int s = 0; s < 4; ++s)
            G[r][s] = __builtin_amdgcn_exp2f(dts[r] * rate[r][s]) * __builtin_fmaf(c[s], ws[r], G[r][s]);
        if ((cut >> i) & 1u) {
#pragma unroll
          for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int s = 0; s < 4; ++s) G[r][s] = 0.0f;
        }
      }
    } else {
      // the state after step i from the one before it
      const auto advance = [&](float(&v)[4][4], int i) {
        float b[4], dts[4], dus[4];
        read4(&s_bc[k.w][i][4 * k.j], b);
        quad_give(dt[i], dts);
        quad_give(dt[i] * x[i], dus);
        if ((cut >> i) & 1u) {
#pragma unroll
          for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int s = 0; s < 4; ++s) v[r][s] = 0.0f;
        }
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int s = 0; s < 4; ++s)
            v[r][s] = __builtin_fmaf(__builtin_amdgcn_exp2f(dts[r] * rate[r][s]), v[r][s], dus[r] * b[s]);
      };
      float y[kUnit], p1[kUnit], p2[kUnit];
      // A lane's own channel of a step, when the sums over its states are known.
      const auto back = [&] {
        ox = walk(ox, -gx.step);
        od = walk(od, -gd.step);
        oz = walk(oz, -gz.step);
      };
      const auto finish = [&](int i) {
        const float dD = __builtin_fmaf(x[i], p1[i], p2[i] * kLn2);
        const float dd = dD * s_slope[k.w][i][k.lane];
        gx.store(ox, 0, t0 + i, __builtin_fmaf(dt[i], p1[i], skip * w[i]));
        gd.store(od, 0, t0 + i, dd);
        if (GATED) gz.store(oz, 0, t0 + i, f[i] * __builtin_fmaf(skip, x[i], y[i]));
        dskip = __builtin_fmaf(w[i], x[i], dskip);
        dbias += dd;
      };
      float v[4][4], held[kHeld][4][4];
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int s = 0; s < 4; ++s) v[r][s] = kept[r][s];
#pragma unroll
      for (int i = 0; i < kUnit; ++i) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          if (i < kHeld) {
            s_held[k.w][i][r][k.lane] = make_float4(v[r][0], v[r][1], v[r][2], v[r][3]);
          } else {
#pragma unroll
            for (int s = 0; s < 4; ++s) held[i < kHeld ? 0 : i - kHeld][r][s] = v[r][s];
          }
        }
        __builtin_amdgcn_sched_barrier(0);
        advance(v, i);
        if (GATED) {
          float c[4], sums[4];
          read4(&s_bc[k.w][i][16 + 4 * k.j], c);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            sums[r] = c[0] * v[r][0];
#pragma unroll
            for (int s = 1; s < 4; ++s) sums[r] = __builtin_fmaf(c[s], v[r][s], sums[r]);
          }
          y[i] = quad_sum(sums);
          if (NB > 1) s_sums[NB > 1 ? k.w : 0][0][i][k.lane] = y[i];
        }
      }
      float odd = 0.0f;  // the second of a pair of steps
#pragma unroll
      for (int i = kUnit - 1; i >= 0; --i) {
        // v: the state after step i; before: the one that a done may cut
        __builtin_amdgcn_sched_barrier(0);
        float before[4][4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          if (i < kHeld) {
            read4(reinterpret_cast<const float*>(&s_held[k.w][i][r][k.lane]), before[r]);
          } else {
#pragma unroll
            for (int s = 0; s < 4; ++s) before[r][s] = held[i < kHeld ? 0 : i - kHeld][r][s];
          }
        }
        float b[4], c[4], dts[4], dus[4], ws[4], db[4], dc[4], s1[4], s2[4];
        read4(&s_bc[k.w][i][4 * k.j], b);
        read4(&s_bc[k.w][i][16 + 4 * k.j], c);
        // (the empty statement keeps the compiler from holding the decays that
        // formed the states, a hundred registers)
        float again = dt[i];
        asm("" : "+v"(again));
        quad_give(again, dts);
        quad_give(dt[i] * x[i], dus);
        quad_give(w[i], ws);
#pragma unroll
        for (int s = 0; s < 4; ++s) db[s] = dc[s] = 0.0f;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          s1[r] = s2[r] = 0.0f;
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            G[r][s] = __builtin_fmaf(c[s], ws[r], G[r][s]);
            dc[s] = __builtin_fmaf(ws[r], v[r][s], dc[s]);
            db[s] = __builtin_fmaf(G[r][s], dus[r], db[s]);
            s1[r] = __builtin_fmaf(G[r][s], b[s], s1[r]);
          }
        }
        if ((cut >> i) & 1u) {
#pragma unroll
          for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int s = 0; s < 4; ++s) G[r][s] = 0.0f;
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int s = 0; s < 4; ++s) {
              G[r][s] *= __builtin_amdgcn_exp2f(dts[r] * rate[r][s]);
              const float p = G[r][s] * before[r][s];
              s2[r] = __builtin_fmaf(rate[r][s], p, s2[r]);
              drate[r][s] = __builtin_fmaf(dts[r], p, drate[r][s]);
            }
        }
        p1[i] = quad_sum(s1);
        p2[i] = quad_sum(s2);
        if constexpr (NB == 1) {
          finish(i);
          back();
        } else {
          s_sums[k.w][1][i][k.lane] = p1[i];
          s_sums[k.w][2][i][k.lane] = p2[i];
        }
        const float met = meet(db, dc, k.lane);
        if (i & 1) {
          odd = met;
        } else {
          const float sum = meet_pair(met, odd, k.lane);
          if (q.shared) {
            row_store<F32>(shared, t0 + i < L ? 256 : 0, met_at, sum);
            shared = walk(shared, -(int64_t)a.rows * a.groups * NB * 64);
          } else {
            if (t0 + i + ((k.lane >> 2) & 1) < L && met_state < S) *own = T::narrow(sum);
            own -= 2 * own_step;
          }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int s = 0; s < 4; ++s) v[r][s] = before[r][s];
        // (the registers of the held states are free from here on)
        if (i == kHeld) fetch(u - 1);
      }
      if constexpr (NB > 1) {
        __syncthreads();
#pragma unroll
        for (int i = kUnit - 1; i >= 0; --i, back()) {
          if (i % NB != k.w) continue;
          y[i] = p1[i] = p2[i] = 0.0f;
#pragma unroll
          for (int o = 0; o < NB; ++o) {
            if (GATED) y[i] += s_sums[o][0][i][k.lane];
            p1[i] += s_sums[o][1][i][k.lane];
            p2[i] += s_sums[o][2][i][k.lane];
          }
          finish(i);
        }
        __syncthreads();
      }
    }
  }

  const int64_t row = (int64_t)k.n * a.width;
  if constexpr (SUMMARY) {
    const int64_t at = (int64_t)k.chunk * a.rows * a.width + row;
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (k.quad_has(q.p, r)) store_states(q.sum.state + (at + k.quad_channel(q.p, r)) * S, k.s0, S, G[r]);
    if (k.mine && k.w == 0) q.sum.total[at + k.channel] = total;
    if (k.block == 0 && k.g == 0 && threadIdx.x == 0)
      q.sum.cut[(int64_t)k.chunk * a.rows + k.n] = any_cut != 0;
  } else {
    float* params = q.params + ((int64_t)k.chunk * a.rows + k.n) * ((int64_t)a.width * (S + 2));
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if (!k.quad_has(q.p, r)) continue;
      store_states(params + (int64_t)k.quad_channel(q.p, r) * S, k.s0, S, drate[r]);
      if (u0 == 0 && g.dstate)
        store_states(g.dstate + (row + k.quad_channel(q.p, r)) * S, k.s0, S, G[r]);
    }
    if constexpr (NB > 1) {
      float4* part = &s_held[0][0][0][0];
      part[k.w * 64 + k.lane] = make_float4(dskip, dbias, 0.0f, 0.0f);
      __syncthreads();
      dskip = dbias = 0.0f;
#pragma unroll
      for (int o = 0; o < NB; ++o) {
        dskip += part[o * 64 + k.lane].x;
        dbias += part[o * 64 + k.lane].y;
      }
    }
    if (k.mine && k.w == 0) {
      params[(int64_t)a.width * S + k.channel] = dskip;
      params[(int64_t)a.width * (S + 1) + k.channel] = dbias;
    }
  }
}

// db and dc: the sums over a group's blocks, rounded.  A thread takes two
// neighbouring states of one kind and step.
template <class T>
__global__ void __launch_bounds__(256) scan_shared_kernel(const GradRun q, int64_t total) {
  const scan_grad_args& g = q.g;
  const scan_args& a = g.f;
  const int32_t wide = q.p.state_blocks * 32;  // couples of states of a pair of steps
  using raw = typename T::raw;
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < total; e += (int64_t)gridDim.x * 256) {
    const int32_t i = (int32_t)(e % wide);
    const int64_t row = e / wide;  // (pair of steps, n, group)
    float s0 = 0.0f, s1 = 0.0f;
    for (int32_t b = 0; b < q.p.blocks; ++b) {
      const float2 v = reinterpret_cast<const float2*>(q.shared)[b * total + e];
      s0 += v.x;
      s1 += v.y;
    }
    const int32_t s = (i / 32) * kBlock + 2 * (i & 7), grp = (int32_t)(row % a.groups);
    const int64_t pn = row / a.groups;
    const int64_t n = pn % a.rows, t = 2 * (pn / a.rows) + ((i >> 4) & 1);
    if (t >= a.steps) continue;
    raw* p = i & 8 ? static_cast<raw*>(g.dc) + t * g.dc_step + n * g.dc_row + grp * g.dc_group
                   : static_cast<raw*>(g.db) + t * g.db_step + n * g.db_row + grp * g.db_group;
    if (s + 1 < a.states) {
      const float v[2] = {s0, s1};
      store_pack<T, 2>(p + s, narrow_pack<T, 2>(v));
    } else if (s < a.states) {
      p[s] = T::narrow(s0);
    }
  }
}

template <class T, int NB, bool GATED>
void launch_backward(const GradRun& q, hipStream_t stream) {
  const dim3 threads(64 * NB);
  if (q.p.chunks > 1)
    scan_backward_kernel<T, NB, GATED, true>
        <<<dim3((uint32_t)(q.p.columns * (q.p.chunks - 1))), threads, 0, stream>>>(q);
  if (q.p.joined)
    scan_join_launch(q.p, q.sum, q.g.f.rows, q.g.f.width, q.g.f.states, q.g.f.rate, nullptr, -1, stream);
  scan_backward_kernel<T, NB, GATED, false>
      <<<dim3((uint32_t)(q.p.columns * q.p.chunks)), threads, 0, stream>>>(q);
  if (q.shared) {
    const int64_t total = (int64_t)q.pairs * q.g.f.rows * q.g.f.groups * NB * 32;
    const int64_t groups = (total + 255) / 256;
    scan_shared_kernel<T><<<dim3((uint32_t)(groups < 16384 ? groups : 16384)), 256, 0, stream>>>(q, total);
  }
}
template <class T, int NB>
void launch_gate(const GradRun& q, hipStream_t stream) {
  q.g.f.gate ? launch_backward<T, NB, true>(q, stream) : launch_backward<T, NB, false>(q, stream);
}
template <class T>
void launch_states(const GradRun& q, hipStream_t stream) {
  if (q.p.state_blocks == 1) return launch_gate<T, 1>(q, stream);
  if (q.p.state_blocks == 2) return launch_gate<T, 2>(q, stream);
  return launch_gate<T, 4>(q, stream);
}

int64_t up(int64_t bytes) { return (bytes + 255) / 256 * 256; }

// The workspace, in order: summaries, shared sums, sums of the parameters'
// gradients, scratch to add those up.
struct Parts {
  int64_t summary, shared, params, scratch;
};
Parts parts_of(const ScanPlan& p, int32_t L, int32_t N, int32_t D, int32_t S, int32_t G) {
  const int64_t rows = (int64_t)p.chunks * N;
  Parts b;
  b.summary = scan_summary_bytes(p, N, D, S);
  b.shared = p.blocks > 1 ? up((int64_t)p.blocks * ((L + 1) / 2) * N * G * p.state_blocks * 64 * 4) : 0;
  b.params = up(rows * D * (S + 2) * 4);
  b.scratch = up(sums_floats(rows, D * (S + 2)) * 4);
  return b;
}

}  // namespace

int64_t scan_grad_workspace_bytes(int32_t L, int32_t N, int32_t D, int32_t S, int32_t G) {
  if (L == 0 || N == 0 || D == 0) return 0;
  const Parts b = parts_of(scan_plan(L, N, D, S, G), L, N, D, S, G);
  return b.summary + b.shared + b.params + b.scratch;
}

hipError_t scan_backward_launch(const scan_grad_args& g, hipStream_t stream) {
  const scan_args& a = g.f;
  const int64_t D = a.width, S = a.states;
  if (a.steps == 0 || a.rows == 0) {
    hipError_t e = copy_or_clear_launch(nullptr, g.drate, D * S * 4, stream);
    if (e == hipSuccess && g.dskip) e = copy_or_clear_launch(nullptr, g.dskip, D * 4, stream);
    if (e == hipSuccess && g.ddelta_bias) e = copy_or_clear_launch(nullptr, g.ddelta_bias, D * 4, stream);
    if (e == hipSuccess && g.dstate && a.rows > 0)
      e = copy_or_clear_launch(g.dnew_state, g.dstate, a.rows * D * S * 4, stream);
    return e;
  }
  GradRun q;
  q.g = g;
  q.p = scan_plan(a.steps, a.rows, a.width, a.states, a.groups);
  q.pairs = (a.steps + 1) / 2;
  const Parts b = parts_of(q.p, a.steps, a.rows, a.width, a.states, a.groups);
  char* w = static_cast<char*>(a.workspace);
  q.sum = scan_summary(q.p, a.rows, a.width, a.states, w);
  q.shared = b.shared ? reinterpret_cast<float*>(w + b.summary) : nullptr;
  q.params = reinterpret_cast<float*>(w + b.summary + b.shared);
  if (a.dtype == POLICY_F32)
    launch_states<F32>(q, stream);
  else if (a.dtype == POLICY_BF16)
    launch_states<BF16>(q, stream);
  else
    launch_states<F16>(q, stream);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int32_t ds = (int32_t)(D * S), d = (int32_t)D;
  const SumsOut out = {{g.drate, g.dskip, g.ddelta_bias}, {ds, ds + d, ds + 2 * d}};
  return sums_launch(q.params, (int64_t)q.p.chunks * a.rows, ds + 2 * d,
                     reinterpret_cast<float*>(w + b.summary + b.shared + b.params), out, stream);
}

}  // namespace rl
