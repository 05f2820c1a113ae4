// Column sums of partial gradients, and copies that a captured graph may hold.
//
// A workgroup takes 64 columns and a run of rows: its four waves the rows
// r, r + 4, ..., eight loads in flight each, and their sums meet in LDS.
// Many rows are cut into runs first, whose sums the same kernel adds up.
// More than 4096 are brought below that before, 64 at a time.
// The order of the additions depends on the two sizes alone, and no summand
// goes through more than 46 of them, whatever the rows: 17 in a run of 64 (15 of
// a wave, 2 in LDS), twice, and 6 in each of at most two times 64 before.
#include <algorithm>

#include "block.hpp"

namespace rl {

namespace {

constexpr int kRun = 64;      // rows of a run, at least
constexpr int kMostRuns = 64;
constexpr int64_t kMostRows = kRun * kMostRuns;

int64_t runs_of(int64_t rows) {
  const int64_t runs = (rows + kRun - 1) / kRun;
  return runs < kMostRuns ? runs : kMostRuns;
}

__global__ void __launch_bounds__(256) sums_kernel(const float* x, int64_t rows, int32_t columns,
                                                   int64_t run, float* partial, SumsOut out) {
  __shared__ float s_sum[4][64];
  const int32_t lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t r0 = blockIdx.y * run, r1 = r0 + run < rows ? r0 + run : rows;
  // (one turn but where there are more columns than a grid holds workgroups)
  for (int64_t c0 = (int64_t)blockIdx.x * 64; c0 < columns; c0 += (int64_t)gridDim.x * 64) {
    const int64_t c = c0 + lane;
    float sum = 0.0f;
    if (c < columns) {
      int64_t r = r0 + w;
      for (; r + 28 < r1; r += 32) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = x[(r + 4 * i) * columns + c];
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += v[i];
      }
      for (; r < r1; r += 4) sum += x[r * columns + c];
    }
    s_sum[w][lane] = sum;
    __syncthreads();
    if (w == 0 && c < columns) {
      sum = (s_sum[0][lane] + s_sum[1][lane]) + (s_sum[2][lane] + s_sum[3][lane]);
      if (partial) {
        partial[(int64_t)blockIdx.y * columns + c] = sum;
      } else {
        const int k = c < out.end[0] ? 0 : c < out.end[1] ? 1 : 2;
        float* p = k == 0 ? out.out[0] : k == 1 ? out.out[1] : out.out[2];
        const int32_t first = k == 0 ? 0 : k == 1 ? out.end[0] : out.end[1];
        if (p) p[c - first] = sum;
      }
    }
    __syncthreads();
  }
}

// partial[run] = the sum of the rows 64 run .. 64 run + 63.  A wave's 16 rows
// are added in pairs, which takes 4 additions on the way of each.
__global__ void __launch_bounds__(256) far_sums_kernel(const float* x, int64_t rows, int32_t columns,
                                                       int64_t blocks, float* partial) {
  __shared__ float s_sum[4][64];
  const int32_t lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int32_t across = (columns + 63) / 64;
  for (int64_t id = blockIdx.x; id < blocks; id += gridDim.x) {
    const int64_t run = id / across;
    const int32_t c = (int32_t)(id % across) * 64 + lane;
    float v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int64_t r = kRun * run + w + 4 * i;
      v[i] = c < columns && r < rows ? x[r * columns + c] : 0.0f;
    }
#pragma unroll
    for (int half = 8; half > 0; half /= 2)
#pragma unroll
      for (int i = 0; i < half; ++i) v[i] += v[i + half];
    s_sum[w][lane] = v[0];
    __syncthreads();
    if (w == 0 && c < columns)
      partial[run * columns + c] = (s_sum[0][lane] + s_sum[1][lane]) + (s_sum[2][lane] + s_sum[3][lane]);
    __syncthreads();
  }
}

__global__ void __launch_bounds__(256) copy_kernel(const uint8_t* src, uint8_t* dst, int64_t bytes) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; 2 * i < bytes; i += (int64_t)gridDim.x * 256)
    reinterpret_cast<uint16_t*>(dst)[i] = src ? reinterpret_cast<const uint16_t*>(src)[i] : (uint16_t)0;
}

}  // namespace

int64_t sums_floats(int64_t rows, int32_t columns) {
  int64_t kept = 0;  // rows
  while (rows > kMostRows) kept += rows = (rows + kRun - 1) / kRun;
  const int64_t runs = runs_of(rows);
  return (kept + (runs > 1 ? runs : 0)) * columns;
}

hipError_t sums_launch(const float* x, int64_t rows, int32_t columns, float* scratch,
                       const SumsOut& out, hipStream_t stream) {
  while (rows > kMostRows) {
    const int64_t fewer = (rows + kRun - 1) / kRun, blocks = fewer * ((columns + 63) / 64);
    far_sums_kernel<<<dim3((uint32_t)std::min(blocks, (int64_t)1 << 20)), 256, 0, stream>>>(
        x, rows, columns, blocks, scratch);
    x = scratch;
    scratch += fewer * columns;
    rows = fewer;
  }
  const int64_t runs = runs_of(rows);
  const uint32_t across = (uint32_t)std::min((columns + 63) / 64, 1 << 20);
  if (runs > 1) {
    const int64_t run = (rows + runs - 1) / runs;
    sums_kernel<<<dim3(across, (uint32_t)runs), 256, 0, stream>>>(x, rows, columns, run, scratch, out);
    x = scratch;
    rows = runs;
  }
  sums_kernel<<<dim3(across, 1), 256, 0, stream>>>(x, rows, columns, rows, nullptr, out);
  return hipGetLastError();
}

hipError_t copy_or_clear_launch(const void* src, void* dst, int64_t bytes, hipStream_t stream) {
  if (bytes == 0) return hipSuccess;
  const int64_t groups = (bytes + 511) / 512;
  copy_kernel<<<dim3((uint32_t)(groups < 4096 ? groups : 4096)), 256, 0, stream>>>(
      static_cast<const uint8_t*>(src), static_cast<uint8_t*>(dst), bytes);
  return hipGetLastError();
}

}  // namespace rl
