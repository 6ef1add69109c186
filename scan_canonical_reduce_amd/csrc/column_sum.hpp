// Column sums of per-chunk partial values (parameter gradients).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace canon {
namespace seq {

constexpr int kColLanes = 16;

// out[(c / np) * n + c % np] = sum over r of part[r * cols + c], for the
// columns c with c % np < n: the rows go to 16 lanes, row r to lane r mod 16,
// each lane is summed in row order and the lanes by the pairwise tree, so the
// value depends on the rows alone.  A workgroup holds 64 columns; its 16
// waves are the lanes.
__global__ __launch_bounds__(1024) static void k_column_sum(const float* __restrict__ part,
                                                            int64_t rows, int64_t cols, int np,
                                                            int n, float* __restrict__ out)
{
    __shared__ float lanes[kColLanes][64];
    const int x = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int64_t c = (int64_t)blockIdx.x * 64 + x;
    float s = 0.f;
    if (c < cols) {
        int64_t r = w;
        for (; r + 3 * kColLanes < rows; r += 4 * kColLanes) {
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = part[(r + i * kColLanes) * cols + c];
#pragma unroll
            for (int i = 0; i < 4; ++i) s += v[i];
        }
        for (; r < rows; r += kColLanes) s += part[r * cols + c];
    }
    lanes[w][x] = s;
    __syncthreads();
    if (w != 0 || c >= cols || c % np >= n) return;
    float v[kColLanes];
#pragma unroll
    for (int i = 0; i < kColLanes; ++i) v[i] = lanes[i][x];
#pragma unroll
    for (int d = 1; d < kColLanes; d *= 2)
#pragma unroll
        for (int i = 0; i < kColLanes; i += 2 * d) v[i] += v[i + d];
    out[c / np * n + c % np] = v[0];
}

inline hipError_t launch_column_sum(const float* part, int64_t rows, int64_t cols, int np, int n,
                                    float* out, hipStream_t st)
{
    if (cols == 0) return hipSuccess;
    k_column_sum<<<dim3((unsigned)((cols + 63) / 64)), dim3(1024), 0, st>>>(part, rows, cols, np,
                                                                           n, out);
    return hipGetLastError();
}

}  // namespace seq
}  // namespace canon
