// Column sums of per-chunk partial values (parameter gradients).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace canon {
namespace seq {

constexpr int kColLanes = 16;

// One result: out[(c / np) * n + c % np] = sum over r of part[r * cols + c], for
// the columns c with c % np < n.
struct ColumnSum {
    const float* part;
    int64_t cols;
    int32_t np, n;
    float* out;  // NULL: not wanted
};

// Up to three results over the same rows in one launch.
struct ColumnSums {
    ColumnSum sum[3];
    int64_t rows;
};

// The rows go to 16 lanes, row r to lane r mod 16; each lane is summed in row
// order and the lanes by the pairwise tree, so the value depends on the rows
// alone.  A workgroup holds 64 columns; its 16 waves are the lanes.
__device__ __forceinline__ void column_sum_block(const ColumnSums& a, int64_t block)
{
    __shared__ float lanes[kColLanes][64];
    const int x = threadIdx.x & 63, w = threadIdx.x >> 6;
    ColumnSum j = a.sum[0];
#pragma unroll
    for (int k = 1; k < 3; ++k) {
        const int64_t blocks = j.out ? (j.cols + 63) / 64 : 0;
        if (block < blocks) break;
        block -= blocks;
        j = a.sum[k];
    }
    const int64_t c = block * 64 + x;
    float s = 0.f;
    if (c < j.cols) {
        const float* p = j.part + c;
        int64_t r = w;
        for (; r + 3 * kColLanes < a.rows; r += 4 * kColLanes) {
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = p[(r + i * kColLanes) * j.cols];
#pragma unroll
            for (int i = 0; i < 4; ++i) s += v[i];
        }
        for (; r < a.rows; r += kColLanes) s += p[r * j.cols];
    }
    lanes[w][x] = s;
    __syncthreads();
    if (w != 0 || c >= j.cols || c % j.np >= j.n) return;
    float v[kColLanes];
#pragma unroll
    for (int i = 0; i < kColLanes; ++i) v[i] = lanes[i][x];
#pragma unroll
    for (int d = 1; d < kColLanes; d *= 2)
#pragma unroll
        for (int i = 0; i < kColLanes; i += 2 * d) v[i] += v[i + d];
    j.out[c / j.np * j.n + c % j.np] = v[0];
}

__global__ __launch_bounds__(1024) static void k_column_sum(ColumnSums a)
{
    column_sum_block(a, blockIdx.x);
}

inline int64_t column_sum_blocks(const ColumnSums& a)
{
    int64_t blocks = 0;
    for (const ColumnSum& j : a.sum) blocks += j.out ? (j.cols + 63) / 64 : 0;
    return blocks;
}

inline hipError_t launch_column_sums(const ColumnSums& a, hipStream_t st)
{
    const int64_t blocks = column_sum_blocks(a);
    if (blocks == 0) return hipSuccess;
    k_column_sum<<<dim3((unsigned)blocks), dim3(1024), 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace seq
}  // namespace canon
