// Launchers of the embedding lookup and its gradient (internal).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "seq_device.hpp"

namespace canon {
namespace seq {

struct EmbedArgs {
    const void* weight;
    int64_t ld_weight, rows, width;
    const void* ids;
    bool ids64, vec;
    int64_t tokens;
    float scale;
    void* out;
    int64_t ld_out;
};

struct EmbedGradArgs {
    const void* dout;
    int64_t ld_dout;
    const void* ids;
    bool ids64, vec, accumulate;
    int64_t tokens, rows, width;
    float scale;
    int64_t padding_id;
    void* dw;
    int64_t ld_dw;
    // workspace
    int32_t *order, *offset;    // tokens by id; the first of each id (rows + 1)
    int4* items;                // row, chunk, offset, tokens of the row; at most one per token
    int32_t *n_items, *n_long, *before;  // per group of ids
    int32_t* longs;
    float *part, *part_last;
    int64_t ld_part;
};

constexpr int kEmbedChunk = 64;  // occurrences that one wave sums

// Ids of a workgroup of the grouping kernel, and the number of workgroups.
inline int64_t ids_per_group(int64_t rows)
{
    const int64_t r = (rows + 255) / 256;
    return r < 16 ? 16 : r > 512 ? 512 : r;  // 16 waves' counts of 512 ids: 32 KiB of LDS
}
inline int64_t id_groups(int64_t rows)
{
    const int64_t r = ids_per_group(rows);
    return (rows + r - 1) / r;
}
// Rows of a gradient's table: the grouping kernel's workgroups, of 1024 threads and
// 512 ids, number below 2^22.
constexpr int64_t kEmbedGradRows = ((int64_t)1 << 31) - 512;

// Accesses per row of width elements of es bytes: 16 bytes each, or single
// elements where a row has fewer; 1024 of them to a workgroup of the lookup.
inline int64_t embed_accesses(int64_t width, size_t es)
{
    const int64_t v = 16 / (int64_t)es;
    return width >= v ? (width + v - 1) / v : width;
}
constexpr int kEmbedGridAccesses = 1024;

constexpr int kGroupWaves = 16;  // of a workgroup that groups tokens by id

// Exclusive sums over the workgroup's 1024 threads, of two pairs of counts at
// once (each pair in the halves of 64 bits); x and y become the sums of all.
struct Pairs {
    uint64_t x, y;
};
__device__ __forceinline__ Pairs block_exclusive(uint64_t& x, uint64_t& y, Pairs* lds)
{
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    Pairs run = {x, y};
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const uint64_t ox = __shfl_up((unsigned long long)run.x, d, 64);
        const uint64_t oy = __shfl_up((unsigned long long)run.y, d, 64);
        if (lane >= d) run.x += ox, run.y += oy;
    }
    if (lane == 63) lds[w] = run;
    __syncthreads();
    Pairs base = {0, 0}, all = {0, 0};
#pragma unroll
    for (int k = 0; k < kGroupWaves; ++k) {
        if (k == w) base = all;
        all.x += lds[k].x, all.y += lds[k].y;
    }
    base.x += run.x - x, base.y += run.y - y;
    x = all.x, y = all.y;
    return base;
}

template <typename T>
hipError_t launch_embedding(const EmbedArgs& a, hipStream_t st);
hipError_t launch_embedding_group(const EmbedGradArgs& a, hipStream_t st);
template <typename T, typename G>
hipError_t launch_embedding_grad(const EmbedGradArgs& a, hipStream_t st);

}  // namespace seq
}  // namespace canon
