// Launchers of the layer norm (internal).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "seq_device.hpp"

namespace canon {
namespace seq {

struct NormArgs {
    int32_t total, rows;  // rows of all sequences, of one
    int32_t width;
    float inv_width, eps;
    canon_rows_t x, residual, sum, out;
    const void *weight, *bias;
    float* stats;
    // backward
    canon_rows_t dout, dsum, dx;
    float *dweight, *dbias;
    float *ws_w, *ws_b;  // per chunk of rows: width
};

// Rows of a chunk of the sums over rows: as many chunks as fill the chip twice (of rows
// wider than kNormGradWide, which are cut into 5 parts or more, a quarter), then longer
// ones, whose partial sums are at most a 24th of the rows' bytes.  Backward passes with
// all chunks and with a quarter: 777 x 20000 float32 65 and 53 us, 1024 x 32768 141 and 87,
// 4096 x 12288 bf16 88 and 77, but 2000 x 8192 float32 44 and 57, 3001 x 1021 bf16 17 and 21.
constexpr int64_t kNormChunks = 512;
constexpr int64_t kNormChunkMost = 64;
constexpr int32_t kNormGradWide = 8192;
inline int64_t norm_chunk(int64_t total, int64_t width)
{
    const int64_t most = width > kNormGradWide ? kNormChunks / 4 : kNormChunks;
    const int64_t n = (total + most - 1) / most;
    return n < 1 ? 1 : n > kNormChunkMost ? kNormChunkMost : n;
}

template <typename T, typename P>
hipError_t launch_layer_norm(const NormArgs& a, hipStream_t st);
template <typename T, typename P>
hipError_t launch_layer_norm_grad(const NormArgs& a, hipStream_t st);

}  // namespace seq
}  // namespace canon
