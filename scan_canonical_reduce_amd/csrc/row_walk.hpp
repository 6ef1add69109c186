// A walk over a run's rows, the next ones on their way while these are computed.
#pragma once

#include <hip/hip_runtime.h>

namespace canon {
namespace seq {

// row(b, u, r) for each r of [0, ROWS), in order and once, r's input in place u
// of buffer b; fetch(b, r0) reads rows [r0, r0 + U) into buffer b, the first U
// before this call.  One loop that the last step leaves early: the same rows as an
// unrolled end spill registers, and a check of each row costs 5 us of 108 in the
// convolution's backward pass (8 x 2048 x 4096, 4 taps, bf16).
template <int ROWS, int U, class Fetch, class Row>
__host__ __device__ __forceinline__ void walk_rows(Fetch&& fetch, Row&& row)
{
    constexpr int REST = ROWS % (2 * U);  // rows of the last, shorter step
    constexpr int REST0 = REST == 0 || REST > U ? U : REST, REST1 = REST > U ? REST - U : U;
#pragma unroll 1
    for (int r0 = 0; r0 < ROWS; r0 += 2 * U) {
        const bool last = REST != 0 && r0 + 2 * U > ROWS;
        if (!last || REST > U) fetch(1, r0 + U);
#pragma unroll
        for (int u = 0; u < REST0; ++u) row(0, u, r0 + u);
        if (last && REST <= U) break;
#pragma unroll
        for (int u = REST0; u < U; ++u) row(0, u, r0 + u);
        if (r0 + 2 * U < ROWS) fetch(0, r0 + 2 * U);
#pragma unroll
        for (int u = 0; u < REST1; ++u) row(1, u, r0 + U + u);
        if (last) break;
#pragma unroll
        for (int u = REST1; u < U; ++u) row(1, u, r0 + U + u);
    }
}

}  // namespace seq
}  // namespace canon
