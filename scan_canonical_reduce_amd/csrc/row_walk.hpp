// A walk over a run's rows, the next ones on their way while these are computed.
#pragma once

#include <hip/hip_runtime.h>

namespace canon {
namespace seq {

// row(b, u, r) for each r of [0, ROWS), in order and once, r's input in place u
// of buffer b; fetch(b, r0) reads rows [r0, r0 + U) into buffer b, the first U
// before this call.  Checks of r, the same in every lane, instead of an unrolled
// end: the compiler would spill registers for that.
template <int ROWS, int U, class Fetch, class Row>
__host__ __device__ __forceinline__ void walk_rows(Fetch&& fetch, Row&& row)
{
#pragma unroll 1
    for (int r0 = 0; r0 < ROWS; r0 += 2 * U) {
        if (r0 + U < ROWS) fetch(1, r0 + U);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (r0 + u < ROWS) row(0, u, r0 + u);
        if (r0 + 2 * U < ROWS) fetch(0, r0 + 2 * U);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (r0 + U + u < ROWS) row(1, u, r0 + U + u);
    }
}

}  // namespace seq
}  // namespace canon
