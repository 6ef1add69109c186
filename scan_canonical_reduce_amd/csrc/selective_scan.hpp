// Launchers of the selective scan (internal).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "seq_device.hpp"

namespace canon {
namespace seq {

// Kernel arguments of the forward and backward passes.
struct ScanArgs {
    Seqs q;
    canon_rows_t u, delta, z, out, B, C;
    const float *A, *D, *bias, *init;
    float *final, *cs;
    int32_t channels, dg, slabs, states;  // dg: channels per group, slabs: per group
    bool softplus, bc_vec, st_vec;  // *_vec: a lane's states load as one vector
    float *ws_state, *ws_dl;  // per slot: channels x NP, channels
    // backward
    canon_rows_t dout, du, ddelta, dz, dB, dC;
    float *dA, *dD, *dbias, *dinit;
    const float* dfinal;
    float *ws_dD, *ws_dbias, *ws_bc;
};

// States per lane (1, 2 or 4: four rows of lanes share a channel's states) and
// the padded states per channel, 4 ks.
inline int scan_ks(int64_t states) { return states <= 4 ? 1 : states <= 8 ? 2 : 4; }

constexpr int kSlab = 64;  // channels of a workgroup: 4 waves of 16
constexpr int kSub = 16;   // rows between saved states, and of a register tile

// Byte offsets within a 16-row tile are 32-bit (below 2^31): fewer than 16 rows
// of a pitch below 2^24 elements, and a column below 2^24 (the host checks both).
constexpr int64_t kMaxPitch = (int64_t)1 << 24;

// Up to this many rows (of all sequences together where they are packed) every
// sequence is walked whole: one launch costs less than three.
constexpr int64_t kShortRows = 2 * CANON_SCAN_CHUNK;

template <typename T>
hipError_t launch_selective_scan(const ScanArgs& a, int64_t groups, hipStream_t st);
template <typename T>
hipError_t launch_selective_scan_grad(const ScanArgs& a, int64_t groups, hipStream_t st);
template <typename T>
hipError_t launch_selective_scan_step(const ScanArgs& a, int64_t groups, hipStream_t st);

}  // namespace seq
}  // namespace canon
