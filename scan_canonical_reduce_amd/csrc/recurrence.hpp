// Launchers of the gated linear recurrence (internal).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/canon_layer.h"
#include "seq_device.hpp"

namespace canon {
namespace seq {

constexpr int kRecurWaves = 16;                               // chunks of a round
constexpr int kRecurRound = kRecurWaves * CANON_RECUR_CHUNK;  // rows between kept states
constexpr int kRecurRounds = CANON_RECUR_BLOCK / kRecurRound;

// Blocks of a sequence up to which each folds those before it itself.
constexpr int64_t kRecurFold = 32;

// Byte offsets within a chunk are 32-bit: row pitches below this many elements.
constexpr int64_t kRecurPitch = (int64_t)1 << 24;

struct RecurArgs {
    Seqs q;
    canon_rows_t x, gate, input, out;
    const float *decay, *init;
    float *final, *kept;  // kept: per slot, kRecurRounds x channels
    int32_t channels;
    int32_t slabs;  // of 64 lanes' channels each; set by the launcher
    bool pairs;     // 16-bit values: two channels a lane, aligned in every row
    float *ws_q, *ws_s, *ws_h;  // per slot: channels; NULL where no sequence has two blocks
    bool carry;  // a launch of its own makes the blocks' start states
    // backward
    canon_rows_t dout, dx, dgate, dinput;
    float *ddecay, *dinit;
    const float* dfinal;
    float* ws_dd;  // per slot: channels
};

template <typename T>
hipError_t launch_recurrence(const RecurArgs& a, hipStream_t st);
template <typename T>
hipError_t launch_recurrence_grad(const RecurArgs& a, hipStream_t st);
template <typename T>
hipError_t launch_recurrence_step(const RecurArgs& a, hipStream_t st);

}  // namespace seq
}  // namespace canon
