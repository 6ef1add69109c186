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

// Blocks of a sequence up to which each folds those before it itself, beyond which a launch
// of its own does.  2048 channels bf16, forward and backward, folded so and by a launch: 16
// blocks 53 + 76 us and 55 + 78, 32 blocks 96 + 140 and 100 + 144, 64 blocks 214 + 293 and
// 219 + 288, 128 blocks 427 + 582 and 414 + 549.
constexpr int64_t kRecurFold = 32;

constexpr int kRecurBlockChunks = kRecurRounds * kRecurWaves;

// Where blocks leave most compute units idle, a workgroup takes a round of one, after a
// launch for the folds of the chunks before it: with no more than 64 slots times 64
// channels, or 128 where there is a launch for the blocks' folds otherwise, and more than
// two rounds.  bf16, forward and backward, a workgroup for each block against each round:
// 512 rows of 4096 channels 18 + 32 us against 16 + 27, of 8192 18 + 33 against 21 + 28;
// 200 rows of 2048 13 + 24 against 17 + 26; 2048 rows of 2048 31 + 44 against 21 + 30, of
// 4096 32 + 46 against 42 + 52.  The bits are the same but for the decay's gradient, which
// is summed by rounds then: so the rule goes by the sizes alone.
constexpr int64_t kRecurSpread = 64, kRecurSpreadBlocks = kRecurWaves - 1;
inline bool recur_spread(int64_t slots, int64_t rows, int64_t channels)
{
    return rows > 2 * kRecurRound && rows <= kRecurSpreadBlocks * CANON_RECUR_BLOCK &&
           slots * ((channels + 63) / 64) <=
               (rows > CANON_RECUR_BLOCK ? 2 * kRecurSpread : kRecurSpread);
}

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
    bool spread;  // a workgroup for each round, with the folds of each chunk:
    float *ws_cq, *ws_cs;  // per slot: kRecurBlockChunks x channels
    // backward
    canon_rows_t dout, dx, dgate, dinput;
    float *ddecay, *dinit;
    const float* dfinal;
    float* ws_dd;  // per slot, or round where they are spread: channels
};

template <typename T>
hipError_t launch_recurrence(const RecurArgs& a, hipStream_t st);
template <typename T>
hipError_t launch_recurrence_grad(const RecurArgs& a, hipStream_t st);
template <typename T>
hipError_t launch_recurrence_step(const RecurArgs& a, hipStream_t st);

}  // namespace seq
}  // namespace canon
