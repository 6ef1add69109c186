// Launcher of the sampling (internal).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/canon_layer.h"
#include "seq_device.hpp"

namespace canon {
namespace seq {

struct SampleArgs {
    const void* logits;
    int64_t ld, rows;
    int32_t vocab, bits;  // weights are multiples of 2^-bits
    int32_t share_bits;   // vocab numbers of so many bits add up to less than 2^32
    const float *u, *temperature, *top_p, *min_p;
    const int32_t* top_k;
    double temperature_all, top_p_all, min_p_all;
    int32_t top_k_all;
    void* ids;
    bool ids64;
};

template <typename T>
hipError_t launch_sample(const SampleArgs& a, hipStream_t st);

}  // namespace seq
}  // namespace canon
