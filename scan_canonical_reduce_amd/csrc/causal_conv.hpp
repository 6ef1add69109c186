// Launchers of the causal convolution (internal).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "seq_device.hpp"

namespace canon {
namespace seq {

struct ConvArgs {
    Seqs q;
    canon_rows_t x, out;
    const void *weight, *bias, *init;
    void* final;
    int32_t channels;
    bool param_f32, silu, vec;  // vec: accesses of four channels are aligned
    // backward
    canon_rows_t dout, dx;
    float *dweight, *dbias;
    const void* dfinal;
    void* dinit;
    float *ws_w, *ws_b;  // per slot: channels x taps, channels
};

template <typename T>
hipError_t launch_causal_conv(const ConvArgs& a, int taps, hipStream_t st);
template <typename T>
hipError_t launch_causal_conv_grad(const ConvArgs& a, int taps, hipStream_t st);
template <typename T>
hipError_t launch_causal_conv_step(const ConvArgs& a, int taps, hipStream_t st);

}  // namespace seq
}  // namespace canon
