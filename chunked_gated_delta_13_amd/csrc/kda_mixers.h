// Host <-> kernel interface of the short convolution, the state space scan and the window
// attention inside libkda (not part of the public C ABI).
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/kda.h"

namespace kda {

struct ConvArgs {
    const void* x;            // [rows, D], row stride x_stride elements (rows = B * T, or N)
    const void* w;            // [D, W]
    const void* bias;         // [D] or nullptr
    const void* state_in;     // [B, W - 1, D] or nullptr (zeros)
    void* state_out;          // [B, W - 1, D] or nullptr
    void* y;                  // [rows, D]
    const int* lens;          // [B] (device, clamped to [0, T]) or nullptr
    long long x_stride;
    int B, T, D;
    int silu;
    int tile;                 // tokens per thread (prompt form)
};

// vec = channels per thread: 16 bytes of them where rows are 16-byte aligned, else 1.
hipError_t launch_conv_prefill(int W, bool f32, bool vec, const ConvArgs& a, hipStream_t s);
hipError_t launch_conv_step(int W, bool f32, bool vec, const ConvArgs& a, hipStream_t s);

}  // namespace kda
