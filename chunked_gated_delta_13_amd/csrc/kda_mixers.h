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
    int streamed;             // 1: outputs larger than the caches, stored past them
};

// vec = channels per thread: 16 bytes of them where rows are 16-byte aligned, else 1.
hipError_t launch_conv_prefill(int W, bool f32, bool vec, const ConvArgs& a, hipStream_t s);
hipError_t launch_conv_step(int W, bool f32, bool vec, const ConvArgs& a, hipStream_t s);

struct SsmArgs {
    const void* x;            // rows of H * p, stride x_stride elements
    const void* dt;           // rows of H
    const float* A;           // [H]
    const void* Bm;           // rows of G * n
    const void* Cm;           // rows of G * n
    const float* D;           // [H] or nullptr
    const void* z;            // rows of H * p or nullptr
    const float* dt_bias;     // [H] or nullptr
    const float* S0;          // [B, H, n, p] or nullptr (zeros)
    const int* lens;          // [B] (device, clamped to [0, T]) or nullptr
    void* y;                  // [rows, H, p]
    float* S_T;               // [B, H, n, p] or nullptr; the token form reads and writes it
    long long x_stride, dt_stride, b_stride, c_stride, z_stride;
    long long T;
    int H, G;
    long long seg_len;        // tokens per segment (whole chunks)
    int n_seg;                // segments of the sequence
    int n_seg_launch;         // segments of this launch (the first ones)
    long long n_units;        // sequences x heads x segments of this launch
    long long per_xcd;
    float* ws_state;          // [B * H, n_seg, n, p] entry states (slot 0 only with keep_S0)
    float* ws_decay;          // [B * H, n_seg] exponents (base 2) of the decay over the segment before
    int keep_S0;              // 1: the first pass copies S0 to slot 0, the second reads it there
};

enum class SsmPass { kStates, kOutputs, kToken };
hipError_t launch_ssm(SsmPass pass, int n, int p, bool f32, const SsmArgs& a, hipStream_t s);
hipError_t launch_ssm_join(int n, int p, int bh, int n_seg, float* ws_state, const float* ws_decay, hipStream_t s);

struct WindowArgs {
    const void* q;            // rows of H * d, stride q_stride elements
    const void* k;            // rows of Hkv * d
    const void* v;
    void* k_cache;            // [B, sinks + window, Hkv, d] or nullptr
    void* v_cache;
    const int* start;         // [B] tokens before the first new one (device) or nullptr (0)
    const int* lens;          // [B] (device, clamped to [0, T]) or nullptr
    void* o;                  // [rows, H, d]
    long long q_stride, k_stride, v_stride;
    int B, T, H, Hkv, window, sinks;
    float scale;
    int few;                  // 1: too few queries for 128 of them per workgroup
    int q_tiles;
    int n_split, split_len;   // ranges of keys (token form: of split_len cache rows)
    long long n_units, per_xcd;
    float* ws_o;              // [rows * H, n_split, d] partial outputs of a split call
    float* ws_ml;             // [rows * H, n_split, 2] their maxima (base 2) and sums
};

hipError_t launch_window_prefill(int d, bool f32, const WindowArgs& a, hipStream_t s);
hipError_t launch_window_step(int d, bool f32, const WindowArgs& a, hipStream_t s);

}  // namespace kda
