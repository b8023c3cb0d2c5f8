// Host <-> kernel interface of the entry points beside KDA inside libkda (not part of the public C ABI).
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

// Groups of waves that share the keys of 64 rows where compute units are left: what LDS holds.
constexpr int attn_groups(int d) { return d == 64 ? 4 : 2; }

struct AttnArgs {
    const void* q;            // [Nq] rows of H * d, stride q_stride elements
    const void* k;            // [Nk] rows of Hkv * d
    const void* v;
    const int* cu_q;          // [B + 1] first rows of the sequences and the last one's end (device)
    const int* cu_k;          // the same of the keys; may be cu_q
    void* o;                  // [Nq, H, d]
    long long q_stride, k_stride, v_stride;
    int B, Nq, Nk, H, Hkv;
    float scale;
    int few;                  // 1: too few rows for 128 of them per workgroup; 2: for 64 of them on every compute unit
    int n_split;              // ranges of keys
    int n_sets;               // sets of kv heads that XCDs share out
    float* ws_o;              // [Nq * H, n_split, d] partial outputs of a split call
    float* ws_ml;             // [Nq * H, n_split, 2] their maxima (base 2) and sums
};

hipError_t launch_attn_prefill(int d, bool f32, const AttnArgs& a, hipStream_t s);

struct CacheArgs {
    const void* k;            // [N] rows of Hkv * d, stride k_stride elements (written ones)
    const void* v;
    void* k_out;              // [N, Hkv, d] (read ones)
    void* v_out;
    uint8_t* k_cache;         // [n_pages, Hkv, page_bytes]
    uint8_t* v_cache;
    const int* pages;         // [B, max_pages]
    const int* cu;            // [B + 1], or nullptr: token i is sequence i's
    const int* start;         // [B] position of each sequence's first token, or nullptr (0)
    long long k_stride, v_stride, page_bytes;
    long long n_units, per_xcd;
    int B, N, Hkv, n_pages, max_pages, page, page_shift;
    int streamed;             // read rows go past the caches
};

hipError_t launch_cache_rows(bool write, int d, bool f32, const CacheArgs& a, hipStream_t s);

struct AttnStepArgs {
    const void* q;            // [N * m] rows of H * d, stride q_stride elements
    const uint8_t* k_cache;   // [n_pages, Hkv, page_bytes]
    const uint8_t* v_cache;
    const int* pages;         // [N, max_pages]
    const int* lens;          // [N] tokens in the cache, the m new ones among them
    void* o;                  // [N, m, H, d]
    long long q_stride, page_bytes;
    int N, m, H, Hkv, n_pages, max_pages, page, page_shift;
    float scale;
    int want, slots;          // slots that the sequences share, and the most there can be
    float* ws_o;              // [slots, m * H, d] partial outputs
    float* ws_ml;             // [slots, m * H, 2] their maxima (base 2) and sums
};

hipError_t launch_attn_step(int d, bool f32, const AttnStepArgs& a, hipStream_t s);

struct DeltaArgs {
    const void* q;            // rows of Hk * dk, stride q_stride elements
    const void* k;
    const void* v;            // rows of H * dv
    const float* g;           // [rows, H] natural log of the decay
    const float* beta;        // [rows, H]
    const int* lens;          // [B] (device, clamped to [0, T]) or nullptr
    void* o;                  // [rows, H, dv]
    const float* S_in;        // entry states: of (b h, segment) at bh * sin_bh + seg * sin_seg, or nullptr (zeros)
    float* S_out;             // final states: of segment out_seg only (at bh * sout_bh), or with out_seg -1 of all; the
                              // token form reads and writes it
    float* M_out;             // [BH, m_bh, dk, dk] transitions of the segments (states' pass)
    int* dead;                // [BH, m_bh] 1: nothing is left of a state over the segment, whose transition is not formed
    long long q_stride, k_stride, v_stride;
    long long sin_bh, sin_seg, sout_bh, sout_seg, m_bh;
    long long T, seg_len;     // tokens, tokens per segment (whole chunks)
    int BH, H, Hk, dv;
    int n_seg_launch, out_seg;
    int slices, id_slices;    // slices of state columns, of the transition's columns
    long long n_units, per_xcd;
};

// One pass over the first n_seg_launch segments, `width` (64 or 128) state columns a workgroup: outputs, or (out false; 128
// columns with dk = dv = 128 only) final states from zero and transitions.
hipError_t launch_delta_prefill(bool out, int dk, bool f32, int width, const DeltaArgs& a, hipStream_t s);
hipError_t launch_delta_join(int dk, int dv, int bh, int n_seg, const float* M, const int* dead, const float* S0, float* S_in, hipStream_t s);
hipError_t launch_delta_step(int dk, bool f32, const DeltaArgs& a, hipStream_t s);

}  // namespace kda
