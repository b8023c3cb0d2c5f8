// Short causal depthwise convolution for gfx950: prompts and single tokens.
//
//   y[t, d] = act(bias[d] + sum_{j < W} w[d, j] x[t - (W - 1) + j, d])
//
// with the W - 1 inputs before the first token taken from the kept history, and act the identity
// or SiLU.  Sums are fp32, rounded once to the output type.
//
// Both forms are bound by HBM: 2 W flops for each element read once and written once.  A thread
// owns one 16-byte group of channels (so that a wave reads and writes 1 KiB runs of a row) and
// walks a tile of consecutive tokens with the last W - 1 inputs in registers, so each input is
// read once per tile and W - 1 more times per tile boundary, from cache.  4 x 8192 tokens of 7424
// channels in bf16 (0.97 GB) take 174 us, 5.6 TB/s, above a device copy's 4.9, in fp32 348 us; one token of
// 256 sequences (30 MB) takes 6.7 us, one token of one sequence 4.6 us a call, 3.4 of them the launch.
// Rows off 16 bytes (a width that is no multiple of 8 in bf16, of 4 in fp32) are taken one channel per
// thread: 4095 channels run at 3.7 TB/s in bf16 and 4.6 in fp32, 4096 in bf16 at 6.1.
#include "kda_device.h"
#include "kda_mixers.h"

namespace kda {

namespace {

constexpr int kConvThreads = 256;

template <typename T, int V> struct ConvVec {
    typedef __attribute__((ext_vector_type(V))) T type;
};
template <typename T> struct ConvVec<T, 1> {
    typedef T type;
};

template <typename T, int V>
__device__ __forceinline__ void conv_widen(float (&out)[V], typename ConvVec<T, V>::type x) {
    if constexpr (V == 1) {
        out[0] = to_f32<T>(x);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) out[i] = to_f32<T>((T)x[i]);
    }
}
template <typename T, int V>
__device__ __forceinline__ void conv_load(float (&out)[V], const T* p) {
    conv_widen<T, V>(out, *reinterpret_cast<const typename ConvVec<T, V>::type*>(p));
}

template <typename T, int V, bool STREAM = false>
__device__ __forceinline__ void conv_store(T* p, const float (&in)[V]) {
    typedef typename ConvVec<T, V>::type vec_t;
    if constexpr (V == 1) {
        *p = from_f32<T>(in[0]);
    } else {
        vec_t x;
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = from_f32<T>(in[i]);
        if constexpr (STREAM) __builtin_nontemporal_store(x, reinterpret_cast<vec_t*>(p));
        else *reinterpret_cast<vec_t*>(p) = x;
    }
}

// x sigmoid(x).  The reciprocal and the exponential are the hardware's (about 1 ulp each).
__device__ __forceinline__ float silu_f32(float x) { return x * __builtin_amdgcn_rcpf(1.0f + __expf(-x)); }

// The weights of V channels, tap by tap, and the bias.
template <typename T, int W, int V>
__device__ __forceinline__ void conv_weights(float (&w)[W][V], float (&b)[V], const ConvArgs& a, int d) {
    const T* wp = reinterpret_cast<const T*>(a.w) + (long long)d * W;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][i] = to_f32<T>(wp[i * W + j]);
#pragma unroll
    for (int i = 0; i < V; ++i) b[i] = 0.0f;
    if (a.bias) conv_load<T, V>(b, reinterpret_cast<const T*>(a.bias) + d);
}

}  // namespace

// grid: (channel groups x token tiles / 256, sequences), groups fastest, so that every lane has work whatever
// the width (workgroups of whole tiles, with idle lanes in each tile's last one: 186 us).  STREAM: outputs go past the caches.
template <typename T, int W, int V, bool STREAM>
__global__ __launch_bounds__(kConvThreads) void kda_conv_prefill_kernel(const ConvArgs a) {
    const uint32_t at = blockIdx.x * kConvThreads + threadIdx.x, groups = (uint32_t)(a.D + V - 1) / V, piece = at / groups;
    const int d = (int)(at - piece * groups) * V;
    const int b = blockIdx.y;
    int len = a.T;
    if (a.lens) {
        const int l = a.lens[b];
        len = l < 0 ? 0 : (l > a.T ? a.T : l);
    }
    const long long t0 = (long long)piece * a.tile;
    if (t0 > 0 && t0 >= len) return;
    const long long t1 = t0 + a.tile < len ? t0 + a.tile : len;
    const T* x = reinterpret_cast<const T*>(a.x) + (long long)b * a.T * a.x_stride + d;
    T* y = reinterpret_cast<T*>(a.y) + (long long)b * a.T * a.D + d;
    const T* past = reinterpret_cast<const T*>(a.state_in);
    if (past) past += (long long)b * (W - 1) * a.D + d;

    // h[i] holds input t - (W - 1) + i of the coming token t
    float h[W][V];
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
        const long long r = t0 - (W - 1) + i;
        if (r >= 0) {
            conv_load<T, V>(h[i], x + r * a.x_stride);
        } else if (past) {
            conv_load<T, V>(h[i], past + (long long)(W - 1 + r) * a.D);
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e) h[i][e] = 0.0f;
        }
    }
    // The thread of the first tile also writes the history kept for the next call: it is the only
    // one that reads state_in, so state_out may be state_in itself.  Row i of the new history is
    // row len + i of (history, inputs).
    if (t0 == 0 && a.state_out) {
        float o[W > 1 ? W - 1 : 1][V];
#pragma unroll
        for (int i = 0; i < W - 1; ++i) {
            const int r = len - (W - 1) + i;
            if (r >= 0) {
                conv_load<T, V>(o[i], x + r * a.x_stride);
            } else {
#pragma unroll
                for (int e = 0; e < V; ++e) o[i][e] = 0.0f;
#pragma unroll
                for (int k = 0; k < W - 1; ++k)   // h[W - 1 + r], indexed without a register array lookup
                    if (k == W - 1 + r) {
#pragma unroll
                        for (int e = 0; e < V; ++e) o[i][e] = h[k][e];
                    }
            }
        }
        T* so = reinterpret_cast<T*>(a.state_out) + (long long)b * (W - 1) * a.D + d;
#pragma unroll
        for (int i = 0; i < W - 1; ++i) conv_store<T, V>(so + (long long)i * a.D, o[i]);
    }
    float w[W][V], bias[V];
    conv_weights<T, W, V>(w, bias, a, d);
    // kRows rows are requested together, so that a wave keeps several loads in flight
    constexpr int kRows = 4;
    auto token = [&](T* out) {   // h[0 .. W - 1] end at the token
        float acc[V];
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] = bias[e];
#pragma unroll
        for (int j = 0; j < W; ++j)
#pragma unroll
            for (int e = 0; e < V; ++e) acc[e] = fmaf(w[j][e], h[j][e], acc[e]);
        if (a.silu) {
#pragma unroll
            for (int e = 0; e < V; ++e) acc[e] = silu_f32(acc[e]);
        }
        conv_store<T, V, STREAM>(out, acc);
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
#pragma unroll
            for (int e = 0; e < V; ++e) h[j][e] = h[j + 1][e];
    };
    long long t = t0;
    for (; t + kRows <= t1; t += kRows) {
        typename ConvVec<T, V>::type v[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) v[i] = *reinterpret_cast<const typename ConvVec<T, V>::type*>(x + (t + i) * a.x_stride);
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            conv_widen<T, V>(h[W - 1], v[i]);
            token(y + (t + i) * a.D);
        }
    }
    for (; t < t1; ++t) {
        conv_load<T, V>(h[W - 1], x + t * a.x_stride);
        token(y + t * a.D);
    }
}

// grid: (channel groups / 256, sequences); the history is shifted in place
template <typename T, int W, int V>
__global__ __launch_bounds__(kConvThreads) void kda_conv_step_kernel(const ConvArgs a) {
    const int d = (int)(blockIdx.x * kConvThreads + threadIdx.x) * V;
    const long long n = blockIdx.y;
    if (d >= a.D) return;
    T* s = reinterpret_cast<T*>(a.state_out) + n * (W - 1) * a.D + d;
    float h[W][V];
#pragma unroll
    for (int i = 0; i < W - 1; ++i) conv_load<T, V>(h[i], s + (long long)i * a.D);
    conv_load<T, V>(h[W - 1], reinterpret_cast<const T*>(a.x) + n * a.x_stride + d);
    float w[W][V], acc[V];
    conv_weights<T, W, V>(w, acc, a, d);
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] = fmaf(w[j][e], h[j][e], acc[e]);
    if (a.silu) {
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] = silu_f32(acc[e]);
    }
    conv_store<T, V>(reinterpret_cast<T*>(a.y) + n * a.D + d, acc);
#pragma unroll
    for (int i = 0; i < W - 1; ++i) conv_store<T, V>(s + (long long)i * a.D, h[i + 1]);
}

namespace {

template <typename T, int W, int V>
hipError_t conv_prefill_wv(const ConvArgs& a, hipStream_t s) {
    const long long groups = (a.D + V - 1) / V;
    const long long tiles = a.T > 0 ? ((long long)a.T + a.tile - 1) / a.tile : 1;
    const dim3 grid((unsigned)((groups * tiles + kConvThreads - 1) / kConvThreads), a.B, 1);
    if (V > 1 && a.streamed) kda_conv_prefill_kernel<T, W, V, (V > 1)><<<grid, kConvThreads, 0, s>>>(a);
    else kda_conv_prefill_kernel<T, W, V, false><<<grid, kConvThreads, 0, s>>>(a);
    return hipGetLastError();
}

template <typename T, int W, int V>
hipError_t conv_step_wv(const ConvArgs& a, hipStream_t s) {
    const int groups = (a.D + V - 1) / V;
    const dim3 grid((groups + kConvThreads - 1) / kConvThreads, a.B, 1);
    kda_conv_step_kernel<T, W, V><<<grid, kConvThreads, 0, s>>>(a);
    return hipGetLastError();
}

template <typename T, int W>
hipError_t conv_w(bool step, bool vec, const ConvArgs& a, hipStream_t s) {
    constexpr int V = 16 / (int)sizeof(T);
    if (step) return vec ? conv_step_wv<T, W, V>(a, s) : conv_step_wv<T, W, 1>(a, s);
    return vec ? conv_prefill_wv<T, W, V>(a, s) : conv_prefill_wv<T, W, 1>(a, s);
}

hipError_t conv_any(int W, bool f32, bool step, bool vec, const ConvArgs& a, hipStream_t s) {
    switch (W) {
        case 2: return f32 ? conv_w<float, 2>(step, vec, a, s) : conv_w<__bf16, 2>(step, vec, a, s);
        case 3: return f32 ? conv_w<float, 3>(step, vec, a, s) : conv_w<__bf16, 3>(step, vec, a, s);
        case 4: return f32 ? conv_w<float, 4>(step, vec, a, s) : conv_w<__bf16, 4>(step, vec, a, s);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace

hipError_t launch_conv_prefill(int W, bool f32, bool vec, const ConvArgs& a, hipStream_t s) {
    return conv_any(W, f32, false, vec, a, s);
}
hipError_t launch_conv_step(int W, bool f32, bool vec, const ConvArgs& a, hipStream_t s) {
    return conv_any(W, f32, true, vec, a, s);
}

}  // namespace kda
