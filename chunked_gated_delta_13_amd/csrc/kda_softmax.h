// Pieces shared by the attention kernels: sums and maxima over the lanes of a query, operands straight
// from memory, stores of four outputs.
#pragma once

#include "kda_tile.h"

namespace kda {

// Over the four lanes 16 apart that share a query.  SWAP: rows of 16 lanes are swapped pairwise, then halves,
// on the vector unit; else the values go round through LDS, which takes longer (ragged prompts of the
// smallest kind 11.8 us instead of 11.4, one token 0.3 us more) but leaves the registers of the
// kernel of 32 queries per wave as they are (the swaps make it spill: 2.55 ms instead of 1.59).
template <bool SWAP, typename F> __device__ __forceinline__ float over_groups(float v, F f) {
    if constexpr (SWAP) {
        const uint32_t u = __float_as_uint(v);
        const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
        const uint32_t w = __float_as_uint(f(__uint_as_float(a[0]), __uint_as_float(a[1])));
        const auto b = __builtin_amdgcn_permlane32_swap(w, w, false, false);
        return f(__uint_as_float(b[0]), __uint_as_float(b[1]));
    } else {
        v = f(v, __shfl_xor(v, 16));
        return f(v, __shfl_xor(v, 32));
    }
}
template <bool SWAP> __device__ __forceinline__ float max_over_groups(float v) {
    return over_groups<SWAP>(v, [](float x, float y) { return fmaxf(x, y); });
}
template <bool SWAP> __device__ __forceinline__ float sum_over_groups(float v) {
    return over_groups<SWAP>(v, [](float x, float y) { return x + y; });
}

// Eight slots of one row in global memory, p at the first one: four at p and four half a row further.
template <int D> __device__ __forceinline__ void global_frag(Frag<__bf16>& f, const __bf16* p) {
    frag_join(f, *reinterpret_cast<const bf16x4_t*>(p), *reinterpret_cast<const bf16x4_t*>(p + D / 2));
}
template <int D> __device__ __forceinline__ void global_frag(Frag<float>& f, const float* p) {
    frag_join(f, *reinterpret_cast<const f32x4_t*>(p), *reinterpret_cast<const f32x4_t*>(p + D / 2));
}
// Eight consecutive elements of one row (slot order 8g .. 8g + 7; both operands use it).
__device__ __forceinline__ void global_frag8(Frag<__bf16>& f, const __bf16* p) {
    f.v = *reinterpret_cast<const bf16x8_t*>(p);
}
__device__ __forceinline__ void global_frag8(Frag<float>& f, const float* p) {
    const f32x4_t lo = *reinterpret_cast<const f32x4_t*>(p);
    const f32x4_t hi = *reinterpret_cast<const f32x4_t*>(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f.v[i] = lo[i];
        f.v[4 + i] = hi[i];
    }
}

// LDS accesses of one wave run in program order; this keeps the compiler from reordering them.
__device__ __forceinline__ void wave_order() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
}

template <typename T> __device__ __forceinline__ void store4(T* p, const f32x4_t& v) {
    typedef __attribute__((ext_vector_type(4))) T vec4;
    vec4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = from_f32<T>(v[i]);
    *reinterpret_cast<vec4*>(p) = o;
}

// Joins n partial outputs of one row: part i's output lies at o + i step D, its maximum (base 2) and sum at ml + 2 i step.  Of
// the workgroup's threads D / 4 own four channels of a part, and groups of as many take parts side by side.
template <int D, typename T, int THREADS>
__device__ __forceinline__ void join_parts(const float* ml, const float* o, int n, long long step, T* out) {
    constexpr int NL = D / 4, NS = THREADS / NL;
    const int tid = threadIdx.x, d = (tid % NL) * 4, i0 = tid / NL;
    o += d;
    // every group keeps a maximum of its own parts
    float M = -INFINITY, L = 0.0f;
    f32x4_t v = zero4();
#pragma unroll 8
    for (int i = i0; i < n; i += NS) {
        const float m = ml[2 * (long long)i * step], l = ml[2 * (long long)i * step + 1];
        const f32x4_t x = *reinterpret_cast<const f32x4_t*>(o + (long long)i * step * D);
        const float top = fmaxf(M, m), base = top == -INFINITY ? 0.0f : top;
        const float f = fast_exp2(M - base), e = fast_exp2(m - base);
        M = top;
        L = fmaf(L, f, e * l);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = fmaf(v[j], f, e * x[j]);
    }
    __shared__ float sM[NS], sL[NS];
    __shared__ __attribute__((aligned(16))) float sv[NS][D];
    *reinterpret_cast<f32x4_t*>(&sv[i0][d]) = v;
    if (d == 0) {
        sM[i0] = M;
        sL[i0] = L;
    }
    __syncthreads();
    if (tid >= NL) return;
    M = -INFINITY;
#pragma unroll
    for (int i = 0; i < NS; ++i) M = fmaxf(M, sM[i]);
    const float base = M == -INFINITY ? 0.0f : M;
    L = 0.0f;
    v = zero4();
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        const float f = fast_exp2(sM[i] - base);
        L = fmaf(f, sL[i], L);
        const f32x4_t x = *reinterpret_cast<const f32x4_t*>(&sv[i][d]);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = fmaf(f, x[j], v[j]);
    }
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] *= inv;
    store4<T>(out + d, v);
}

}  // namespace kda
