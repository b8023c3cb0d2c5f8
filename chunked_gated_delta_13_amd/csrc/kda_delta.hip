// The gated delta rule with one decay per head and token, for gfx950: prompts in chunks, and single tokens.
//
// Per sequence and head, with a state S (dk x dv, fp32), a_t = e^(g_t), and key heads shared by groups of value heads:
//     S <- a_t S + beta_t k_t (v_t - a_t S^T k_t)^T,    o_t = S^T q_t          read after the write
//
// Chunks of C tokens.  With c_i the sum of the exponents (base 2) up to token i of the chunk and S0 its entry state:
//     A_ij = beta_i 2^(c_i - c_j) (k_i . k_j)  for j < i,     T = (I + A)^-1
//     R = diag(beta) (V - diag(2^c) K S0),     U = T R
//     O = diag(2^c) Q S0 + B U,                B_ij = 2^(c_i - c_j) (q_i . k_j)  for j <= i
//     S <- 2^(c_C) S0 + K^T diag(2^(c_C - c_j)) U
// With one decay per token the differences of exponents are formed directly, never above 0 for decays: nothing has to be
// scaled apart and together again.  T is formed by 16 x 16 blocks in fp32.
//
// Numerics.  bf16 keys and queries are exact operands.  On the state's path S, T, R and U enter the products as three
// bf16 parts (24 bits; the six products of two such factors above 2^-24 are formed), so that states are as exact as with
// fp32 operands, at three to six bf16 products instead of the sixteen that one in fp32 takes.  The outputs, rounded to
// bf16 anyway, take S in one part, U in two and B in one.  fp32 inputs use fp32 products throughout.
#include "kda_mixers.h"
#include "kda_tile.h"

namespace kda {

namespace {

// The inputs' types: tokens of a chunk, parts of a factor on the state's path.
template <typename T> struct DeltaTraits;
template <> struct DeltaTraits<__bf16> { static constexpr int C = 64, NP = 3; };
template <> struct DeltaTraits<float> { static constexpr int C = 32, NP = 1; };

constexpr float kLeastExponent = -160.0f;   // 2^-160 of any state is below fp32's range: the same as nothing

// Straight from memory to LDS, 16 bytes a lane, without the compiler's waits (see barrier_all): it would wait for
// every such request before the next read of LDS.  `lds` is uniform.
__device__ __forceinline__ void dma16(const void* src, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(src), "s"(lds) : "memory");
}
__device__ __forceinline__ uint32_t lds_address(const void KDA_LDS* p) { return (uint32_t)(size_t)p; }

// An operand kept as the wave holds it: 8 elements a lane, lane after lane.
template <typename T> __device__ __forceinline__ void frag_get(Frag<T>& f, const KDA_LDS T* p) {
    typedef typename Vec4<T>::type vec4;
    frag_join(f, *reinterpret_cast<const KDA_LDS vec4*>(p), *reinterpret_cast<const KDA_LDS vec4*>(p + 4));
}
template <> __device__ __forceinline__ void frag_get(Frag<__bf16>& f, const KDA_LDS __bf16* p) {
    f.v = *reinterpret_cast<const KDA_LDS bf16x8_t*>(p);
}

// Two stacked accumulator tiles as an operand in NP parts, the first one largest.
template <typename T, int NP> __device__ __forceinline__ void parts_of(Frag<T> (&f)[NP], f32x4_t lo, f32x4_t hi) {
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        acc_pair_frag<T>(f[p], lo, hi, true);
        if (p + 1 < NP) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                lo[j] -= f[p].get(j);
                hi[j] -= f[p].get(4 + j);
            }
        }
    }
}

// acc + a b for factors in parts: the products above 2^-24, the smallest first.
template <typename T, int NP>
__device__ __forceinline__ f32x4_t mma_parts(const Frag<T> (&a)[NP], const Frag<T> (&b)[NP], f32x4_t c) {
#pragma unroll
    for (int s = NP - 1; s >= 0; --s)
#pragma unroll
        for (int p = 0; p <= s; ++p) c = mma(a[p], b[s - p], c);
    return c;
}

// A 16 x 16 by 16 x 16 product in fp32: slots 4 g + j of either operand.
__device__ __forceinline__ f32x4_t mma16(f32x4_t a, f32x4_t b, f32x4_t c) {
#pragma unroll
    for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[j], b[j], c, 0, 0, 0);
    return c;
}

__device__ __forceinline__ double shfl_up_f64(double x, int s) {
    const unsigned long long u = __builtin_bit_cast(unsigned long long, x);
    const uint32_t lo = __shfl_up((uint32_t)u, s), hi = __shfl_up((uint32_t)(u >> 32), s);
    return __builtin_bit_cast(double, (unsigned long long)hi << 32 | lo);
}
__device__ __forceinline__ double lane_f64(double x, int lane) {
    const unsigned long long u = __builtin_bit_cast(unsigned long long, x);
    const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)u, lane), hi = __builtin_amdgcn_readlane((uint32_t)(u >> 32), lane);
    return __builtin_bit_cast(double, (unsigned long long)hi << 32 | lo);
}

template <typename T> __device__ __forceinline__ void store4_t(T* p, const f32x4_t& v) {
    typename Vec4<T>::type o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = from_f32<T>(v[i]);
    *reinterpret_cast<typename Vec4<T>::type*>(p) = o;
}

}  // namespace

// Prompt.  A workgroup runs one (sequence, head, segment, slice of 64 NCT state columns) with two roles: four state
// waves hold the slice (16 NCT columns each, fp32, in the accumulators' layout) and run chunk c; four chunk waves
// prepare what chunk c + 1 needs and does not depend on the state.  A SIMD hosts one of each.  Three workgroup barriers a
// chunk:
//     interval   state waves, chunk c             chunk waves, chunk n = c + 1
//     1          X = K S0, Q S0                   A (fp32), B
//     2          R, U = T R                       inverses of A's diagonal blocks; K and Q of n + 1 requested
//     3          V of c + 1 requested; O, S       T by blocks, row by row; exponents of n + 1
// K has three buffers (chunks c, n and the one in flight), Q, B and the exponents' tables two or three, T and V one: each is
// overwritten only in an interval after its last reader's.
//
// OUT: outputs are formed (else only states).
template <typename T, int DK, int NCT, bool OUT>
__global__ __launch_bounds__(512) void kda_delta_prefill_kernel(const DeltaArgs a) {
    constexpr int C = DeltaTraits<T>::C, NP = DeltaTraits<T>::NP, NA = C / 16, NQ = C / 32;   // token tiles, pairs of them
    constexpr int NT = DK / 16, NKB = DK / 32, DVS = 64 * NCT;
    constexpr int KT = C * DK, VT = C * DVS;                     // elements of a tile
    constexpr int NF = NQ * (NQ + 1);                            // operands of a lower triangle
    constexpr int FR = 64 * 8;                                   // elements of an operand
    constexpr int ARR = 5 * C + 16;                              // exponents (high, low parts), 2^c, 2^(c_C - c), beta, 2^c_C
    constexpr int NLOW = NA * (NA - 1) / 2;
    struct Shared {
        T k[3][KT], q[OUT ? 2 : 1][KT], v[VT];
        T t[NP][NF * FR], b[2][OUT ? NF * FR : 8];
        float low[NLOW * 256], diag[NA * 256], rows[NA * 256];   // A below the diagonal; its diagonal blocks, then T's by columns; T's by rows
        float arr[3][ARR];
    };
    static_assert(sizeof(Shared) <= 160 * 1024, "LDS of a compute unit");
    __shared__ __attribute__((aligned(16))) Shared sh_;
    KDA_LDS Shared* sh = (KDA_LDS Shared*)&sh_;
    auto frag_at = [](int i, int q) { return (i / 2) * (i / 2 + 1) + (i & 1) * (i / 2 + 1) + q; };   // of token tile i, pair q

    // unit = (sequence, head, segment, slice): consecutive units share keys, and an XCD takes a contiguous range
    uint32_t unit = (blockIdx.x & 7) * (uint32_t)a.per_xcd + (blockIdx.x >> 3);
    if (unit >= (uint32_t)a.n_units) return;
    const int slices = a.slices + a.id_slices;
    int slice = (int)(unit % (uint32_t)slices);
    unit /= (uint32_t)slices;
    const int seg = (int)(unit % (uint32_t)a.n_seg_launch);
    unit /= (uint32_t)a.n_seg_launch;
    const int h = (int)(unit % (uint32_t)a.H), b = (int)(unit / (uint32_t)a.H), hk = h / (a.H / a.Hk);
    const long long bh = (long long)b * a.H + h;
    const bool ident = slice >= a.slices;   // the transition's columns: from the identity, without values
    if (ident) slice -= a.slices;

    long long len = a.T;
    if (a.lens) {
        const int l = a.lens[b];
        len = l < 0 ? 0 : (l > a.T ? a.T : l);
    }
    const long long begin = seg * a.seg_len;
    long long todo = len - begin;           // tokens of this unit
    todo = todo < 0 ? 0 : (todo < a.seg_len ? todo : a.seg_len);
    const int nc = (int)((todo + C - 1) / C);

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, r = lane & 15;

    // Rows of one tile from memory: step i of `steps` covers 1 KB; rows past the unit's take its last one (finite, and of
    // no weight: their beta is 0).
    auto fetch = [&](const T* base, long long stride, int chunk, KDA_LDS T* tile, int i, int nb) {
        const int group = i / nb, block = i % nb;
        const int row16 = group * TileStep<T>::ROWS + TileStep<T>::row(lane);
        const long long at = (long long)chunk * C + row16, row = at < todo ? at : todo - 1;
        const T* p = base + row * stride + tile_dma_piece<T>(row16, lane) * TileStep<T>::ELEMS + 32 * block;
        dma16(p, lds_address(tile + block * C * 32 + group * TileStep<T>::ROWS * 32));
    };
    constexpr int GROUPS = C / TileStep<T>::ROWS;
    const long long tok0 = (long long)b * a.T + begin;

    if (wave < 4) {
        // ------------------------------------------------------------------------------------------ state waves
        const T* vp = reinterpret_cast<const T*>(a.v) + tok0 * a.v_stride + (long long)h * a.dv + slice * DVS;
        constexpr int VSTEPS = GROUPS * (DVS / 32) / 4;
        auto fetch_v = [&](int chunk) {
            if (ident) return;
#pragma unroll
            for (int i = 0; i < VSTEPS; ++i) fetch(vp, a.v_stride, chunk, sh->v, wave * VSTEPS + i, DVS / 32);
        };
        if (nc > 0) fetch_v(0);

        const int col = slice * DVS + wave * 16 * NCT + r;   // this lane's column of tile 0
        const int width = ident ? DK : a.dv;
        f32x4_t S[NT][NCT];
        const float* s_in = ident ? nullptr : (a.S_in ? a.S_in + bh * a.sin_bh + seg * a.sin_seg : nullptr);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int c = 0; c < NCT; ++c)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int row = 16 * t + 4 * g + j;
                    S[t][c][j] = s_in ? s_in[(long long)row * width + col + 16 * c] : (ident && row == col + 16 * c ? 1.0f : 0.0f);
                }
        TileRows<T, C, DK> rk, rq;
        TileCols<T, C> ck, cvt[NCT];
        rk.set(sh->k[0], lane);
        rq.set(sh->q[0], lane);
        ck.set(sh->k[0], lane);
#pragma unroll
        for (int c = 0; c < NCT; ++c) cvt[c].set_tile(sh->v, lane, wave * NCT + c);
        const KDA_LDS T* tf = lds_pin(&sh->t[0][0] + lane * 8);

        barrier_all();
        if (nc > 0) {
            barrier_lds();
            barrier_lds();
            barrier_lds();
        }
        T* op = OUT ? reinterpret_cast<T*>(a.o) + (tok0 * a.H + h) * a.dv + slice * DVS + wave * 16 * NCT + 4 * g : nullptr;
        for (int n = 0; n < nc; ++n) {
            const int kb3 = n % 3;
            const TileRows<T, C, DK> k_rows = rk.at_delta(kb3 * KT);
            const TileRows<T, C, DK> q_rows = rq.at_delta((OUT ? n & 1 : 0) * KT);
            const KDA_LDS float* arr = &sh->arr[kb3][0];

            // 1: X = K S0 and (transposed) S0^T Q^T, contraction block by contraction block
            f32x4_t X[NA][NCT], O[NA][NCT];
#pragma unroll
            for (int i = 0; i < NA; ++i)
#pragma unroll
                for (int c = 0; c < NCT; ++c) X[i][c] = O[i][c] = zero4();
#pragma unroll
            for (int kb = 0; kb < NKB; ++kb) {
                Frag<T> s[NCT][NP];
#pragma unroll
                for (int c = 0; c < NCT; ++c) parts_of<T, NP>(s[c], S[kb][c], S[kb + NKB][c]);
#pragma unroll
                for (int i = 0; i < NA; ++i) {
                    Frag<T> f;
                    k_rows.frag(f, 0, i, kb);
#pragma unroll
                    for (int p = NP - 1; p >= 0; --p)
#pragma unroll
                        for (int c = 0; c < NCT; ++c) X[i][c] = mma(f, s[c][p], X[i][c]);
                    if constexpr (OUT) {
                        q_rows.frag(f, 0, i, kb);
#pragma unroll
                        for (int c = 0; c < NCT; ++c) O[i][c] = mma(s[c][0], f, O[i][c]);
                    }
                }
            }
            barrier_all();   // (V has arrived, for every wave)

            // 2: R = beta (V - 2^c X) in X's place, then U = T R
#pragma unroll
            for (int q = 0; q < NQ; ++q)
#pragma unroll
                for (int c = 0; c < NCT; ++c) {
                    Frag<T> v;
                    if (!ident) cvt[c].frag(v, 0, 0, q);
                    else v.zero();
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int i = q + x * NQ;
                        const f32x4_t grow = *reinterpret_cast<const KDA_LDS f32x4_t*>(arr + 2 * C + 16 * i + 4 * g);
                        const f32x4_t beta = *reinterpret_cast<const KDA_LDS f32x4_t*>(arr + 4 * C + 16 * i + 4 * g);
#pragma unroll
                        for (int j = 0; j < 4; ++j) X[i][c][j] = beta[j] * fmaf(-grow[j], X[i][c][j], v.get(4 * x + j));
                    }
                }
            f32x4_t U[NA][NCT];
#pragma unroll
            for (int i = 0; i < NA; ++i)
#pragma unroll
                for (int c = 0; c < NCT; ++c) U[i][c] = zero4();
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
                Frag<T> rr[NCT][NP];
#pragma unroll
                for (int c = 0; c < NCT; ++c) parts_of<T, NP>(rr[c], X[2 * q][c], X[2 * q + 1][c]);
#pragma unroll
                for (int i = 2 * q; i < NA; ++i) {
                    Frag<T> tt[NP];
#pragma unroll
                    for (int p = 0; p < NP; ++p) frag_get<T>(tt[p], tf + (p * NF + frag_at(i, q)) * FR);
#pragma unroll
                    for (int c = 0; c < NCT; ++c) U[i][c] = mma_parts<T, NP>(tt, rr[c], U[i][c]);
                }
            }
            barrier_lds();

            // 3: outputs, then the state
            if (n + 1 < nc) fetch_v(n + 1);
            if constexpr (OUT) {
                const KDA_LDS T* bf = lds_pin(&sh->b[n & 1][0] + lane * 8);
#pragma unroll
                for (int i = 0; i < NA; ++i) {
                    const float grow = arr[2 * C + 16 * i + r];
#pragma unroll
                    for (int c = 0; c < NCT; ++c)
#pragma unroll
                        for (int j = 0; j < 4; ++j) O[i][c][j] *= grow;
                }
                constexpr int UP = NP > 1 ? 2 : 1;
#pragma unroll
                for (int q = 0; q < NQ; ++q) {
                    Frag<T> uu[NCT][UP];
#pragma unroll
                    for (int c = 0; c < NCT; ++c) parts_of<T, UP>(uu[c], U[2 * q][c], U[2 * q + 1][c]);
#pragma unroll
                    for (int i = 2 * q; i < NA; ++i) {
                        Frag<T> f;
                        frag_get<T>(f, bf + frag_at(i, q) * FR);
#pragma unroll
                        for (int p = UP - 1; p >= 0; --p)
#pragma unroll
                            for (int c = 0; c < NCT; ++c) O[i][c] = mma(uu[c][p], f, O[i][c]);
                    }
                }
#pragma unroll
                for (int i = 0; i < NA; ++i) {
                    const long long at = (long long)n * C + 16 * i + r;
                    if (at < todo) {
#pragma unroll
                        for (int c = 0; c < NCT; ++c) store4_t<T>(op + at * a.H * a.dv + 16 * c, O[i][c]);
                    }
                }
            }
            const float dec = arr[5 * C];
#pragma unroll
            for (int i = 0; i < NA; ++i) {
                const f32x4_t late = *reinterpret_cast<const KDA_LDS f32x4_t*>(arr + 3 * C + 16 * i + 4 * g);
#pragma unroll
                for (int c = 0; c < NCT; ++c)
#pragma unroll
                    for (int j = 0; j < 4; ++j) U[i][c][j] *= late[j];
            }
            const TileCols<T, C> k_cols = ck.at_delta(kb3 * KT);
            Frag<T> uu[NQ][NCT][NP];
#pragma unroll
            for (int q = 0; q < NQ; ++q)
#pragma unroll
                for (int c = 0; c < NCT; ++c) parts_of<T, NP>(uu[q][c], U[q][c], U[q + NQ][c]);
            // (a chunk's sum starts from zero and joins the decayed state with one rounding)
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                f32x4_t add[NCT];
#pragma unroll
                for (int c = 0; c < NCT; ++c) add[c] = zero4();
#pragma unroll
                for (int q = 0; q < NQ; ++q) {
                    Frag<T> f;
                    k_cols.frag(f, 0, t, q);
#pragma unroll
                    for (int p = NP - 1; p >= 0; --p)
#pragma unroll
                        for (int c = 0; c < NCT; ++c) add[c] = mma(f, uu[q][c][p], add[c]);
                }
#pragma unroll
                for (int c = 0; c < NCT; ++c)
#pragma unroll
                    for (int j = 0; j < 4; ++j) S[t][c][j] = fmaf(S[t][c][j], dec, add[c][j]);
            }
            barrier_lds();
        }
        float* s_out = ident ? a.M_out + (bh * a.m_bh + seg) * (long long)(DK * DK)
                             : (a.S_out && (a.out_seg < 0 || a.out_seg == seg) ? a.S_out + bh * a.sout_bh + (a.out_seg < 0 ? seg : 0) * a.sout_seg : nullptr);
        if (s_out) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int c = 0; c < NCT; ++c)
#pragma unroll
                    for (int j = 0; j < 4; ++j) s_out[(long long)(16 * t + 4 * g + j) * width + col + 16 * c] = S[t][c][j];
        }
        return;
    }

    // ---------------------------------------------------------------------------------------------- chunk waves
    const int cw = wave - 4;
    const T* kp = reinterpret_cast<const T*>(a.k) + tok0 * a.k_stride + (long long)hk * DK;
    const T* qp = reinterpret_cast<const T*>(a.q) + tok0 * a.q_stride + (long long)hk * DK;
    constexpr int KSTEPS = GROUPS * NKB / 4;
    auto fetch_kq = [&](int chunk) {
#pragma unroll
        for (int i = 0; i < KSTEPS; ++i) fetch(kp, a.k_stride, chunk, sh->k[chunk % 3], cw * KSTEPS + i, NKB);
        if constexpr (OUT) {
#pragma unroll
            for (int i = 0; i < KSTEPS; ++i) fetch(qp, a.q_stride, chunk, sh->q[chunk & 1], cw * KSTEPS + i, NKB);
        }
    };
    // exponents and beta of a chunk's tokens, one a lane (wave 0)
    float g_next = 0.0f, beta_next = 0.0f;
    auto request_arr = [&](int chunk) {
        const long long at = (long long)chunk * C + lane;
        const bool there = lane < C && at < todo;
        g_next = there ? a.g[(tok0 + at) * a.H + h] : 0.0f;
        beta_next = there ? a.beta[(tok0 + at) * a.H + h] : 0.0f;
    };
    auto put_arr = [&](int chunk) {
        // sums in 64 bits: the decay between two tokens is the difference of two of them
        double e = (double)g_next * 1.4426950408889634;
        if (e < (double)kLeastExponent) e = (double)kLeastExponent;
#pragma unroll
        for (int s = 1; s < C; s <<= 1) {
            const double y = shfl_up_f64(e, s);
            if (lane >= s) e += y;
        }
        const double all = lane_f64(e, C - 1);
        KDA_LDS float* arr = &sh->arr[chunk % 3][0];
        if (lane < C) {
            const float hi = (float)e;
            arr[lane] = hi;
            arr[C + lane] = (float)(e - (double)hi);
            arr[2 * C + lane] = fast_exp2(hi);
            arr[3 * C + lane] = fast_exp2((float)(all - e));
            arr[4 * C + lane] = beta_next;
            if (lane == 0) arr[5 * C] = fast_exp2((float)all);
        }
    };
    TileRows<T, C, DK> rk, rq;
    rk.set(sh->k[0], lane);
    rq.set(sh->q[0], lane);

    if (nc > 0) {
        fetch_kq(0);
        if (cw == 0) {
            request_arr(0);
            put_arr(0);
        }
        // the halves of operands that lie above the diagonal stay zero
        for (int i = tid - 256; i < NP * NF * FR; i += 256) (&sh->t[0][0])[i] = (T)0.0f;
        if constexpr (OUT)
            for (int i = tid - 256; i < 2 * NF * FR; i += 256) (&sh->b[0][0])[i] = (T)0.0f;
    }
    barrier_all();
    for (int n = 0; n < nc; ++n) {
        const bool more = n + 1 < nc;
        if (cw == 0 && more) request_arr(n + 1);
        const KDA_LDS float* arr = &sh->arr[n % 3][0];
        // 1: tiles of K K^T (rows by block of rows i, columns by j) and of K Q^T (the transposed ones)
        const TileRows<T, C, DK> k_rows = rk.at_delta((n % 3) * KT);
        const TileRows<T, C, DK> q_rows = rq.at_delta((OUT ? n & 1 : 0) * KT);
        static_for<0, (NA * (NA + 1) / 2 + 3) / 4>([&](auto step) {
            const int idx = decltype(step)::value * 4 + cw;
            int i = 0, j = idx;   // (wave-uniform)
            while (j > i) j -= ++i;
            if (i >= NA) return;
            const KDA_LDS float* ai = arr + 16 * i;
            const KDA_LDS float* aj = arr + 16 * j;
            const TileRows<T, C, DK> ki = k_rows.at_delta(16 * 32 * i), kj = k_rows.at_delta(16 * 32 * j), qi = q_rows.at_delta(16 * 32 * i);
            f32x4_t G = zero4(), P = zero4();
#pragma unroll
            for (int kb = 0; kb < NKB; ++kb) {
                Frag<T> x, y;
                ki.frag(x, 0, 0, kb);
                kj.frag(y, 0, 0, kb);
                G = mma(x, y, G);
                if constexpr (OUT) {
                    qi.frag(x, 0, 0, kb);
                    P = mma(y, x, P);
                }
            }
            {   // rows 4 g .. of block i, column r of block j
                const f32x4_t hi = *reinterpret_cast<const KDA_LDS f32x4_t*>(ai + 4 * g), lo = *reinterpret_cast<const KDA_LDS f32x4_t*>(ai + C + 4 * g);
                const f32x4_t beta = *reinterpret_cast<const KDA_LDS f32x4_t*>(ai + 4 * C + 4 * g);
                const float hj = aj[r], lj = aj[C + r];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const float w = fast_exp2((hi[x] - hj) + (lo[x] - lj));
                    G[x] = i == j && r >= 4 * g + x ? 0.0f : beta[x] * w * G[x];
                }
                KDA_LDS float* to = (i == j ? &sh->diag[i * 256] : &sh->low[(i * (i - 1) / 2 + j) * 256]) + lane * 4;
                *reinterpret_cast<KDA_LDS f32x4_t*>(to) = G;
            }
            if constexpr (OUT) {   // row r of block i, columns 4 g .. of block j
                const f32x4_t hi = *reinterpret_cast<const KDA_LDS f32x4_t*>(aj + 4 * g), lo = *reinterpret_cast<const KDA_LDS f32x4_t*>(aj + C + 4 * g);
                const float hj = ai[r], lj = ai[C + r];
                typename Vec4<T>::type o;
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const float w = fast_exp2((hj - hi[x]) + (lj - lo[x]));
                    o[x] = from_f32<T>(i == j && 4 * g + x > r ? 0.0f : w * P[x]);
                }
                *reinterpret_cast<KDA_LDS typename Vec4<T>::type*>(&sh->b[n & 1][frag_at(i, j >> 1) * FR + lane * 8 + (j & 1) * 4]) = o;
            }
        });
        barrier_lds();

        // 2: (I + A_ii)^-1 of all diagonal blocks at once, a block per 16 lanes, a column per lane
        if (more) fetch_kq(n + 1);
        if (cw == 0) {
            const int blk = g < NA ? g : 0;
            const KDA_LDS float* L = &sh->diag[blk * 256];
            f32x4_t x[4];
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i >> 2][i & 3] = i == r ? 1.0f : 0.0f;
#pragma unroll
            for (int j = 0; j < 15; ++j) {
                const float xj = x[j >> 2][j & 3];
#pragma unroll
                for (int y = (j + 1) >> 2; y < 4; ++y) {
                    const f32x4_t l = *reinterpret_cast<const KDA_LDS f32x4_t*>(L + (16 * y + j) * 4);   // rows 4 y .. of column j
#pragma unroll
                    for (int z = 0; z < 4; ++z)
                        if (4 * y + z > j) x[y][z] = fmaf(-l[z], xj, x[y][z]);
                }
            }
            if (g < NA) {
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    *reinterpret_cast<KDA_LDS f32x4_t*>(&sh->diag[g * 256 + (16 * y + r) * 4]) = x[y];   // rows 4 y .. of column r
#pragma unroll
                    for (int z = 0; z < 4; ++z) sh->rows[g * 256 + (16 * (r >> 2) + 4 * y + z) * 4 + (r & 3)] = x[y][z];
                }
            }
        }
        barrier_lds();

        // 3: T_ij = -(sum_{j < m <= i} T_im A_mj) T_jj, transposed, from the diagonal outwards; wave i has row i
        static_for<0, NA>([&](auto row) {
            constexpr int I = decltype(row)::value;
            if (cw != I) return;
            f32x4_t t[I + 1];
            t[I] = *reinterpret_cast<const KDA_LDS f32x4_t*>(&sh->rows[I * 256 + lane * 4]);
#pragma unroll
            for (int j = I - 1; j >= 0; --j) {
                f32x4_t s = zero4();
#pragma unroll
                for (int m = I; m > j; --m) s = mma16(*reinterpret_cast<const KDA_LDS f32x4_t*>(&sh->low[(m * (m - 1) / 2 + j) * 256 + lane * 4]), t[m], s);
                s = mma16(*reinterpret_cast<const KDA_LDS f32x4_t*>(&sh->diag[j * 256 + lane * 4]), s, zero4());
#pragma unroll
                for (int x = 0; x < 4; ++x) t[j][x] = -s[x];
            }
#pragma unroll
            for (int j = 0; j <= I; ++j) {
                f32x4_t v = t[j];
#pragma unroll
                for (int p = 0; p < NP; ++p) {
                    typename Vec4<T>::type o;
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        o[x] = from_f32<T>(v[x]);
                        v[x] -= to_f32<T>(o[x]);
                    }
                    *reinterpret_cast<KDA_LDS typename Vec4<T>::type*>(&sh->t[p][frag_at(I, j >> 1) * FR + lane * 8 + (j & 1) * 4]) = o;
                }
            }
        });
        if (cw == 0 && more) put_arr(n + 1);
        barrier_all();   // (K and Q of n + 1 have arrived)
    }
    if (nc > 0) {
        barrier_lds();
        barrier_lds();
        barrier_lds();
    }
}

// Entry states of a split's segments: S_in(s + 1) = M_s S_in(s) + H_s in fp32.  H lies in the place of S_in(s + 1); M_s
// is dk x dk.  A workgroup owns 16 columns of one (sequence, head), in LDS; a thread sums a row's part of them.
template <int DK>
__global__ __launch_bounds__(256) void kda_delta_join_kernel(const float* M, const float* S0, float* S_in, int n_seg, int dv) {
    constexpr int TPR = 256 / DK, CPT = 16 / TPR;   // threads of a row, columns of a thread
    const long long bh = blockIdx.x;
    const int row = threadIdx.x / TPR, c0 = (threadIdx.x % TPR) * CPT, col = blockIdx.y * 16 + c0;
    __shared__ __attribute__((aligned(16))) float cur[DK][16];
    float* at = S_in + bh * n_seg * (long long)(DK * dv) + (long long)row * dv + col;
    const float* m = M + bh * (n_seg - 1) * (long long)(DK * DK) + (long long)row * DK;
    f32x4_t s[CPT / 4];
#pragma unroll
    for (int x = 0; x < CPT / 4; ++x)
        s[x] = S0 ? *reinterpret_cast<const f32x4_t*>(S0 + (bh * DK + row) * dv + col + 4 * x) : zero4();
    for (int seg = 0; seg < n_seg; ++seg) {
#pragma unroll
        for (int x = 0; x < CPT / 4; ++x) {
            if (seg == 0) *reinterpret_cast<f32x4_t*>(at + 4 * x) = s[x];
            *reinterpret_cast<f32x4_t*>(&cur[row][c0 + 4 * x]) = s[x];
        }
        __syncthreads();
        if (seg + 1 < n_seg) {
            at += (long long)DK * dv;
#pragma unroll
            for (int x = 0; x < CPT / 4; ++x) s[x] = *reinterpret_cast<const f32x4_t*>(at + 4 * x);
#pragma unroll 4
            for (int k = 0; k < DK; k += 4) {
                const f32x4_t w = *reinterpret_cast<const f32x4_t*>(m + k);
#pragma unroll
                for (int y = 0; y < 4; ++y)
#pragma unroll
                    for (int x = 0; x < CPT / 4; ++x) {
                        const f32x4_t v = *reinterpret_cast<const f32x4_t*>(&cur[k + y][c0 + 4 * x]);
#pragma unroll
                        for (int j = 0; j < 4; ++j) s[x][j] = fmaf(w[y], v[j], s[x][j]);
                    }
            }
#pragma unroll
            for (int x = 0; x < CPT / 4; ++x) *reinterpret_cast<f32x4_t*>(at + 4 * x) = s[x];
            m += DK * DK;
        }
        __syncthreads();
    }
}

// One token, bound by HBM (about 7 flops per 8 bytes of state moved): one streaming pass over the state without matrix
// products.  With p = S^T k and r = S^T q of the old state:
//     u = beta (v - a p),     S <- a S + k u^T,     o = a r + (k . q) u
// A workgroup owns one (sequence, head): dv / 4 column groups of four (a state's row is one contiguous run) x 16 row
// groups, and takes states so that an XCD streams one contiguous range of them.
template <int DK, int DV, typename T>
__global__ __launch_bounds__(4 * DV) void kda_delta_step_kernel(const DeltaArgs a) {
    constexpr int NCG = DV / 4, NRG = 16, NW = NCG * NRG / 64, RPT = DK / NRG;
    const long long nh = (long long)(blockIdx.x & 7) * a.per_xcd + (blockIdx.x >> 3);
    if (nh >= a.n_units) return;
    const int n = (int)(nh / a.H), h = (int)(nh % a.H), hk = h / (a.H / a.Hk);
    const int tid = threadIdx.x, cg = tid % NCG, rg = tid / NCG, lane = tid & 63, wave = tid >> 6, col = 4 * cg;

    float* Sp = a.S_out + nh * (long long)(DK * DV) + (long long)rg * DV + col;
    f32x4_t s[RPT];
#pragma unroll
    for (int m = 0; m < RPT; ++m) s[m] = __builtin_nontemporal_load(reinterpret_cast<const f32x4_t*>(Sp + (long long)(NRG * m) * DV));
    const T* kp = reinterpret_cast<const T*>(a.k) + n * a.k_stride + (long long)hk * DK + rg;
    const T* qp = reinterpret_cast<const T*>(a.q) + n * a.q_stride + (long long)hk * DK + rg;
    const T* vp = reinterpret_cast<const T*>(a.v) + n * a.v_stride + (long long)h * DV + col;
    float kk[RPT], qq[RPT];
#pragma unroll
    for (int m = 0; m < RPT; ++m) {
        kk[m] = to_f32<T>(kp[NRG * m]);
        qq[m] = to_f32<T>(qp[NRG * m]);
    }
    const typename Vec4<T>::type vv = *reinterpret_cast<const typename Vec4<T>::type*>(vp);
    const float al = fast_exp2(a.g[nh] * kLog2e), beta = a.beta[nh];

    f32x4_t p = zero4(), q = zero4();
    float kq = 0.0f;
#pragma unroll
    for (int m = 0; m < RPT; ++m) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            p[j] = fmaf(s[m][j], kk[m], p[j]);
            q[j] = fmaf(s[m][j], qq[m], q[j]);
        }
        kq = fmaf(kk[m], qq[m], kq);
    }
#pragma unroll
    for (int x = NCG; x < 64; x <<= 1) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            p[j] += __shfl_xor(p[j], x);
            q[j] += __shfl_xor(q[j], x);
        }
        kq += __shfl_xor(kq, x);
    }
    __shared__ __attribute__((aligned(16))) float part[NW][2 * DV + 4];
    if (lane < NCG) {
        *reinterpret_cast<f32x4_t*>(&part[wave][col]) = p;
        *reinterpret_cast<f32x4_t*>(&part[wave][DV + col]) = q;
    }
    if (lane == 0) part[wave][2 * DV] = kq;
    __syncthreads();
    p = *reinterpret_cast<const f32x4_t*>(&part[0][col]);
#pragma unroll
    for (int w = 1; w < NW; ++w) {
        const f32x4_t x = *reinterpret_cast<const f32x4_t*>(&part[w][col]);
#pragma unroll
        for (int j = 0; j < 4; ++j) p[j] += x[j];
    }
    f32x4_t u;
#pragma unroll
    for (int j = 0; j < 4; ++j) u[j] = beta * fmaf(-al, p[j], to_f32<T>(vv[j]));
    if (rg == 0) {
        q = zero4();
        kq = 0.0f;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const f32x4_t x = *reinterpret_cast<const f32x4_t*>(&part[w][DV + col]);
#pragma unroll
            for (int j = 0; j < 4; ++j) q[j] += x[j];
            kq += part[w][2 * DV];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) q[j] = fmaf(al, q[j], kq * u[j]);
        store4_t<T>(reinterpret_cast<T*>(a.o) + nh * DV + col, q);
    }
#pragma unroll
    for (int m = 0; m < RPT; ++m) {
#pragma unroll
        for (int j = 0; j < 4; ++j) s[m][j] = fmaf(al, s[m][j], kk[m] * u[j]);
        __builtin_nontemporal_store(s[m], reinterpret_cast<f32x4_t*>(Sp + (long long)(NRG * m) * DV));
    }
}

namespace {

template <typename T, int DK, int NCT, bool OUT> hipError_t run_chunks(DeltaArgs a, hipStream_t s) {
    a.slices = a.dv / (64 * NCT);
    a.id_slices = OUT ? 0 : DK / (64 * NCT);
    a.n_units = (long long)a.BH * a.n_seg_launch * (a.slices + a.id_slices);
    a.per_xcd = (a.n_units + 7) / 8;
    if (a.n_units > (1LL << 22)) return hipErrorInvalidValue;
    kda_delta_prefill_kernel<T, DK, NCT, OUT><<<dim3((unsigned)(8 * a.per_xcd)), 512, 0, s>>>(a);
    return hipGetLastError();
}
template <typename T, int DK> hipError_t prefill_t(bool out, int nct, const DeltaArgs& a, hipStream_t s) {
    if (out) return nct == 2 ? run_chunks<T, DK, 2, true>(a, s) : run_chunks<T, DK, 1, true>(a, s);
    return run_chunks<T, DK, 1, false>(a, s);
}
template <int DK, int DV, typename T> hipError_t step_t(DeltaArgs a, hipStream_t s) {
    a.per_xcd = (a.n_units + 7) / 8;
    kda_delta_step_kernel<DK, DV, T><<<dim3((unsigned)(8 * a.per_xcd)), 4 * DV, 0, s>>>(a);
    return hipGetLastError();
}
template <typename T> hipError_t step_of(int dk, const DeltaArgs& a, hipStream_t s) {
    if (dk == 64) return a.dv == 64 ? step_t<64, 64, T>(a, s) : step_t<64, 128, T>(a, s);
    return a.dv == 64 ? step_t<128, 64, T>(a, s) : step_t<128, 128, T>(a, s);
}

}  // namespace

hipError_t launch_delta_prefill(bool out, int dk, bool f32, int nct, const DeltaArgs& a, hipStream_t s) {
    if (dk == 64) return f32 ? prefill_t<float, 64>(out, nct, a, s) : prefill_t<__bf16, 64>(out, nct, a, s);
    return f32 ? prefill_t<float, 128>(out, nct, a, s) : prefill_t<__bf16, 128>(out, nct, a, s);
}
hipError_t launch_delta_join(int dk, int dv, int bh, int n_seg, const float* M, const float* S0, float* S_in, hipStream_t s) {
    const dim3 grid((unsigned)bh, (unsigned)(dv / 16));
    if (dk == 64) kda_delta_join_kernel<64><<<grid, 256, 0, s>>>(M, S0, S_in, n_seg, dv);
    else kda_delta_join_kernel<128><<<grid, 256, 0, s>>>(M, S0, S_in, n_seg, dv);
    return hipGetLastError();
}
hipError_t launch_delta_step(int dk, bool f32, const DeltaArgs& a, hipStream_t s) {
    return f32 ? step_of<float>(dk, a, s) : step_of<__bf16>(dk, a, s);
}

}  // namespace kda
