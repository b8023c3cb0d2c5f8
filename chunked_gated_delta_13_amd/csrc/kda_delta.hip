// The gated delta rule with one decay per head and token, for gfx950: prompts in chunks, and single tokens.
//
// Per sequence and head, with a state S (dk x dv, fp32), a_t = e^(g_t), and key heads shared by groups of value heads:
//     S <- a_t S + beta_t k_t (v_t - a_t S^T k_t)^T,    o_t = S^T q_t          read after the write
//
// Chunks of C tokens.  With c_i the sum of the exponents (base 2) up to token i of the chunk and S0 its entry state:
//     A_ij = beta_i 2^(c_i - c_j) (k_i . k_j)  for j < i,     T = (I + A)^-1
//     R = V - diag(2^c) K S0,     U = T diag(beta) R
//     O = diag(2^c) Q S0 + B U,                B_ij = 2^(c_i - c_j) (q_i . k_j)  for j <= i
//     S <- 2^(c_C) S0 + K^T diag(2^(c_C - c_j)) U
// With one decay per token the differences of exponents are formed directly, never above 0 for decays: nothing has to be
// scaled apart and together again.  T is formed by 16 x 16 blocks in fp32.
//
// Numerics.  bf16 keys and queries are exact operands.  On the state's path S, T, R and U enter the products as three
// bf16 parts (24 bits; the six products of two such factors above 2^-24 are formed), so that states are as exact as with
// fp32 operands, at three to six bf16 products instead of the sixteen that one in fp32 takes.  The outputs, rounded to
// bf16 anyway, take S, U and B in two (in one part S and B leave them 2.5e-3 off where their own rounding is 1.7e-3, and
// the few outputs of a token or two up to 4e-3; it costs 8%).  fp32 inputs use fp32 products throughout.
#include "kda_mixers.h"
#include "kda_softmax.h"

namespace kda {

namespace {

// The inputs' types: tokens of a chunk, parts of a factor on the state's path.
template <typename T> struct DeltaTraits;
template <> struct DeltaTraits<__bf16> { static constexpr int C = 64, NP = 3; };
template <> struct DeltaTraits<float> { static constexpr int C = 32, NP = 1; };

constexpr float kDeadExponent = -126.0f;    // a segment's transition that leaves nothing of its entry state
constexpr float kDeadSlack = 2.0f;          // what decays leave for updates that expand a little
constexpr float kLeastExponent = -160.0f;   // 2^-160 of any state is below fp32's range: the same as nothing

// An operand kept as the wave holds it: 8 elements a lane, lane after lane.
__device__ __forceinline__ void frag_get(Frag<float>& f, const KDA_LDS float* p) {
    frag_join(f, *reinterpret_cast<const KDA_LDS f32x4_t*>(p), *reinterpret_cast<const KDA_LDS f32x4_t*>(p + 4));
}
__device__ __forceinline__ void frag_get(Frag<__bf16>& f, const KDA_LDS __bf16* p) {
    f.v = *reinterpret_cast<const KDA_LDS bf16x8_t*>(p);
}

// Four elements in NP parts, the first one largest.
template <int NP> __device__ __forceinline__ void parts4(bf16x4_t (&o)[NP], f32x4_t v) {
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const bf16x2_t u = {(__bf16)v[2 * j], (__bf16)v[2 * j + 1]};
            uint32_t w = __builtin_bit_cast(uint32_t, u);
            if (p + 1 < NP) asm("" : "+v"(w));   // (as in parts_of)
            const bf16x2_t y = __builtin_bit_cast(bf16x2_t, w);
            o[p][2 * j] = y[0];
            o[p][2 * j + 1] = y[1];
            if (p + 1 < NP) {
                v[2 * j] -= __uint_as_float(w << 16);
                v[2 * j + 1] -= __uint_as_float(w & 0xffff0000u);
            }
        }
}
template <int NP> __device__ __forceinline__ void parts4(f32x4_t (&o)[NP], f32x4_t v) {
    static_assert(NP == 1, "fp32 operands are whole");
    o[0] = v;
}

// c += a b of two rows of tiles for factors in parts: the products above 2^-24, the smallest first.
template <typename T, int NP>
__device__ __forceinline__ void mma_parts(const Frag<T> (&a)[2][NP], const Frag<T> (&b)[NP], f32x4_t& c0, f32x4_t& c1) {
#pragma unroll
    for (int s = NP - 1; s >= 0; --s)
#pragma unroll
        for (int p = 0; p <= s; ++p) {
            c0 = mma(a[0][p], b[s - p], c0);
            c1 = mma(a[1][p], b[s - p], c1);
        }
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

// Values of lane I of each quad.
template <int I> __device__ __forceinline__ f32x4_t quad_lane(const f32x4_t& v) {
    f32x4_t o;
#pragma unroll
    for (int x = 0; x < 4; ++x) o[x] = __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v[x]), I * 0x55, 0xF, 0xF, true));
    return o;
}

}  // namespace

// Chunk waves: eight beside four state waves in bf16, of which four form the inverses and T, the others A's other blocks and B: a
// lone wave of a SIMD issues an instruction every eight cycles at best (16 heads of 128, one chunk 12.9 -> 11.7 us, ten 49.8 ->
// 47.4; in fp32, whose products take longer, 31.1 and 31.8 for 3 prompts of 301 tokens).
template <typename T> constexpr int chunk_waves(int nsw) { return nsw == 4 && sizeof(T) == 2 ? 8 : 4; }

// Prompt.  A workgroup runs one (sequence, head, segment, slice of 16 NSW state columns) with two roles: NSW state
// waves hold the slice (16 columns each, fp32, in the accumulators' layout) and run chunk c; the chunk waves
// prepare what chunk c + 1 needs and does not depend on the state.  With eight state waves a SIMD hosts two of them and a
// chunk wave.  Three workgroup barriers a chunk:
//     interval   state waves, chunk c             chunk waves, chunk n = c + 1
//     1          X = K S0, Q S0                   A (fp32) and the inverses of its diagonal blocks
//     2          R, U = T R                       K and Q of n + 1 requested; the first products of T's other blocks
//     3          O, S; V of c + 1 requested       T's other blocks, T's parts to LDS; B; exponents of n + 1
// K has three buffers (chunks c, n and the one in flight), Q, B and the exponents' tables two or three, T and V one: each is
// overwritten only in an interval after its last reader's.
//
// Bound by issue: 4 prompts of 16384 tokens, 56 heads on 28 of 128 in 1600 to 1660 us, 13500 cycles a chunk; products take 16.7
// cycles, two vector instructions beside each are free and further ones take 4, which makes 10000 cycles for a chunk's.
// Products are busy in 54% of the cycles, vector instructions, these among them, issued in 57%, LDS busy in 35%; HBM moves
// 1.7 TB/s.
//
// OUT: outputs are formed (else only states).
template <typename T, int DK, int NSW, bool OUT>
__global__ __launch_bounds__(64 * (NSW + chunk_waves<T>(NSW))) void kda_delta_prefill_kernel(const DeltaArgs a) {
    constexpr int C = DeltaTraits<T>::C, NP = DeltaTraits<T>::NP, NA = C / 16, NQ = C / 32;   // token tiles, pairs of them
    constexpr int NT = DK / 16, NKB = DK / 32, DVS = 16 * NSW;
    constexpr int KT = C * DK, VT = C * DVS;                     // elements of a tile
    constexpr int NF = NQ * (NQ + 1);                            // operands of a lower triangle
    constexpr int FR = 64 * 8;                                   // elements of an operand
    constexpr int ARR = 5 * C + 16;                              // exponents (high, low parts), 2^c, 2^(c_C - c), beta, 2^c_C
    constexpr int NLOW = NA * (NA - 1) / 2;
    constexpr int OP = NP > 1 ? 2 : 1;                           // parts of a factor of the outputs
    constexpr int NCW = chunk_waves<T>(NSW), CS = NCW / 4;       // chunk waves; those that share a group of rows
    static_assert(NCW == 4 || NA == 4, "eight chunk waves share four rows of blocks");
    struct Shared {
        T k[3][KT], q[OUT ? 2 : 1][KT], v[VT];
        T t[NP][NF * FR], b[2][OP][OUT ? NF * FR : 8];
        float low[NLOW * 256], diag[NA * 256], rows[NA * 256], pair[512];   // A's blocks below the diagonal, transposed; T's on it, as they
                                                                            // are and transposed; two of T's below it
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
    long long todo_ = len - begin;          // tokens of this unit (a segment has fewer than 2^31)
    todo_ = todo_ < 0 ? 0 : (todo_ < a.seg_len ? todo_ : a.seg_len);
    const int todo = (int)todo_, nc = (todo + C - 1) / C;
    int first = 0;                          // chunk to start from

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, r = lane & 15;

    // Rows of one tile from memory: step i covers 1 KB, rows of a group and a block of 32 columns; nb blocks.  `off` is the
    // lane's offset in a whole chunk.  Rows past the unit's take its last one (finite, and of no weight: their beta is 0).
    constexpr int GROUPS = C / TileStep<T>::ROWS, ES = (int)sizeof(T);
    auto lane_off = [&](long long stride, int group, int last) {
        int row = group * TileStep<T>::ROWS + TileStep<T>::row(lane);
        const int piece = tile_dma_piece<T>(row, lane);
        row = row < last ? row : last;
        return (uint32_t)row * (uint32_t)(stride * ES) + (uint32_t)(piece * 16);
    };
    auto fetch = [&](const T* base, uint32_t off, KDA_LDS T* tile, int group, int block) {
        dma16(base + 32 * block, off, lds_address(tile + block * C * 32 + group * TileStep<T>::ROWS * 32));
    };
    const long long tok0 = (long long)b * a.T + begin;

    if constexpr (!OUT) {
        // Where the transitions from some chunk to the segment's end together leave less than 2^-126 of a state, nothing before
        // that chunk matters: the state from zero is run from there, and the transition is dead (marked, not formed).  A token's
        // transition a (I - beta k k^T) has the norm a max(1, |1 - beta |k|^2|).  The chunk is found by the decays (sums of 64
        // chunks at a time from the end backwards, 8 or 16 of them a wave); then what all of the segment's updates expand, where
        // beta |k|^2 passes 2 or is negative, is added, and if that is too much the whole segment and its transition are
        // formed (20001 tokens, 16 heads 353 -> 363 us; by the decays alone expanding updates lost what they had kept).  A few short
        // segments are not looked at: forming all transitions, each on a compute unit of its own, takes less than that (in fp32 3
        // prompts of 301 tokens 33.4 -> 30.6 us, 4 of 333 46.3 -> 42.7; in bf16 3 of 602 tokens 35.1 -> 32.8, with d = 128 59.4 -> 53.4).
        constexpr int NW = NSW + NCW;
        KDA_LDS float* sums = &sh->low[0];
        bool dead = false;
        float total = 0.0f;
        for (int last = nc <= 4 && a.n_seg_launch < 8 ? 0 : nc; last > 0 && !dead; last -= 64) {
            for (int i = wave; i < 64; i += NW) {
                const int c = last - 1 - i, at = c * C + lane;
                float e = 0.0f;
                if (c >= 0 && lane < C && at < todo) e = a.g[(tok0 + at) * a.H + h] * kLog2e;
                if (e < kLeastExponent) e = kLeastExponent;   // (a NaN stays one, and kills nothing)
#pragma unroll
                for (int x = 1; x < 64; x <<= 1) e += __shfl_xor(e, x);
                if (lane == 0) sums[i] = e;
            }
            barrier_lds();
            float e = sums[lane];
#pragma unroll
            for (int x = 1; x < 64; x <<= 1) {
                const float y = __shfl_up(e, x);
                if (lane >= x) e += y;
            }
            e += total;
            const unsigned long long past = __ballot(e <= kDeadExponent - kDeadSlack);
            if (past) {
                dead = true;
                first = last - 1 - __builtin_ctzll(past);
            }
            total = __shfl(e, past ? __builtin_ctzll(past) : 63);
            barrier_lds();
        }
        if (dead) {
            constexpr int LE = 16 / (int)sizeof(T), LR = DK / LE, RL = 64 / LR, NL = C / RL;   // elements of a lane, lanes of a row, rows
            typedef __attribute__((ext_vector_type(LE))) T piece_t;                            // of a load, loads of a chunk
            const T* kr = reinterpret_cast<const T*>(a.k) + tok0 * a.k_stride + (long long)hk * DK + (lane % LR) * LE;
            float more = 0.0f;
            for (int c = wave; c < nc; c += NW) {
                piece_t x[NL];
                float beta[NL];
#pragma unroll
                for (int i = 0; i < NL; ++i) {   // (rows past the unit's: the last one again, without a weight)
                    const int row = c * C + i * RL + lane / LR, at = row < todo ? row : todo - 1;
                    x[i] = *reinterpret_cast<const piece_t*>(kr + at * a.k_stride);
                    beta[i] = a.beta[(tok0 + at) * a.H + h];
                }
#pragma unroll
                for (int i = 0; i < NL; ++i) {
                    float n = 0.0f;
#pragma unroll
                    for (int j = 0; j < LE; ++j) n = fmaf((float)x[i][j], (float)x[i][j], n);
#pragma unroll
                    for (int s = 1; s < LR; s <<= 1) n += __shfl_xor(n, s);
                    const float f = fabsf(fmaf(-beta[i], n, 1.0f));
                    // (base 2; a NaN kills nothing either)
                    if (c * C + i * RL + lane / LR < todo && !(f <= 1.0f)) more += __builtin_amdgcn_logf(f);
                }
            }
#pragma unroll
            for (int x = LR; x < 64; x <<= 1) more += __shfl_xor(more, x);
            if (lane == 0) sums[wave] = more;
            barrier_lds();
#pragma unroll
            for (int i = 0; i < NW; ++i) total += sums[i];
            if (!__all(total <= kDeadExponent)) {   // (the same in every lane)
                dead = false;
                first = 0;
            }
        }
        if (ident) {
            if (slice == 0 && tid == 0) a.dead[bh * a.m_bh + seg] = dead ? 1 : 0;
            if (dead) return;
            first = 0;
        }
    }

    if (wave < NSW) {
        // ------------------------------------------------------------------------------------------ state waves
        const T* vp = reinterpret_cast<const T*>(a.v) + tok0 * a.v_stride + (long long)h * a.dv + slice * DVS;
        constexpr int NB = DVS / 32, VG = NSW / GROUPS;   // blocks of a row; waves that share a group of rows
        const int v_group = wave / VG;
        const uint32_t v_off = lane_off(a.v_stride, v_group, C);
        auto fetch_v = [&](int chunk) {
            if (ident) return;
            const int left = todo - chunk * C;
            const uint32_t off = left >= C ? v_off : lane_off(a.v_stride, v_group, left - 1);
            const T* base = vp + (long long)chunk * C * a.v_stride;
#pragma unroll
            for (int i = 0; i < NB / VG; ++i) fetch(base, off, sh->v, v_group, (wave % VG) * (NB / VG) + i);
        };
        if (nc > 0) fetch_v(first);

        const int col = slice * DVS + wave * 16 + r;   // this lane's column
        const int width = ident ? DK : a.dv;
        f32x4_t S[NT];
        if (!ident && a.S_in) {
            const float* s_in = a.S_in + bh * a.sin_bh + seg * a.sin_seg + (long long)(4 * g) * width + col;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j) S[t][j] = s_in[(16 * t + j) * width];
        } else {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j) S[t][j] = ident && 16 * t + 4 * g + j == col ? 1.0f : 0.0f;
        }
        // Waves of one SIMD are served the oldest first: the second state wave of one ended an interval 2000 cycles after the
        // first.  It goes first, and a chunk wave before either but in interval 3, where it has time (1700 -> 1652 us).
        if (wave >= 4) __builtin_amdgcn_s_setprio(2);
        else __builtin_amdgcn_s_setprio(1);
        TileRows<T, C, DK> rk, rq;
        TileCols<T, C> ck, cvt;
        rk.set(sh->k[0], lane);
        rq.set(sh->q[0], lane);
        ck.set(sh->k[0], lane);
        cvt.set_tile(sh->v, lane, wave);
        const KDA_LDS T* tf = lds_pin(&sh->t[0][0] + lane * 8);
        const int o_step = a.H * a.dv;   // (at most 2^22)
        T* op = OUT ? reinterpret_cast<T*>(a.o) + (tok0 * a.H + h) * a.dv + slice * DVS + wave * 16 : nullptr;
        const uint32_t o_off = (uint32_t)((r * o_step + 4 * g) * ES);

        barrier_all();
        if (nc > 0) {
            barrier_lds();
            barrier_lds();
            barrier_lds();
        }
        for (int n = first; n < nc; ++n) {
            const int kb3 = n % 3;
            const TileRows<T, C, DK> k_rows = rk.at_delta(kb3 * KT);
            const TileRows<T, C, DK> q_rows = rq.at_delta((OUT ? n & 1 : 0) * KT);
            const KDA_LDS float* arr = &sh->arr[kb3][0];

            // 1: X = K S0 and (transposed) S0^T Q^T, contraction block by contraction block; the parts of the next
            // block's state are formed between the products of this one
            f32x4_t X[NA], O[NA];
#pragma unroll
            for (int i = 0; i < NA; ++i) X[i] = O[i] = zero4();
            {
                Frag<T> kf[2][NA], qf[NA], s[2][NP];
#pragma unroll
                for (int i = 0; i < NA; ++i) k_rows.frag(kf[0][i], 0, i, 0);
                parts_of<NP>(s[0], S[0], S[NKB]);
#pragma unroll
                for (int kb = 0; kb < NKB; ++kb) {
                    __builtin_amdgcn_sched_barrier(0);
                    if constexpr (OUT) {
#pragma unroll
                        for (int i = 0; i < NA; ++i) q_rows.frag(qf[i], 0, i, kb);
                    }
                    if (kb + 1 < NKB) {
#pragma unroll
                        for (int i = 0; i < NA; ++i) k_rows.frag(kf[(kb + 1) & 1][i], 0, i, kb + 1);
                        parts_of<NP>(s[(kb + 1) & 1], S[kb + 1], S[kb + 1 + NKB]);
                    }
#pragma unroll
                    for (int p = NP - 1; p >= 0; --p)
#pragma unroll
                        for (int i = 0; i < NA; ++i) X[i] = mma(kf[kb & 1][i], s[kb & 1][p], X[i]);
                    if constexpr (OUT) {
#pragma unroll
                        for (int p = OP - 1; p >= 0; --p)
#pragma unroll
                            for (int i = 0; i < NA; ++i) O[i] = mma(s[kb & 1][p], qf[i], O[i]);
                    }
                }
            }
            barrier_all();   // (V has arrived, for every wave)

            // 2: R = V - 2^c X in X's place, then U = (T diag(beta)) R
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
                Frag<T> v;
                if (!ident) cvt.frag(v, 0, 0, q);
                else v.zero();
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int i = q + x * NQ;
                    const f32x4_t grow = *reinterpret_cast<const KDA_LDS f32x4_t*>(arr + 2 * C + 16 * i + 4 * g);
#pragma unroll
                    for (int j = 0; j < 4; ++j) X[i][j] = fmaf(-grow[j], X[i][j], v.get(4 * x + j));
                }
            }
            f32x4_t U[NA];
#pragma unroll
            for (int i = 0; i < NA; ++i) U[i] = zero4();
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
                Frag<T> rr[NP];
                parts_of<NP>(rr, X[2 * q], X[2 * q + 1]);
#pragma unroll
                for (int i = 2 * q; i < NA; i += 2) {
                    Frag<T> tt[2][NP];
#pragma unroll
                    for (int y = 0; y < 2; ++y)
#pragma unroll
                        for (int p = 0; p < NP; ++p) frag_get(tt[y][p], tf + (p * NF + frag_at(i + y, q)) * FR);
                    mma_parts<T, NP>(tt, rr, U[i], U[i + 1]);
                }
            }
            barrier_lds();

            // 3: outputs, then the state
            if constexpr (OUT) {
                const KDA_LDS T* bf = lds_pin(&sh->b[n & 1][0][0] + lane * 8);
                Frag<T> f[2][NF], uu[NQ][OP];
#pragma unroll
                for (int i = 0; i < NF; ++i) frag_get(f[(OP - 1) & 1][i], bf + ((OP - 1) * NF + i) * FR);
#pragma unroll
                for (int i = 0; i < NA; ++i) {
                    const float grow = arr[2 * C + 16 * i + r];
#pragma unroll
                    for (int j = 0; j < 4; ++j) O[i][j] *= grow;
                }
#pragma unroll
                for (int q = 0; q < NQ; ++q) parts_of<OP>(uu[q], U[2 * q], U[2 * q + 1]);
                // (the product of the two second parts is left out)
#pragma unroll
                for (int y = OP - 1; y >= 0; --y) {
                    if (y > 0) {
#pragma unroll
                        for (int i = 0; i < NF; ++i) frag_get(f[0][i], bf + i * FR);
                    }
#pragma unroll
                    for (int p = OP - 1 - y; p >= 0; --p)
#pragma unroll
                        for (int q = 0; q < NQ; ++q)
#pragma unroll
                            for (int i = 2 * q; i < NA; ++i) O[i] = mma(uu[q][p], f[y][frag_at(i, q)], O[i]);
                }
#pragma unroll
                for (int i = 0; i < NA; ++i)
                    if (n * C + 16 * i + r < todo) store4<T>(at_byte(op + (long long)(n * C + 16 * i) * o_step, pinned_u(o_off)), O[i]);
            }
            const float dec = arr[5 * C];
#pragma unroll
            for (int i = 0; i < NA; ++i) {
                const f32x4_t late = *reinterpret_cast<const KDA_LDS f32x4_t*>(arr + 3 * C + 16 * i + 4 * g);
#pragma unroll
                for (int j = 0; j < 4; ++j) U[i][j] *= late[j];
            }
            const TileCols<T, C> k_cols = ck.at_delta(kb3 * KT);
            Frag<T> uu[NQ][NP];
#pragma unroll
            for (int q = 0; q < NQ; ++q) parts_of<NP>(uu[q], U[q], U[q + NQ]);
            // (a chunk's sum starts from zero and joins the decayed state with one rounding)
            Frag<T> kc[2][2][NQ];
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
                for (int q = 0; q < NQ; ++q) k_cols.frag(kc[0][y][q], 0, y, q);
#pragma unroll
            for (int t = 0; t < NT; t += 2) {
                if (t + 2 < NT) {
#pragma unroll
                    for (int y = 0; y < 2; ++y)
#pragma unroll
                        for (int q = 0; q < NQ; ++q) k_cols.frag(kc[(t / 2 + 1) & 1][y][q], 0, t + 2 + y, q);
                }
                f32x4_t add[2] = {zero4(), zero4()};
#pragma unroll
                for (int p = NP - 1; p >= 0; --p)
#pragma unroll
                    for (int q = 0; q < NQ; ++q)
#pragma unroll
                        for (int y = 0; y < 2; ++y) add[y] = mma(kc[(t / 2) & 1][y][q], uu[q][p], add[y]);
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                    for (int j = 0; j < 4; ++j) S[t + y][j] = fmaf(S[t + y][j], dec, add[y][j]);
            }
            if (n + 1 < nc) fetch_v(n + 1);
            barrier_lds();
        }
        float* s_out = ident ? a.M_out + (bh * a.m_bh + seg) * (long long)(DK * DK)
                             : (a.S_out && (a.out_seg < 0 || a.out_seg == seg) ? a.S_out + bh * a.sout_bh + (a.out_seg < 0 ? seg : 0) * a.sout_seg : nullptr);
        if (s_out) {
            s_out += (long long)(4 * g) * width + col;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j) s_out[(16 * t + j) * width] = S[t][j];
        }
        return;
    }

    // ---------------------------------------------------------------------------------------------- chunk waves
    const int cw = wave - NSW;
    const T* kp = reinterpret_cast<const T*>(a.k) + tok0 * a.k_stride + (long long)hk * DK;
    const T* qp = reinterpret_cast<const T*>(a.q) + tok0 * a.q_stride + (long long)hk * DK;
    static_assert(GROUPS == 4 && NKB % CS == 0, "chunk waves share groups of rows");
    const int rows_of = cw & 3, block0 = (cw >> 2) * (NKB / CS);
    const uint32_t k_off = lane_off(a.k_stride, rows_of, C), q_off = lane_off(a.q_stride, rows_of, C);
    auto fetch_kq = [&](int chunk) {
        const int left = todo - chunk * C;
        const uint32_t ko = left >= C ? k_off : lane_off(a.k_stride, rows_of, left - 1);
        const T* base = kp + (long long)chunk * C * a.k_stride;
#pragma unroll
        for (int i = 0; i < NKB / CS; ++i) fetch(base, ko, sh->k[chunk % 3], rows_of, block0 + i);
        if constexpr (OUT) {
            const uint32_t qo = left >= C ? q_off : lane_off(a.q_stride, rows_of, left - 1);
            base = qp + (long long)chunk * C * a.q_stride;
#pragma unroll
            for (int i = 0; i < NKB / CS; ++i) fetch(base, qo, sh->q[chunk & 1], rows_of, block0 + i);
        }
    };
    // exponents and beta of a chunk's tokens, one a lane (the last wave)
    float g_next = 0.0f, beta_next = 0.0f;
    auto request_arr = [&](int chunk) {
        const int at = chunk * C + lane;
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
        fetch_kq(first);
        if (cw == NCW - 1) {
            request_arr(first);
            put_arr(first);
        }
        // the halves of operands that lie above the diagonal stay zero
        for (int i = tid - 64 * NSW; i < NP * NF * FR; i += 64 * NCW) (&sh->t[0][0])[i] = (T)0.0f;
        if constexpr (OUT)
            for (int i = tid - 64 * NSW; i < 2 * OP * NF * FR; i += 64 * NCW) (&sh->b[0][0][0])[i] = (T)0.0f;
    }
    barrier_all();
    for (int n = first; n < nc; ++n) {
        const bool more = n + 1 < nc;
        if (cw == NCW - 1 && more) request_arr(n + 1);
        const KDA_LDS float* arr = &sh->arr[n % 3][0];
        const TileRows<T, C, DK> k_rows = rk.at_delta((n % 3) * KT);
        const TileRows<T, C, DK> q_rows = rq.at_delta((OUT ? n & 1 : 0) * KT);
        // 2^(c_i - c_j) of row r of block i, columns 4 g .. of block j
        auto decays = [&](int i, int j) {
            const KDA_LDS float *ai = arr + 16 * i + r, *aj = arr + 16 * j + 4 * g;
            const f32x4_t hj = *reinterpret_cast<const KDA_LDS f32x4_t*>(aj), lj = *reinterpret_cast<const KDA_LDS f32x4_t*>(aj + C);
            const float hi = ai[0], lo = ai[C];
            f32x4_t w;
#pragma unroll
            for (int x = 0; x < 4; ++x) w[x] = fast_exp2((hi - hj[x]) + (lo - lj[x]));
            return w;
        };
        // rows j of K by rows i of `rows`, for one tile
        auto product = [&](const TileRows<T, C, DK>& rows, int i, int j) {
            const TileRows<T, C, DK> x = k_rows.at_delta(16 * 32 * j), y = rows.at_delta(16 * 32 * i);
            Frag<T> fx[NKB], fy[NKB];
#pragma unroll
            for (int kb = 0; kb < NKB; ++kb) {
                x.frag(fx[kb], 0, 0, kb);
                y.frag(fy[kb], 0, 0, kb);
            }
            f32x4_t p = zero4();
#pragma unroll
            for (int kb = 0; kb < NKB; ++kb) p = mma(fx[kb], fy[kb], p);
            return p;
        };
        auto dumped = [&](const KDA_LDS float* p) { return *reinterpret_cast<const KDA_LDS f32x4_t*>(p + lane * 4); };
        auto dump = [&](KDA_LDS float* p, const f32x4_t& v) { *reinterpret_cast<KDA_LDS f32x4_t*>(p + lane * 4) = v; };
        auto low = [&](int i, int j) { return &sh->low[(i * (i - 1) / 2 + j) * 256]; };
        auto below = [&](int i, int j) {   // A_ij, i > j, transposed
            f32x4_t G = product(k_rows, i, j);
            const f32x4_t w = decays(i, j);
            const float beta = arr[4 * C + 16 * i + r];
#pragma unroll
            for (int x = 0; x < 4; ++x) G[x] *= beta * w[x];
            dump(low(i, j), G);
            return w;
        };

        __builtin_amdgcn_s_setprio(3);
        // 1: A by tiles of K K^T.  Wave i forms the inverse of the diagonal one of row i.
        f32x4_t Dt = zero4(), up = zero4(), w1 = zero4(), w2 = zero4();   // T_ii transposed; decays, for A and for B
        if (cw < NA) {
            const f32x4_t G = product(k_rows, cw, cw);
            up = decays(cw, cw);
            const float br = arr[4 * C + 16 * cw + r], hj = arr[16 * cw + r], lj = arr[C + 16 * cw + r];
            const f32x4_t hi = *reinterpret_cast<const KDA_LDS f32x4_t*>(arr + 16 * cw + 4 * g), lo = *reinterpret_cast<const KDA_LDS f32x4_t*>(arr + C + 16 * cw + 4 * g);
            const f32x4_t beta = *reinterpret_cast<const KDA_LDS f32x4_t*>(arr + 4 * C + 16 * cw + 4 * g);
            // L = A_ii and its transpose, both in the accumulators' layout.  (K K^T is symmetric.)
            f32x4_t L, Lt, D;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                L[x] = 4 * g + x > r ? G[x] * beta[x] * fast_exp2((hi[x] - hj) + (lo[x] - lj)) : 0.0f;
                Lt[x] = 4 * g + x < r ? G[x] * br * up[x] : 0.0f;
                D[x] = Dt[x] = 4 * g + x == r ? 1.0f : 0.0f;
            }
            // The 4 x 4 blocks on its diagonal, whose columns are the lanes of a quad: column r of the inverse by
            // substitution from above, and its row r (the transpose's column) from the right.
            const f32x4_t l0 = quad_lane<0>(L), l1 = quad_lane<1>(L), l2 = quad_lane<2>(L);
            if ((r >> 2) == g) {
#pragma unroll
                for (int x = 1; x < 4; ++x) D[x] = fmaf(-l0[x], D[0], D[x]);
#pragma unroll
                for (int x = 2; x < 4; ++x) D[x] = fmaf(-l1[x], D[1], D[x]);
                D[3] = fmaf(-l2[3], D[2], D[3]);
                Dt[2] = fmaf(-l2[3], Dt[3], Dt[2]);
                Dt[1] = fmaf(-l1[2], Dt[2], fmaf(-l1[3], Dt[3], Dt[1]));
                Dt[0] = fmaf(-l0[1], Dt[1], fmaf(-l0[2], Dt[2], fmaf(-l0[3], Dt[3], Dt[0])));
            }
            // Blocks of 8 and of 16 rows from halves: D - D M D, M the part of L between the halves.  An accumulator is
            // the operand of its own matrix from the right, and of its transpose from the left.
            KDA_LDS float* turn = &sh->rows[cw * 256];
#pragma unroll
            for (int w = 4; w <= 8; w *= 2) {
                f32x4_t Mt;
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int row = r, col = 4 * g + x;   // of M; Mt holds it transposed
                    Mt[x] = row / (2 * w) == col / (2 * w) && row / w != col / w ? -Lt[x] : 0.0f;
                }
                D = mma16(Dt, mma16(Mt, D, zero4()), D);
#pragma unroll
                for (int x = 0; x < 4; ++x) turn[(16 * (r >> 2) + 4 * g + x) * 4 + (r & 3)] = D[x];   // row 4 g + x, column r
                wave_order();
                Dt = dumped(turn);
                wave_order();
            }
            dump(&sh->diag[cw * 256], D);
        }
        if constexpr (NCW == 8) {
            const int x = cw - 4;
            if (x >= 0) w1 = below(x < 2 ? 3 : (x == 2 ? 2 : 1), x == 2 ? 1 : (x == 1 ? 2 : 0));   // (3,0) (3,2) (2,1) (1,0)
            if (x == 0) w2 = below(2, 0);
            if (x == 3) w2 = below(3, 1);
        } else if constexpr (NA == 4) {
            w1 = below(cw < 2 ? 3 : (cw == 2 ? 2 : 1), cw == 2 ? 1 : (cw == 1 ? 2 : 0));   // (3,0) (3,2) (2,1) (1,0)
            if (cw == 0) below(2, 0);
            if (cw == 3) w2 = below(3, 1);
        } else {
            if (cw == 2) w1 = below(1, 0);
        }
        barrier_lds();

        // 2: T below the diagonal.  Of a 2 x 2 block matrix that is T_ij = -T_ii A_ij T_jj: first inside the pairs of rows
        // (0, 1) and (2, 3), then between the pairs (columns 0 and 1, a wave each).
        if (more) fetch_kq(n + 1);
        f32x4_t x0 = zero4(), x1 = zero4();
        auto negated = [](f32x4_t v) { return f32x4_t{-v[0], -v[1], -v[2], -v[3]}; };
        if (cw == 1 || (NA == 4 && cw == 3)) {
            const f32x4_t Q = mma16(dumped(low(cw, cw - 1)), dumped(&sh->diag[(cw - 1) * 256]), zero4());
            x0 = negated(mma16(Q, Dt, zero4()));                           // T_10 or T_32, transposed
            if constexpr (NA == 4) {
                if (cw == 1) dump(&sh->pair[0], negated(mma16(Dt, Q, zero4())));   // T_10
                else dump(&sh->pair[256], x0);
            }
        } else if (NA == 4 && cw < 4) {   // A_2x T_xx, A_3x T_xx for x = cw / 2
            const f32x4_t D = dumped(&sh->diag[(cw >> 1) * 256]);
            x0 = mma16(dumped(low(2, cw >> 1)), D, zero4());
            x1 = mma16(dumped(low(3, cw >> 1)), D, zero4());
        }
        barrier_lds();

        __builtin_amdgcn_s_setprio(0);
        // 3: the rest of T, and all of it to the state waves, which have read the last one; B
        auto put = [&](int i, int j, f32x4_t v) {   // with beta: U = (T diag(beta)) (V - 2^c X)
            const f32x4_t beta = *reinterpret_cast<const KDA_LDS f32x4_t*>(arr + 4 * C + 16 * j + 4 * g);
#pragma unroll
            for (int x = 0; x < 4; ++x) v[x] *= beta[x];
            typename Vec4<T>::type o[NP];
            parts4<NP>(o, v);
#pragma unroll
            for (int p = 0; p < NP; ++p)
                *reinterpret_cast<KDA_LDS typename Vec4<T>::type*>(&sh->t[p][frag_at(i, j >> 1) * FR + lane * 8 + (j & 1) * 4]) = o[p];
        };
        auto weights = [&](int i, int j, const f32x4_t& w) {   // B_ij, from its decays
            const f32x4_t P = product(q_rows, i, j);
            f32x4_t e;
#pragma unroll
            for (int x = 0; x < 4; ++x) e[x] = i == j && 4 * g + x > r ? 0.0f : w[x] * P[x];
            typename Vec4<T>::type o[OP];
            parts4<OP>(o, e);
#pragma unroll
            for (int p = 0; p < OP; ++p)
                *reinterpret_cast<KDA_LDS typename Vec4<T>::type*>(&sh->b[n & 1][p][frag_at(i, j >> 1) * FR + lane * 8 + (j & 1) * 4]) = o[p];
        };
        if (cw < NA) put(cw, cw, Dt);
        if (cw == 1 || (NA == 4 && cw == 3)) {
            put(cw, cw - 1, x0);
        } else if (NA == 4 && cw < 4) {
            if (cw == 0) {
                const f32x4_t T10 = dumped(&sh->pair[0]);
                x0 = mma16(dumped(low(2, 1)), T10, x0);
                x1 = mma16(dumped(low(3, 1)), T10, x1);
            }
            const f32x4_t D2 = dumped(&sh->rows[2 * 256]), D3 = dumped(&sh->rows[3 * 256]), T32 = dumped(&sh->pair[256]);
            put(2, cw >> 1, negated(mma16(x0, D2, zero4())));
            put(3, cw >> 1, negated(mma16(x1, D3, mma16(x0, T32, zero4()))));
        }
        if constexpr (OUT) {   // B, from the decays at hand where a wave has formed them
            if constexpr (NCW == 8) {
                if (cw == 4) {
                    weights(3, 0, w1);
                    weights(2, 0, w2);
                    weights(0, 0, decays(0, 0));
                } else if (cw == 5) {
                    weights(3, 2, w1);
                    weights(1, 1, decays(1, 1));
                    weights(3, 3, decays(3, 3));
                } else if (cw == 6) {
                    weights(2, 1, w1);
                    weights(2, 2, decays(2, 2));
                } else if (cw == 7) {
                    weights(1, 0, w1);
                    weights(3, 1, w2);
                }
            } else if constexpr (NA == 4) {
                if (cw == 0) {
                    weights(3, 0, w1);
                } else if (cw == 1) {
                    weights(0, 0, decays(0, 0));
                    weights(1, 1, up);
                    weights(2, 0, decays(2, 0));
                    weights(3, 2, w1);
                } else if (cw == 2) {
                    weights(2, 1, w1);
                    weights(2, 2, up);
                } else {
                    weights(1, 0, w1);
                    weights(3, 1, w2);
                    weights(3, 3, up);
                }
            } else {
                if (cw < 2) weights(cw, cw, up);
                if (cw == 2) weights(1, 0, w1);
            }
        }
        if (cw == NCW - 1 && more) put_arr(n + 1);
        barrier_all();   // (K and Q of n + 1 have arrived)
    }
    if (nc > 0) {
        barrier_lds();
        barrier_lds();
        barrier_lds();
    }
}

// Entry states of a split's segments: S_in(s + 1) = M_s S_in(s) + H_s in fp32.  H lies in the place of S_in(s + 1); M_s
// is dk x dk, and a dead one leaves nothing to do.  A workgroup owns 16 columns of one (sequence, head), a wave one tile of
// rows, which it forms from the tiles of the state in LDS (as the accumulators hold them, which is how an operand does); what
// the next step reads is requested a step ahead.
template <int DK>
__global__ __launch_bounds__(4 * DK) void kda_delta_join_kernel(const float* M, const int* dead, const float* S0, float* S_in, int n_seg, int dv) {
    constexpr int NT = DK / 16;   // row tiles, a wave each
    const long long bh = blockIdx.x;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), g = lane >> 4, r = lane & 15;
    __shared__ __attribute__((aligned(16))) float cur[2][NT * 256];
    float* at = S_in + bh * n_seg * (long long)(DK * dv) + (long long)(16 * wave + 4 * g) * dv + blockIdx.y * 16 + r;
    const float* s0 = S0 ? S0 + bh * (long long)(DK * dv) + (at - (S_in + bh * n_seg * (long long)(DK * dv))) : nullptr;
    const float* m = M + (bh * (n_seg - 1) * DK + 16 * wave + r) * (long long)DK + 4 * g;
    dead += bh * (n_seg - 1);
    const long long step = (long long)DK * dv;
    f32x4_t s, next[2] = {zero4(), zero4()}, w[2][NT];
    auto request = [&](int seg, bool alive, f32x4_t& n, f32x4_t (&t)[NT]) {   // the step after segment `seg`: its H, its transition
#pragma unroll
        for (int j = 0; j < 4; ++j) n[j] = at[(seg + 1) * step + j * dv];
        if (alive) {
#pragma unroll
            for (int k = 0; k < NT; ++k) t[k] = *reinterpret_cast<const f32x4_t*>(m + (long long)seg * (DK * DK) + 16 * k);
        }
    };
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        s[j] = s0 ? s0[j * dv] : 0.0f;
        at[j * dv] = s[j];
    }
    int turn = 0;
    for (int from = 0; from + 1 < n_seg; from += 64) {   // 64 segments' marks at a time
        const int end = from + 64 < n_seg - 1 ? from + 64 : n_seg - 1;
        const unsigned long long live = __ballot(from + lane < end && dead[from + lane < end ? from + lane : from] == 0);
        request(from, live & 1, next[0], w[0]);
        for (int seg0 = from; seg0 < end; seg0 += 2)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int seg = seg0 + y;
                if (seg >= end) break;
                const bool alive = live >> (seg - from) & 1;   // (uniform over the workgroup)
                if (seg + 1 < end) request(seg + 1, live >> (seg + 1 - from) & 1, next[y ^ 1], w[y ^ 1]);
                if (alive) {
                    // (two buffers in turn: a wave reaches the barrier before it overwrites one with its last reads of it done)
                    KDA_LDS float* c = (KDA_LDS float*)cur[turn];
                    turn ^= 1;
                    *reinterpret_cast<KDA_LDS f32x4_t*>(c + wave * 256 + lane * 4) = s;
                    barrier_lds();
                    f32x4_t p[2] = {zero4(), zero4()};
#pragma unroll
                    for (int k = 0; k < NT; ++k) p[k & 1] = mma16(w[y][k], *reinterpret_cast<const KDA_LDS f32x4_t*>(c + k * 256 + lane * 4), p[k & 1]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        s[j] = next[y][j] + (p[0][j] + p[1][j]);
                        at[(seg + 1) * step + j * dv] = s[j];
                    }
                } else {
                    s = next[y];
                }
            }
    }
}

// One token, bound by HBM (about 7 flops per 8 bytes of state moved): one streaming pass over the state without matrix
// products.  With p = S^T k and r = S^T q of the old state:
//     u = beta (v - a p),     S <- a S + k u^T,     o = a r + (k . q) u
// A workgroup owns one (sequence, head): dv / 4 column groups of four (a state's row is one contiguous run) x 16 row
// groups, and takes states so that an XCD streams one contiguous range of them.  256 sequences of 56 heads of 128: 304 us, 6.2
// TB/s, the rate of the best plain read-modify-write.
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
        store4<T>(reinterpret_cast<T*>(a.o) + nh * DV + col, q);
    }
#pragma unroll
    for (int m = 0; m < RPT; ++m) {
#pragma unroll
        for (int j = 0; j < 4; ++j) s[m][j] = fmaf(al, s[m][j], kk[m] * u[j]);
        __builtin_nontemporal_store(s[m], reinterpret_cast<f32x4_t*>(Sp + (long long)(NRG * m) * DV));
    }
}

namespace {

template <typename T, int DK, int NSW, bool OUT> hipError_t run_chunks(DeltaArgs a, hipStream_t s) {
    a.slices = a.dv / (16 * NSW);
    a.id_slices = OUT ? 0 : DK / (16 * NSW);
    a.n_units = (long long)a.BH * a.n_seg_launch * (a.slices + a.id_slices);
    a.per_xcd = (a.n_units + 7) / 8;
    if (a.n_units > (1LL << 22)) return hipErrorInvalidValue;
    kda_delta_prefill_kernel<T, DK, NSW, OUT><<<dim3((unsigned)(8 * a.per_xcd)), 64 * (NSW + chunk_waves<T>(NSW)), 0, s>>>(a);
    return hipGetLastError();
}
template <typename T, int DK> hipError_t prefill_t(bool out, int width, const DeltaArgs& a, hipStream_t s) {
    if (out) return width == 128 ? run_chunks<T, DK, 8, true>(a, s) : run_chunks<T, DK, 4, true>(a, s);
    if constexpr (DK == 128)
        if (width == 128) return run_chunks<T, DK, 8, false>(a, s);
    return run_chunks<T, DK, 4, false>(a, s);
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

hipError_t launch_delta_prefill(bool out, int dk, bool f32, int width, const DeltaArgs& a, hipStream_t s) {
    if (dk == 64) return f32 ? prefill_t<float, 64>(out, width, a, s) : prefill_t<__bf16, 64>(out, width, a, s);
    return f32 ? prefill_t<float, 128>(out, width, a, s) : prefill_t<__bf16, 128>(out, width, a, s);
}
hipError_t launch_delta_join(int dk, int dv, int bh, int n_seg, const float* M, const int* dead, const float* S0, float* S_in, hipStream_t s) {
    const dim3 grid((unsigned)bh, (unsigned)(dv / 16));
    if (dk == 64) kda_delta_join_kernel<64><<<grid, 256, 0, s>>>(M, dead, S0, S_in, n_seg, dv);
    else kda_delta_join_kernel<128><<<grid, 512, 0, s>>>(M, dead, S0, S_in, n_seg, dv);
    return hipGetLastError();
}
hipError_t launch_delta_step(int dk, bool f32, const DeltaArgs& a, hipStream_t s) {
    return f32 ? step_of<float>(dk, a, s) : step_of<__bf16>(dk, a, s);
}

}  // namespace kda
