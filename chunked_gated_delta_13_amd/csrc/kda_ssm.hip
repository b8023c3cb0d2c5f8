// Selective state space scan for gfx950: prompts and single tokens.
//
// Per sequence and head, with a state S (n x p, fp32), dt_t = softplus(raw_t + bias), decay
// a_t = dt_t A (one number per head and token):
//   S <- e^{a_t} S + dt_t B_t x_t^T,      y_t = (S^T C_t + D x_t) silu(z_t)
//
// Prompt.  Tokens run in chunks of 64.  With c_i the sum of a over the chunk up to token i,
//   y_i  = sum_{j <= i} e^{c_i - c_j} dt_j (C_i . B_j) x_j + e^{c_i} S^T C_i
//   S   <- e^{c_63} S + sum_j B_j (e^{c_63 - c_j} dt_j x_j)^T
// which are products for the matrix cores.  Every exponent is a sum of a's of consecutive tokens,
// never a quotient of large factors, so nothing overflows that the recurrence itself does not.
// One workgroup of p/16 waves runs a (sequence, head, segment) with the state in registers: a wave holds
// 16 columns of S as accumulator tiles, which are at once the operand of S^T C (with S rounded to bf16
// for that product only).  The weights M_ij of x_j are rounded to bf16 as the other operand that forms y:
// in two parts they would need a second set of LDS tiles, for which the wide form has no room (151 of 160 KB),
// and the product again.  Both roundings leave y 2.2e-3 off, 1.7e-3 of it the output's own; S alone in two
// parts leaves 2.0e-3 and takes 1067 us instead of 1007 for the prompts below.  x, B and C are staged once per chunk in LDS and read there both row by row
// and transposed.  The update must not lose the state's 32 bits: x and B are exact in bf16 and the
// weighted x is fed as three bf16 parts (24 bits of it), three products instead of one.
// A long sequence is split into segments where there are fewer (sequence, head) pairs than the GPU holds
// workgroups: a first pass forms every segment's final state from zero, a small kernel joins them (the
// transition of a segment is one number per head), and the second pass runs every segment from its entry
// state.
// What bounds it: 4 x 16384 tokens of 56 heads, n = p = 128, bf16, take 1.01 ms, 297 TFLOP/s of the
// formulas' products; the 2.87 GB they cannot do without take 0.58 ms.  A SIMD holds two waves, each a
// chain LDS - matrix cores - vector unit - LDS, and of 8000 cycles a chunk issues vector instructions in
// 4300 and products in 2430; the 224 sequences and heads leave 32 of 256 compute units without work.  One sequence of 20001 tokens, 16 heads, n = 128, p = 64 takes 90 us, 26 of
// them the first pass, 9 the join between two launches, 55 the outputs (ten chunks one after the other).
// In fp32, 4 x 4096 tokens of 56 heads take 861 us at n = p = 128 (matrix cores busy in 72% of the cycles; the
// formulas' products at a library product's 154 TFLOP/s would take 488), 616 at p = 64 and 390 at n = p = 64.
//
// Token.  One streaming pass over the state, bound by HBM: 8 bytes of traffic per state element.
#include "kda_mixers.h"
#include "kda_tile.h"

namespace kda {

namespace {

constexpr int kC = 64;             // tokens per chunk
constexpr float kDecayMin = -160;  // exponents of 2 at or below this give zero

// log(1 + e^v).  With w = 1 + u rounded, log(w) u / (w - 1) is log(1 + u) to fp32 also for small u.
__device__ __forceinline__ float softplus_f32(float v) {
    const float u = __expf(-fabsf(v)), w = 1.0f + u;
    const float l = w == 1.0f ? u : __logf(w) * (u * __builtin_amdgcn_rcpf(w - 1.0f));
    return fmaxf(v, 0.0f) + l;
}
__device__ __forceinline__ float silu_f32(float x) { return x * __builtin_amdgcn_rcpf(1.0f + __expf(-x)); }

// v of the lane that a DPP control names, 0 where there is none (or where the row mask leaves out).
template <int CTRL, int ROWS> __device__ __forceinline__ double dpp_f64(double v) {
    const u32x2_t u = __builtin_bit_cast(u32x2_t, v);
    const u32x2_t w = {(unsigned)__builtin_amdgcn_update_dpp(0, (int)u[0], CTRL, ROWS, 0xF, true),
                       (unsigned)__builtin_amdgcn_update_dpp(0, (int)u[1], CTRL, ROWS, 0xF, true)};
    return __builtin_bit_cast(double, w);
}

// Running sum over the 64 lanes of a wave, by data-parallel moves: inside rows of 16 lanes (shifts by 1, 2,
// 4, 8), then the last lane of a row into the next row, and of the lower half into the upper one.  In 64
// bits: decays of neighbouring tokens are differences of these sums, which may be large.
__device__ __forceinline__ double wave_prefix(double v) {
    v += dpp_f64<0x111, 0xF>(v);
    v += dpp_f64<0x112, 0xF>(v);
    v += dpp_f64<0x114, 0xF>(v);
    v += dpp_f64<0x118, 0xF>(v);
    v += dpp_f64<0x142, 0xA>(v);
    v += dpp_f64<0x143, 0xC>(v);
    return v;
}
__device__ __forceinline__ double last_lane(double v) {
    const u32x2_t u = __builtin_bit_cast(u32x2_t, v);
    const u32x2_t w = {(unsigned)__builtin_amdgcn_readlane((int)u[0], 63), (unsigned)__builtin_amdgcn_readlane((int)u[1], 63)};
    return __builtin_bit_cast(double, w);
}

// x times w (per contraction slot) as a sum of operands.  bf16: the fp32 product is cut into three parts
// of 8 bits, high halves of its bit pattern and of what is left, which loses nothing but the last bit.
__device__ __forceinline__ void weigh(Frag<__bf16> (&f)[3], const Frag<__bf16>& x, const float (&w)[8]) {
    union { bf16x8_t v; uint32_t u[4]; } in, out[3];
    in.v = x.v;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float a = __uint_as_float(in.u[j] << 16) * w[2 * j], b = __uint_as_float(in.u[j] & 0xffff0000u) * w[2 * j + 1];
        const uint32_t a0 = __float_as_uint(a), b0 = __float_as_uint(b);
        const float a1 = a - __uint_as_float(a0 & 0xffff0000u), b1 = b - __uint_as_float(b0 & 0xffff0000u);
        const uint32_t a1u = __float_as_uint(a1), b1u = __float_as_uint(b1);
        const float a2 = a1 - __uint_as_float(a1u & 0xffff0000u), b2 = b1 - __uint_as_float(b1u & 0xffff0000u);
        out[0].u[j] = __builtin_amdgcn_perm(b0, a0, 0x07060302u);
        out[1].u[j] = __builtin_amdgcn_perm(b1u, a1u, 0x07060302u);
        out[2].u[j] = __builtin_amdgcn_perm(__float_as_uint(b2), __float_as_uint(a2), 0x07060302u);
    }
#pragma unroll
    for (int i = 0; i < 3; ++i) f[i].v = out[i].v;
}
__device__ __forceinline__ void weigh(Frag<float> (&f)[1], const Frag<float>& x, const float (&w)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[0].v[j] = x.v[j] * w[j];
}

template <typename T> struct Parts { static constexpr int n = 3; };
template <> struct Parts<float> { static constexpr int n = 1; };

// A wave's share of 64 rows of WIDTH elements: requested one chunk ahead into registers, put into the
// tile when the last chunk's readers are done.  Rows past a partial chunk's last one lie past the
// buffer's end and come as zeros.
template <typename T, int WIDTH, int NW> struct Stage {
    typedef TileSteps<T, kC, WIDTH, NW> Steps;
    static constexpr uint32_t ES = sizeof(T);
    u32x4_t v[Steps::N];
    __device__ __forceinline__ void load(const T* base, uint32_t step, int rows, int wave, int lane) {
        const buffer_t buf = make_rows(base, rows, step, WIDTH * ES);
        const uint32_t off = TileStep<T>::row(lane) * step + 16u * TileStep<T>::piece(lane);
        const uint32_t first = Steps::group0(wave) * TileStep<T>::ROWS * step + Steps::block0(wave) * 32 * ES;
#pragma unroll
        for (int i = 0; i < Steps::N; ++i)
            v[i] = buffer_load16(buf, off, first + Steps::group(i) * TileStep<T>::ROWS * step + Steps::block(i) * 32 * ES);
    }
    __device__ __forceinline__ void put(KDA_LDS T* tile, int wave, int lane) const {
        TilePut<T, kC> p;
        p.set(tile + Steps::block0(wave) * kC * 32, Steps::group0(wave), lane);
#pragma unroll
        for (int i = 0; i < Steps::N; ++i) p.put(Steps::group(i), Steps::block(i), v[i]);
    }
};

// The weights of token tiles kb and kb + 2 at this lane's slots.
__device__ __forceinline__ void load_weights(float (&w)[8], const KDA_LDS float* p) {
    const f32x4_t lo = *reinterpret_cast<const KDA_LDS f32x4_t*>(p);
    const f32x4_t hi = *reinterpret_cast<const KDA_LDS f32x4_t*>(p + 32);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w[i] = lo[i];
        w[4 + i] = hi[i];
    }
}

// A uniform value that the compiler may not carry over from an earlier use.
__device__ __forceinline__ int pinned_s(int x) {
    asm volatile("" : "+s"(x));
    return x;
}

// Numbers of one chunk.
struct ChunkDecay {
    float hi[kC];      // sum of the exponents (base 2) up to this token
    float lo[kC];      // what `hi` leaves of that sum
    float dt[kC];      // fp32: dt; bf16: lo - log2 dt
    float e[kC];       // factor of S^T C: 2^sum
    float w[kC];       // weight of the token in the state's update
    float sum;         // of the whole chunk
    float factor;      // 2^sum of the whole chunk
};

// By one wave, lane = token.  OUT: with the numbers that outputs take.
template <typename T, bool OUT>
__device__ __forceinline__ void chunk_decay(KDA_LDS ChunkDecay* c, float raw, bool live, float A2, int lane) {
    const float d = live ? softplus_f32(raw) : 0.0f;
    const double s = wave_prefix(live ? (double)fmaxf(d * A2, kDecayMin) : 0.0);
    const double end = last_lane(s);
    const float hi = (float)s;
    if constexpr (OUT) {
        const float lo = (float)(s - (double)hi);
        c->hi[lane] = hi;
        c->lo[lane] = lo;
        // bf16: 2^(c_i - c_j) dt_j as one exponential; dt = 0 gives +inf here and a factor of 0
        c->dt[lane] = sizeof(T) == 4 ? d : lo - __log2f(d);
        c->e[lane] = fast_exp2(hi);
    }
    c->w[lane] = fast_exp2((float)(end - s)) * d;
    if (lane == 0) {
        c->sum = (float)end;
        c->factor = fast_exp2((float)end);
    }
}

// A lane's place in the tiles of one workgroup, and the three parts of a chunk's work.  N x P state, NW
// waves of P / NW columns each.  LDS tiles have kC rows.
template <int N, int P, typename T, int NW> struct Mixer {
    static constexpr int WC = P / NW, NCT = WC / 16, NT = N / 16, NP = Parts<T>::n;
    typedef typename Vec4<T>::type vec4;
    typedef f32x4_t State[NT][NCT];
    TileRows<T, kC, N> rb, rc;    // rows of B and of C
    TileCols<T, kC> cb;           // columns of B
    TileRows<T, kC, kC> rm;       // rows of M
    TileCols<T, kC> cx[NCT];      // this wave's column tiles of x
    KDA_LDS T* xrow[NCT];         // its four columns of row r of x

    __device__ __forceinline__ void set_bc(KDA_LDS T* sB, KDA_LDS T* sC, int lane) {
        rb.set(sB, lane);
        rc.set(sC, lane);
    }
    __device__ __forceinline__ void set_x(KDA_LDS T* sX, int wave, int lane) {
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct) {
            cx[ct].set_tile(sX, lane, wave * NCT + ct);
            xrow[ct] = lds_pin(sX + tile_at<T, kC>(lane & 15, 4 * (wave * NCT + ct) + (lane >> 4)));
        }
    }

    // M[i][j] = e^{c_i - c_j} dt_j (C_i . B_j) for j <= i, rounded to T: K of the ten lower 16 x 16 tiles side by side
    // (pair 0 .. 9, row by row), each a chain from LDS through the matrix cores and an exponential
    template <int K>
    __device__ __forceinline__ void mix(KDA_LDS T* sM, const KDA_LDS ChunkDecay* cd, const int (&pair)[K], int lane) const {
        constexpr int Q = N / 32;
        const int g = lane >> 4, r = lane & 15;
        Frag<T> fb[K][Q], fc[K][Q];
        int ti[K], tj[K];
        float ci[K], li[K];
        f32x4_t cj[K], dj[K];
#pragma unroll
        for (int p = 0; p < K; ++p) {
            ti[p] = pair[p] < 1 ? 0 : (pair[p] < 3 ? 1 : (pair[p] < 6 ? 2 : 3));
            tj[p] = pair[p] - ti[p] * (ti[p] + 1) / 2;
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                rb.frag(fb[p][q], 16 * 32 * tj[p], 0, q);
                rc.frag(fc[p][q], 16 * 32 * ti[p], 0, q);
            }
            ci[p] = cd->hi[16 * ti[p] + r];
            li[p] = cd->lo[16 * ti[p] + r];
            cj[p] = *reinterpret_cast<const KDA_LDS f32x4_t*>(cd->hi + 16 * tj[p] + 4 * g);
            dj[p] = *reinterpret_cast<const KDA_LDS f32x4_t*>(cd->dt + 16 * tj[p] + 4 * g);
        }
        __builtin_amdgcn_sched_barrier(0);
        f32x4_t acc[K];   // acc[p][k]: token j = 16 tj + 4 g + k against i = 16 ti + r
#pragma unroll
        for (int q = 0; q < Q; ++q)
#pragma unroll
            for (int p = 0; p < K; ++p) acc[p] = mma(fb[p][q], fc[p][q], q == 0 ? zero4() : acc[p]);
#pragma unroll
        for (int p = 0; p < K; ++p) {
            float m[4];
            // sums of a chunk may be large and the decay between two of its tokens small: differences of the
            // high parts (exact where they are near each other) and of the low parts
            if constexpr (sizeof(T) == 4) {
                const f32x4_t lj = *reinterpret_cast<const KDA_LDS f32x4_t*>(cd->lo + 16 * tj[p] + 4 * g);
#pragma unroll
                for (int k = 0; k < 4; ++k) m[k] = acc[p][k] * (fast_exp2((ci[p] - cj[p][k]) + (li[p] - lj[k])) * dj[p][k]);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) m[k] = acc[p][k] * fast_exp2((ci[p] - cj[p][k]) + (li[p] - dj[p][k]));
            }
            if (ti[p] == tj[p]) {
#pragma unroll
                for (int k = 0; k < 4; ++k) m[k] = 4 * g + k <= r ? m[k] : 0.0f;
            }
            lds_store_run<4>(sM + 16 * 32 * ti[p] + tile_at<T, kC>(r, 4 * tj[p] + g), m);
        }
    }
    // The tiles first, first + step, .., K at a time
    template <int K>
    __device__ __forceinline__ void mix_every(KDA_LDS T* sM, const KDA_LDS ChunkDecay* cd, int first, int step, int lane) const {
        int pair = first;
        if constexpr (K == 2)
            for (; pair + step < 10; pair += 2 * step) mix<2>(sM, cd, {pair, pair + step}, lane);
        for (; pair < 10; pair += step) mix<1>(sM, cd, {pair}, lane);
    }

    // x of this wave's columns, transposed: contraction over tokens
    __device__ __forceinline__ void load_x(Frag<T> (&xt)[2][NCT]) const {
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) cx[ct].frag(xt[q][ct], 0, 0, q);
    }

    // y^T = (S^T C^T) e^{c_i} + x^T M^T, the skip term and the gate: columns are tokens, rows p
    __device__ __forceinline__ void outputs(const State& S, const Frag<T> (&xt)[2][NCT], const vec4 (&zv)[4][NCT], bool gated,
                                            float Dh, const KDA_LDS ChunkDecay* cd, buffer_t ybuf, uint32_t y_off,
                                            uint32_t y_step, int lane) const {
        const int r = lane & 15;
        constexpr int Q = N / 32;
        f32x4_t y[4][NCT];
        Frag<T> fc[2][4], fm[4][2];
        float e[4];
        vec4 xv[4][NCT];
        // operands are requested one block ahead of the products that use them
#pragma unroll
        for (int ti = 0; ti < 4; ++ti) rc.frag(fc[0][ti], 0, ti, 0);
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            if (q + 1 < Q) {
#pragma unroll
                for (int ti = 0; ti < 4; ++ti) rc.frag(fc[(q + 1) & 1][ti], 0, ti, q + 1);
            } else {
#pragma unroll
                for (int ti = 0; ti < 4; ++ti) {
                    e[ti] = cd->e[16 * ti + r];
                    // token tiles 0 and 2, then 1 and 3, as far as they reach
                    if (ti < 2) rm.frag_lo(fm[ti][0], 0, ti, 0);
                    else rm.frag(fm[ti][0], 0, ti, 0);
                    if (ti == 3) rm.frag(fm[ti][1], 0, ti, 1);
                    else if (ti > 0) rm.frag_lo(fm[ti][1], 0, ti, 1);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
            Frag<T> fs[NCT];
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) acc_pair_frag<T>(fs[ct], S[q][ct], S[q + NT / 2][ct], true);
#pragma unroll
            for (int ti = 0; ti < 4; ++ti)
#pragma unroll
                for (int ct = 0; ct < NCT; ++ct) y[ti][ct] = mma(fs[ct], fc[q & 1][ti], q == 0 ? zero4() : y[ti][ct]);
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int ti = 0; ti < 4; ++ti)
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) xv[ti][ct] = *reinterpret_cast<const volatile KDA_LDS vec4*>(xrow[ct] + 16 * 32 * ti);
#pragma unroll
        for (int ti = 0; ti < 4; ++ti)
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) {
#pragma unroll
                for (int k = 0; k < 4; ++k) y[ti][ct][k] *= e[ti];
                y[ti][ct] = mma(xt[0][ct], fm[ti][0], y[ti][ct]);
                if (ti > 0) y[ti][ct] = mma(xt[1][ct], fm[ti][1], y[ti][ct]);
            }
#pragma unroll
        for (int ti = 0; ti < 4; ++ti)
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) {
                f32x4_t o;
#pragma unroll
                for (int k = 0; k < 4; ++k) o[k] = fmaf(Dh, to_f32<T>((T)xv[ti][ct][k]), y[ti][ct][k]);
                if (gated) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) o[k] *= silu_f32(to_f32<T>((T)zv[ti][ct][k]));
                }
                vec4 ov;
#pragma unroll
                for (int k = 0; k < 4; ++k) ov[k] = from_f32<T>(o[k]);
                buffer_store4(ov, ybuf, y_off, 16 * ti * y_step + 16 * ct * (uint32_t)sizeof(T));
            }
    }

    // S <- e^{c_63} S + B^T (w x).  The chunk's sum starts from zero and is added to the decayed state with
    // one rounding: the matrix cores drop low bits when they add to a large accumulator, always towards
    // zero, which a state that decays slowly would collect over many chunks.
    __device__ __forceinline__ void update(State& S, const Frag<T> (&xt)[2][NCT], const KDA_LDS ChunkDecay* cd, int lane) const {
        const float f = cd->factor;
        // groups of NG row tiles of the state; a group's columns of B are requested while the products of the
        // group before run, and its sums join the state beside the products of the next one
        constexpr int NG = 2, NGR = NT / NG;
        Frag<T> fb[2][NG][2], xs[2][NCT][NP];
        float w[2][8];
        load_weights(w[0], cd->w + 4 * (lane >> 4));
        load_weights(w[1], cd->w + 16 + 4 * (lane >> 4));
#pragma unroll
        for (int i = 0; i < NG; ++i)
#pragma unroll
            for (int q = 0; q < 2; ++q) cb.frag(fb[0][i][q], 0, i, q);
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) weigh(xs[q][ct], xt[q][ct], w[q]);
        f32x4_t acc[2][NG][NCT];
        auto join = [&](int j) {
#pragma unroll
            for (int i = 0; i < NG; ++i)
#pragma unroll
                for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
                    for (int k = 0; k < 4; ++k) S[j * NG + i][ct][k] = fmaf(f, S[j * NG + i][ct][k], acc[j & 1][i][ct][k]);
        };
#pragma unroll
        for (int j = 0; j < NGR; ++j) {
            if (j + 1 < NGR) {
#pragma unroll
                for (int i = 0; i < NG; ++i)
#pragma unroll
                    for (int q = 0; q < 2; ++q) cb.frag(fb[(j + 1) & 1][i][q], 0, (j + 1) * NG + i, q);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int k = NP - 1; k >= 0; --k)
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                    for (int i = 0; i < NG; ++i)
#pragma unroll
                        for (int ct = 0; ct < NCT; ++ct)
                            acc[j & 1][i][ct] =
                                mma(fb[j & 1][i][q], xs[q][ct][k], k == NP - 1 && q == 0 ? zero4() : acc[j & 1][i][ct]);
            if (j > 0) join(j - 1);
        }
        join(NGR - 1);
    }

    // A state in memory, p as the lane's element of row tile 0, column tile 0 (byte offset `off`).
    __device__ __forceinline__ static uint32_t state_off(int wave, int lane) {
        return (uint32_t)((4 * (lane >> 4) * P + wave * WC + (lane & 15)) * sizeof(float));
    }
    __device__ __forceinline__ static void load_state(State& S, const float* p, uint32_t off) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) S[nt][ct] = zero4();
        if (p) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
                    for (int k = 0; k < 4; ++k) S[nt][ct][k] = *at_byte(p + (16 * nt + k) * P + 16 * ct, off);
        }
    }
    __device__ __forceinline__ static void store_state(const State& S, float* p, uint32_t off) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
                for (int k = 0; k < 4; ++k) *at_byte(p + (16 * nt + k) * P + 16 * ct, off) = S[nt][ct][k];
    }
};

}  // namespace

// OUT: with outputs (the pass that runs every segment from its entry state), else final states only: two
// sets of tiles and one barrier per chunk.
// AHEAD: M of the next chunk is formed beside the outputs of this one, over three sets of B and C tiles,
// two of x and two of M: one barrier per chunk, and every wave has independent work for the matrix
// cores, the vector unit and the LDS all through it.  It takes most of the LDS, so one workgroup runs per
// compute unit: taken for p = 128 in bf16, whose eight waves fill it alone (1.01 ms for the long prompts
// above, 1.22 with the plain schedule of three barriers).  The plain one leaves room for a second
// workgroup, which p = 64 needs; fp32 tiles leave no room for more sets.
template <int N, int P, typename T, bool OUT, int NW, bool AHEAD>
__global__ __launch_bounds__(64 * NW, sizeof(T) == 2 ? 2 : 1) void kda_ssm_prefill_kernel(const SsmArgs a) {
    typedef Mixer<N, P, T, NW> Mix;
    typedef typename Mix::vec4 vec4;
    constexpr int WC = Mix::WC, NCT = Mix::NCT;
    constexpr uint32_t ES = sizeof(T), ROW_P = P * ES;
    constexpr int NBC = AHEAD ? 3 : (OUT ? 1 : 2), NXM = AHEAD || !OUT ? 2 : 1, ND = AHEAD ? 3 : 2 * NW;
    // LDS: B, C (with outputs), M (likewise), x tiles (elements), then the numbers of two or three chunks
    constexpr int oC = NBC * kC * N, oM = OUT ? 2 * oC : oC, oX = oM + (OUT ? NXM * kC * kC : 0), oEnd = oX + NXM * kC * P;
    __shared__ __attribute__((aligned(16))) T smem[oEnd];
    __shared__ __attribute__((aligned(16))) ChunkDecay sD_[ND];
    KDA_LDS T* sB = (KDA_LDS T*)smem;
    KDA_LDS T* sC = sB + oC;
    KDA_LDS T* sM = sB + oM;
    KDA_LDS T* sX = sB + oX;
    KDA_LDS ChunkDecay* sD = (KDA_LDS ChunkDecay*)sD_;

    // unit = (b, segment, h), heads fastest: the heads of a segment share B and C, and each XCD takes a
    // contiguous range of units
    const uint32_t unit = (blockIdx.x & 7) * (uint32_t)a.per_xcd + (blockIdx.x >> 3);
    if (unit >= (uint32_t)a.n_units) return;
    const int h = (int)(unit % (uint32_t)a.H);
    const uint32_t bs = unit / (uint32_t)a.H;
    const int s = (int)(bs % (uint32_t)a.n_seg_launch);
    const int b = (int)(bs / (uint32_t)a.n_seg_launch);
    const long long bh = (long long)b * a.H + h;
    const int grp = (int)((uint32_t)h / ((uint32_t)a.H / (uint32_t)a.G));

    long long len = a.T;
    if (a.lens) {
        const int l = a.lens[b];
        len = l < 0 ? 0 : (l > a.T ? a.T : l);
    }
    const long long t_begin = (long long)s * a.seg_len;
    long long t_end = t_begin + a.seg_len < len ? t_begin + a.seg_len : len;
    if (t_end < t_begin) t_end = t_begin;
    const bool last = OUT && s == a.n_seg - 1;
    if (OUT && t_end == t_begin && !(last && a.S_T)) return;

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, r = lane & 15;

    // the current row of every input, and the bytes between rows
    const long long row0 = (long long)b * a.T + t_begin;
    const T* xp = reinterpret_cast<const T*>(a.x) + row0 * a.x_stride + (long long)h * P;
    const T* bp = reinterpret_cast<const T*>(a.Bm) + row0 * a.b_stride + (long long)grp * N;
    const T* cp = reinterpret_cast<const T*>(a.Cm) + row0 * a.c_stride + (long long)grp * N;
    const T* dp = reinterpret_cast<const T*>(a.dt) + row0 * a.dt_stride + h;
    const T* zp = reinterpret_cast<const T*>(a.z);
    const bool gated = OUT && zp != nullptr;
    if (gated) zp += row0 * a.z_stride + (long long)h * P;
    T* yp = OUT ? reinterpret_cast<T*>(a.y) + (row0 * a.H + h) * P : nullptr;
    const uint32_t x_step = (uint32_t)a.x_stride * ES, b_step = (uint32_t)a.b_stride * ES, c_step = (uint32_t)a.c_stride * ES;
    const uint32_t dt_step = (uint32_t)a.dt_stride * ES, z_step = (uint32_t)a.z_stride * ES, y_step = (uint32_t)a.H * ROW_P;
    const uint32_t z_off = r * z_step + (wave * WC + 4 * g) * ES, y_off = r * y_step + (wave * WC + 4 * g) * ES;
    const float A2 = a.A[h] * kLog2e;
    const float bias = a.dt_bias ? a.dt_bias[h] : 0.0f;
    const float Dh = a.D ? a.D[h] : 0.0f;

    // entry state
    typename Mix::State S;
    const uint32_t s_off = Mix::state_off(wave, lane);
    const float* sin = nullptr;
    if (s == 0 && !(OUT && a.keep_S0)) {
        if (a.S0) sin = a.S0 + bh * (long long)(N * P);
    } else if (OUT) {
        sin = a.ws_state + (bh * a.n_seg + s) * (long long)(N * P);
    }
    Mix::load_state(S, sin, s_off);
    // S_T is S0: the other pass's last segment overwrites it
    if (!OUT && s == 0 && a.keep_S0) Mix::store_state(S, a.ws_state + bh * a.n_seg * (long long)(N * P), s_off);

    float total = 0.0f;   // exponent (base 2) of the segment's decay
    Mix mx;
    // Rows of B, C and x are requested into registers a chunk or more before they are put into their
    // tiles; the raw steps (one wave) a chunk before their sums, a long chain that this wave forms while
    // others work on M.  Requests past the end name empty buffers instead of being skipped: straight code
    // lets every wait count the requests behind it.
    Stage<T, P, NW> gx;
    Stage<T, N, NW> gb, gc;
    float gdt = 0.0f;
    int left = (int)(t_end - t_begin);   // tokens left, from the chunk at hand on
    auto rows_at = [&](int ahead) { return left - ahead < kC ? left - ahead : kC; };
    auto request_bc = [&](int ahead) {   // the chunk `ahead` tokens from the one at hand
        gb.load(bp + ahead * a.b_stride, b_step, rows_at(ahead), wave, lane);
        if constexpr (OUT) gc.load(cp + ahead * a.c_stride, c_step, rows_at(ahead), wave, lane);
    };
    auto put_bc = [&](int buf) {
        gb.put(sB + buf * kC * N, wave, lane);
        if constexpr (OUT) gc.put(sC + buf * kC * N, wave, lane);
    };
    auto request_x = [&](int ahead) { gx.load(xp + ahead * a.x_stride, x_step, rows_at(ahead), wave, lane); };
    auto request_dt = [&](int ahead) {
        gdt = buffer_load1(dp, make_rows(dp + ahead * a.dt_stride, rows_at(ahead), dt_step, ES), lane * dt_step);
    };
    auto decay = [&](int ahead, int buf) { chunk_decay<T, OUT>(sD + buf, gdt + bias, ahead + lane < left, A2, lane); };
    vec4 zv[4][NCT];
    auto request_z = [&](int ahead) {
        const buffer_t zbuf = make_rows(zp + ahead * a.z_stride, gated ? rows_at(ahead) : 0, z_step, ROW_P);
#pragma unroll
        for (int ti = 0; ti < 4; ++ti)
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) buffer_load4(zv[ti][ct], zbuf, z_off, 16 * ti * z_step + 16 * ct * ES);
    };
    auto y_buffer = [&]() { return make_rows(yp, rows_at(0), y_step, ROW_P); };
    auto advance = [&]() {
        xp += kC * a.x_stride;
        bp += kC * a.b_stride;
        cp += kC * a.c_stride;
        dp += kC * a.dt_stride;
        if (gated) zp += kC * a.z_stride;
        if constexpr (OUT) yp += (long long)kC * a.H * P;
        left -= kC;
    };
    if constexpr (!AHEAD) {
        // Decays are a long chain on one wave: NW chunks' at a time, a chunk per wave, NW chunks ahead.  (By one
        // wave chunk by chunk, while the others wait: 92 us for 20001 tokens of 16 heads.)
        auto decay_many = [&](int c) {
            decay((NW + wave) * kC, (c + NW + wave) & (2 * NW - 1));
            request_dt((2 * NW + wave) * kC);
        };
        if (left > 0) {
            request_dt(wave * kC);
            decay(wave * kC, wave);
            request_dt((NW + wave) * kC);
            request_bc(0);
            request_x(0);
        }
        if constexpr (!OUT) {
            // two sets of tiles: one barrier per chunk
            if (left > 0) {
                put_bc(0);
                gx.put(sX, wave, lane);
                request_bc(kC);
                request_x(kC);
                __syncthreads();
            }
            for (int c = 0, par = 0; left > 0; ++c, par ^= 1) {
                const KDA_LDS ChunkDecay* cd = sD + (c & (2 * NW - 1));
                put_bc(par ^ 1);
                gx.put(sX + (par ^ 1) * kC * P, wave, lane);
                request_bc(2 * kC);
                request_x(2 * kC);
                mx.cb.set(sB + par * kC * N, lane);
                mx.set_x(sX + par * kC * P, wave, lane);
                Frag<T> xt[2][NCT];
                mx.load_x(xt);
                mx.update(S, xt, cd, lane);
                if ((c & (NW - 1)) == 0) decay_many(c);
                total += cd->sum;
                __syncthreads();
                advance();
            }
        } else {
            mx.set_bc(sB, sC, lane);
            mx.cb.set(sB, lane);
            mx.rm.set(sM, lane);
            mx.set_x(sX, wave, lane);
            for (int c = 0; left > 0; ++c) {
                const KDA_LDS ChunkDecay* cd = sD + (c & (2 * NW - 1));
                put_bc(0);
                gx.put(sX, wave, lane);
                __syncthreads();
                request_z(0);
                // (the first tile is taken as new in every chunk: its addresses are not worth registers)
                mx.template mix_every<2>(sM, cd, pinned_s(wave), NW, lane);
                if ((c & (NW - 1)) == 0) decay_many(c);
                __syncthreads();
                Frag<T> xt[2][NCT];
                mx.load_x(xt);
                mx.outputs(S, xt, zv, gated, Dh, cd, y_buffer(), y_off, y_step, lane);
                // requested here, where the outputs' registers are free again
                request_bc(kC);
                request_x(kC);
                mx.update(S, xt, cd, lane);
                total += cd->sum;
                __syncthreads();
                advance();
            }
        }
    } else if (left > 0) {
        // The wave that forms the decays, and the waves 0 .. MW - 1 that form M.  Of two waves on a SIMD the
        // older one is served first and has time left at the barrier: with all eight sharing this work, waves
        // 0 - 3 waited 3000 of 9300 cycles a chunk for waves 4 - 7.
        constexpr int DW = NW / 2 - 1, MW = DW;
        // chunks 0 and 1 of B and C, chunk 0 of x, M of chunk 0
        request_bc(0);
        request_x(0);
        if (wave == DW) {
            request_dt(0);
            decay(0, 0);
            request_dt(kC);
            decay(kC, 1);
            request_dt(2 * kC);
        }
        put_bc(0);
        gx.put(sX, wave, lane);
        request_bc(kC);
        request_x(kC);
        put_bc(1);
        __syncthreads();
        mx.set_bc(sB, sC, lane);
        mx.template mix_every<1>(sM, sD, wave, NW, lane);
        request_bc(2 * kC);
        request_z(0);
        __syncthreads();
        int c3 = 0, n3 = 1, f3 = 2;   // tiles of this chunk, the next one, and the one after it
        for (int par = 0; left > 0; par ^= 1) {
            const KDA_LDS ChunkDecay* cd = sD + c3;
            put_bc(f3);
            gx.put(sX + (par ^ 1) * kC * P, wave, lane);
            request_bc(3 * kC);
            request_x(2 * kC);
            mx.rc.set(sC + c3 * kC * N, lane);
            mx.cb.set(sB + c3 * kC * N, lane);
            mx.rm.set(sM + par * kC * kC, lane);
            mx.set_x(sX + par * kC * P, wave, lane);
            Frag<T> xt[2][NCT];
            mx.load_x(xt);
            mx.outputs(S, xt, zv, gated, Dh, cd, y_buffer(), y_off, y_step, lane);
            request_z(kC);
            mx.update(S, xt, cd, lane);
            total += cd->sum;
            mx.set_bc(sB + n3 * kC * N, sC + n3 * kC * N, lane);
            if (wave < MW) mx.template mix_every<1>(sM + (par ^ 1) * kC * kC, sD + n3, pinned_s(wave), MW, lane);
            if (wave == DW) {
                decay(2 * kC, f3);
                request_dt(3 * kC);
            }
            __syncthreads();
            advance();
            const int t3 = c3;
            c3 = n3;
            n3 = f3;
            f3 = t3;
        }
    }

    float* so = nullptr;
    if (OUT) {
        if (last && a.S_T) so = a.S_T + bh * (long long)(N * P);
    } else {
        so = a.ws_state + (bh * a.n_seg + s + 1) * (long long)(N * P);
        if (tid == 0) a.ws_decay[bh * a.n_seg + s + 1] = total;
    }
    if (so) Mix::store_state(S, so, s_off);
}

// Entry states from the segments' final states, in place: slot s + 1 holds the final state of segment s
// from zero (segment 0: from its entry state) and becomes the entry state of segment s + 1.  A thread
// owns two elements and requests kAhead segments at a time: the chain is one multiply-add per segment,
// the loads do not wait for it.
// grid: sequences x heads x (state elements / 512)
__global__ __launch_bounds__(256) void kda_ssm_join_kernel(float* ws, const float* decay, int n_seg, int np) {
    constexpr int kAhead = 8;
    typedef __attribute__((ext_vector_type(2))) float f32x2_t;
    const int per = np / 512;
    const long long bh = blockIdx.x / per;
    const int e = ((int)(blockIdx.x % per) * 256 + threadIdx.x) * 2;
    float* p = ws + (bh * n_seg + 1) * (long long)np + e;
    const float* d = decay + bh * n_seg;
    f32x2_t S = *reinterpret_cast<const f32x2_t*>(p);
    for (int s = 2; s < n_seg; s += kAhead) {
        f32x2_t h[kAhead];
        float f[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int t = s + i < n_seg ? s + i : n_seg - 1;
            h[i] = *reinterpret_cast<const f32x2_t*>(p + (long long)(t - 1) * np);
            f[i] = d[t];
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (s + i >= n_seg) break;
            const float x = fast_exp2(f[i]);
            S[0] = fmaf(x, S[0], h[i][0]);
            S[1] = fmaf(x, S[1], h[i][1]);
            *reinterpret_cast<f32x2_t*>(p + (long long)(s + i - 1) * np) = S;
        }
    }
}

// One token: a workgroup owns one (sequence, head) state, P/4 groups of four columns x 16 row groups, so that
// each XCD streams a contiguous range of states, past the caches.  A thread's rows are all requested
// before the first is used and stored together after the last: 256 sequences of 56 heads, n = p = 128
// (1.89 GB) take 307 us, 6.2 TB/s; each row stored as soon as it is ready, reads and writes mix in
// memory and it takes 329.
template <int N, int P, typename T>
__global__ __launch_bounds__(4 * P) void kda_ssm_step_kernel(const SsmArgs a) {
    constexpr int NCG = P / 4, NRG = 16, NTH = NCG * NRG, NW = NTH / 64, RPT = N / NRG;
    const uint32_t unit = (blockIdx.x & 7) * (uint32_t)a.per_xcd + (blockIdx.x >> 3);
    if (unit >= (uint32_t)a.n_units) return;
    const long long nh = unit, n = unit / (uint32_t)a.H;
    const int h = (int)(unit % (uint32_t)a.H), grp = (int)((uint32_t)h / ((uint32_t)a.H / (uint32_t)a.G));
    const int tid = threadIdx.x, cg = tid % NCG, rg = tid / NCG, lane = tid & 63, wave = tid >> 6, col = 4 * cg;
    float* Sb = a.S_T + nh * (long long)(N * P) + col;
    f32x4_t S[RPT];
#pragma unroll
    for (int m = 0; m < RPT; ++m)
        S[m] = __builtin_nontemporal_load(reinterpret_cast<const f32x4_t*>(Sb + (long long)(rg + NRG * m) * P));
    const T* bp = reinterpret_cast<const T*>(a.Bm) + n * a.b_stride + (long long)grp * N;
    const T* cp = reinterpret_cast<const T*>(a.Cm) + n * a.c_stride + (long long)grp * N;
    const T* xp = reinterpret_cast<const T*>(a.x) + n * a.x_stride + (long long)h * P + col;
    const float raw = to_f32<T>(reinterpret_cast<const T*>(a.dt)[n * a.dt_stride + h]) + (a.dt_bias ? a.dt_bias[h] : 0.0f);
    const float dt = softplus_f32(raw);
    const float dec = fast_exp2(fmaxf(dt * (a.A[h] * kLog2e), kDecayMin));
    typedef __attribute__((ext_vector_type(4))) T vec4;
    const vec4 xv = *reinterpret_cast<const vec4*>(xp);
    f32x4_t x, y = zero4();
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = to_f32<T>((T)xv[j]);
#pragma unroll
    for (int m = 0; m < RPT; ++m) {
        const int i = rg + NRG * m;
        const float bi = dt * to_f32<T>(bp[i]), ci = to_f32<T>(cp[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            S[m][j] = fmaf(dec, S[m][j], bi * x[j]);
            y[j] = fmaf(ci, S[m][j], y[j]);
        }
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int m = 0; m < RPT; ++m)
        __builtin_nontemporal_store(S[m], reinterpret_cast<f32x4_t*>(Sb + (long long)(rg + NRG * m) * P));
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int o = NCG; o < 64; o <<= 1)
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] += __shfl_xor(y[j], o);
    __shared__ __attribute__((aligned(16))) float part[NW][P];
    if (lane < NCG) *reinterpret_cast<f32x4_t*>(&part[wave][col]) = y;
    __syncthreads();
    if (rg == 0) {
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = 0.0f;
#pragma unroll
        for (int w = 0; w < NW; ++w)
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] += part[w][col + j];
        const float Dh = a.D ? a.D[h] : 0.0f;
        vec4 o;
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = fmaf(Dh, x[j], y[j]);
        if (a.z) {
            const vec4 z = *reinterpret_cast<const vec4*>(reinterpret_cast<const T*>(a.z) + n * a.z_stride + (long long)h * P + col);
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] *= silu_f32(to_f32<T>((T)z[j]));
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = from_f32<T>(y[j]);
        *reinterpret_cast<vec4*>(reinterpret_cast<T*>(a.y) + nh * P + col) = o;
    }
}

namespace {

template <int N, int P, typename T>
hipError_t ssm_launch(SsmPass pass, SsmArgs a, hipStream_t s) {
    constexpr int NW = P / 16;
    constexpr bool AHEAD = P == 128 && sizeof(T) == 2;
    a.per_xcd = (a.n_units + 7) / 8;
    const dim3 grid((unsigned)(8 * a.per_xcd));
    switch (pass) {
        case SsmPass::kStates: kda_ssm_prefill_kernel<N, P, T, false, NW, false><<<grid, 64 * NW, 0, s>>>(a); break;
        case SsmPass::kOutputs: kda_ssm_prefill_kernel<N, P, T, true, NW, AHEAD><<<grid, 64 * NW, 0, s>>>(a); break;
        case SsmPass::kToken: kda_ssm_step_kernel<N, P, T><<<grid, 4 * P, 0, s>>>(a); break;
    }
    return hipGetLastError();
}

template <int N, int P>
hipError_t ssm_type(SsmPass pass, bool f32, const SsmArgs& a, hipStream_t s) {
    return f32 ? ssm_launch<N, P, float>(pass, a, s) : ssm_launch<N, P, __bf16>(pass, a, s);
}

}  // namespace

hipError_t launch_ssm(SsmPass pass, int n, int p, bool f32, const SsmArgs& a, hipStream_t s) {
    if (n == 64 && p == 64) return ssm_type<64, 64>(pass, f32, a, s);
    if (n == 64 && p == 128) return ssm_type<64, 128>(pass, f32, a, s);
    if (n == 128 && p == 64) return ssm_type<128, 64>(pass, f32, a, s);
    if (n == 128 && p == 128) return ssm_type<128, 128>(pass, f32, a, s);
    return hipErrorInvalidValue;
}

hipError_t launch_ssm_join(int n, int p, int bh, int n_seg, float* ws_state, const float* ws_decay, hipStream_t s) {
    kda_ssm_join_kernel<<<dim3((unsigned)bh * (n * p / 512)), 256, 0, s>>>(ws_state, ws_decay, n_seg, n * p);
    return hipGetLastError();
}

}  // namespace kda
