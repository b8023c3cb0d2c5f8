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
// One workgroup of four waves runs a (sequence, head, segment) with the state in registers: wave w
// holds p/4 columns of S as accumulator tiles, which are at once the operand of S^T C (with S rounded
// to bf16 for that product only).  x, B and C are staged once per chunk in LDS and read there both row
// by row and transposed.  The update must not lose the state's 32 bits: x and B are exact in bf16 and
// the weighted x is fed as three bf16 parts (24 bits of it), three products instead of one.
// A long sequence is split into segments: a first pass forms every segment's final state from zero, a
// small kernel joins them (the transition of a segment is one number per head), and the second pass
// runs every segment from its entry state.
//
// Token.  One streaming pass over the state, bound by HBM: 8 bytes of traffic per state element.
#include "kda_mixers.h"
#include "kda_tile.h"

namespace kda {

namespace {

constexpr int kC = 64;             // tokens per chunk
constexpr float kDecayMin = -160;  // exponents of 2 at or below this give zero

__device__ __forceinline__ float softplus_f32(float v) { return fmaxf(v, 0.0f) + log1pf(__expf(-fabsf(v))); }
__device__ __forceinline__ float silu_f32(float x) { return x * __builtin_amdgcn_rcpf(1.0f + __expf(-x)); }

// Running sum over the 64 lanes of a wave.  In 64 bits: decays of neighbouring tokens are differences of
// these sums, which may be large.
__device__ __forceinline__ double wave_prefix(double v, int lane) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const double u = __shfl_up(v, o);
        if (lane >= o) v += u;
    }
    return v;
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
        const buffer_t buf = make_buffer(base, (uint32_t)(rows - 1) * step + WIDTH * ES);
        const uint32_t off = TileStep<T>::row(lane) * step + 16u * TileStep<T>::piece(lane);
        const uint32_t first = Steps::group0(wave) * TileStep<T>::ROWS * step + Steps::block0(wave) * 32 * ES;
#pragma unroll
        for (int i = 0; i < Steps::N; ++i)
            v[i] = buffer_load16(buf, off, first + Steps::group(i) * TileStep<T>::ROWS * step + Steps::block(i) * 32 * ES);
    }
    __device__ __forceinline__ void put(KDA_LDS T* tile, int wave, int lane) const {
        TilePut<T, kC> p;
        p.set(tile + (Steps::block0(wave) * kC + Steps::group0(wave) * TileStep<T>::ROWS) * 32, lane);
#pragma unroll
        for (int i = 0; i < Steps::N; ++i) p.put((Steps::block(i) * kC + Steps::group(i) * TileStep<T>::ROWS) * 32, v[i]);
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

// Per-token numbers of one chunk: sums of the exponents (base 2, high and low part), steps, and the
// weights of the state's update; `last` is the sum over the whole chunk.
struct ChunkDecay {
    float hi[kC], lo[kC], dt[kC], w[kC];
};

__device__ __forceinline__ void chunk_decay(KDA_LDS ChunkDecay* c, float raw, bool live, float A2, int lane) {
    const float d = live ? softplus_f32(raw) : 0.0f;
    const double s = wave_prefix(live ? (double)fmaxf(d * A2, kDecayMin) : 0.0, lane);
    const double end = __shfl(s, 63);
    const float hi = (float)s;
    c->hi[lane] = hi;
    c->lo[lane] = (float)(s - (double)hi);
    c->dt[lane] = d;
    c->w[lane] = fast_exp2((float)(end - s)) * d;
}

}  // namespace

// OUT: with outputs (the pass that runs every segment from its entry state), else final states only.
template <int N, int P, typename T, bool OUT, int NW>
__global__ __launch_bounds__(64 * NW, sizeof(T) == 2 ? 2 : 1) void kda_ssm_prefill_kernel(const SsmArgs a) {
    constexpr int NTH = 64 * NW;
    constexpr int WC = P / NW;       // state columns per wave
    constexpr int NCT = WC / 16;     // column tiles per wave
    constexpr int NT = N / 16;       // row tiles of the state
    constexpr int NP = Parts<T>::n;
    typedef __attribute__((ext_vector_type(4))) T vec4;
    // LDS: B, C, M, x tiles (elements), then the decays of two chunks
    constexpr int oC = kC * N, oM = OUT ? 2 * kC * N : kC * N, oX = oM + (OUT ? kC * kC : 0), oEnd = oX + kC * P;
    __shared__ __attribute__((aligned(16))) T smem[oEnd];
    __shared__ __attribute__((aligned(16))) ChunkDecay sD_[2];
    KDA_LDS T* sB = (KDA_LDS T*)smem;
    KDA_LDS T* sC = sB + oC;
    KDA_LDS T* sM = sB + oM;
    KDA_LDS T* sX = sB + oX;
    KDA_LDS ChunkDecay* sD = (KDA_LDS ChunkDecay*)sD_;

    // unit = (b, segment, h), heads fastest: the heads of a segment share B and C, and each XCD takes a
    // contiguous range of units
    const long long unit = (long long)(blockIdx.x & 7) * a.per_xcd + (blockIdx.x >> 3);
    if (unit >= a.n_units) return;
    const int h = (int)(unit % a.H);
    const long long bs = unit / a.H;
    const int s = (int)(bs % a.n_seg_launch);
    const int b = (int)(bs / a.n_seg_launch);
    const long long bh = (long long)b * a.H + h;
    const int grp = h / (a.H / a.G);

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
    TileRows<T, kC, N> rn;    // rows of B (and of C, oC further)
    TileCols<T, kC> cn;       // columns of B
    TileRows<T, kC, kC> rm;   // rows of M
    cn.set(sB, lane);
    if constexpr (OUT) {
        rn.set(sB, lane);
        rm.set(sM, lane);
    }
    // this lane's four columns of row r of x, column tile ct of the wave
    KDA_LDS T* xrow[NCT];
#pragma unroll
    for (int ct = 0; ct < NCT; ++ct) xrow[ct] = lds_pin(sX + tile_at<T, kC>(r, 4 * (wave * NCT + ct) + g));

    // row t_begin of every input, and the bytes between rows
    const long long row0 = (long long)b * a.T + t_begin;
    const T* xp = reinterpret_cast<const T*>(a.x) + row0 * a.x_stride + (long long)h * P;
    const T* bp = reinterpret_cast<const T*>(a.Bm) + row0 * a.b_stride + (long long)grp * N;
    const T* cp = reinterpret_cast<const T*>(a.Cm) + row0 * a.c_stride + (long long)grp * N;
    const T* dp = reinterpret_cast<const T*>(a.dt) + row0 * a.dt_stride + h;
    const T* zp = reinterpret_cast<const T*>(a.z);
    const bool gated = OUT && zp != nullptr;
    if (gated) zp += row0 * a.z_stride + (long long)h * P;
    T* yp = OUT ? reinterpret_cast<T*>(a.y) + (row0 * a.H + h) * P : nullptr;
    constexpr uint32_t ES = sizeof(T), ROW_P = P * ES;
    const uint32_t x_step = (uint32_t)a.x_stride * ES, b_step = (uint32_t)a.b_stride * ES, c_step = (uint32_t)a.c_stride * ES;
    const uint32_t z_step = (uint32_t)a.z_stride * ES, y_step = (uint32_t)a.H * ROW_P;
    const uint32_t z_off = r * z_step + (wave * WC + 4 * g) * ES, y_off = r * y_step + (wave * WC + 4 * g) * ES;
    const float A2 = a.A[h] * kLog2e;
    const float bias = a.dt_bias ? a.dt_bias[h] : 0.0f;
    const float Dh = a.D ? a.D[h] : 0.0f;

    // entry state
    f32x4_t S[NT][NCT];
    const float* sin = nullptr;
    if (s == 0 && !(OUT && a.keep_S0)) {
        if (a.S0) sin = a.S0 + bh * (long long)(N * P);
    } else if (OUT) {
        sin = a.ws_state + (bh * a.n_seg + s) * (long long)(N * P);
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct) S[nt][ct] = zero4();
    // this lane's element of row tile 0, column tile 0 of a state
    const uint32_t s_off = (uint32_t)((4 * g * P + wave * WC + r) * sizeof(float));
    if (sin) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
                for (int i = 0; i < 4; ++i) S[nt][ct][i] = *at_byte(sin + (16 * nt + i) * P + 16 * ct, s_off);
    }
    if (!OUT && s == 0 && a.keep_S0) {   // S_T is S0: the other pass's last segment overwrites it
        float* keep = a.ws_state + bh * a.n_seg * (long long)(N * P);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
                for (int i = 0; i < 4; ++i) *at_byte(keep + (16 * nt + i) * P + 16 * ct, s_off) = S[nt][ct][i];
    }
    float total = 0.0f;   // exponent (base 2) of the segment's decay

    // Inputs are requested one chunk ahead, the raw steps (last wave) two chunks ahead: their running sum
    // is a long chain, formed while the other waves work on M.
    Stage<T, P, NW> gx;
    Stage<T, N, NW> gb, gc;
    float gdt = 0.0f;
    // tokens left in the segment (32 bits: at most seg_len)
    int left = (int)(t_end - t_begin);
    auto request = [&](int rows) {   // the chunk at xp, bp, cp
        gx.load(xp, x_step, rows, wave, lane);
        gb.load(bp, b_step, rows, wave, lane);
        if constexpr (OUT) gc.load(cp, c_step, rows, wave, lane);
    };
    auto request_dt = [&](int ahead) {
        const int t = ahead + lane < left ? ahead + lane : left - 1;
        gdt = to_f32<T>(dp[t * a.dt_stride]);
    };
    if (left > 0) {
        if (wave == NW - 1) {
            request_dt(0);
            chunk_decay(sD, gdt + bias, lane < left, A2, lane);
            request_dt(kC);
        }
        request(left < kC ? left : kC);
    }

    // columns 16 (wave NCT + ct) .. of x, transposed (the tile index is the wave's: addresses of its own)
    TileCols<T, kC> cx[NCT];
#pragma unroll
    for (int ct = 0; ct < NCT; ++ct) cx[ct].set_tile(sX, lane, wave * NCT + ct);
    auto cx_frag = [&](Frag<T>& f, int ct, int kb) { cx[ct].frag(f, 0, 0, kb); };

    for (int par = 0; left > 0; left -= kC, par ^= 1) {
        const int rows = left < kC ? left : kC;
        const KDA_LDS ChunkDecay* cd = sD + par;
        gx.put(sX, wave, lane);
        gb.put(sB, wave, lane);
        if constexpr (OUT) gc.put(sC, wave, lane);
        __syncthreads();
        vec4 zv[4][NCT];
        if (gated) {
            const buffer_t zbuf = make_buffer(zp, (uint32_t)(rows - 1) * z_step + ROW_P);
#pragma unroll
            for (int ti = 0; ti < 4; ++ti)
#pragma unroll
                for (int ct = 0; ct < NCT; ++ct) buffer_load4(zv[ti][ct], zbuf, z_off, 16 * ti * z_step + 16 * ct * ES);
            zp += kC * a.z_stride;
        }
        if constexpr (OUT) {
            // M[i][j] = e^{c_i - c_j} dt_j (C_i . B_j) for j <= i: the ten lower 16 x 16 tiles
            // (the pair is taken as new in every chunk: its addresses are not worth registers)
            for (int pair = pinned_s(wave); pair < 10; pair += NW) {
                {
                    const int ti = pair < 1 ? 0 : (pair < 3 ? 1 : (pair < 6 ? 2 : 3));
                    const int tj = pair - ti * (ti + 1) / 2;
                    f32x4_t acc = zero4();
#pragma unroll
                    for (int kb = 0; kb < N / 32; ++kb) {
                        Frag<T> fb, fc;
                        rn.frag(fb, 16 * 32 * tj, 0, kb);
                        rn.frag(fc, oC + 16 * 32 * ti, 0, kb);
                        acc = mma(fb, fc, acc);   // acc[q]: token j = 16 tj + 4 g + q against i = 16 ti + r
                    }
                    const float ci = cd->hi[16 * ti + r], cil = cd->lo[16 * ti + r];
                    const f32x4_t cj = *reinterpret_cast<const KDA_LDS f32x4_t*>(cd->hi + 16 * tj + 4 * g);
                    const f32x4_t cjl = *reinterpret_cast<const KDA_LDS f32x4_t*>(cd->lo + 16 * tj + 4 * g);
                    const f32x4_t dj = *reinterpret_cast<const KDA_LDS f32x4_t*>(cd->dt + 16 * tj + 4 * g);
                    float m[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float v = acc[q] * (fast_exp2((ci - cj[q]) + (cil - cjl[q])) * dj[q]);
                        m[q] = tj < ti || 4 * g + q <= r ? v : 0.0f;
                    }
                    lds_store_run<4>(sM + 16 * 32 * ti + tile_at<T, kC>(r, 4 * tj + g), m);
                }
            }
        }
        if (left > kC && wave == NW - 1) {
            chunk_decay(sD + (par ^ 1), gdt + bias, kC + lane < left, A2, lane);
            request_dt(2 * kC);
            dp += kC * a.dt_stride;
        }
        if constexpr (OUT) __syncthreads();

        // x of this wave's columns, transposed: contraction over tokens
        Frag<T> xt[2][NCT];
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) cx_frag(xt[kb][ct], ct, kb);

        if constexpr (OUT) {
            // y^T = (S^T C^T) e^{c_i} + x^T M^T: columns are tokens, rows p
            f32x4_t y[4][NCT];
            const buffer_t ybuf = make_buffer(yp, (uint32_t)(rows - 1) * y_step + ROW_P);
            yp += (long long)kC * a.H * P;
#pragma unroll
            for (int kb = 0; kb < N / 32; ++kb) {
                Frag<T> fs[NCT];
#pragma unroll
                for (int ct = 0; ct < NCT; ++ct) acc_pair_frag<T>(fs[ct], S[kb][ct], S[kb + NT / 2][ct], true);
#pragma unroll
                for (int ti = 0; ti < 4; ++ti) {
                    Frag<T> fc;
                    rn.frag(fc, oC, ti, kb);
#pragma unroll
                    for (int ct = 0; ct < NCT; ++ct) y[ti][ct] = mma(fs[ct], fc, kb == 0 ? zero4() : y[ti][ct]);
                }
            }
#pragma unroll
            for (int ti = 0; ti < 4; ++ti) {
                __builtin_amdgcn_sched_barrier(0);
                const float e = fast_exp2(cd->hi[16 * ti + r]);
#pragma unroll
                for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
                    for (int q = 0; q < 4; ++q) y[ti][ct][q] *= e;
#pragma unroll
                for (int kb = 0; kb < (ti < 1 ? 1 : 2); ++kb) {   // token tiles kb and kb + 2, as far as they reach
                    Frag<T> fm;
                    if (kb + 2 > ti) rm.frag_lo(fm, 0, ti, kb);
                    else rm.frag(fm, 0, ti, kb);
#pragma unroll
                    for (int ct = 0; ct < NCT; ++ct) y[ti][ct] = mma(xt[kb][ct], fm, y[ti][ct]);
                }
#pragma unroll
                for (int ct = 0; ct < NCT; ++ct) {
                    const vec4 xv = *reinterpret_cast<const KDA_LDS vec4*>(xrow[ct] + 16 * 32 * ti);
                    f32x4_t o;
#pragma unroll
                    for (int q = 0; q < 4; ++q) o[q] = fmaf(Dh, to_f32<T>((T)xv[q]), y[ti][ct][q]);
                    if (gated) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) o[q] *= silu_f32(to_f32<T>((T)zv[ti][ct][q]));
                    }
                    vec4 ov;
#pragma unroll
                    for (int q = 0; q < 4; ++q) ov[q] = from_f32<T>(o[q]);
                    buffer_store4(ov, ybuf, y_off, 16 * ti * y_step + 16 * ct * ES);
                }
            }
        }

        // the next chunk's rows are requested here, where the outputs' registers are free again
        if (left > kC) {
            xp += kC * a.x_stride;
            bp += kC * a.b_stride;
            cp += kC * a.c_stride;
            request(left - kC < kC ? left - kC : kC);
        }

        // S <- e^{c_63} S + B^T (w x)
        __builtin_amdgcn_sched_barrier(0);
        {
            const float cl = cd->hi[kC - 1];
            const float eL = fast_exp2(cl);
            total += cl;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
                    for (int q = 0; q < 4; ++q) S[nt][ct][q] *= eL;
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
                __builtin_amdgcn_sched_barrier(0);
                float w[8];
                load_weights(w, cd->w + 16 * kb + 4 * g);
                Frag<T> xs[NCT][NP];
#pragma unroll
                for (int ct = 0; ct < NCT; ++ct) weigh(xs[ct], xt[kb][ct], w);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    Frag<T> fb;
                    cn.frag(fb, 0, nt, kb);
#pragma unroll
                    for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
                        for (int q = NP - 1; q >= 0; --q) S[nt][ct] = mma(fb, xs[ct][q], S[nt][ct]);
                }
            }
        }
        __syncthreads();
    }

    float* so = nullptr;
    if (OUT) {
        if (last && a.S_T) so = a.S_T + bh * (long long)(N * P);
    } else {
        so = a.ws_state + (bh * a.n_seg + s + 1) * (long long)(N * P);
        if (tid == 0) a.ws_decay[bh * a.n_seg + s + 1] = total;
    }
    if (so) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
                for (int i = 0; i < 4; ++i) *at_byte(so + (16 * nt + i) * P + 16 * ct, s_off) = S[nt][ct][i];
    }
}

// Entry states from the segments' final states, in place: slot s + 1 holds the final state of segment s
// from zero (segment 0: from its entry state) and becomes the entry state of segment s + 1.
// grid: sequences x heads x (state elements / 1024)
__global__ __launch_bounds__(256) void kda_ssm_join_kernel(float* ws, const float* decay, int n_seg, int np) {
    const int per = np / 1024;
    const long long bh = blockIdx.x / per;
    const int e = ((int)(blockIdx.x % per) * 256 + threadIdx.x) * 4;
    float* p = ws + (bh * n_seg + 1) * (long long)np + e;
    const float* d = decay + bh * n_seg;
    f32x4_t S = *reinterpret_cast<const f32x4_t*>(p);
    for (int s = 2; s < n_seg; ++s) {
        p += np;
        const f32x4_t hs = *reinterpret_cast<const f32x4_t*>(p);
        const float f = fast_exp2(d[s]);
#pragma unroll
        for (int i = 0; i < 4; ++i) S[i] = fmaf(f, S[i], hs[i]);
        *reinterpret_cast<f32x4_t*>(p) = S;
    }
}

// One token: a workgroup owns one (sequence, head) state, P/4 groups of four columns x 16 row groups.
template <int N, int P, typename T>
__global__ __launch_bounds__(4 * P) void kda_ssm_step_kernel(const SsmArgs a) {
    constexpr int NCG = P / 4, NRG = 16, NTH = NCG * NRG, NW = NTH / 64, RPT = N / NRG;
    const long long nh = (long long)(blockIdx.x & 7) * a.per_xcd + (blockIdx.x >> 3);
    if (nh >= a.n_units) return;
    const long long n = nh / a.H;
    const int h = (int)(nh % a.H), grp = h / (a.H / a.G);
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
        __builtin_nontemporal_store(S[m], reinterpret_cast<f32x4_t*>(Sb + (long long)i * P));
    }
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
    a.per_xcd = (a.n_units + 7) / 8;
    const dim3 grid((unsigned)(8 * a.per_xcd));
    switch (pass) {
        case SsmPass::kStates: kda_ssm_prefill_kernel<N, P, T, false, NW><<<grid, 64 * NW, 0, s>>>(a); break;
        case SsmPass::kOutputs: kda_ssm_prefill_kernel<N, P, T, true, NW><<<grid, 64 * NW, 0, s>>>(a); break;
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
    kda_ssm_join_kernel<<<dim3((unsigned)bh * (n * p / 1024)), 256, 0, s>>>(ws_state, ws_decay, n_seg, n * p);
    return hipGetLastError();
}

}  // namespace kda
