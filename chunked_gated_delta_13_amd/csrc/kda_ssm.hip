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

// Running sum over the 64 lanes of a wave.
__device__ __forceinline__ float wave_prefix(float v, int lane) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const float u = __shfl_up(v, o);
        if (lane >= o) v += u;
    }
    return v;
}

// v as a sum of NPART operands (bf16: three parts of 8 bits each; fp32: itself).
__device__ __forceinline__ void split_parts(Frag<__bf16> (&f)[3], int j, float v) {
    const __bf16 a = (__bf16)v;
    const float r1 = v - (float)a;
    const __bf16 b = (__bf16)r1;
    f[0].v[j] = a;
    f[1].v[j] = b;
    f[2].v[j] = (__bf16)(r1 - (float)b);
}
__device__ __forceinline__ void split_parts(Frag<float> (&f)[1], int j, float v) { f[0].v[j] = v; }

template <typename T> struct Parts { static constexpr int n = 3; };
template <> struct Parts<float> { static constexpr int n = 1; };

// A wave's share of 64 rows of WIDTH elements: requested one chunk ahead into registers, put into the
// tile when the last chunk's readers are done.
template <typename T, int WIDTH> struct Stage {
    static constexpr int PER_ROW = WIDTH * (int)sizeof(T) / 16;
    static constexpr int N = kC * PER_ROW / 256;
    static constexpr int ROWS = 256 / PER_ROW;   // rows per step
    u32x4_t v[N];
    __device__ __forceinline__ void load(const T* base, long long stride, int rows, int tid) {
        const int m = tid % PER_ROW, r0 = tid / PER_ROW;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int r = r0 + i * ROWS;
            v[i] = u32x4_t{0, 0, 0, 0};
            if (r < rows) v[i] = *reinterpret_cast<const u32x4_t*>(base + r * stride + m * (16 / (int)sizeof(T)));
        }
    }
    __device__ __forceinline__ void put(KDA_LDS T* tile, int tid) const {
        const int m = tid % PER_ROW, r0 = tid / PER_ROW;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int r = r0 + i * ROWS;
            tile_put(tile + r * WIDTH, m, r & 15, v[i]);
        }
    }
};

}  // namespace

// OUT: with outputs (the pass that runs every segment from its entry state), else final states only.
template <int N, int P, typename T, bool OUT>
__global__ __launch_bounds__(256) void kda_ssm_prefill_kernel(const SsmArgs a) {
    constexpr int WC = P / 4;        // state columns per wave
    constexpr int NCT = WC / 16;     // column tiles per wave
    constexpr int NT = N / 16;       // row tiles of the state
    constexpr int NP = Parts<T>::n;
    __shared__ __attribute__((aligned(16))) T sX_[kC * P], sB_[kC * N], sC_[OUT ? kC * N : 16], sM_[OUT ? kC * kC : 16];
    __shared__ __attribute__((aligned(16))) float sCum_[kC], sDt_[kC], sW_[kC];
    KDA_LDS T* sX = (KDA_LDS T*)sX_;
    KDA_LDS T* sB = (KDA_LDS T*)sB_;
    KDA_LDS T* sC = (KDA_LDS T*)sC_;
    KDA_LDS T* sM = (KDA_LDS T*)sM_;
    KDA_LDS float* sCum = (KDA_LDS float*)sCum_;
    KDA_LDS float* sDt = (KDA_LDS float*)sDt_;
    KDA_LDS float* sW = (KDA_LDS float*)sW_;

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
    TileLane<T, N> ln;
    TileLane<T, P> lp;
    TileLane<T, kC> lm;
    ln.set(lane);
    lp.set(lane);
    if constexpr (OUT) lm.set(lane);

    const T* xb = reinterpret_cast<const T*>(a.x) + (long long)b * a.T * a.x_stride + (long long)h * P;
    const T* bb = reinterpret_cast<const T*>(a.Bm) + (long long)b * a.T * a.b_stride + (long long)grp * N;
    const T* cb = reinterpret_cast<const T*>(a.Cm) + (long long)b * a.T * a.c_stride + (long long)grp * N;
    const T* zb = reinterpret_cast<const T*>(a.z);
    if (OUT && zb) zb += (long long)b * a.T * a.z_stride + (long long)h * P;
    const T* db = reinterpret_cast<const T*>(a.dt) + (long long)b * a.T * a.dt_stride + h;
    T* yb = OUT ? reinterpret_cast<T*>(a.y) + ((long long)b * a.T * a.H + h) * P : nullptr;
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
        for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                S[nt][ct][i] = sin ? sin[(16 * nt + 4 * g + i) * P + wave * WC + 16 * ct + r] : 0.0f;
    if (!OUT && s == 0 && a.keep_S0) {   // S_T is S0: the other pass's last segment overwrites it
        float* keep = a.ws_state + bh * a.n_seg * (long long)(N * P);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
                for (int i = 0; i < 4; ++i) keep[(16 * nt + 4 * g + i) * P + wave * WC + 16 * ct + r] = S[nt][ct][i];
    }
    float total = 0.0f;   // exponent (base 2) of the segment's decay

    Stage<T, P> gx;
    Stage<T, N> gb, gc;
    float gdt = 0.0f;
    auto request = [&](long long t0) {
        const int rows = t_end - t0 < kC ? (int)(t_end - t0) : kC;
        gx.load(xb + t0 * a.x_stride, a.x_stride, rows, tid);
        gb.load(bb + t0 * a.b_stride, a.b_stride, rows, tid);
        if constexpr (OUT) gc.load(cb + t0 * a.c_stride, a.c_stride, rows, tid);
        if (wave == 0) gdt = lane < rows ? to_f32<T>(db[(t0 + lane) * a.dt_stride]) : 0.0f;
    };
    if (t_begin < t_end) request(t_begin);

    for (long long t0 = t_begin; t0 < t_end; t0 += kC) {
        const int rows = t_end - t0 < kC ? (int)(t_end - t0) : kC;
        gx.put(sX, tid);
        gb.put(sB, tid);
        if constexpr (OUT) gc.put(sC, tid);
        if (wave == 0) {
            const float d = lane < rows ? softplus_f32(gdt + bias) : 0.0f;
            const float c = wave_prefix(lane < rows ? fmaxf(d * A2, kDecayMin) : 0.0f, lane);
            const float cl = __shfl(c, 63);
            sCum[lane] = c;
            sDt[lane] = d;
            sW[lane] = fast_exp2(cl - c) * d;
        }
        __syncthreads();
        if (t0 + kC < t_end) request(t0 + kC);

        if constexpr (OUT) {
            // M[i][j] = e^{c_i - c_j} dt_j (C_i . B_j) for j <= i: the ten lower 16 x 16 tiles
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                const int pair = wave + 4 * k;
                if (pair < 10) {
                    const int ti = pair < 1 ? 0 : (pair < 3 ? 1 : (pair < 6 ? 2 : 3));
                    const int tj = pair - ti * (ti + 1) / 2;
                    f32x4_t acc = zero4();
#pragma unroll
                    for (int kb = 0; kb < N / 32; ++kb) {
                        Frag<T> fb, fc;
                        tile_row_frag<T, N>(fb, sB, ln, tj, kb);
                        tile_row_frag<T, N>(fc, sC, ln, ti, kb);
                        acc = mma(fb, fc, acc);   // acc[q]: token j = 16 tj + 4 g + q against i = 16 ti + r
                    }
                    const float ci = sCum[16 * ti + r];
                    const f32x4_t cj = *reinterpret_cast<const KDA_LDS f32x4_t*>(sCum + 16 * tj + 4 * g);
                    const f32x4_t dj = *reinterpret_cast<const KDA_LDS f32x4_t*>(sDt + 16 * tj + 4 * g);
                    float m[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float v = acc[q] * (fast_exp2(ci - cj[q]) * dj[q]);
                        m[q] = tj < ti || 4 * g + q <= r ? v : 0.0f;
                    }
                    lds_store_run<4>(sM + (16 * ti + r) * kC + (((4 * tj + g) ^ tile_f(r)) << 2), m);
                }
            }
            __syncthreads();
        }

        // x of this wave's columns, transposed: contraction over tokens
        Frag<T> xt[2][NCT];
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) tile_tr_frag<T, P>(xt[kb][ct], sX, lp, wave * NCT + ct, kb, lane);

        if constexpr (OUT) {
            // y^T = (S^T C^T) e^{c_i} + x^T M^T: columns are tokens, rows p
            f32x4_t y[4][NCT];
#pragma unroll
            for (int ti = 0; ti < 4; ++ti)
#pragma unroll
                for (int ct = 0; ct < NCT; ++ct) y[ti][ct] = zero4();
#pragma unroll
            for (int kb = 0; kb < N / 32; ++kb) {
                Frag<T> fs[NCT];
#pragma unroll
                for (int ct = 0; ct < NCT; ++ct) acc_pair_frag<T>(fs[ct], S[2 * kb][ct], S[2 * kb + 1][ct], true);
#pragma unroll
                for (int ti = 0; ti < 4; ++ti) {
                    Frag<T> fc;
                    tile_row_frag<T, N>(fc, sC, ln, ti, kb);
#pragma unroll
                    for (int ct = 0; ct < NCT; ++ct) y[ti][ct] = mma(fs[ct], fc, y[ti][ct]);
                }
            }
#pragma unroll
            for (int ti = 0; ti < 4; ++ti) {
                const float e = fast_exp2(sCum[16 * ti + r]);
#pragma unroll
                for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
                    for (int q = 0; q < 4; ++q) y[ti][ct][q] *= e;
#pragma unroll
                for (int kb = 0; kb <= ti / 2; ++kb) {
                    Frag<T> fm;
                    if (2 * kb + 1 > ti) tile_row_frag_lo<T, kC>(fm, sM, lm, ti, kb);
                    else tile_row_frag<T, kC>(fm, sM, lm, ti, kb);
#pragma unroll
                    for (int ct = 0; ct < NCT; ++ct) y[ti][ct] = mma(xt[kb][ct], fm, y[ti][ct]);
                }
                const int i = 16 * ti + r;
                if (i < rows) {
#pragma unroll
                    for (int ct = 0; ct < NCT; ++ct) {
                        const int p0 = wave * WC + 16 * ct + 4 * g;
                        const KDA_LDS T* xr = sX + i * P + (((p0 >> 2) ^ tile_f(r)) << 2);
                        float o[4];
#pragma unroll
                        for (int q = 0; q < 4; ++q) o[q] = fmaf(Dh, to_f32<T>(xr[q]), y[ti][ct][q]);
                        if (zb) {
                            typedef __attribute__((ext_vector_type(4))) T vec4;
                            const vec4 zv = *reinterpret_cast<const vec4*>(zb + (t0 + i) * a.z_stride + p0);
#pragma unroll
                            for (int q = 0; q < 4; ++q) o[q] *= silu_f32(to_f32<T>((T)zv[q]));
                        }
                        typedef __attribute__((ext_vector_type(4))) T vec4;
                        vec4 ov;
#pragma unroll
                        for (int q = 0; q < 4; ++q) ov[q] = from_f32<T>(o[q]);
                        *reinterpret_cast<vec4*>(yb + (t0 + i) * (long long)a.H * P + p0) = ov;
                    }
                }
            }
        }

        // S <- e^{c_63} S + B^T (w x)
        {
            const float cl = sCum[kC - 1];
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
                float w[8];
                f32x8_ld(w, sW + 32 * kb + 4 * g);
                Frag<T> xs[NCT][NP];
#pragma unroll
                for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
                    for (int j = 0; j < 8; ++j) split_parts(xs[ct], j, xt[kb][ct].get(j) * w[j]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    Frag<T> fb;
                    tile_tr_frag<T, N>(fb, sB, ln, nt, kb, lane);
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
                for (int i = 0; i < 4; ++i) so[(16 * nt + 4 * g + i) * P + wave * WC + 16 * ct + r] = S[nt][ct][i];
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
    a.per_xcd = (a.n_units + 7) / 8;
    const dim3 grid((unsigned)(8 * a.per_xcd));
    switch (pass) {
        case SsmPass::kStates: kda_ssm_prefill_kernel<N, P, T, false><<<grid, 256, 0, s>>>(a); break;
        case SsmPass::kOutputs: kda_ssm_prefill_kernel<N, P, T, true><<<grid, 256, 0, s>>>(a); break;
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
