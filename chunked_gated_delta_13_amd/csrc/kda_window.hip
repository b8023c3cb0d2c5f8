// Attention with a sliding window and a few first tokens that stay visible, for gfx950: prompts and
// single tokens over a ring cache of fixed size.
//
// The query at position t sees key j <= t when t - j < window or j < sinks.  The cache of a sequence
// holds sinks + window rows per kv head; token p lies in row p for p < sinks and in row
// sinks + (p - sinks) mod window after that, so a row is overwritten just when it leaves the window.
//
// Both forms run one pass over the visible keys with the running maximum and sum of the softmax (fp32,
// exponentials of base 2).  Scores are formed transposed, K Q^T with keys as rows: a lane then holds
// four keys of one query, the statistics of a query stay in its lanes, and the probabilities are at
// once the operand of V^T P^T.  For that product only they are rounded to the input type in the prompt
// form: outputs are 2.0 to 2.3e-3 off in bf16, 1.7e-3 of it their own rounding.  P in two parts leaves only the
// latter, but adds half the products again: a prompt of model width takes 4050 us instead of 1614 (the operands
// spill), 2048 tokens of 8 heads 30.5 instead of 26.3, short pieces 12.4 instead of 11.5.  The one-token form,
// bound by HBM, feeds bf16 ones as two parts.
#include "kda_mixers.h"
#include "kda_softmax.h"

namespace kda {

namespace {

constexpr int kKeys = 64;   // keys per tile of the prompt form

// Row of the cache for position p (32 bits hold every position: starts are int32, prompts at most 2^29).
__device__ __forceinline__ int ring_row(uint32_t p, int sinks, int window) {
    return p < (uint32_t)sinks ? (int)p : sinks + (int)((p - (uint32_t)sinks) % (uint32_t)window);
}

}  // namespace

// Prompt.  A workgroup of four waves runs 64 NQ queries of one (sequence, head); each wave holds
// 16 NQ queries and their outputs in registers.  The keys come tile by tile straight from memory into
// one of two LDS tiles, one tile ahead, and two workgroups share a compute unit: while one wave of a
// SIMD forms exponentials, the other feeds the matrix cores.  (Through registers, written to LDS a tile
// later, the same keys take 1.83 ms instead of 1.68.)
// What bounds it: 16384 tokens, 56 heads on 8, d = 128, window 4096 in bf16 take 1.59 to 1.65 ms by card, 1.02
// to 1.06 PFLOP/s of the visible products; a large library product reaches 1.23 to 1.35.  Matrix instructions and exponentials of
// the two waves do not overlap without gaps, and tiles at the window's two edges are multiplied whole.
// Pieces of a few hundred tokens (5 sequences of up to 333, window 200, d = 64) take 11.4 us, bound by
// the chain of a workgroup: lengths, first keys, five tiles, and the launch that keeps the new rows.
// In fp32, 8192 tokens, 16 heads on 4, window 1024 take 740 us at d = 128 and 344 at d = 64, 87 and 94 TFLOP/s
// of the 154 that a library product reaches: the matrix cores are busy in 68 and 73% of the cycles, and at d =
// 128 two pairs of tiles (128 KB) leave room for one wave a SIMD, with nothing beside its exponentials.
//
// The running maximum only has to keep exponentials in range.  A tile that every query of the wave sees
// whole is taken with the maximum at hand, without forming its own; only if a sum of its exponentials
// passes kSumMax (a score far above that maximum) is the maximum brought up to date.
constexpr float kSumMax = 16384.0f;

// SPLIT: a workgroup takes one of n_split ranges of its queries' tiles and leaves partial outputs with their
// maxima and sums, which kda_window_join_kernel joins.
template <int D, typename T, int NQ, bool SPLIT>
__global__ __launch_bounds__(256, sizeof(T) == 2 ? 2 : 1) void kda_window_prefill_kernel(const WindowArgs a) {
    constexpr int BM = 64 * NQ, TILE = kKeys * D;
    typedef TileSteps<T, kKeys, D, 4> Steps;
    constexpr int NG = Steps::N / Steps::NB;   // row groups per wave
    static_assert(NG * Steps::NB == Steps::N, "a wave takes whole rows");
    __shared__ __attribute__((aligned(16))) T smem[2 * 2 * TILE];   // two pairs of a tile of keys and one of values
    KDA_LDS T* sK = (KDA_LDS T*)smem;

    // unit = (b, kv head, query tile, head of the group): consecutive units share keys, and each XCD
    // takes a contiguous range of them
    uint32_t unit = (blockIdx.x & 7) * (uint32_t)a.per_xcd + (blockIdx.x >> 3);
    if (unit >= (uint32_t)a.n_units) return;
    int split = 0;
    if constexpr (SPLIT) {
        split = (int)(unit % (uint32_t)a.n_split);
        unit /= (uint32_t)a.n_split;
    }
    const uint32_t R = (uint32_t)a.H / (uint32_t)a.Hkv;
    const int hr = (int)(unit % R);
    unit /= R;
    const int q0 = (int)(unit % (uint32_t)a.q_tiles) * BM;
    unit /= (uint32_t)a.q_tiles;
    const int hk = (int)(unit % (uint32_t)a.Hkv), b = (int)(unit / (uint32_t)a.Hkv), h = hk * (int)R + hr;

    // (both asked for before either is waited for)
    int len = a.lens ? a.lens[b] : a.T;
    int s = a.start ? a.start[b] : 0;
    len = len < 0 ? 0 : (len > a.T ? a.T : len);
    if (s < 0) s = 0;
    if (q0 >= len) return;
    const int window = a.window, sinks = a.sinks;

    // Keys in relative positions (0 = the first new token): nsink first tokens, then lo .. hi
    const int hi = (q0 + BM < len ? q0 + BM : len) - 1;
    const int lo = sinks - s > q0 - window + 1 ? sinks - s : q0 - window + 1;
    const int nsink = s >= sinks ? sinks : (sinks < hi + 1 + s ? sinks : hi + 1 + s);
    const int total = nsink + (hi >= lo ? hi - lo + 1 : 0);
    int t_first = 0, t_end = total;   // this workgroup's part of them
    if constexpr (SPLIT) {
        const int tiles = (total + kKeys - 1) / kKeys, per = (int)((uint32_t)(tiles + a.n_split - 1) / (uint32_t)a.n_split);
        t_first = split * per * kKeys < total ? split * per * kKeys : total;
        t_end = t_first + per * kKeys < total ? t_first + per * kKeys : total;
    }
    const int base0 = s > sinks ? (int)((uint32_t)(s - sinks) % (uint32_t)window) : 0;

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, r = lane & 15;
    TileRows<T, kKeys, D> rk0;
    TileCols<T, kKeys> cv0;
    rk0.set(sK, lane);
    cv0.set(sK + TILE, lane);

    const T* kn = reinterpret_cast<const T*>(a.k) + (long long)b * a.T * a.k_stride + (long long)hk * D;
    const T* vn = reinterpret_cast<const T*>(a.v) + (long long)b * a.T * a.v_stride + (long long)hk * D;
    const long long crow = (long long)a.Hkv * D;
    const T* kc = reinterpret_cast<const T*>(a.k_cache);
    const T* vc = reinterpret_cast<const T*>(a.v_cache);
    if (kc) {
        kc += (long long)b * (sinks + window) * crow + (long long)hk * D;
        vc += (long long)b * (sinks + window) * crow + (long long)hk * D;
    }

    // A lane's key rows of a tile: one (bf16) or two (fp32) per wave, 16 bytes of each block of 32 columns.
    // Places past the last key take the last key again: they are masked, and their values are finite.
    auto fetch = [&](int t0, int buf) {
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            const int row16 = (Steps::group0(wave) + j) * TileStep<T>::ROWS + TileStep<T>::row(lane);
            const int pcol = tile_dma_piece<T>(row16, lane) * TileStep<T>::ELEMS;
            const int at = t0 + row16, idx = at < total ? at : total - 1;
            const int rel = idx < nsink ? idx - s : lo + (idx - nsink);
            const T *kp = kn + (long long)rel * a.k_stride, *vp = vn + (long long)rel * a.v_stride;
            if (rel < 0) {
                int row = idx;
                if (idx >= nsink) {
                    row = base0 + rel;
                    row = sinks + (row < 0 ? row + window : row);
                }
                kp = kc + row * crow;
                vp = vc + row * crow;
            }
            KDA_LDS T* dst = sK + buf * (2 * TILE) + (Steps::group0(wave) + j) * TileStep<T>::ROWS * 32;
#pragma unroll
            for (int i = 0; i < Steps::NB; ++i) {
                lds_dma16(reinterpret_cast<const float*>(kp + pcol + 32 * i), dst + i * kKeys * 32);
                lds_dma16(reinterpret_cast<const float*>(vp + pcol + 32 * i), dst + TILE + i * kKeys * 32);
            }
        }
    };
    fetch(t_first, 0);

    // queries of this wave
    const int wq = q0 + wave * 16 * NQ;
    Frag<T> fq[NQ][D / 32];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        const int i = wq + 16 * n + r;
        const T* qp = reinterpret_cast<const T*>(a.q) + ((long long)b * a.T + i) * a.q_stride + (long long)h * D + 4 * g;
#pragma unroll
        for (int kb = 0; kb < D / 32; ++kb) {
            if (i < len) global_frag<D>(fq[n][kb], qp + 16 * kb);
            else fq[n][kb].zero();
        }
    }

    f32x4_t O[D / 16][NQ];
    float m[NQ], l[NQ];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        m[n] = -INFINITY;
        l[n] = 0.0f;
#pragma unroll
        for (int t = 0; t < D / 16; ++t) O[t][n] = zero4();
    }
    const float sc = a.scale * kLog2e;
    bool ready = false;   // every query of the wave has a maximum
    barrier_all();

    for (int t0 = t_first, buf = 0; t0 < t_end; t0 += kKeys, buf ^= 1) {
        const TileRows<T, kKeys, D> rk = rk0.at_delta(buf * (2 * TILE));
        const TileCols<T, kKeys> cv = cv0.at_delta(buf * (2 * TILE));

        // scores, operands one contraction block ahead
        f32x4_t sT[4][NQ];
        Frag<T> fk[2][4];
#pragma unroll
        for (int kt = 0; kt < 4; ++kt) rk.frag(fk[0][kt], 0, kt, 0);
#pragma unroll
        for (int kb = 0; kb < D / 32; ++kb) {
            if (kb + 1 < D / 32) {
#pragma unroll
                for (int kt = 0; kt < 4; ++kt) rk.frag(fk[(kb + 1) & 1][kt], 0, kt, kb + 1);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int kt = 0; kt < 4; ++kt)
#pragma unroll
                for (int n = 0; n < NQ; ++n) sT[kt][n] = mma(fk[kb & 1][kt], fq[n][kb], kb == 0 ? zero4() : sT[kt][n]);
            __builtin_amdgcn_sched_barrier(0);
        }
        // The first values are read ahead of the exponentials, and the next tile is requested behind them: a
        // transposed read waits for every request to LDS before it (asked for before the scores, the tile
        // would be waited for here: 2.4% slower).
        Frag<T> fv[2][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) cv.frag(fv[0][i], 0, i, 0);
        __builtin_amdgcn_sched_barrier(0);
        if (t0 + kKeys < t_end) fetch(t0 + kKeys, buf ^ 1);
        __builtin_amdgcn_sched_barrier(0);

        const int w0 = lo + (t0 - nsink);   // relative position of the tile's first window key
        const bool whole = t0 >= nsink && t0 + kKeys <= total && w0 + kKeys - 1 <= wq && wq + 16 * NQ - 1 - w0 < window;
        Frag<T> fp[2][NQ];
        bool done = false;
        if (whole && ready) {
            float sum[NQ];
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
                f32x4_t p[4];
                sum[n] = 0.0f;
#pragma unroll
                for (int kt = 0; kt < 4; ++kt)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        p[kt][j] = fast_exp2(fmaf(sT[kt][n][j], sc, -m[n]));
                        sum[n] += p[kt][j];
                    }
#pragma unroll
                for (int kb = 0; kb < 2; ++kb) acc_pair_frag<T>(fp[kb][n], p[kb], p[kb + 2], true);
            }
            float big = sum[0];
#pragma unroll
            for (int n = 1; n < NQ; ++n) big += sum[n];
            done = !__any(!(big < kSumMax));
            if (done) {
#pragma unroll
                for (int n = 0; n < NQ; ++n) l[n] += sum[n];
            }
        }
        if (!done) {
            if (!whole) {
                // Query i sees the keys from..to of the list, and the first tokens below `first`; all three
                // from this lane's first key on.
#pragma unroll
                for (int n = 0; n < NQ; ++n) {
                    int i = wq + 16 * n + r;
                    asm volatile("" : "+v"(i));   // (formed here: not worth registers through the loop)
                    const int at = t0 + 4 * g;
                    const int out = i - window + 1 - lo, end = nsink + i - lo;
                    const int from = nsink + (out > 0 ? out : 0) - at, to = (end < total - 1 ? end : total - 1) - at;
                    const int first = (i + 1 < nsink - s ? i + 1 + s : nsink) - at;
#pragma unroll
                    for (int kt = 0; kt < 4; ++kt)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int x = 16 * kt + j;
                            sT[kt][n][j] = (x >= from && x <= to) || x < first ? sT[kt][n][j] : -INFINITY;
                        }
                }
            }
            bool got = true;
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
                float mx = -INFINITY;
#pragma unroll
                for (int kt = 0; kt < 4; ++kt)
#pragma unroll
                    for (int j = 0; j < 4; ++j) mx = fmaxf(mx, sT[kt][n][j]);
                mx = fmaxf(m[n], max_over_groups<NQ == 1>(mx) * sc);
                const float base = mx == -INFINITY ? 0.0f : mx;   // nothing visible yet: all exponentials are 0
                const float al = fast_exp2(m[n] - base);
                m[n] = mx;
                got = got && mx != -INFINITY;
                float sum = 0.0f;
#pragma unroll
                for (int kt = 0; kt < 4; ++kt)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float p = fast_exp2(fmaf(sT[kt][n][j], sc, -base));
                        sT[kt][n][j] = p;
                        sum += p;
                    }
                l[n] = l[n] * al + sum;
#pragma unroll
                for (int t = 0; t < D / 16; ++t)
#pragma unroll
                    for (int j = 0; j < 4; ++j) O[t][n][j] *= al;
#pragma unroll
                for (int kb = 0; kb < 2; ++kb) acc_pair_frag<T>(fp[kb][n], sT[kb][n], sT[kb + 2][n], true);
            }
            ready = __all(got);
        }

        // groups of four tiles of the head's channels, keys (0, 2) then (1, 3), a group ahead
        constexpr int GR = D / 64;
#pragma unroll
        for (int j = 0; j < 2 * GR; ++j) {
            const int kb = j / GR, d0 = (j % GR) * 4;
            if (j + 1 < 2 * GR) {
#pragma unroll
                for (int i = 0; i < 4; ++i) cv.frag(fv[(j + 1) & 1][i], 0, ((j + 1) % GR) * 4 + i, (j + 1) / GR);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int n = 0; n < NQ; ++n) O[d0 + i][n] = mma(fv[j & 1][i], fp[kb][n], O[d0 + i][n]);
            __builtin_amdgcn_sched_barrier(0);
        }
        barrier_all();   // the next tile has arrived, and nobody reads this one any more
    }

#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        const int i = wq + 16 * n + r;
        const float sum = sum_over_groups<NQ == 1>(l[n]);
        if (SPLIT && i < len) {
            const long long part = (((long long)b * a.T + i) * a.H + h) * a.n_split + split;
#pragma unroll
            for (int t = 0; t < D / 16; ++t) *reinterpret_cast<f32x4_t*>(a.ws_o + part * D + 16 * t + 4 * g) = O[t][n];
            if (g == 0) {
                a.ws_ml[2 * part] = m[n];
                a.ws_ml[2 * part + 1] = sum;
            }
        }
        const float inv = 1.0f / sum;
        if (!SPLIT && i < len) {
            T* op = reinterpret_cast<T*>(a.o) + (((long long)b * a.T + i) * a.H + h) * D + 4 * g;
#pragma unroll
            for (int t = 0; t < D / 16; ++t) {
                f32x4_t v = O[t][n];
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] *= inv;
                store4<T>(op + 16 * t, v);
            }
        }
    }
}

// The new tokens that stay in the cache: the first ones, and the last `window` ones.  It runs after
// the attention, which reads the rows overwritten here.  A copy, 2 to 4 us for a few hundred tokens.
// grid: (candidate rows / rows per workgroup, sequences); a row is 2^k or more threads wide
template <typename T>
__global__ __launch_bounds__(256) void kda_window_keep_kernel(const WindowArgs a, int row_bytes, int recent, int shift) {
    const int b = blockIdx.y;
    const uint32_t lane = threadIdx.x & ((1u << shift) - 1);
    const uint32_t c = blockIdx.x * (256u >> shift) + (threadIdx.x >> shift);
    if (c >= (uint32_t)(a.sinks + recent)) return;
    int len = a.T;
    if (a.lens) {
        const int l = a.lens[b];
        len = l < 0 ? 0 : (l > a.T ? a.T : l);
    }
    int s = a.start ? a.start[b] : 0;
    if (s < 0) s = 0;
    const bool first = c < (uint32_t)a.sinks;
    const int i = first ? (int)c - s : len - recent + (int)(c - a.sinks);
    if (i < 0 || i >= len) return;
    const uint32_t p = (uint32_t)s + (uint32_t)i;
    if (!first && p < (uint32_t)a.sinks) return;   // a first token: written by its own candidate
    const long long slot = (long long)b * (a.sinks + a.window) + ring_row(p, a.sinks, a.window), row = (long long)b * a.T + i;
    char* kd = reinterpret_cast<char*>(a.k_cache) + slot * row_bytes;
    char* vd = reinterpret_cast<char*>(a.v_cache) + slot * row_bytes;
    const char* ks = reinterpret_cast<const char*>(reinterpret_cast<const T*>(a.k) + row * a.k_stride);
    const char* vs = reinterpret_cast<const char*>(reinterpret_cast<const T*>(a.v) + row * a.v_stride);
    for (uint32_t o = 16 * lane; o < (uint32_t)row_bytes; o += 16u << shift) {
        *reinterpret_cast<u32x4_t*>(kd + o) = *reinterpret_cast<const u32x4_t*>(ks + o);
        *reinterpret_cast<u32x4_t*>(vd + o) = *reinterpret_cast<const u32x4_t*>(vs + o);
    }
}

// One token, bound by HBM: every visible key and value is read once (64 sequences, 8 kv heads, d = 128, 4100
// rows in bf16: 1.08 GB in 197 us, 5.5 TB/s; a plain read of the same memory reaches 6.9; in fp32 370 us, 5.8
// TB/s).  One sequence takes 10.2 us (16.5 in fp32), a chain of two launches, positions, keys and values.  A workgroup of four waves runs up to
// 16 query heads of one (sequence, kv head) over one
// range of cache rows; each wave takes every fourth tile of 32 rows with statistics of its own, and the
// waves (then the ranges) are joined at the end.  Keys go from memory straight into the operand; values
// pass through a tile of the wave's own in LDS to be transposed.
template <int D, typename T>
__global__ __launch_bounds__(256) void kda_window_step_kernel(const WindowArgs a) {
    constexpr int TK = 32;                                     // rows per tile
    constexpr int PER_ROW = D * (int)sizeof(T) / 16, EPP = 16 / (int)sizeof(T);
    typedef TileSteps<T, TK, D, 1> Steps;
    constexpr int NG = Steps::N / Steps::NB;                   // row groups per tile
    constexpr int OP = D + 4;                                  // pitch of the partial outputs
    constexpr int PP = sizeof(T) == 2 ? 2 : 1;                 // parts of a probability
    constexpr int REGION = TK * D * (int)sizeof(T) > 16 * OP * 4 ? TK * D * (int)sizeof(T) : 16 * OP * 4;
    __shared__ __attribute__((aligned(16))) char sV_[4][REGION];
    __shared__ float sm[4][16], sl[4][16];

    uint32_t unit = (blockIdx.x & 7) * (uint32_t)a.per_xcd + (blockIdx.x >> 3);
    if (unit >= (uint32_t)a.n_units) return;
    const int split = (int)(unit % (uint32_t)a.n_split);
    unit /= (uint32_t)a.n_split;
    const int R = (int)((uint32_t)a.H / (uint32_t)a.Hkv), RT = (R + 15) / 16;
    const int rt = (int)(unit % (uint32_t)RT);
    unit /= (uint32_t)RT;
    const int hk = (int)(unit % (uint32_t)a.Hkv);
    const long long b = unit / (uint32_t)a.Hkv;
    const int heads = R - 16 * rt < 16 ? R - 16 * rt : 16;
    const int h0 = hk * R + 16 * rt;

    long long pos = a.start[b];
    if (pos < 0) pos = 0;
    const int slots = a.sinks + a.window;
    const int fresh = ring_row((uint32_t)pos, a.sinks, a.window);   // the new token's row
    const int filled = pos + 1 < slots ? (int)pos + 1 : slots;
    const int k0 = split * a.split_len;
    const int k1 = k0 + a.split_len < filled ? k0 + a.split_len : filled;

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, r = lane & 15;
    KDA_LDS T* sV = (KDA_LDS T*)(KDA_LDS char*)sV_[wave];
    TileCols<T, TK> cv;
    cv.set(sV, lane);
    TilePut<T, TK> put;
    put.set(sV, 0, lane);

    const T* kn = reinterpret_cast<const T*>(a.k) + b * a.k_stride + (long long)hk * D;
    const T* vn = reinterpret_cast<const T*>(a.v) + b * a.v_stride + (long long)hk * D;
    const long long crow = (long long)a.Hkv * D;
    T* kc = reinterpret_cast<T*>(a.k_cache) + b * slots * crow + (long long)hk * D;
    T* vc = reinterpret_cast<T*>(a.v_cache) + b * slots * crow + (long long)hk * D;
    // The one workgroup whose range holds the new token's row writes it; nobody reads that row from the
    // cache in this call.
    if (rt == 0 && fresh >= k0 && fresh < k0 + a.split_len && tid < 2 * PER_ROW) {
        const int m = tid % PER_ROW;
        if (tid < PER_ROW) *reinterpret_cast<u32x4_t*>(kc + fresh * crow + m * EPP) = *reinterpret_cast<const u32x4_t*>(kn + m * EPP);
        else *reinterpret_cast<u32x4_t*>(vc + fresh * crow + m * EPP) = *reinterpret_cast<const u32x4_t*>(vn + m * EPP);
    }

    Frag<T> fq[D / 32];
    {
        const T* qp = reinterpret_cast<const T*>(a.q) + b * a.q_stride + (long long)(h0 + r) * D + 8 * g;
#pragma unroll
        for (int kb = 0; kb < D / 32; ++kb) {
            if (r < heads) global_frag8(fq[kb], qp + 32 * kb);
            else fq[kb].zero();
        }
    }
    f32x4_t O[D / 16];
#pragma unroll
    for (int t = 0; t < D / 16; ++t) O[t] = zero4();
    float m = -INFINITY, l = 0.0f;
    const float sc = a.scale * kLog2e;

    // Rows past the filled ones stand for the new token and are masked: memory that no token has written
    // is never read.  A tile's keys are requested as soon as the products with the last one's are issued,
    // its values as soon as the last one's are in LDS.
    u32x4_t gv[Steps::N];
    Frag<T> fk[2][D / 32];
    auto request_k = [&](int t0) {
#pragma unroll
        for (int kt = 0; kt < 2; ++kt) {
            const int row = t0 + 16 * kt + r;
            const T* kp = (row >= k1 || row == fresh ? kn : kc + row * crow) + 8 * g;
#pragma unroll
            for (int kb = 0; kb < D / 32; ++kb) global_frag8(fk[kt][kb], kp + 32 * kb);
        }
    };
    auto request_v = [&](int t0) {
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            const int row = t0 + j * TileStep<T>::ROWS + TileStep<T>::row(lane);
            const T* vp = (row >= k1 || row == fresh ? vn : vc + row * crow) + TileStep<T>::piece(lane) * EPP;
#pragma unroll
            for (int i = 0; i < Steps::NB; ++i) gv[j * Steps::NB + i] = *reinterpret_cast<const u32x4_t*>(vp + 32 * i);
        }
    };
    request_k(k0 + TK * wave);
    request_v(k0 + TK * wave);
    for (int t0 = k0 + TK * wave; t0 < k1; t0 += 4 * TK) {
        f32x4_t sT[2];
#pragma unroll
        for (int kt = 0; kt < 2; ++kt) {
            sT[kt] = zero4();
#pragma unroll
            for (int kb = 0; kb < D / 32; ++kb) sT[kt] = mma(fk[kt][kb], fq[kb], sT[kt]);
        }
        __builtin_amdgcn_sched_barrier(0);
        request_k(t0 + 4 * TK);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < Steps::N; ++i) put.put(Steps::group(i), Steps::block(i), gv[i]);
        __builtin_amdgcn_sched_barrier(0);
        request_v(t0 + 4 * TK);
        __builtin_amdgcn_sched_barrier(0);
        float mx = -INFINITY;
#pragma unroll
        for (int kt = 0; kt < 2; ++kt)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (t0 + 16 * kt + 4 * g + j >= k1) sT[kt][j] = -INFINITY;
                mx = fmaxf(mx, sT[kt][j]);
            }
        mx = fmaxf(m, max_over_groups<true>(mx) * sc);
        const float base = mx == -INFINITY ? 0.0f : mx;   // every score so far is below fp32's range: no weight
        const float al = fast_exp2(m - base);
        m = mx;
        float sum = 0.0f;
#pragma unroll
        for (int kt = 0; kt < 2; ++kt)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                sT[kt][j] = fast_exp2(fmaf(sT[kt][j], sc, -base));
                sum += sT[kt][j];
            }
        l = l * al + sum;
        // Probabilities as operands: in bf16 as two parts, which hold 16 bits of them.  The products are a few
        // percent of the time that the loads take, so rounding them to 8 bits would buy nothing here.
        Frag<T> fp[PP];
        acc_pair_frag<T>(fp[0], sT[0], sT[1], true);
        if constexpr (PP == 2) {
#pragma unroll
            for (int kt = 0; kt < 2; ++kt)
#pragma unroll
                for (int j = 0; j < 4; ++j) sT[kt][j] -= fp[0].get(4 * kt + j);
            acc_pair_frag<T>(fp[1], sT[0], sT[1], true);
        }
        wave_order();
#pragma unroll
        for (int t = 0; t < D / 16; ++t) {
            Frag<T> fv;
            cv.frag(fv, 0, t, 0);
#pragma unroll
            for (int j = 0; j < 4; ++j) O[t][j] *= al;
#pragma unroll
            for (int i = PP - 1; i >= 0; --i) O[t] = mma(fv, fp[i], O[t]);
        }
        wave_order();
    }
    l = sum_over_groups<true>(l);

    // join the waves: every wave's outputs go to its own region as [head][d]
    KDA_LDS float* sO = (KDA_LDS float*)(KDA_LDS char*)sV_[wave];
#pragma unroll
    for (int t = 0; t < D / 16; ++t) *reinterpret_cast<KDA_LDS f32x4_t*>(sO + r * OP + 16 * t + 4 * g) = O[t];
    if (g == 0) {
        sm[wave][r] = m;
        sl[wave][r] = l;
    }
    __syncthreads();
    for (int e = tid; e < heads * (D / 4); e += 256) {
        const int hh = e / (D / 4), d = (e % (D / 4)) * 4;
        float M = -INFINITY, L = 0.0f;
#pragma unroll
        for (int w = 0; w < 4; ++w) M = fmaxf(M, sm[w][hh]);
        f32x4_t v = zero4();
        const float base = M == -INFINITY ? 0.0f : M;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const float f = fast_exp2(sm[w][hh] - base);
            L = fmaf(f, sl[w][hh], L);
            const f32x4_t x = *reinterpret_cast<const KDA_LDS f32x4_t*>((KDA_LDS float*)(KDA_LDS char*)sV_[w] + hh * OP + d);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = fmaf(f, x[j], v[j]);
        }
        const long long row = b * a.H + h0 + hh;
        if (a.n_split == 1) {
            const float inv = 1.0f / L;
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] *= inv;
            store4<T>(reinterpret_cast<T*>(a.o) + row * D + d, v);
        } else {
            *reinterpret_cast<f32x4_t*>(a.ws_o + (row * a.n_split + split) * D + d) = v;
            if (d == 0) {
                a.ws_ml[2 * (row * a.n_split + split)] = M;
                a.ws_ml[2 * (row * a.n_split + split) + 1] = L;
            }
        }
    }
}

// Joins the ranges of a split call.  grid: (sequence, token, head) rows; one wave: D / 4 lanes own four
// channels of a range, and 64 / (D / 4) ranges are taken side by side.
template <int D, typename T>
__global__ __launch_bounds__(64) void kda_window_join_kernel(const WindowArgs a) {
    constexpr int NL = D / 4, NS = 64 / NL;
    const long long row = blockIdx.x;
    if (a.lens) {   // rows behind a sequence's end have no parts
        const uint32_t token = blockIdx.x / (uint32_t)a.H, b = token / (uint32_t)a.T;
        if ((int)(token - b * (uint32_t)a.T) >= a.lens[b]) return;
    }
    const int lane = threadIdx.x, d = (lane % NL) * 4, i0 = lane / NL;
    const float* ml = a.ws_ml + 2 * row * a.n_split;
    const float* o = a.ws_o + row * a.n_split * D + d;
    float M = -INFINITY;
    for (int i = lane; i < a.n_split; i += 64) M = fmaxf(M, ml[2 * i]);
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) M = fmaxf(M, __shfl_xor(M, x));
    float L = 0.0f;
    f32x4_t v = zero4();
#pragma unroll 4
    for (int i = i0; i < a.n_split; i += NS) {
        const float f = fast_exp2(ml[2 * i] - M);
        L = fmaf(f, ml[2 * i + 1], L);
        const f32x4_t x = *reinterpret_cast<const f32x4_t*>(o + (long long)i * D);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = fmaf(f, x[j], v[j]);
    }
#pragma unroll
    for (int x = NL; x < 64; x <<= 1) {
        L += __shfl_xor(L, x);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] += __shfl_xor(v[j], x);
    }
    const float inv = 1.0f / L;
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] *= inv;
    if (i0 == 0) store4<T>(reinterpret_cast<T*>(a.o) + row * D + d, v);
}

namespace {

template <int D, typename T, int NQ, bool SPLIT>
hipError_t window_attend(WindowArgs a, hipStream_t s) {
    a.q_tiles = (a.T + 64 * NQ - 1) / (64 * NQ);
    a.n_units = (long long)a.B * a.H * a.q_tiles * (SPLIT ? a.n_split : 1);
    a.per_xcd = (a.n_units + 7) / 8;
    if (a.per_xcd > 0x0fffffff) return hipErrorInvalidValue;
    kda_window_prefill_kernel<D, T, NQ, SPLIT><<<dim3((unsigned)(8 * a.per_xcd)), 256, 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (!SPLIT || e != hipSuccess) return e;
    kda_window_join_kernel<D, T><<<dim3((unsigned)((long long)a.B * a.T * a.H)), 64, 0, s>>>(a);
    return hipGetLastError();
}

template <int D, typename T>
hipError_t window_prefill_t(const WindowArgs& a, hipStream_t s) {
    // 128 queries per workgroup read each key once for twice the products; 64 where there are too few
    // queries to give every compute unit a workgroup (and for fp32, whose operands take twice the
    // registers).
    hipError_t e;
    if (a.n_split > 1) e = window_attend<D, T, 1, true>(a, s);
    else if (sizeof(T) == 2 && !a.few) e = window_attend<D, T, sizeof(T) == 2 ? 2 : 1, false>(a, s);
    else e = window_attend<D, T, 1, false>(a, s);
    if (e != hipSuccess || !a.k_cache) return e;
    const int recent = a.window < a.T ? a.window : a.T;
    const int row_bytes = a.Hkv * D * (int)sizeof(T);
    int shift = 3;   // threads per row: a power of two of 16-byte pieces, at most the workgroup
    while (shift < 8 && (16 << shift) < row_bytes) ++shift;
    const int per = 256 >> shift;
    kda_window_keep_kernel<T><<<dim3((unsigned)((a.sinks + recent + per - 1) / per), a.B), 256, 0, s>>>(a, row_bytes, recent, shift);
    return hipGetLastError();
}

template <int D, typename T>
hipError_t window_step_t(WindowArgs a, hipStream_t s) {
    a.n_units = (long long)a.B * a.Hkv * ((a.H / a.Hkv + 15) / 16) * a.n_split;
    a.per_xcd = (a.n_units + 7) / 8;
    if (a.per_xcd > 0x0fffffff) return hipErrorInvalidValue;
    kda_window_step_kernel<D, T><<<dim3((unsigned)(8 * a.per_xcd)), 256, 0, s>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.n_split == 1) return e;
    kda_window_join_kernel<D, T><<<dim3((unsigned)((long long)a.B * a.H)), 64, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_window_prefill(int d, bool f32, const WindowArgs& a, hipStream_t s) {
    if (d == 64) return f32 ? window_prefill_t<64, float>(a, s) : window_prefill_t<64, __bf16>(a, s);
    return f32 ? window_prefill_t<128, float>(a, s) : window_prefill_t<128, __bf16>(a, s);
}
hipError_t launch_window_step(int d, bool f32, const WindowArgs& a, hipStream_t s) {
    if (d == 64) return f32 ? window_step_t<64, float>(a, s) : window_step_t<64, __bf16>(a, s);
    return f32 ? window_step_t<128, float>(a, s) : window_step_t<128, __bf16>(a, s);
}

}  // namespace kda
