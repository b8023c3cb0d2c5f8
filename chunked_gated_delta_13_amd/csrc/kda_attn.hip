// Causal attention over packed prompts, for gfx950.
//
// The queries of a sequence are the last nq of its nk tokens: query i sees the keys j <= i + nk - nq (one that
// sees none gets zeros).  The H / Hkv query heads of a kv head are rows beside each other: row i R + h of a
// sequence is its query i of head h of the group, so a few queries of a piece fill a matrix tile, and rows
// that share keys share the tile's edge on the diagonal.
//
// One pass over the visible keys with the running maximum and sum of the softmax (fp32, exponentials of base
// 2).  Scores are formed transposed, K Q^T with keys as rows: a lane then holds four keys of one query, the
// statistics of a query stay in its lanes, and the probabilities are at once the operand of V^T P^T.  For that
// product only they are rounded to the input type (bf16 outputs are 2.0 to 2.3e-3 off then, 1.7e-3 of it
// their own rounding).
#include "kda_mixers.h"
#include "kda_softmax.h"

namespace kda {

namespace {

constexpr int kKeys = 64;   // keys per tile

// A sequence of the packed batch: its first row, its length.  Ends outside the tensor are clamped, a sequence
// that ends before its start is empty.
__device__ __forceinline__ void packed(const int* cu, int b, int n, int* first, int* len) {
    int x = cu[b], y = cu[b + 1];
    x = x < 0 ? 0 : (x > n ? n : x);
    y = y < x ? x : (y > n ? n : y);
    *first = x;
    *len = y - x;
}

}  // namespace

// A workgroup of four waves runs 64 NQ rows of one (sequence, kv head); each wave holds 16 NQ rows and their
// outputs in registers.  The keys come tile by tile straight from memory into one of two LDS tiles, one tile
// ahead, and two workgroups share a compute unit: while one wave of a SIMD forms exponentials, the other feeds
// the matrix cores.
//
// The running maximum only has to keep exponentials in range.  A tile that every row of the wave sees whole is
// taken with the maximum at hand, without forming its own; only if a sum of its exponentials passes kSumMax (a
// score far above that maximum) is the maximum brought up to date.
constexpr float kSumMax = 16384.0f;

// SPLIT: a workgroup takes one of n_split ranges of its rows' tiles and leaves partial outputs with their
// maxima and sums, which kda_attn_join_kernel joins.
template <int D, typename T, int NQ, bool SPLIT>
__global__ __launch_bounds__(256, sizeof(T) == 2 ? 2 : 1) void kda_attn_prefill_kernel(const AttnArgs a) {
    constexpr int BM = 64 * NQ, TILE = kKeys * D;
    typedef TileSteps<T, kKeys, D, 4> Steps;
    constexpr int NG = Steps::N / Steps::NB;   // row groups per wave
    static_assert(NG * Steps::NB == Steps::N, "a wave takes whole rows");
    __shared__ __attribute__((aligned(16))) T smem[2 * 2 * TILE];   // two pairs of a tile of keys and one of values
    KDA_LDS T* sK = (KDA_LDS T*)smem;

    // unit = (kv head, eighth of the row tiles, range): the workgroups of an XCD take every eighth tile, so
    // that each XCD gets early and late tiles, whose keys differ in number
    uint32_t unit = blockIdx.x >> 3;
    int split = 0;
    if constexpr (SPLIT) {
        split = (int)(unit % (uint32_t)a.n_split);
        unit /= (uint32_t)a.n_split;
    }
    const int hk = (int)(unit / (uint32_t)a.per_xcd);
    int x = (int)(unit % (uint32_t)a.per_xcd) * 8 + (int)(blockIdx.x & 7);
    const int R = (int)((uint32_t)a.H / (uint32_t)a.Hkv);

    // Tile x, counted from the last sequence's last tile (the longest of each sequence come first): 64
    // sequences at a time, a lane each, their tiles summed over the lanes.
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int b = -1, q_first = 0, nq = 0, tile = 0;
    for (int b0 = a.B - 1; b0 >= 0; b0 -= 64) {
        int first = 0, len = 0;
        if (b0 - lane >= 0) packed(a.cu_q, b0 - lane, a.Nq, &first, &len);
        const int tiles = (int)(((long long)len * R + BM - 1) / BM);
        int sum = tiles;
#pragma unroll
        for (int s = 1; s < 64; s <<= 1) {
            const int y = __shfl_up(sum, s);
            if (lane >= s) sum += y;
        }
        const unsigned long long past = __ballot(sum > x);
        if (past) {
            const int at = __builtin_ctzll(past);
            b = b0 - at;
            q_first = __builtin_amdgcn_readlane(first, at);
            nq = __builtin_amdgcn_readlane(len, at);
            tile = __builtin_amdgcn_readlane(sum, at) - 1 - x;
            break;
        }
        x -= __builtin_amdgcn_readlane(sum, 63);
    }
    if (b < 0) return;
    int k_first = q_first, nk = nq;
    if (a.cu_k != a.cu_q) packed(a.cu_k, b, a.Nk, &k_first, &nk);
    const int off = nk - nq;                      // keys before the first query
    const int row0 = tile * BM, rows = nq * R;    // (B tiles of 64 rows fit 32 bits: checked on the host)
    const int row1 = row0 + BM < rows ? row0 + BM : rows;
    int total = (int)((uint32_t)(row1 - 1) / (uint32_t)R) + off + 1;   // keys that the last row sees
    if (total < 0) total = 0;
    int t_first = 0, t_end = total;   // this workgroup's part of them
    if constexpr (SPLIT) {
        const int tiles = (total + kKeys - 1) / kKeys, per = (int)((uint32_t)(tiles + a.n_split - 1) / (uint32_t)a.n_split);
        t_first = split * per * kKeys < total ? split * per * kKeys : total;
        t_end = t_first + per * kKeys < total ? t_first + per * kKeys : total;
    }

    const int g = lane >> 4, r = lane & 15;
    TileRows<T, kKeys, D> rk0;
    TileCols<T, kKeys> cv0;
    rk0.set(sK, lane);
    cv0.set(sK + TILE, lane);

    const T* kn = reinterpret_cast<const T*>(a.k) + (long long)k_first * a.k_stride + (long long)hk * D;
    const T* vn = reinterpret_cast<const T*>(a.v) + (long long)k_first * a.v_stride + (long long)hk * D;

    // A lane's key rows of a tile: one (bf16) or two (fp32) per wave, 16 bytes of each block of 32 columns.
    // Places past the last key take the last key again: they are masked, and their values are finite.
    auto fetch = [&](int t0, int buf) {
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            const int row16 = (Steps::group0(wave) + j) * TileStep<T>::ROWS + TileStep<T>::row(lane);
            const int pcol = tile_dma_piece<T>(row16, lane) * TileStep<T>::ELEMS;
            const int at = t0 + row16, idx = at < total ? at : total - 1;
            const T *kp = kn + (long long)idx * a.k_stride, *vp = vn + (long long)idx * a.v_stride;
            KDA_LDS T* dst = sK + buf * (2 * TILE) + (Steps::group0(wave) + j) * TileStep<T>::ROWS * 32;
#pragma unroll
            for (int i = 0; i < Steps::NB; ++i) {
                lds_dma16(reinterpret_cast<const float*>(kp + pcol + 32 * i), dst + i * kKeys * 32);
                lds_dma16(reinterpret_cast<const float*>(vp + pcol + 32 * i), dst + TILE + i * kKeys * 32);
            }
        }
    };
    if (t_first < t_end) fetch(t_first, 0);

    // this wave's rows, and the last key that each sees
    const int w_row = row0 + wave * 16 * NQ;
    const int w_sees = (int)((uint32_t)w_row / (uint32_t)R) + off;   // of its first row
    Frag<T> fq[NQ][D / 32];
    int sees[NQ];
    long long place[NQ];   // row of the outputs: query and head
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        const int row = w_row + 16 * n + r;
        const int i = (int)((uint32_t)row / (uint32_t)R), h = hk * R + (row - i * R);
        sees[n] = i + off;
        place[n] = (long long)(q_first + i) * a.H + h;
        const T* qp = reinterpret_cast<const T*>(a.q) + (long long)(q_first + i) * a.q_stride + (long long)h * D + 4 * g;
#pragma unroll
        for (int kb = 0; kb < D / 32; ++kb) {
            if (row < row1) global_frag<D>(fq[n][kb], qp + 16 * kb);
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
    bool ready = false;   // every row of the wave has a maximum
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
        // transposed read waits for every request to LDS before it.
        Frag<T> fv[2][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) cv.frag(fv[0][i], 0, i, 0);
        __builtin_amdgcn_sched_barrier(0);
        if (t0 + kKeys < t_end) fetch(t0 + kKeys, buf ^ 1);
        __builtin_amdgcn_sched_barrier(0);

        const bool whole = t0 + kKeys - 1 <= w_sees;
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
#pragma unroll
                for (int n = 0; n < NQ; ++n) {
                    const int to = (sees[n] < total - 1 ? sees[n] : total - 1) - t0 - 4 * g;
#pragma unroll
                    for (int kt = 0; kt < 4; ++kt)
#pragma unroll
                        for (int j = 0; j < 4; ++j) sT[kt][n][j] = 16 * kt + j <= to ? sT[kt][n][j] : -INFINITY;
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
        const float sum = sum_over_groups<NQ == 1>(l[n]);
        if (w_row + 16 * n + r >= row1) continue;
        if constexpr (SPLIT) {
            const long long part = place[n] * a.n_split + split;
#pragma unroll
            for (int t = 0; t < D / 16; ++t) *reinterpret_cast<f32x4_t*>(a.ws_o + part * D + 16 * t + 4 * g) = O[t][n];
            if (g == 0) {
                a.ws_ml[2 * part] = m[n];
                a.ws_ml[2 * part + 1] = sum;
            }
        } else {
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
            T* op = reinterpret_cast<T*>(a.o) + place[n] * D + 4 * g;
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

// Joins the ranges of a split call.  grid: (query, head) rows; one wave: D / 4 lanes own four channels of a
// range, and 64 / (D / 4) ranges are taken side by side.  Rows outside the sequences have no parts.
template <int D, typename T>
__global__ __launch_bounds__(64) void kda_attn_join_kernel(const AttnArgs a) {
    constexpr int NL = D / 4, NS = 64 / NL;
    const long long row = blockIdx.x;
    const int lane = threadIdx.x, d = (lane % NL) * 4, i0 = lane / NL;
    const int query = (int)(blockIdx.x / (uint32_t)a.H);
    bool in = false;
    for (int b = lane; b < a.B; b += 64) {
        int first = 0, len = 0;
        packed(a.cu_q, b, a.Nq, &first, &len);
        in = in || (query >= first && query - first < len);
    }
    if (!__any(in)) return;
    const float* ml = a.ws_ml + 2 * row * a.n_split;
    const float* o = a.ws_o + row * a.n_split * D + d;
    float M = -INFINITY;
    for (int i = lane; i < a.n_split; i += 64) M = fmaxf(M, ml[2 * i]);
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) M = fmaxf(M, __shfl_xor(M, x));
    const float base = M == -INFINITY ? 0.0f : M;
    float L = 0.0f;
    f32x4_t v = zero4();
#pragma unroll 4
    for (int i = i0; i < a.n_split; i += NS) {
        const float f = fast_exp2(ml[2 * i] - base);
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
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] *= inv;
    if (i0 == 0) store4<T>(reinterpret_cast<T*>(a.o) + row * D + d, v);
}

namespace {

template <int D, typename T, int NQ, bool SPLIT>
hipError_t attend(AttnArgs a, hipStream_t s) {
    // every sequence adds at most one tile that is not full
    const long long rows = (long long)a.Nq * (a.H / a.Hkv), tiles = rows / (64 * NQ) + a.B;
    a.per_xcd = (tiles + 7) / 8;
    const long long blocks = 8 * a.per_xcd * a.Hkv * (SPLIT ? a.n_split : 1);
    if (blocks > 0x7fffffff / 256 * 2) return hipErrorInvalidValue;
    kda_attn_prefill_kernel<D, T, NQ, SPLIT><<<dim3((unsigned)blocks), 256, 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (!SPLIT || e != hipSuccess) return e;
    kda_attn_join_kernel<D, T><<<dim3((unsigned)((long long)a.Nq * a.H)), 64, 0, s>>>(a);
    return hipGetLastError();
}

template <int D, typename T>
hipError_t attn_prefill_t(const AttnArgs& a, hipStream_t s) {
    if (a.n_split > 1) return attend<D, T, 1, true>(a, s);
    if constexpr (sizeof(T) == 2) {
        if (!a.few) return attend<D, T, 2, false>(a, s);
    }
    return attend<D, T, 1, false>(a, s);
}

}  // namespace

hipError_t launch_attn_prefill(int d, bool f32, const AttnArgs& a, hipStream_t s) {
    if (d == 64) return f32 ? attn_prefill_t<64, float>(a, s) : attn_prefill_t<64, __bf16>(a, s);
    return f32 ? attn_prefill_t<128, float>(a, s) : attn_prefill_t<128, __bf16>(a, s);
}

}  // namespace kda
