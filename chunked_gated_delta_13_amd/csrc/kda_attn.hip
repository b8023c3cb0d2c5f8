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

// What a workgroup does: BM rows of one sequence and kv head, from row0 up to row1, over the keys from t_first up to t_end
// (SPLIT: a range of them).  The last row sees `total` keys, a sequence's query i the keys up to i + off.
struct AttnUnit {
    int R, hk, split, q_first, k_first, off, row0, row1, total, t_first, t_end;
};

// An XCD serves every `n_sets`-th kv head (n_sets: the greatest common divisor of their count and 8), so that what it reads
// is read again from its own L2; XCDs with the same heads take turns at their row tiles.  Long tiles are started
// first, whatever their head: with one head after the other six prompts of up to 2000 tokens took half as long again.  The
// ranges of a split, whose keys few workgroups share, go to the XCDs in turn.
template <int BM, bool SPLIT> __device__ __forceinline__ bool attn_unit(const AttnArgs& a, int lane, AttnUnit& u) {
    int x;
    if constexpr (SPLIT) {
        uint32_t unit = blockIdx.x;
        u.split = (int)(unit % (uint32_t)a.n_split);
        unit /= (uint32_t)a.n_split;
        u.hk = (int)(unit % (uint32_t)a.Hkv);
        x = (int)(unit / (uint32_t)a.Hkv);
    } else {
        const uint32_t unit = blockIdx.x >> 3, xcd = blockIdx.x & 7, sets = (uint32_t)a.n_sets, heads = (uint32_t)a.Hkv / sets;
        u.split = 0;
        u.hk = (int)(unit % heads * sets + xcd % sets);
        x = (int)(unit / heads * (8 / sets) + xcd / sets);
    }
    const int R = (int)((uint32_t)a.H / (uint32_t)a.Hkv);
    u.R = R;

    // Tile x, counted from the last sequence's last tile (the longest of each sequence come first): 64
    // sequences at a time, a lane each, their tiles summed over the lanes.
    int b = -1, nq = 0, tile = 0;
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
            u.q_first = __builtin_amdgcn_readlane(first, at);
            nq = __builtin_amdgcn_readlane(len, at);
            tile = __builtin_amdgcn_readlane(sum, at) - 1 - x;
            break;
        }
        x -= __builtin_amdgcn_readlane(sum, 63);
    }
    if (b < 0) return false;
    int k_first = u.q_first, nk = nq;
    if (a.cu_k != a.cu_q) packed(a.cu_k, b, a.Nk, &k_first, &nk);
    u.k_first = k_first;
    u.off = nk - nq;                              // keys before the first query
    u.row0 = tile * BM;
    const int rows = nq * R;                      // (B tiles of 64 rows fit 32 bits: checked on the host)
    u.row1 = u.row0 + BM < rows ? u.row0 + BM : rows;
    int total = (int)((uint32_t)(u.row1 - 1) / (uint32_t)R) + u.off + 1;   // keys that the last row sees
    if (total < 0) total = 0;
    u.total = total;
    u.t_first = 0;
    u.t_end = total;
    if constexpr (SPLIT) {
        const int tiles = (total + kKeys - 1) / kKeys, per = (int)((uint32_t)(tiles + a.n_split - 1) / (uint32_t)a.n_split);
        u.t_first = u.split * per * kKeys < total ? u.split * per * kKeys : total;
        u.t_end = u.t_first + per * kKeys < total ? u.t_first + per * kKeys : total;
    }
    return true;
}

// Groups of four waves that hold the same rows: their outputs, maxima and sums, joined by group 0 (true).  Every wave of
// the workgroup calls it, behind its last use of LDS and a barrier.
template <int D, int KG>
__device__ __forceinline__ bool join_groups(KDA_LDS f32x4_t* room, f32x4_t (&O)[D / 16][1], float& m, float& sum, int wave, int group,
                                            int lane) {
    constexpr int NT = D / 16;
    KDA_LDS f32x4_t* at = room + wave * (NT + 1) * 64 + lane;
    if (group > 0) {
        KDA_LDS f32x4_t* to = at + (group - 1) * 4 * (NT + 1) * 64;
#pragma unroll
        for (int t = 0; t < NT; ++t) to[64 * t] = O[t][0];
        to[64 * NT] = f32x4_t{m, sum, 0.0f, 0.0f};
    }
    barrier_lds();
    if (group > 0) return false;
    float mx = m;
    f32x4_t ml[KG - 1];
#pragma unroll
    for (int i = 0; i < KG - 1; ++i) {
        ml[i] = at[(i * 4 * (NT + 1) + NT) * 64];
        mx = fmaxf(mx, ml[i][0]);
    }
    const float base = mx == -INFINITY ? 0.0f : mx, f0 = fast_exp2(m - base);
    sum *= f0;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) O[t][0][j] *= f0;
#pragma unroll
    for (int i = 0; i < KG - 1; ++i) {
        const float f = fast_exp2(ml[i][0] - base);
        sum = fmaf(f, ml[i][1], sum);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const f32x4_t x = at[(i * 4 * (NT + 1) + t) * 64];
#pragma unroll
            for (int j = 0; j < 4; ++j) O[t][0][j] = fmaf(f, x[j], O[t][0][j]);
        }
    }
    m = mx;
    return true;
}

}  // namespace

// A workgroup of four waves runs 64 NQ rows of one (sequence, kv head); each wave holds 16 NQ rows and their
// outputs in registers.  The keys come tile by tile straight from memory into one of two LDS tiles, one tile
// ahead, and two workgroups share a compute unit: while one wave of a SIMD forms exponentials, the other feeds
// the matrix cores.
//
// Bound by the issue of products and of the exponentials between them: prompts of 333 to 16384 tokens, 56 heads on 8 of 128,
// 3.54 to 3.72 ms by card, 1.12 to 1.17 PFLOP/s (a large library product 1.40).  Products are busy in 56% of the cycles, and
// vector instructions, these among them, are issued in 47%; scores of the next tile formed beside the exponentials of this one
// in the same wave were slower (4.9 ms), since their registers leave no room.
//
// The running maximum only has to keep exponentials in range.  A tile that every row of the wave sees whole is
// taken with the maximum at hand, without forming its own; only if a sum of its exponentials passes kSumMax (a
// score far above that maximum) is the maximum brought up to date.
constexpr float kSumMax = 16384.0f;

// SPLIT: a workgroup takes one of n_split ranges of its rows' tiles and leaves partial outputs with their
// maxima and sums, which kda_attn_join_kernel joins.
//
// KG: with workgroups for less than the compute units, KG groups of four waves hold the same rows and take every KG-th
// tile of keys; their outputs are joined at the end, in LDS.  Five pieces of up to 77 queries behind up to 1500 keys, 8 heads
// on 2 of 64: 13.2 us in four groups, 17.6 in one; a step of the groups takes 1.3 us.
template <int D, int NQ, int KG, bool SPLIT>
__global__ __launch_bounds__(256 * KG, KG == 1 ? 2 : KG) void kda_attn_prefill_kernel(const AttnArgs a) {
    typedef __bf16 T;
    constexpr int BM = 64 * NQ, TILE = kKeys * D, STEP = KG * kKeys;
    typedef TileSteps<T, kKeys, D, 4> Steps;
    constexpr int NG = Steps::N / Steps::NB;   // row groups per wave
    static_assert(NG * Steps::NB == Steps::N, "a wave takes whole rows");
    static_assert(KG == 1 || NQ == 1, "the groups' outputs fit in LDS");
    __shared__ __attribute__((aligned(16))) T smem[KG * 2 * 2 * TILE];   // two pairs of a tile of keys and one of values each
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6) & 3, group = __builtin_amdgcn_readfirstlane(tid >> 8);
    KDA_LDS T* sK = (KDA_LDS T*)smem + group * (2 * 2 * TILE);

    AttnUnit u;
    if (!attn_unit<BM, SPLIT>(a, lane, u)) return;
    const int R = u.R, hk = u.hk, split = u.split, q_first = u.q_first, off = u.off, row0 = u.row0, row1 = u.row1;
    const int total = u.total, t_first = u.t_first, t_end = u.t_end;

    const int g = lane >> 4, r = lane & 15;
    TileRows<T, kKeys, D> rk0;
    TileCols<T, kKeys> cv0;
    rk0.set(sK, lane);
    cv0.set(sK + TILE, lane);

    const T* kn = reinterpret_cast<const T*>(a.k) + (long long)u.k_first * a.k_stride + (long long)hk * D;
    const T* vn = reinterpret_cast<const T*>(a.v) + (long long)u.k_first * a.v_stride + (long long)hk * D;

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
                dma16(kp + pcol + 32 * i, lds_address(dst + i * kKeys * 32));
                dma16(vp + pcol + 32 * i, lds_address(dst + TILE + i * kKeys * 32));
            }
        }
    };
    const int own0 = t_first + group * kKeys;   // this group's first tile
    if (own0 < t_end) fetch(own0, 0);

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

    for (int t0 = own0, buf = 0; t0 - group * kKeys < t_end; t0 += STEP, buf ^= 1) {
        if (KG > 1 && t0 >= t_end) {   // (the other groups' last barrier)
            barrier_all();
            break;
        }
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
        if (t0 + STEP < t_end) fetch(t0 + STEP, buf ^ 1);
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
        float sum = sum_over_groups<NQ == 1>(l[n]);
        if constexpr (KG > 1) {
            if (!join_groups<D, KG>((KDA_LDS f32x4_t*)smem, O, m[n], sum, wave, group, lane)) return;
        }
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

// fp32.  The matrix cores multiply bf16 at sixteen times the rate of fp32, so every operand is taken in three bf16 parts
// (x = h + m + l to 2^-24 of x, or to 2^-126, where bf16's normal numbers end) and of a product of two operands the six
// largest products of parts, from h h down to l h, m m and h l: what is left out is below 2^-23 of it.  A wave's queries
// are split once; keys and values once per workgroup and tile, on their way from registers to LDS.
//
// Eight waves run 64 rows: 16 rows each, waves 4 to 7 the same rows as 0 to 3 over the other half of each tile's keys, so
// that a long prompt's chain of tiles is half as long; the halves are joined at the end.  A tile takes two phases: the values
// are split while the scores are formed, the next keys while the values are summed, so that one copy of each (96 KB at
// d = 128) is enough and splitting runs beside the products.  Of the two waves of a SIMD one splits first, one last.  Prompts of
// up to 2000 tokens, 16 heads on 4 of 128: 131 to 134 us (fp32 products 259), 3.6 us a tile; bound by issue (products busy in 39%
// of the cycles, vector instructions, these among them, issued in 42%) and by the longest prompt's tiles one after the other.
template <int D, bool SPLIT>
__global__ __launch_bounds__(512) void kda_attn_prefill_f32_kernel(const AttnArgs a) {
    constexpr int BM = 64, TILE = kKeys * D, NT = D / 16;
    typedef TileSteps<__bf16, kKeys, D, 8> Steps;
    __shared__ __attribute__((aligned(16))) __bf16 smem[6 * TILE];   // three parts of the keys, three of the values
    KDA_LDS __bf16* sK = (KDA_LDS __bf16*)smem;

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int half = wave >> 2;
    AttnUnit u;
    if (!attn_unit<BM, SPLIT>(a, lane, u)) return;
    const int g = lane >> 4, r = lane & 15;

    TileRows<__bf16, kKeys, D> rk;
    TileCols<__bf16, kKeys> cv;
    TilePut<__bf16, kKeys> put;
    rk.set(sK, lane);
    cv.set(sK + 3 * TILE, lane);
    put.set(sK + Steps::block0(wave) * kKeys * 32, Steps::group0(wave), lane);

    // A lane's share of a tile: eight columns of one row, Steps::N times.  Places past the last key take the last key
    // again: they are masked, and their values are finite.
    const int krow = Steps::group0(wave) * TileStep<__bf16>::ROWS + TileStep<__bf16>::row(lane);
    const int col = Steps::block0(wave) * 32 + TileStep<__bf16>::piece(lane) * 8;
    const float* kn = reinterpret_cast<const float*>(a.k) + (long long)u.k_first * a.k_stride + (long long)u.hk * D + col;
    const float* vn = reinterpret_cast<const float*>(a.v) + (long long)u.k_first * a.v_stride + (long long)u.hk * D + col;
    f32x4_t xk[Steps::N][2], xv[Steps::N][2];
    auto fetch = [&](f32x4_t (&x)[Steps::N][2], const float* p, long long stride, int t0) {
        const int at = t0 + krow, idx = at < u.total ? at : u.total - 1;
        p += (long long)idx * stride;
#pragma unroll
        for (int i = 0; i < Steps::N; ++i) {
            x[i][0] = *reinterpret_cast<const f32x4_t*>(p + 32 * i);
            x[i][1] = *reinterpret_cast<const f32x4_t*>(p + 32 * i + 4);
        }
    };
    auto keep = [&](const f32x4_t (&x)[Steps::N][2], int base) {
#pragma unroll
        for (int i = 0; i < Steps::N; ++i) {
            Frag<__bf16> f[3];
            parts_of<3>(f, x[i][0], x[i][1]);
#pragma unroll
            for (int p = 0; p < 3; ++p)
                *reinterpret_cast<KDA_LDS u32x4_t*>(put.at[0] + (base + p) * TILE + i * kKeys * 32) = __builtin_bit_cast(u32x4_t, f[p].v);
        }
    };
    static_assert(Steps::N <= Steps::NB, "a wave's steps lie in one group of rows");
    if (u.t_first < u.t_end) {
        fetch(xk, kn, a.k_stride, u.t_first);
        fetch(xv, vn, a.v_stride, u.t_first);
    }

    // this wave's rows, and the last key that each sees
    const int w_row = u.row0 + (wave & 3) * 16, row = w_row + r;
    const int w_sees = (int)((uint32_t)w_row / (uint32_t)u.R) + u.off;   // of its first row
    const int qi = (int)((uint32_t)row / (uint32_t)u.R), h = u.hk * u.R + (row - qi * u.R), sees = qi + u.off;
    const long long place = (long long)(u.q_first + qi) * a.H + h;   // row of the outputs: query and head
    Frag<__bf16> fq[D / 32][3];
    {
        const float* qp = reinterpret_cast<const float*>(a.q) + (long long)(u.q_first + qi) * a.q_stride + (long long)h * D + 4 * g;
#pragma unroll
        for (int kb = 0; kb < D / 32; ++kb) {
            f32x4_t lo = zero4(), hi = zero4();
            if (row < u.row1) {
                lo = *reinterpret_cast<const f32x4_t*>(qp + 16 * kb);
                hi = *reinterpret_cast<const f32x4_t*>(qp + 16 * kb + D / 2);
            }
            parts_of<3>(fq[kb], lo, hi);
        }
    }

    f32x4_t O[NT][1];
    float m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int t = 0; t < NT; ++t) O[t][0] = zero4();
    const float sc = a.scale * kLog2e;
    bool ready = false;   // every row of the wave has a maximum
    if (u.t_first < u.t_end) {
        keep(xk, 0);
        if (u.t_first + kKeys < u.t_end) fetch(xk, kn, a.k_stride, u.t_first + kKeys);
    }

    for (int t0 = u.t_first; t0 < u.t_end; t0 += kKeys) {
        const bool more = t0 + kKeys < u.t_end;
        barrier_lds();   // the keys' parts are there, and nobody reads the values before them any more
        if (half == 0) {
            keep(xv, 3);
            if (more) fetch(xv, vn, a.v_stride, t0 + kKeys);
        }

        // key tiles half and half + 2: their rows are the contraction block `half` of the product with the values
        f32x4_t s[2] = {zero4(), zero4()};
        Frag<__bf16> fk[2][2][3];
        auto keys = [&](int kb) {
#pragma unroll
            for (int kt = 0; kt < 2; ++kt)
#pragma unroll
                for (int p = 0; p < 3; ++p) rk.frag(fk[kb & 1][kt][p], p * TILE, half + 2 * kt, kb);
        };
        keys(0);
#pragma unroll
        for (int kb = 0; kb < D / 32; ++kb) {
            if (kb + 1 < D / 32) keys(kb + 1);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int x = 0; x < 6; ++x) {
                constexpr int A[6] = {2, 0, 1, 1, 0, 0}, B[6] = {0, 2, 1, 0, 1, 0};
#pragma unroll
                for (int kt = 0; kt < 2; ++kt) s[kt] = mma(fk[kb & 1][kt][A[x]], fq[kb][B[x]], s[kt]);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        const bool whole = t0 + kKeys - 1 <= w_sees;
        bool done = false;
        Frag<__bf16> fp[3];
        if (whole && ready) {
            f32x4_t e[2];
            float sum = 0.0f;
#pragma unroll
            for (int kt = 0; kt < 2; ++kt)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    e[kt][j] = fast_exp2(fmaf(s[kt][j], sc, -m));
                    sum += e[kt][j];
                }
            done = !__any(!(sum < kSumMax));
            if (done) {
                l += sum;
                parts_of<3>(fp, e[0], e[1]);
            }
        }
        if (!done) {
            if (!whole) {
                const int to = (sees < u.total - 1 ? sees : u.total - 1) - t0 - 16 * half - 4 * g;
#pragma unroll
                for (int kt = 0; kt < 2; ++kt)
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[kt][j] = 32 * kt + j <= to ? s[kt][j] : -INFINITY;
            }
            float mx = -INFINITY;
#pragma unroll
            for (int kt = 0; kt < 2; ++kt)
#pragma unroll
                for (int j = 0; j < 4; ++j) mx = fmaxf(mx, s[kt][j]);
            mx = fmaxf(m, max_over_groups<true>(mx) * sc);
            const float base = mx == -INFINITY ? 0.0f : mx;   // nothing visible yet: all exponentials are 0
            const float al = fast_exp2(m - base);
            m = mx;
            ready = __all(mx != -INFINITY);
            float sum = 0.0f;
#pragma unroll
            for (int kt = 0; kt < 2; ++kt)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[kt][j] = fast_exp2(fmaf(s[kt][j], sc, -base));
                    sum += s[kt][j];
                }
            l = l * al + sum;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j) O[t][0][j] *= al;
            parts_of<3>(fp, s[0], s[1]);
        }
        if (half == 1) {
            keep(xv, 3);
            if (more) fetch(xv, vn, a.v_stride, t0 + kKeys);
        }
        barrier_lds();   // the values' parts are there, and nobody reads the keys any more
        if (half == 0 && more) {
            keep(xk, 0);
            if (t0 + 2 * kKeys < u.t_end) fetch(xk, kn, a.k_stride, t0 + 2 * kKeys);
        }
        Frag<__bf16> fv[2][2][3];
        auto values = [&](int t) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int p = 0; p < 3; ++p) cv.frag(fv[(t >> 1) & 1][i][p], p * TILE, t + i, half);
        };
        values(0);
#pragma unroll
        for (int t = 0; t < NT; t += 2) {
            if (t + 2 < NT) values(t + 2);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int x = 0; x < 6; ++x) {
                constexpr int A[6] = {2, 0, 1, 1, 0, 0}, B[6] = {0, 2, 1, 0, 1, 0};
#pragma unroll
                for (int i = 0; i < 2; ++i) O[t + i][0] = mma(fv[(t >> 1) & 1][i][A[x]], fp[B[x]], O[t + i][0]);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if (half == 1 && more) {
            keep(xk, 0);
            if (t0 + 2 * kKeys < u.t_end) fetch(xk, kn, a.k_stride, t0 + 2 * kKeys);
        }
    }

    l = sum_over_groups<true>(l);
    barrier_lds();
    if (!join_groups<D, 2>((KDA_LDS f32x4_t*)smem, O, m, l, wave & 3, half, lane) || row >= u.row1) return;
    const float inv = SPLIT ? 1.0f : (l == 0.0f ? 0.0f : 1.0f / l);
    const long long to = SPLIT ? place * a.n_split + u.split : place;
    float* op = (SPLIT ? a.ws_o : reinterpret_cast<float*>(a.o)) + to * D + 4 * g;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int j = 0; j < 4; ++j) O[t][0][j] *= inv;
        *reinterpret_cast<f32x4_t*>(op + 16 * t) = O[t][0];
    }
    if (SPLIT && g == 0) {
        a.ws_ml[2 * to] = m;
        a.ws_ml[2 * to + 1] = l;
    }
}

// Joins the ranges of a split call.  grid: (query, head) rows.  Rows outside the sequences have no parts.
template <int D, typename T>
__global__ __launch_bounds__(256) void kda_attn_join_kernel(const AttnArgs a) {
    const long long row = blockIdx.x;
    const int query = (int)(blockIdx.x / (uint32_t)a.H);
    bool in = false;
    for (int b = threadIdx.x & 63; b < a.B; b += 64) {
        int first = 0, len = 0;
        packed(a.cu_q, b, a.Nq, &first, &len);
        in = in || (query >= first && query - first < len);
    }
    if (!__any(in)) return;   // (every wave finds the same)
    const long long first = row * a.n_split;
    join_parts<D, T, 256>(a.ws_ml + 2 * first, a.ws_o + first * D, a.n_split, 1, reinterpret_cast<T*>(a.o) + row * D);
}

namespace {

// NQ: 16 NQ rows per wave.  KG: groups of waves (bf16).
template <int D, typename T, int NQ, int KG, bool SPLIT>
hipError_t attend(AttnArgs a, hipStream_t s) {
    // every sequence adds at most one tile that is not full
    constexpr int THREADS = sizeof(T) == 4 ? 512 : 256 * KG;
    const long long rows = (long long)a.Nq * (a.H / a.Hkv), tiles = rows / (64 * NQ) + a.B;
    a.n_sets = 1;
    while (a.n_sets < 8 && a.Hkv % (2 * a.n_sets) == 0) a.n_sets *= 2;
    const long long turns = 8 / a.n_sets, per_xcd = (tiles + turns - 1) / turns;
    const long long blocks = SPLIT ? tiles * a.Hkv * a.n_split : 8 * per_xcd * (a.Hkv / a.n_sets);
    if (blocks > 0xffffffffLL / THREADS) return hipErrorInvalidValue;
    if constexpr (sizeof(T) == 4) kda_attn_prefill_f32_kernel<D, SPLIT><<<dim3((unsigned)blocks), THREADS, 0, s>>>(a);
    else kda_attn_prefill_kernel<D, NQ, KG, SPLIT><<<dim3((unsigned)blocks), THREADS, 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (!SPLIT || e != hipSuccess) return e;
    kda_attn_join_kernel<D, T><<<dim3((unsigned)((long long)a.Nq * a.H)), 256, 0, s>>>(a);   // (few rows: see the plan)
    return hipGetLastError();
}

template <int D, typename T>
hipError_t attn_prefill_t(const AttnArgs& a, hipStream_t s) {
    if constexpr (sizeof(T) == 2) {
        constexpr int KG = attn_groups(D);
        if (a.n_split > 1) return attend<D, T, 1, KG, true>(a, s);
        if (a.few > 1) return attend<D, T, 1, KG, false>(a, s);
        return a.few ? attend<D, T, 1, 1, false>(a, s) : attend<D, T, 2, 1, false>(a, s);
    } else {
        return a.n_split > 1 ? attend<D, T, 1, 1, true>(a, s) : attend<D, T, 1, 1, false>(a, s);
    }
}

}  // namespace

hipError_t launch_attn_prefill(int d, bool f32, const AttnArgs& a, hipStream_t s) {
    if (d == 64) return f32 ? attn_prefill_t<64, float>(a, s) : attn_prefill_t<64, __bf16>(a, s);
    return f32 ? attn_prefill_t<128, float>(a, s) : attn_prefill_t<128, __bf16>(a, s);
}

}  // namespace kda
