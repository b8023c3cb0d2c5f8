// A paged cache of keys and values in 4 bits an element, for gfx950: written, read back, and attended to.
//
// The form is the open microscaling one: 32 channels of a row share a power of two 2^e, kept as the byte
// e + 127, and an element is a sign, two bits of exponent and one of fraction (0, .5, 1, 1.5, 2, 3, 4, 6).
// e is the smallest integer from -125 to 95 with max |x| <= 7 2^e: the largest element, at most half a step above
// the last value, is then rounded no more coarsely than the others (above 7 2^95 elements are kept as 6 2^95, 2.4e29).
// Elements are rounded to the nearest value, ties to the even fraction.  A block that holds a NaN or an infinity has
// the byte 255 and reads as NaN.  Every value is exact in bf16, and none is subnormal in fp32.
//
// A page holds P rows (a power of two from 16 on) of one kv head: P d/2 bytes of elements, row after row, even
// channels in the low halves of their bytes, then P d/32 bytes of exponents.  Page p of kv head h lies at
// (p Hkv + h) P (d/2 + d/32).  A sequence's table names the page of each P positions.  An entry outside the pool is
// never followed: its tokens are not written, read back as zeros, and are not seen.
#include "kda_mixers.h"
#include "kda_softmax.h"

namespace kda {

namespace {

// Bytes of the smallest and largest powers of two, 2^-125 and 2^95: no value is subnormal, and the conversions of
// this GPU are right (from the byte 223 on the second of two elements came back as the first).
constexpr uint32_t kLeastExp = 2, kMostExp = 222;

__device__ __forceinline__ float block_scale(uint32_t e) { return __uint_as_float(e << 23); }

// Eight elements of a dword, widened with their block's power of two.
__device__ __forceinline__ void widen8(bf16x8_t& v, uint32_t c, float s) {
    const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 0), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 1);
    const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 2), e = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 3);
    v = bf16x8_t{a[0], a[1], b[0], b[1], d[0], d[1], e[0], e[1]};
}

// Eight elements of a row as they lie in memory (16 bytes are aligned).
template <typename T> struct Eight { typedef bf16x8_t type; };
template <> struct Eight<float> { typedef __attribute__((ext_vector_type(8), aligned(16))) float type; };

__device__ __forceinline__ void load8(float (&x)[8], const __bf16* p) {
    const bf16x8_t v = *reinterpret_cast<const bf16x8_t*>(p);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (float)v[i];
}
__device__ __forceinline__ void load8(float (&x)[8], const float* p) {
    const f32x4_t a = *reinterpret_cast<const f32x4_t*>(p), b = *reinterpret_cast<const f32x4_t*>(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[i] = a[i];
        x[4 + i] = b[i];
    }
}
template <bool STREAMED> __device__ __forceinline__ void store8(__bf16* p, const bf16x8_t& v) {
    bf16x8_t* to = reinterpret_cast<bf16x8_t*>(p);
    if constexpr (STREAMED) __builtin_nontemporal_store(v, to);
    else *to = v;
}
template <bool STREAMED> __device__ __forceinline__ void store8(float* p, const bf16x8_t& v) {
    f32x4_t* to = reinterpret_cast<f32x4_t*>(p);
    const f32x4_t lo = {(float)v[0], (float)v[1], (float)v[2], (float)v[3]}, hi = {(float)v[4], (float)v[5], (float)v[6], (float)v[7]};
    if constexpr (STREAMED) {
        __builtin_nontemporal_store(lo, to);
        __builtin_nontemporal_store(hi, to + 1);
    } else {
        to[0] = lo;
        to[1] = hi;
    }
}

// Largest of the four lanes of a quad.
__device__ __forceinline__ uint32_t quad_max(uint32_t x) {
    const uint32_t a = (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0xB1, 0xF, 0xF, true);   // lanes 1 0 3 2
    x = a > x ? a : x;
    const uint32_t b = (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x4E, 0xF, 0xF, true);   // lanes 2 3 0 1
    return b > x ? b : x;
}

// Eight channels of a block of 32 whose other ones are in the lanes of the quad: their elements, and the
// block's exponent byte.
__device__ __forceinline__ uint32_t narrow8(const float (&x)[8], uint32_t* byte) {
    uint32_t most = 0;   // by their bits, which also order infinities and NaN above all numbers
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t u = __float_as_uint(x[i]) & 0x7fffffffu;
        most = u > most ? u : most;
    }
    most = quad_max(most);
    const int ex = (int)(most >> 23);
    int e = ex - 2 + ((most & 0x7fffffu) > 0x600000u ? 1 : 0);   // 7 = 1.75 * 2^2
    e = e < (int)kLeastExp ? (int)kLeastExp : (e > (int)kMostExp ? (int)kMostExp : e);
    *byte = ex == 255 ? 255u : (uint32_t)e;
    const float s = block_scale((uint32_t)e);
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[0], x[1], s, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[2], x[3], s, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[4], x[5], s, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[6], x[7], s, 3);
    return ex == 255 ? 0u : c;
}

// The place of packed token i in the cache, in rows of one head's page: false where it has none.  b0 is a
// sequence at or before the token's.  Ends outside the tensor are clamped: 0 <= i < N, so only a first row below 0
// has to be seen to.
__device__ __forceinline__ bool place_of(const CacheArgs& a, int i, int b0, long long* page, int* row, bool* inside) {
    int b = b0;
    long long pos = 0;
    *inside = true;
    if (a.cu) {
        while (b < a.B && a.cu[b + 1] <= i) ++b;
        int first = b < a.B ? a.cu[b] : i + 1;
        if (first < 0) first = 0;
        if (i < first) {
            *inside = false;
            return false;
        }
        pos = i - first;
    } else {
        b = i;
    }
    if (a.start) {
        const int s = a.start[b];
        pos += s > 0 ? s : 0;
    }
    const long long at = pos >> a.page_shift;
    if (at >= a.max_pages) return false;
    const int p = a.pages[(long long)b * a.max_pages + at];
    if (p < 0 || p >= a.n_pages) return false;
    *page = p;
    *row = (int)(pos & (a.page - 1));
    return true;
}

// How many sequences end at or before token i.
__device__ __forceinline__ int ended_before(const CacheArgs& a, int i, int lane) {
    if (!a.cu) return 0;
    int n = 0;
    for (int b = 0; b < a.B; b += 64) {
        const unsigned long long past = __ballot(b + lane < a.B && a.cu[b + lane + 1] <= i);
        n += __builtin_popcountll(past);
        if (past != ~0ull) break;
    }
    return n;
}

}  // namespace

// Writing and reading back, bound by HBM.  A thread owns eight channels of a token's key and value: 16 bytes of
// them in bf16, one dword of elements.  A workgroup takes 16 (d = 128) or 32 tokens of one kv head, whose elements
// lie beside each other in a page; the heads of the same tokens follow on the same XCD, so that whole rows of the packed
// tensors are read or written at about the same time.
//
// STREAMED: rows are read back past the last-level cache, from half its size of them on, where what else is in use passes the
// rest.  8 heads of 128 in bf16, alone and with attention of 16 queries that reads them next: 65536 tokens (256 MiB) 89 and
// 341 us with plain stores, 50 and 349 us streamed; 32768 tokens 28 and 188, 25 and 179 us; 16384 tokens 15 and 92, 12 and
// 104 us.  Write and read of 48000 tokens (187 MiB of results) 105 and 99 us on other data each time, 104 and 57 on the same.
template <int D, typename T, bool WRITE, bool STREAMED>
__global__ __launch_bounds__(256) void kda_cache_rows_kernel(const CacheArgs a) {
    constexpr int LPR = D / 8, TB = 256 / LPR;
    const uint32_t unit = (blockIdx.x & 7) * (uint32_t)a.per_xcd + (blockIdx.x >> 3);
    if (unit >= (uint32_t)a.n_units) return;
    const int lane = threadIdx.x & 63, c = threadIdx.x % LPR, hk = (int)(unit % (uint32_t)a.Hkv);
    const int i0 = (int)(unit / (uint32_t)a.Hkv) * TB, i = i0 + threadIdx.x / LPR;
    const bool there = i < a.N;
    // Rows are requested before their places are looked up, four loads one after the other (write and read of 48000 tokens of 8
    // heads whose rows lie in the last-level cache: 59 -> 56 us; on other data each time 97 to 99 either way; two or four tokens a
    // thread are no faster).
    typedef typename Eight<T>::type eight_t;
    eight_t xs = {}, ys = {};
    if constexpr (WRITE) {
        if (there) {
            xs = *reinterpret_cast<const eight_t*>(reinterpret_cast<const T*>(a.k) + (long long)i * a.k_stride + (long long)hk * D + 8 * c);
            ys = *reinterpret_cast<const eight_t*>(reinterpret_cast<const T*>(a.v) + (long long)i * a.v_stride + (long long)hk * D + 8 * c);
        }
    }
    const int b0 = ended_before(a, i0, lane);
    long long page = 0;
    int row = 0;
    bool inside = false, has = false;
    if (there) has = place_of(a, i, b0, &page, &row, &inside);
    const long long base = (page * a.Hkv + hk) * a.page_bytes;
    const long long at = base + (long long)row * (D / 2) + 4 * c;
    const long long at_e = base + (long long)a.page * (D / 2) + (long long)row * (D / 32) + c / 4;
    if constexpr (WRITE) {
        if (has) {   // (the four lanes of a quad hold one block, and have a place or none together)
            float x[8], y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[j] = (float)xs[j];
                y[j] = (float)ys[j];
            }
            uint32_t ex, ey;
            const uint32_t cx = narrow8(x, &ex), cy = narrow8(y, &ey);
            *reinterpret_cast<uint32_t*>(a.k_cache + at) = cx;
            *reinterpret_cast<uint32_t*>(a.v_cache + at) = cy;
            if (c % 4 == 0) {
                a.k_cache[at_e] = (uint8_t)ex;
                a.v_cache[at_e] = (uint8_t)ey;
            }
        }
    } else {
        if (!inside) return;
        bf16x8_t x = {}, y = {};
        if (has) {
            const uint32_t cx = *reinterpret_cast<const uint32_t*>(a.k_cache + at), ex = a.k_cache[at_e];
            const uint32_t cy = *reinterpret_cast<const uint32_t*>(a.v_cache + at), ey = a.v_cache[at_e];
            widen8(x, cx, block_scale(ex));
            widen8(y, cy, block_scale(ey));
        }
        const long long to = ((long long)i * a.Hkv + hk) * D + 8 * c;
        store8<STREAMED>(reinterpret_cast<T*>(a.k_out) + to, x);
        store8<STREAMED>(reinterpret_cast<T*>(a.v_out) + to, y);
    }
}

namespace {

// Sequences' shares of a call: in tiles of 128 keys, `per` of them a slot, so that the slots of all sequences
// are alike whatever their lengths; each sequence has one slot at least.
constexpr int kSlotKeys = 128;
constexpr float kSumMax = 16384.0f;

__device__ __forceinline__ int seq_len(const AttnStepArgs& a, int b) {
    const int n = a.lens[b];
    const long long most = (long long)a.max_pages << a.page_shift;
    return n < 0 ? 0 : (n > most ? (int)most : n);
}
__device__ __forceinline__ int seq_tiles(const AttnStepArgs& a, int b) {
    return b < a.N ? (int)(((long long)seq_len(a, b) + kSlotKeys - 1) / kSlotKeys) : 0;
}
__device__ __forceinline__ int seq_slots(int tiles, int per) {
    const int n = (int)((uint32_t)(tiles + per - 1) / (uint32_t)per);
    return n > 1 ? n : 1;
}
__device__ __forceinline__ int wave_sum(int x) {
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) x += __shfl_xor(x, s);
    return x;
}
__device__ __forceinline__ int tiles_per_slot(const AttnStepArgs& a, int lane) {
    int all = 0;
    if (a.N == 1) all = seq_tiles(a, 0);
    else
        for (int b = 0; b < a.N; b += 64) all += wave_sum(seq_tiles(a, b + lane));
    const int per = (int)(((long long)all + a.want - 1) / a.want);
    return per > 1 ? per : 1;
}

}  // namespace

// One token, or a few drafted ones, per sequence over the cache, bound by HBM: every visible row is read once, 17
// bits for 32 of bf16's.  A workgroup of four waves runs up to 16 rows (query and head of the group) of one
// (sequence, kv head) over one slot's keys; each wave takes every fourth tile of 32 rows with statistics of its
// own, and the waves (then the slots) are joined at the end.  A lane holds a quarter of a row's channels: those of
// keys are widened straight into the operand (bf16 holds every value), those of values go through a tile of the
// wave's own in LDS to be transposed.  Queries of fp32 are fed as three bf16 parts, probabilities as two, or three
// for fp32 outputs: the products take a fifth of the time that the loads do.  64 sequences of 1000 to 16384 tokens, 56 heads
// on 8 of 128: 87 us and 5 for the join, 4.1 TB/s in all (loads of the same pages alone 88, in order of addresses 69); one
// of 32777 tokens 12.4 and 4.7 us.
template <int D, typename T>
__global__ __launch_bounds__(256, D == 128 && sizeof(T) == 4 ? 3 : 4) void kda_attn_step_kernel(const AttnStepArgs a) {
    constexpr int TK = 32;                        // rows per tile
    constexpr int CH = D / 4, KB = D / 32;        // channels of a lane, dwords of them
    constexpr int OP = D + 4;                     // pitch of the partial outputs
    constexpr int QP = sizeof(T) == 2 ? 1 : 3, PP = sizeof(T) == 2 ? 2 : 3;   // parts of a query, of a probability
    constexpr int REGION = TK * D * 2 > 16 * OP * 4 ? TK * D * 2 : 16 * OP * 4;
    __shared__ __attribute__((aligned(16))) char sV_[4][REGION];
    __shared__ float sm[4][16], sl[4][16];
    typedef __attribute__((ext_vector_type(KB))) uint32_t codes_t;

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    uint32_t unit = blockIdx.x;
    const int hk = (int)(unit % (uint32_t)a.Hkv);
    unit /= (uint32_t)a.Hkv;
    const int R = (int)((uint32_t)a.H / (uint32_t)a.Hkv), rows = a.m * R, RT = (rows + 15) / 16;
    const int rt = (int)(unit % (uint32_t)RT), slot = (int)(unit / (uint32_t)RT);

    // the slot's sequence and its part of it
    const int per = tiles_per_slot(a, lane);
    int b = -1, split = slot, n_split = 0;
    if (a.N == 1) {
        n_split = seq_slots(seq_tiles(a, 0), per);
        if (slot < n_split) b = 0;
    } else for (int b0 = 0; b0 < a.N; b0 += 64) {
        const int mine = b0 + lane < a.N ? seq_slots(seq_tiles(a, b0 + lane), per) : 0;
        int sum = mine;
#pragma unroll
        for (int s = 1; s < 64; s <<= 1) {
            const int y = __shfl_up(sum, s);
            if (lane >= s) sum += y;
        }
        const unsigned long long past = __ballot(sum > split);
        if (past) {
            const int at = __builtin_ctzll(past);
            b = b0 + at;
            n_split = __builtin_amdgcn_readlane(mine, at);
            split -= __builtin_amdgcn_readlane(sum, at) - n_split;
            break;
        }
        split -= __builtin_amdgcn_readlane(sum, 63);
    }
    if (b < 0) return;
    const int len = __builtin_amdgcn_readfirstlane(seq_len(a, b));

    const int g = lane >> 4, r = lane & 15;
    const int row = 16 * rt + r, t = (int)((uint32_t)row / (uint32_t)R), h = hk * R + (row - t * R);
    const int sees = len - a.m + 1 + t;           // keys that this lane's row sees
    const int last = 16 * rt + 15 < rows ? 16 * rt + 15 : rows - 1;
    int total = len - a.m + 1 + (int)((uint32_t)last / (uint32_t)R);
    if (total < 0) total = 0;
    const long long first = (long long)split * per * kSlotKeys, past = first + (long long)per * kSlotKeys;
    const int k0 = first < total ? (int)first : total, k1 = past < total ? (int)past : total;

    KDA_LDS __bf16* sV = (KDA_LDS __bf16*)(KDA_LDS char*)sV_[wave];
    TileCols<__bf16, TK> cv;
    cv.set(sV, lane);
    KDA_LDS __bf16* put[KB];
#pragma unroll
    for (int p = 0; p < KB; ++p) put[p] = lds_pin(sV + tile_at<__bf16, TK>(r, CH / 4 * g + 2 * p));

    Frag<__bf16> fq[QP][KB];
    {
        const T* qp = reinterpret_cast<const T*>(a.q) + ((long long)b * a.m + t) * a.q_stride + (long long)h * D + CH * g;
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            float x[8];
            if (row < rows) {
                load8(x, qp + 8 * kb);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = 0.0f;
            }
            Frag<__bf16> f[QP];
            parts_of<QP>(f, f32x4_t{x[0], x[1], x[2], x[3]}, f32x4_t{x[4], x[5], x[6], x[7]});
#pragma unroll
            for (int i = 0; i < QP; ++i) fq[i][kb] = f[i];
        }
    }
    f32x4_t O[D / 16];
#pragma unroll
    for (int i = 0; i < D / 16; ++i) O[i] = zero4();
    float m = -INFINITY, l = 0.0f;
    bool ready = false;                           // every row has a maximum
    const float sc = a.scale * kLog2e;
    const int all_see = len - a.m + 1 + (int)((uint32_t)(16 * rt) / (uint32_t)R) < k1 ? len - a.m + 1 + (int)((uint32_t)(16 * rt) / (uint32_t)R) : k1;

    const int* table = a.pages + (long long)b * a.max_pages;
    const long long head = (long long)hk * a.page_bytes, pages_step = (long long)a.Hkv * a.page_bytes;
    const int in_page = a.page - 1, exps_at = a.page * (D / 2);

    // Pages of this wave's next 32 tiles, two groups of 16 rows each: lane 2 i + x has group x of tile i.
    int page_of = 0, page_t0 = 0;
    auto request_pages = [&](int t0) {
        page_t0 = t0;
        const long long at = (long long)t0 + (lane >> 1) * (4 * TK) + (lane & 1) * 16;
        page_of = at < k1 ? table[at >> a.page_shift] : -1;
    };
    // A tile's elements and exponents.  Rows without a page, or past the slot's, are read from the pool's start,
    // not seen, and have a finite exponent.
    codes_t ck[2], cw[2];
    uint32_t ek[2], ew[2];
    bool ok[2];
    auto request = [&](int t0) {
        if (t0 - page_t0 >= 32 * 4 * TK) request_pages(t0);
        const int i = (int)((uint32_t)(t0 - page_t0) / (4 * TK));
#pragma unroll
        for (int kt = 0; kt < 2; ++kt) {
            int p = __builtin_amdgcn_readlane(page_of, 2 * i + kt);
            ok[kt] = p >= 0 && p < a.n_pages;
            if (!ok[kt]) p = 0;
            const long long base = p * pages_step + head;
            const int at = ((t0 + 16 * kt) & in_page) + r;
            const uint32_t off = (uint32_t)at * (D / 2) + g * (D / 8), off_e = exps_at + (uint32_t)at * (D / 32) + (uint32_t)(CH * g) / 32;
            ck[kt] = *reinterpret_cast<const codes_t*>(a.k_cache + base + off);
            cw[kt] = *reinterpret_cast<const codes_t*>(a.v_cache + base + off);
            ek[kt] = a.k_cache[base + off_e];
            ew[kt] = a.v_cache[base + off_e];
        }
    };
    const int start = k0 + TK * wave;
    if (start < k1) {
        request_pages(start);
        request(start);
    }
    for (int t0 = start; t0 < k1; t0 += 4 * TK) {
        // values to LDS, then the scores: their codes are in registers for as short as can be
#pragma unroll
        for (int kt = 0; kt < 2; ++kt) {
            const float sv = block_scale(ok[kt] && t0 + 16 * kt + r < k1 ? ew[kt] : kLeastExp);
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                bf16x8_t w;
                widen8(w, cw[kt][kb], sv);
                *reinterpret_cast<KDA_LDS bf16x8_t*>(put[kb] + 16 * 32 * kt) = w;
            }
        }
        f32x4_t sT[2];
        bool live[2];
#pragma unroll
        for (int kt = 0; kt < 2; ++kt) {
            live[kt] = ok[kt];
            const float s = block_scale(ek[kt]);
            sT[kt] = zero4();
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                Frag<__bf16> fk;
                widen8(fk.v, ck[kt][kb], s);
#pragma unroll
                for (int i = QP - 1; i >= 0; --i) sT[kt] = mma(fk, fq[i][kb], sT[kt]);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        if (t0 + 4 * TK < k1) request(t0 + 4 * TK);
        __builtin_amdgcn_sched_barrier(0);

        // The maximum only has to keep exponentials in range.  A tile that every row sees whole is taken with the maximum
        // at hand; where a sum of its exponentials passes kSumMax, and for the others, it is brought up to date.
        const bool whole = t0 + TK <= all_see && live[0] && live[1];
        bool done = false;
        if (whole && ready) {
            f32x4_t p[2];
            float sum = 0.0f;
#pragma unroll
            for (int kt = 0; kt < 2; ++kt)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    p[kt][j] = fast_exp2(fmaf(sT[kt][j], sc, -m));
                    sum += p[kt][j];
                }
            done = !__any(!(sum < kSumMax));
            if (done) {
                l += sum;
                sT[0] = p[0];
                sT[1] = p[1];
            }
        }
        if (!done) {
            const int to = (sees < k1 ? sees : k1) - t0 - 4 * g;
            float mx = -INFINITY;
#pragma unroll
            for (int kt = 0; kt < 2; ++kt)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (!whole) sT[kt][j] = live[kt] && 16 * kt + j < to ? sT[kt][j] : -INFINITY;
                    mx = fmaxf(mx, sT[kt][j]);
                }
            mx = fmaxf(m, max_over_groups<true>(mx) * sc);
            const float base = mx == -INFINITY ? 0.0f : mx;   // nothing seen so far, or scores below fp32's range: no weight
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
            ready = __all(mx != -INFINITY);
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) O[i][j] *= al;
        }
        Frag<__bf16> fp[PP];
        parts_of<PP>(fp, sT[0], sT[1]);
        wave_order();
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            Frag<__bf16> fv;
            cv.frag(fv, 0, i, 0);
#pragma unroll
            for (int x = PP - 1; x >= 0; --x) O[i] = mma(fv, fp[x], O[i]);
        }
        wave_order();
    }
    l = sum_over_groups<true>(l);

    // join the waves: every wave's outputs go to its own region as [row][d]
    KDA_LDS float* sO = (KDA_LDS float*)(KDA_LDS char*)sV_[wave];
#pragma unroll
    for (int i = 0; i < D / 16; ++i) *reinterpret_cast<KDA_LDS f32x4_t*>(sO + r * OP + 16 * i + 4 * g) = O[i];
    if (g == 0) {
        sm[wave][r] = m;
        sl[wave][r] = l;
    }
    __syncthreads();
    const int n_rows = rows - 16 * rt < 16 ? rows - 16 * rt : 16;
    for (int e = tid; e < n_rows * (D / 4); e += 256) {
        const int rr = e / (D / 4), d = (e % (D / 4)) * 4;
        float M = -INFINITY, L = 0.0f;
#pragma unroll
        for (int w = 0; w < 4; ++w) M = fmaxf(M, sm[w][rr]);
        f32x4_t v = zero4();
        const float base = M == -INFINITY ? 0.0f : M;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const float f = fast_exp2(sm[w][rr] - base);
            L = fmaf(f, sl[w][rr], L);
            const f32x4_t x = *reinterpret_cast<const KDA_LDS f32x4_t*>((KDA_LDS float*)(KDA_LDS char*)sV_[w] + rr * OP + d);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = fmaf(f, x[j], v[j]);
        }
        const int rho = 16 * rt + rr, tt = (int)((uint32_t)rho / (uint32_t)R);
        const long long place = (long long)tt * a.H + hk * R + (rho - tt * R);   // among the sequence's m H rows
        if (n_split == 1) {
            const float inv = L == 0.0f ? 0.0f : 1.0f / L;
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] *= inv;
            store4<T>(reinterpret_cast<T*>(a.o) + ((long long)b * a.m * a.H + place) * D + d, v);
        } else {
            const long long part = (long long)slot * a.m * a.H + place;
            *reinterpret_cast<f32x4_t*>(a.ws_o + part * D + d) = v;
            if (d == 0) {
                a.ws_ml[2 * part] = M;
                a.ws_ml[2 * part + 1] = L;
            }
        }
    }
}

// Joins the slots of a sequence that has more than one.  grid: (sequence, query, head) rows.
template <int D, typename T, int THREADS>
__global__ __launch_bounds__(THREADS) void kda_attn_step_join_kernel(const AttnStepArgs a) {
    const int lane = threadIdx.x & 63;
    const uint32_t mh = (uint32_t)a.m * (uint32_t)a.H;
    const int b = (int)(blockIdx.x / mh);
    const uint32_t place = blockIdx.x - (uint32_t)b * mh;
    const int per = tiles_per_slot(a, lane);
    int before = 0, n = 1;
    if (a.N == 1) before = n = seq_slots(seq_tiles(a, 0), per);
    else for (int b0 = 0; b0 <= b; b0 += 64) {
        const int mine = b0 + lane <= b ? seq_slots(seq_tiles(a, b0 + lane), per) : 0;
        before += wave_sum(mine);
        if (b - b0 < 64) n = __builtin_amdgcn_readlane(mine, b - b0);
    }
    before -= n;
    if (n == 1) return;
    const long long first = (long long)before * mh + place;
    join_parts<D, T, THREADS>(a.ws_ml + 2 * first, a.ws_o + first * D, n, mh, reinterpret_cast<T*>(a.o) + (long long)blockIdx.x * D);
}

namespace {

template <int D, typename T> hipError_t cache_rows_t(bool write, CacheArgs a, hipStream_t s) {
    constexpr int TB = 256 / (D / 8);
    a.n_units = ((long long)a.N + TB - 1) / TB * a.Hkv;
    a.per_xcd = (a.n_units + 7) / 8;
    const dim3 grid((unsigned)(8 * a.per_xcd));
    if (write) kda_cache_rows_kernel<D, T, true, false><<<grid, 256, 0, s>>>(a);
    else if (a.streamed) kda_cache_rows_kernel<D, T, false, true><<<grid, 256, 0, s>>>(a);
    else kda_cache_rows_kernel<D, T, false, false><<<grid, 256, 0, s>>>(a);
    return hipGetLastError();
}

template <int D, typename T> hipError_t attn_step_t(const AttnStepArgs& a, hipStream_t s) {
    const int rt = (a.m * (a.H / a.Hkv) + 15) / 16;
    kda_attn_step_kernel<D, T><<<dim3((unsigned)((long long)a.slots * rt * a.Hkv)), 256, 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.slots == a.N) return e;
    // Four waves a row where its sequence can have many slots (one of 128 of them 4.9 us, 8.9 with one wave), one where rows are
    // many and slots few (64 sequences 8.3 us with four, 5.0 with one).
    const dim3 rows((unsigned)((long long)a.N * a.m * a.H));
    if (a.want >= 8LL * a.N) kda_attn_step_join_kernel<D, T, 256><<<rows, 256, 0, s>>>(a);
    else kda_attn_step_join_kernel<D, T, 64><<<rows, 64, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_cache_rows(bool write, int d, bool f32, const CacheArgs& a, hipStream_t s) {
    if (d == 64) return f32 ? cache_rows_t<64, float>(write, a, s) : cache_rows_t<64, __bf16>(write, a, s);
    return f32 ? cache_rows_t<128, float>(write, a, s) : cache_rows_t<128, __bf16>(write, a, s);
}
hipError_t launch_attn_step(int d, bool f32, const AttnStepArgs& a, hipStream_t s) {
    if (d == 64) return f32 ? attn_step_t<64, float>(a, s) : attn_step_t<64, __bf16>(a, s);
    return f32 ? attn_step_t<128, float>(a, s) : attn_step_t<128, __bf16>(a, s);
}

}  // namespace kda
