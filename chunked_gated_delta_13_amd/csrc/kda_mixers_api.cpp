// Host side of the token mixers beside KDA: argument validation, launch plans and launches of the
// short convolution, the state space scan and the window attention.  Nothing here allocates
// memory or synchronises the host with the device.
#include <math.h>
#include <string.h>

#include <atomic>

#include <hip/hip_runtime.h>

#include "../../include/kda.h"
#include "kda_host.h"
#include "kda_mixers.h"

using namespace kda::host;

namespace kda {
namespace host {

// Compute units of the current device (256 where the runtime does not say).
int cu_count() {
    static std::atomic<int> cached[64];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) {
        (void)hipGetLastError();
        return 256;
    }
    int n = cached[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0) {
            (void)hipGetLastError();
            n = 256;
        }
        cached[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

}  // namespace host
}  // namespace kda

namespace {

constexpr size_t kStreamedBytes = (size_t)192 << 20;   // outputs that do not stay in the 256 MB last-level cache

kda_status_t check_conv(const void* x, const void* w, const void* bias, int rows_b, int T, int D, int W,
                        long long x_stride, kda_dtype_t dt) {
    if (rows_b < 0 || T < 0 || D < 0) return KDA_ERR_INVALID_ARGUMENT;
    if (dt != KDA_BF16 && dt != KDA_F32) return KDA_ERR_INVALID_ARGUMENT;
    if (W < 1) return KDA_ERR_INVALID_ARGUMENT;
    if (W < 2 || W > 4) return KDA_ERR_UNSUPPORTED;
    if (!stride_ok((long long)rows_b * T, D, x_stride)) return KDA_ERR_INVALID_ARGUMENT;
    if (D > (1 << 28) || rows_b > kMaxGridYZ) return KDA_ERR_UNSUPPORTED;
    long long n = 0;
    if (!mul_ok((long long)rows_b * (T > W ? T : W), D, &n) || n >= (1LL << 58)) return KDA_ERR_INVALID_ARGUMENT;
    if (rows_b == 0 || D == 0) return KDA_OK;
    const size_t esz = elem_size(dt);
    if (!w || (T > 0 && !x)) return KDA_ERR_INVALID_ARGUMENT;
    if (!aligned(w, esz) || !aligned(x, esz) || !aligned(bias, esz)) return KDA_ERR_INVALID_ARGUMENT;
    return KDA_OK;
}

// Whole 16-byte groups of channels: every row of every tensor starts on a 16-byte boundary.
bool conv_vec(const void* x, const void* bias, const void* s0, const void* s1, const void* y, int D,
              long long x_stride, kda_dtype_t dt) {
    const int v = dt == KDA_BF16 ? 8 : 4;
    return D % v == 0 && x_stride % v == 0 && aligned(x, 16) && aligned(bias, 16) && aligned(s0, 16) &&
           aligned(s1, 16) && aligned(y, 16);
}

constexpr int kSsmChunk = 64;

kda_status_t check_ssm_shape(int rows_b, int T, int H, int G, int n, int p, kda_dtype_t dt) {
    if (rows_b < 0 || T < 0 || H < 0 || G < 0) return KDA_ERR_INVALID_ARGUMENT;
    if (dt != KDA_BF16 && dt != KDA_F32) return KDA_ERR_INVALID_ARGUMENT;
    if (n <= 0 || p <= 0) return KDA_ERR_INVALID_ARGUMENT;
    if ((n != 64 && n != 128) || (p != 64 && p != 128)) return KDA_ERR_UNSUPPORTED;
    if (H > 0 && (G == 0 || H % G != 0)) return KDA_ERR_INVALID_ARGUMENT;
    long long a = 0, b = 0;
    if (!mul_ok((long long)rows_b * T, (long long)H * p, &a) || a >= (1LL << 58)) return KDA_ERR_INVALID_ARGUMENT;
    if (!mul_ok((long long)rows_b * H, (long long)n * p, &b) || b >= (1LL << 58)) return KDA_ERR_INVALID_ARGUMENT;
    if ((long long)rows_b * H > kMaxUnits) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

// Segments of seg_in tokens (whole chunks), or as many as take the least time (seg_in 0).  Where there are
// fewer sequences and heads than workgroups at once (two per compute unit; one where the tiles fill the
// LDS: p = 128, or fp32 with n = 128), a split shortens the chain of chunks.  In microseconds, measured: a chunk of the
// outputs takes 3.3 (n = 128) or 2.5 (n = 64) in bf16 and 6 to 13 in fp32, half as much again beside a
// second workgroup; the states of a chunk 0.4 of that; the two further launches 4; and every segment's
// state is written and read twice, at 6 TB/s together.  8 heads, n = p = 128: 300 tokens 19 us in segments
// of a chunk, 22 in one piece (fp32 31 and 69); 128 heads, 300 tokens: 30 in two, 25 in one.
kda_status_t ssm_plan(int B, int T, int H, int n, int p, kda_dtype_t dt, int seg_in, long long* seg_len, int* n_seg) {
    if (seg_in < 0 || seg_in % kSsmChunk != 0) return KDA_ERR_INVALID_ARGUMENT;
    const long long chunks = ((long long)T + kSsmChunk - 1) / kSsmChunk;
    const long long units = (long long)B * H;
    long long per = seg_in > 0 ? seg_in / kSsmChunk : chunks;
    const bool f32 = dt == KDA_F32;
    const long long cus = seg_in == 0 && units > 0 ? cu_count() : 0, at_once = p == 128 || (f32 && n == 128) ? cus : 2 * cus;
    if (cus > 0 && at_once >= 2 * units) {
        const double chunk = f32 ? 0.05 * n + 0.06 * p - 1.0 : 1.75 + 0.0117 * n;
        const double segment = (double)units * n * p * 16 / 6e6;
        double best = (double)chunks * chunk;
        const long long most = at_once / units < chunks ? at_once / units : chunks;
        for (long long ns = 2; ns <= most; ++ns) {
            const long long c = (chunks + ns - 1) / ns;
            const double us = (double)c * chunk * 1.4 * (units * ns > cus ? 1.45 : 1.0) + (double)ns * segment + 4.0;
            if (us < best) {
                best = us;
                per = c;
            }
        }
    }
    if (per < 1) per = 1;
    const long long ns = chunks > 0 ? (chunks + per - 1) / per : 1;
    // a split's join runs n p / 512 (at most 32) workgroups of 256 threads per sequence and head
    if (units * ns > (ns > 1 ? kMaxUnits / 4 : kMaxUnits)) return KDA_ERR_UNSUPPORTED;
    *seg_len = per * kSsmChunk;
    *n_seg = (int)ns;
    return KDA_OK;
}

// Workspace of a split: the segments' entry states [B * H, n_seg, n, p], then decays [B * H, n_seg],
// fp32, padded to 16 bytes.
size_t ssm_workspace(int B, int H, int n, int p, int n_seg) {
    if (n_seg <= 1) return 0;
    const size_t slots = (size_t)B * H * (size_t)n_seg;
    return slots * (size_t)n * p * sizeof(float) + (slots * sizeof(float) + 15) / 16 * 16;
}

struct SsmPtrs {
    const void *x, *dt;
    const float* A;
    const void *Bm, *Cm;
    const float* D;
    const void* z;
    const float* dt_bias;
    const int* lens;
    long long x_stride, dt_stride, b_stride, c_stride, z_stride;
};

// Pointer, stride and overlap checks shared by the prompt and the token form.  S_in is NULL where the
// state is updated in place.
kda_status_t check_ssm_ptrs(const SsmPtrs& q, const float* S_in, const void* y, const float* S_out, int rows_b, int T, int H,
                            int G, int n, int p, kda_dtype_t dt) {
    const size_t esz = elem_size(dt);
    const long long rows = (long long)rows_b * T;
    if (!q.A || (rows > 0 && (!q.x || !q.dt || !q.Bm || !q.Cm || !y))) return KDA_ERR_INVALID_ARGUMENT;
    if (!wide_rows_ok(q.x, rows, (long long)H * p, q.x_stride, esz) ||
        !wide_rows_ok(q.Bm, rows, (long long)G * n, q.b_stride, esz) ||
        !wide_rows_ok(q.Cm, rows, (long long)G * n, q.c_stride, esz) ||
        (q.z && !wide_rows_ok(q.z, rows, (long long)H * p, q.z_stride, esz)) || !stride_ok(rows, H, q.dt_stride))
        return KDA_ERR_INVALID_ARGUMENT;
    // offsets inside a chunk are 32-bit: 64 rows of at most 2^22 elements
    const long long widest = 1LL << 22;
    if ((long long)H * p > widest || (rows > 1 && (q.x_stride > widest || q.b_stride > widest || q.c_stride > widest ||
                                                   q.dt_stride > widest || (q.z && q.z_stride > widest))))
        return KDA_ERR_UNSUPPORTED;
    if (!aligned(q.dt, esz) || !aligned(q.A, 4) || !aligned(q.D, 4) || !aligned(q.dt_bias, 4) || !aligned(q.lens, 4) ||
        !aligned(y, 16) || !aligned(S_in, 16) || !aligned(S_out, 16))
        return KDA_ERR_INVALID_ARGUMENT;
    const size_t state = (size_t)rows_b * H * n * p * sizeof(float);
    const Range ry = range_of(y, (size_t)rows * H * p * esz), rs = range_of(S_out, S_out ? state : 0);
    const Range ri = range_of(S_in, S_in ? state : 0);
    const Range ins[] = {rows_range(q.x, rows, (long long)H * p, q.x_stride, esz),
                         rows_range(q.dt, rows, H, q.dt_stride, esz),
                         rows_range(q.Bm, rows, (long long)G * n, q.b_stride, esz),
                         rows_range(q.Cm, rows, (long long)G * n, q.c_stride, esz),
                         rows_range(q.z, rows, (long long)H * p, q.z_stride, esz),
                         range_of(q.A, (size_t)H * 4), range_of(q.D, q.D ? (size_t)H * 4 : 0),
                         range_of(q.dt_bias, q.dt_bias ? (size_t)H * 4 : 0),
                         range_of(q.lens, q.lens ? (size_t)rows_b * 4 : 0)};
    for (const Range& r : ins)
        if (overlap(ry, r) || overlap(rs, r)) return KDA_ERR_INVALID_ARGUMENT;
    if (overlap(ry, ri) || overlap(ry, rs)) return KDA_ERR_INVALID_ARGUMENT;
    if (S_in != S_out && overlap(rs, ri)) return KDA_ERR_INVALID_ARGUMENT;
    return KDA_OK;
}

kda::SsmArgs ssm_args(const SsmPtrs& q) {
    kda::SsmArgs a;
    memset(&a, 0, sizeof(a));
    a.x = q.x;
    a.dt = q.dt;
    a.A = q.A;
    a.Bm = q.Bm;
    a.Cm = q.Cm;
    a.D = q.D;
    a.z = q.z;
    a.dt_bias = q.dt_bias;
    a.lens = q.lens;
    a.x_stride = q.x_stride;
    a.dt_stride = q.dt_stride;
    a.b_stride = q.b_stride;
    a.c_stride = q.c_stride;
    a.z_stride = q.z_stride;
    return a;
}

kda_status_t check_window_shape(int rows_b, int T, int H, int Hkv, int d, int window, int sinks, kda_dtype_t dt) {
    if (rows_b < 0 || T < 0 || H < 0 || Hkv < 0 || d <= 0) return KDA_ERR_INVALID_ARGUMENT;
    if (dt != KDA_BF16 && dt != KDA_F32) return KDA_ERR_INVALID_ARGUMENT;
    if (window < 1 || sinks < 0) return KDA_ERR_INVALID_ARGUMENT;
    if (d != 64 && d != 128) return KDA_ERR_UNSUPPORTED;
    if (H > 0 && (Hkv == 0 || H % Hkv != 0)) return KDA_ERR_INVALID_ARGUMENT;
    if ((long long)window + sinks > (1 << 29) || T > (1 << 29)) return KDA_ERR_UNSUPPORTED;   // 32-bit relative positions
    if (rows_b > kMaxGridYZ || H > (1 << 16)) return KDA_ERR_UNSUPPORTED;
    long long a = 0, b = 0;
    if (!mul_ok((long long)rows_b * T, (long long)H * d, &a) || a >= (1LL << 58)) return KDA_ERR_INVALID_ARGUMENT;
    if (!mul_ok((long long)rows_b * (window + sinks), (long long)Hkv * d, &b) || b >= (1LL << 58)) return KDA_ERR_INVALID_ARGUMENT;
    if ((long long)rows_b * H * (T / 64 + 1) > 2 * kMaxUnits) return KDA_ERR_UNSUPPORTED;   // workgroups of 256 threads
    return KDA_OK;
}

// Pointer, stride and overlap checks shared by the prompt and the token form.
kda_status_t check_window_ptrs(const void* q, const void* k, const void* v, const void* kc, const void* vc, const int* start,
                               const int* lens, const void* o, const void* ws, size_t ws_bytes, int rows_b, int T, int H,
                               int Hkv, int d, int window, int sinks, long long q_stride, long long k_stride,
                               long long v_stride, kda_dtype_t dt) {
    const size_t esz = elem_size(dt);
    const long long rows = (long long)rows_b * T;
    if (rows > 0 && (!q || !k || !v || !o)) return KDA_ERR_INVALID_ARGUMENT;
    if ((kc == nullptr) != (vc == nullptr)) return KDA_ERR_INVALID_ARGUMENT;
    if (start && !kc) return KDA_ERR_INVALID_ARGUMENT;   // earlier tokens live in the cache only
    if (!wide_rows_ok(q, rows, (long long)H * d, q_stride, esz) || !wide_rows_ok(k, rows, (long long)Hkv * d, k_stride, esz) ||
        !wide_rows_ok(v, rows, (long long)Hkv * d, v_stride, esz))
        return KDA_ERR_INVALID_ARGUMENT;
    if (!aligned(kc, 16) || !aligned(vc, 16) || !aligned(o, 16) || !aligned(start, 4) || !aligned(lens, 4) || !aligned(ws, 16))
        return KDA_ERR_INVALID_ARGUMENT;
    const size_t cache = kc ? (size_t)rows_b * (window + sinks) * Hkv * d * esz : 0;
    const Range outs[] = {range_of(o, (size_t)rows * H * d * esz), range_of(kc, cache), range_of(vc, cache),
                          range_of(ws, ws ? ws_bytes : 0)};
    const Range ins[] = {rows_range(q, rows, (long long)H * d, q_stride, esz),
                         rows_range(k, rows, (long long)Hkv * d, k_stride, esz),
                         rows_range(v, rows, (long long)Hkv * d, v_stride, esz),
                         range_of(start, start ? (size_t)rows_b * 4 : 0), range_of(lens, lens ? (size_t)rows_b * 4 : 0)};
    for (int i = 0; i < 4; ++i) {
        for (const Range& r : ins)
            if (overlap(outs[i], r)) return KDA_ERR_INVALID_ARGUMENT;
        for (int j = i + 1; j < 4; ++j)
            if (overlap(outs[i], outs[j])) return KDA_ERR_INVALID_ARGUMENT;
    }
    return KDA_OK;
}

// Ranges of cache rows of a step: enough workgroups for two per compute unit, each at least one tile for
// every wave (one sequence of 8 kv heads over 4100 rows: 10.3 us with ranges of 128 rows, 11.3 with 256).
void window_step_plan(int N, int H, int Hkv, int window, int sinks, int* n_split, int* split_len) {
    const long long slots = (long long)window + sinks;
    const long long units = (long long)N * Hkv * ((H / Hkv + 15) / 16);
    long long want = units > 0 ? 2LL * cu_count() / units : 1;
    if (want > slots / 128) want = slots / 128;
    if (want < 1) want = 1;
    const long long len = ((slots + want - 1) / want + 127) / 128 * 128;   // whole tiles of the four waves
    *n_split = (int)((slots + len - 1) / len);
    *split_len = (int)len;
}

// Partial outputs of `rows` queries' H heads, their maxima and sums, padded to 16 bytes.
size_t window_workspace(long long rows, int H, int d, int n_split) {
    return n_split <= 1 ? 0 : (size_t)rows * H * n_split * ((size_t)d + 4) * sizeof(float);
}

// A prompt's workgroups take 128 queries each where that gives every compute unit one, else 64.  Where these
// are few too, the keys of a workgroup (at most its window, its queries and the first tokens; without
// earlier tokens no more than T) are split into ranges of at least two tiles (one in fp32), for at most
// two workgroups per compute unit (one in fp32), if that shortens the chain: in microseconds, a tile
// takes 0.65 (d = 64) or 0.9 (d = 128) in bf16 and 2.6 or 4.8 in fp32, the join 3, and a range's outputs
// are written and read at 3.7 TB/s, so that the best count is the root of tiles / outputs.  Measured with
// 8 heads on 2, d = 128, bf16: 64 tokens over a window of 4000 65 us in one range, 16 in the 20 taken; 1024 tokens
// over 1000 26 us in one, 27 in four (stays one); 64 tokens over 200 13.4 us either way.
void window_prefill_plan(int B, int T, int H, int d, int window, int sinks, kda_dtype_t dt, bool continued, int* few,
                         int* n_split) {
    const int cus = cu_count();
    const bool f32 = dt == KDA_F32;
    const long long heads = (long long)B * H;
    *few = heads * ((T + 127LL) / 128) < cus ? 1 : 0;
    *n_split = 1;
    const long long units = heads * ((T + 63LL) / 64);
    if (!*few || units == 0) return;
    long long keys = (long long)window + sinks + 64;
    if (!continued && keys > T) keys = T;
    const long long tiles = (keys + 63) / 64;
    const double tile_us = f32 ? 0.4 + 0.034 * d : 0.42 + 0.0036 * d, part_us = (double)heads * T * d * 8 / 3.7e6;
    long long n = (f32 ? 1LL : 2LL) * cus / units;
    if (n > tiles / (f32 ? 1 : 2)) n = tiles / (f32 ? 1 : 2);
    const double best = sqrt((double)tiles * tile_us / part_us);
    if (best < (double)n) n = (long long)best;
    if (n < 2) return;
    const double whole = (double)tiles * tile_us, split = (double)((tiles + n - 1) / n) * tile_us + (double)n * part_us + 3.0;
    if (split < whole) *n_split = (int)n;
}

}  // namespace

extern "C" {

kda_status_t kda_conv_prefill(const void* x, const void* w, const void* bias, const void* state_in, const int* lens,
                              void* y, void* state_out, int B, int T, int D, int W, long long x_stride, int silu,
                              kda_dtype_t dt, void* stream) {
    const kda_status_t st = check_conv(x, w, bias, B, T, D, W, x_stride, dt);
    if (st != KDA_OK || B == 0 || D == 0) return st;
    const size_t esz = elem_size(dt);
    if ((T > 0 && !y) || !aligned(y, esz) || !aligned(state_in, esz) || !aligned(state_out, esz) || !aligned(lens, 4))
        return KDA_ERR_INVALID_ARGUMENT;
    const size_t keep = (size_t)B * (W - 1) * D * esz;
    const Range ry = range_of(y, (size_t)B * T * D * esz), rso = range_of(state_out, state_out ? keep : 0);
    const Range rsi = range_of(state_in, state_in ? keep : 0);
    const Range ins[] = {rows_range(x, (long long)B * T, D, x_stride, esz), range_of(w, (size_t)D * W * esz),
                         range_of(bias, bias ? (size_t)D * esz : 0), range_of(lens, lens ? (size_t)B * 4 : 0)};
    for (const Range& r : ins)
        if (overlap(ry, r) || overlap(rso, r)) return KDA_ERR_INVALID_ARGUMENT;
    if (overlap(ry, rsi) || overlap(ry, rso)) return KDA_ERR_INVALID_ARGUMENT;
    if (state_out != state_in && overlap(rso, rsi)) return KDA_ERR_INVALID_ARGUMENT;
    if (T == 0 && !state_out) return KDA_OK;

    kda::ConvArgs a;
    memset(&a, 0, sizeof(a));
    a.x = x;
    a.w = w;
    a.bias = bias;
    a.state_in = state_in;
    a.state_out = state_out;
    a.y = y;
    a.lens = lens;
    a.x_stride = x_stride;
    a.B = B;
    a.T = T;
    a.D = D;
    a.silu = silu ? 1 : 0;
    const bool vec = conv_vec(x, bias, state_in, state_out, y, D, x_stride, dt);
    // Tokens per thread.  Every tile re-reads W - 1 rows, from cache: 8 or 16 tokens and streamed stores take
    // 32768 rows of 7424 channels in bf16 in 174 us, 32 tokens 184, 64 tokens 204; with plain stores 16 take
    // 185.  Short inputs halve the tile until there are about 16 waves per compute unit of 256.
    const long long groups = (D + (vec ? (dt == KDA_BF16 ? 8 : 4) : 1) - 1) / (vec ? (dt == KDA_BF16 ? 8 : 4) : 1);
    int tile = 16;
    while (tile > 4 && groups * B * (((long long)T + tile - 1) / tile) < 64LL * 4096) tile >>= 1;
    a.streamed = (size_t)B * T * D * esz > kStreamedBytes ? 1 : 0;
    while (groups * (((long long)T + tile - 1) / tile) > (1LL << 31)) tile <<= 1;   // threads of a launch
    a.tile = tile;
    (void)hipGetLastError();
    if (kda::launch_conv_prefill(W, dt == KDA_F32, vec, a, reinterpret_cast<hipStream_t>(stream)) != hipSuccess)
        return KDA_ERR_DEVICE;
    return KDA_OK;
}

kda_status_t kda_conv_step(const void* x, const void* w, const void* bias, void* state, void* y, int N, int D, int W,
                           long long x_stride, int silu, kda_dtype_t dt, void* stream) {
    const kda_status_t st = check_conv(x, w, bias, N, 1, D, W, x_stride, dt);
    if (st != KDA_OK || N == 0 || D == 0) return st;
    const size_t esz = elem_size(dt);
    if (!state || !y || !aligned(state, esz) || !aligned(y, esz)) return KDA_ERR_INVALID_ARGUMENT;
    const Range ry = range_of(y, (size_t)N * D * esz), rs = range_of(state, (size_t)N * (W - 1) * D * esz);
    const Range ins[] = {rows_range(x, N, D, x_stride, esz), range_of(w, (size_t)D * W * esz),
                         range_of(bias, bias ? (size_t)D * esz : 0)};
    for (const Range& r : ins)
        if (overlap(ry, r) || overlap(rs, r)) return KDA_ERR_INVALID_ARGUMENT;
    if (overlap(ry, rs)) return KDA_ERR_INVALID_ARGUMENT;
    kda::ConvArgs a;
    memset(&a, 0, sizeof(a));
    a.x = x;
    a.w = w;
    a.bias = bias;
    a.state_in = state;
    a.state_out = state;
    a.y = y;
    a.x_stride = x_stride;
    a.B = N;
    a.T = 1;
    a.D = D;
    a.silu = silu ? 1 : 0;
    (void)hipGetLastError();
    if (kda::launch_conv_step(W, dt == KDA_F32, conv_vec(x, bias, state, state, y, D, x_stride, dt), a,
                              reinterpret_cast<hipStream_t>(stream)) != hipSuccess)
        return KDA_ERR_DEVICE;
    return KDA_OK;
}

size_t kda_ssm_prefill_workspace_bytes(int B, int T, int H, int G, int n, int p, kda_dtype_t dt, int seg_len) {
    long long sl = 0;
    int ns = 1;
    if (check_ssm_shape(B, T, H, G, n, p, dt) != KDA_OK || ssm_plan(B, T, H, n, p, dt, seg_len, &sl, &ns) != KDA_OK) return 0;
    return ssm_workspace(B, H, n, p, ns);
}

kda_status_t kda_ssm_prefill(const void* x, const void* dt, const float* A, const void* Bm, const void* Cm, const float* D,
                             const void* z, const float* dt_bias, const float* S0, const int* lens, void* y, float* S_T,
                             int B, int T, int H, int G, int n, int p, long long x_stride, long long dt_stride,
                             long long b_stride, long long c_stride, long long z_stride, kda_dtype_t dtype, int seg_len,
                             void* workspace, size_t workspace_bytes, void* stream) {
    kda_status_t st = check_ssm_shape(B, T, H, G, n, p, dtype);
    if (st != KDA_OK) return st;
    long long sl = 0;
    int ns = 1;
    st = ssm_plan(B, T, H, n, p, dtype, seg_len, &sl, &ns);
    if (st != KDA_OK || B == 0 || H == 0) return st;
    const SsmPtrs q = {x, dt, A, Bm, Cm, D, z, dt_bias, lens, x_stride, dt_stride, b_stride, c_stride, z_stride};
    st = check_ssm_ptrs(q, S0, y, S_T, B, T, H, G, n, p, dtype);
    if (st != KDA_OK) return st;
    const size_t need = ssm_workspace(B, H, n, p, ns);
    if (need > 0) {
        if (!workspace || workspace_bytes < need) return KDA_ERR_WORKSPACE;
        if (!aligned(workspace, 16)) return KDA_ERR_INVALID_ARGUMENT;
        const size_t esz = elem_size(dtype);
        const long long rows = (long long)B * T;
        const size_t state = (size_t)B * H * n * p * sizeof(float);
        const Range rw = range_of(workspace, need);
        const Range others[] = {rows_range(x, rows, (long long)H * p, x_stride, esz), rows_range(dt, rows, H, dt_stride, esz),
                                rows_range(Bm, rows, (long long)G * n, b_stride, esz),
                                rows_range(Cm, rows, (long long)G * n, c_stride, esz),
                                rows_range(z, rows, (long long)H * p, z_stride, esz), range_of(A, (size_t)H * 4),
                                range_of(D, D ? (size_t)H * 4 : 0), range_of(dt_bias, dt_bias ? (size_t)H * 4 : 0),
                                range_of(lens, lens ? (size_t)B * 4 : 0), range_of(y, (size_t)rows * H * p * esz),
                                range_of(S0, S0 ? state : 0), range_of(S_T, S_T ? state : 0)};
        for (const Range& r : others)
            if (overlap(rw, r)) return KDA_ERR_INVALID_ARGUMENT;
    }
    if (T == 0 && !S_T) return KDA_OK;
    const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const bool f32 = dtype == KDA_F32;
    kda::SsmArgs a = ssm_args(q);
    a.S0 = S0;
    a.y = y;
    a.S_T = S_T;
    a.T = T;
    a.H = H;
    a.G = G;
    a.seg_len = sl;
    a.n_seg = ns;
    (void)hipGetLastError();
    if (ns > 1) {
        a.ws_state = reinterpret_cast<float*>(workspace);
        a.ws_decay = a.ws_state + (size_t)B * H * (size_t)ns * n * p;
        a.keep_S0 = S_T && S_T == S0 ? 1 : 0;
        a.n_seg_launch = ns - 1;
        a.n_units = (long long)B * H * (ns - 1);
        if (kda::launch_ssm(kda::SsmPass::kStates, n, p, f32, a, s) != hipSuccess) return KDA_ERR_DEVICE;
        if (ns > 2 && kda::launch_ssm_join(n, p, B * H, ns, a.ws_state, a.ws_decay, s) != hipSuccess) return KDA_ERR_DEVICE;
    }
    a.n_seg_launch = ns;
    a.n_units = (long long)B * H * ns;
    if (kda::launch_ssm(kda::SsmPass::kOutputs, n, p, f32, a, s) != hipSuccess) return KDA_ERR_DEVICE;
    return KDA_OK;
}

kda_status_t kda_ssm_step(const void* x, const void* dt, const float* A, const void* Bm, const void* Cm, const float* D,
                          const void* z, const float* dt_bias, float* S, void* y, int N, int H, int G, int n, int p,
                          long long x_stride, long long dt_stride, long long b_stride, long long c_stride,
                          long long z_stride, kda_dtype_t dtype, void* stream) {
    kda_status_t st = check_ssm_shape(N, 1, H, G, n, p, dtype);
    if (st != KDA_OK || N == 0 || H == 0) return st;
    if (!S) return KDA_ERR_INVALID_ARGUMENT;
    const SsmPtrs q = {x, dt, A, Bm, Cm, D, z, dt_bias, nullptr, x_stride, dt_stride, b_stride, c_stride, z_stride};
    st = check_ssm_ptrs(q, nullptr, y, S, N, 1, H, G, n, p, dtype);
    if (st != KDA_OK) return st;
    kda::SsmArgs a = ssm_args(q);
    a.y = y;
    a.S_T = S;
    a.T = 1;
    a.H = H;
    a.G = G;
    a.n_units = (long long)N * H;
    (void)hipGetLastError();
    if (kda::launch_ssm(kda::SsmPass::kToken, n, p, dtype == KDA_F32, a, reinterpret_cast<hipStream_t>(stream)) != hipSuccess)
        return KDA_ERR_DEVICE;
    return KDA_OK;
}

size_t kda_window_prefill_workspace_bytes(int B, int T, int H, int Hkv, int d, int window, int sinks, kda_dtype_t dt,
                                          int continued) {
    if (check_window_shape(B, T, H, Hkv, d, window, sinks, dt) != KDA_OK) return 0;
    int few = 0, ns = 1;
    window_prefill_plan(B, T, H, d, window, sinks, dt, continued != 0, &few, &ns);
    return window_workspace((long long)B * T, H, d, ns);
}

kda_status_t kda_window_prefill(const void* q, const void* k, const void* v, void* k_cache, void* v_cache, const int* start,
                                const int* lens, void* o, int B, int T, int H, int Hkv, int d, int window, int sinks,
                                float scale, long long q_stride, long long k_stride, long long v_stride, kda_dtype_t dt,
                                void* workspace, size_t workspace_bytes, void* stream) {
    kda_status_t st = check_window_shape(B, T, H, Hkv, d, window, sinks, dt);
    if (st == KDA_OK && !scale_ok(scale)) st = KDA_ERR_INVALID_ARGUMENT;
    if (st != KDA_OK || B == 0 || H == 0) return st;
    int few = 0, n_split = 1;
    window_prefill_plan(B, T, H, d, window, sinks, dt, start != nullptr, &few, &n_split);
    if (!workspace) n_split = 1;
    const size_t need = window_workspace((long long)B * T, H, d, n_split);
    st = check_window_ptrs(q, k, v, k_cache, v_cache, start, lens, o, need ? workspace : nullptr, need, B, T, H, Hkv, d,
                           window, sinks, q_stride, k_stride, v_stride, dt);
    if (st != KDA_OK || T == 0) return st;
    if (workspace_bytes < need) return KDA_ERR_WORKSPACE;
    // the launch that keeps a sequence's rows has a thread for 16 bytes of each, fewer than 2^32 after rounding up
    const long long kept = (long long)sinks + (window < T ? window : T);
    if (k_cache && kept * ((long long)Hkv * d * (long long)elem_size(dt) / 16) > (1LL << 31)) return KDA_ERR_UNSUPPORTED;
    kda::WindowArgs a;
    memset(&a, 0, sizeof(a));
    a.q = q;
    a.k = k;
    a.v = v;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.start = start;
    a.lens = lens;
    a.o = o;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.B = B;
    a.T = T;
    a.H = H;
    a.Hkv = Hkv;
    a.window = window;
    a.sinks = sinks;
    a.scale = scale;
    a.few = few;
    a.n_split = n_split;
    if (need > 0) {
        a.ws_o = reinterpret_cast<float*>(workspace);
        a.ws_ml = a.ws_o + (size_t)B * T * H * n_split * d;
    }
    (void)hipGetLastError();
    if (kda::launch_window_prefill(d, dt == KDA_F32, a, reinterpret_cast<hipStream_t>(stream)) != hipSuccess)
        return KDA_ERR_DEVICE;
    return KDA_OK;
}

size_t kda_window_step_workspace_bytes(int N, int H, int Hkv, int d, int window, int sinks, kda_dtype_t dt) {
    if (check_window_shape(N, 1, H, Hkv, d, window, sinks, dt) != KDA_OK || N == 0 || H == 0) return 0;
    int ns = 1, len = 0;
    window_step_plan(N, H, Hkv, window, sinks, &ns, &len);
    return window_workspace(N, H, d, ns);
}

kda_status_t kda_window_step(const void* q, const void* k, const void* v, void* k_cache, void* v_cache, const int* pos,
                             void* o, int N, int H, int Hkv, int d, int window, int sinks, float scale,
                             long long q_stride, long long k_stride, long long v_stride, kda_dtype_t dt, void* workspace,
                             size_t workspace_bytes, void* stream) {
    kda_status_t st = check_window_shape(N, 1, H, Hkv, d, window, sinks, dt);
    if (st == KDA_OK && !scale_ok(scale)) st = KDA_ERR_INVALID_ARGUMENT;
    if (st != KDA_OK || N == 0 || H == 0) return st;
    if (!k_cache || !v_cache || !pos) return KDA_ERR_INVALID_ARGUMENT;
    kda::WindowArgs a;
    memset(&a, 0, sizeof(a));
    window_step_plan(N, H, Hkv, window, sinks, &a.n_split, &a.split_len);
    const size_t need = window_workspace(N, H, d, a.n_split);
    st = check_window_ptrs(q, k, v, k_cache, v_cache, pos, nullptr, o, need ? workspace : nullptr, need, N, 1, H, Hkv, d,
                           window, sinks, q_stride, k_stride, v_stride, dt);
    if (st != KDA_OK) return st;
    if (need > 0) {
        if (!workspace || workspace_bytes < need) return KDA_ERR_WORKSPACE;
        a.ws_o = reinterpret_cast<float*>(workspace);
        a.ws_ml = a.ws_o + (size_t)N * H * a.n_split * d;
    }
    a.q = q;
    a.k = k;
    a.v = v;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.start = pos;
    a.o = o;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.B = N;
    a.T = 1;
    a.H = H;
    a.Hkv = Hkv;
    a.window = window;
    a.sinks = sinks;
    a.scale = scale;
    (void)hipGetLastError();
    if (kda::launch_window_step(d, dt == KDA_F32, a, reinterpret_cast<hipStream_t>(stream)) != hipSuccess)
        return KDA_ERR_DEVICE;
    return KDA_OK;
}

}  // extern "C"
