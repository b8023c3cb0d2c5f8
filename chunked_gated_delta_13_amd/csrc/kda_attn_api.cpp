// Host side of the packed causal attention and of the 4-bit paged cache: argument validation, launch plans and
// launches.  Nothing here allocates memory or synchronises the host with the device.
#include <math.h>
#include <string.h>

#include <hip/hip_runtime.h>

#include "../../include/kda.h"
#include "kda_host.h"
#include "kda_mixers.h"

using namespace kda::host;

namespace {

constexpr size_t kStreamedBytes = (size_t)128 << 20;   // half of the last-level cache: what else is in use passes the rest
constexpr long long kMaxRows = 1LL << 30;   // rows and keys that 32 bits count, with room for a tile more

kda_status_t check_heads(int H, int Hkv, int d, kda_dtype_t dt) {
    if (H < 0 || Hkv < 0 || d <= 0) return KDA_ERR_INVALID_ARGUMENT;
    if (dt != KDA_BF16 && dt != KDA_F32) return KDA_ERR_INVALID_ARGUMENT;
    if (d != 64 && d != 128) return KDA_ERR_UNSUPPORTED;
    if (H > 0 && (Hkv == 0 || H % Hkv != 0)) return KDA_ERR_INVALID_ARGUMENT;
    if (H > (1 << 16) || Hkv > (1 << 16)) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

kda_status_t check_attn_shape(int B, int Nq, int Nk, int H, int Hkv, int d, kda_dtype_t dt) {
    if (B < 0 || Nq < 0 || Nk < 0) return KDA_ERR_INVALID_ARGUMENT;
    const kda_status_t st = check_heads(H, Hkv, d, dt);
    if (st != KDA_OK) return st;
    if (H == 0) return KDA_OK;
    const long long rows = (long long)Nq * (H / Hkv);
    if (rows > kMaxRows || Nk > kMaxRows) return KDA_ERR_UNSUPPORTED;
    if ((rows / 64 + B + 8) * Hkv > 2 * kMaxUnits) return KDA_ERR_UNSUPPORTED;   // workgroups of 256 threads
    return KDA_OK;
}

// A prompt's workgroups take 128 rows (query and head of a group) each where that gives every compute unit one, else 64.
// Where 64 rows do not give every compute unit one either, groups of waves share the rows' keys (bf16), and the keys are
// split into ranges, with at most one workgroup per compute unit, if that shortens the chain: in microseconds, a step of
// the groups takes 1.3 in bf16, and 1.5 (d = 64) or 2.75 (d = 128) in fp32, the join 3, and a range's outputs are written
// and read at 3.7 TB/s, so that the best count is the root of steps / outputs.  Lengths are on the device: the
// sequences are taken to be alike.
void attn_plan(int B, int Nq, int Nk, int H, int Hkv, int d, kda_dtype_t dt, int* few, int* n_split) {
    const int cus = cu_count();
    const bool f32 = dt == KDA_F32;
    const long long rows = (long long)Nq * (H / Hkv);
    *few = Hkv * (rows / 128 + (B + 1) / 2) < cus ? 1 : 0;
    *n_split = 1;
    const long long units = Hkv * (rows / 64 + (B + 1) / 2);
    if (units > cus || Nq == 0 || B == 0) return;
    *few = 2;
    const int kg = f32 ? 1 : kda::attn_groups(d);
    const long long tiles = ((long long)Nk / B + 63) / 64, steps = (tiles + kg - 1) / kg;
    const double step_us = f32 ? 0.25 + 0.0195 * d : 1.3, part_us = (double)Nq * H * d * 8 / 3.7e6;
    long long n = cus / units;
    if (n > steps) n = steps;
    const double best = sqrt((double)steps * step_us / part_us);
    if (best < (double)n) n = (long long)best;
    if (n < 2) return;
    const double whole = (double)steps * step_us, split = (double)((steps + n - 1) / n) * step_us + (double)n * part_us + 3.0;
    if (split < whole) *n_split = (int)n;
}

// Partial outputs, their maxima and sums, padded to 16 bytes.
size_t parts_bytes(long long parts, int d) { return (size_t)parts * ((size_t)d + 4) * sizeof(float); }

kda_status_t check_cache(int B, int Hkv, int d, int n_pages, int max_pages, int page, kda_dtype_t dt) {
    if (B < 0 || n_pages < 0 || max_pages < 0 || page <= 0) return KDA_ERR_INVALID_ARGUMENT;
    const kda_status_t st = check_heads(Hkv, Hkv, d, dt);
    if (st != KDA_OK) return st;
    if (page & (page - 1)) return KDA_ERR_INVALID_ARGUMENT;
    if (page < 16 || page > (1 << 16)) return KDA_ERR_UNSUPPORTED;
    if ((long long)max_pages * page > kMaxRows || Hkv > kMaxGridYZ) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}
long long page_bytes(int d, int page) { return (long long)page * (d / 2 + d / 32); }
int shift_of(int page) {
    int s = 4;
    while ((1 << s) < page) ++s;
    return s;
}

kda::CacheArgs cache_args(const int* pages, const int* cu, const int* start, int B, int N, int Hkv, int d, int n_pages,
                          int max_pages, int page) {
    kda::CacheArgs a;
    memset(&a, 0, sizeof(a));
    a.pages = pages;
    a.cu = cu;
    a.start = start;
    a.B = B;
    a.N = N;
    a.Hkv = Hkv;
    a.n_pages = n_pages;
    a.max_pages = max_pages;
    a.page = page;
    a.page_shift = shift_of(page);
    a.page_bytes = page_bytes(d, page);
    return a;
}

// The shape checks shared by writing and reading, and the pointers that both have.
kda_status_t check_cache_rows(const void* k_cache, const void* v_cache, const int* pages, const int* cu, const int* start, int B,
                              int N, int Hkv, int d, int n_pages, int max_pages, int page, kda_dtype_t dt) {
    if (N < 0) return KDA_ERR_INVALID_ARGUMENT;
    const kda_status_t st = check_cache(B, Hkv, d, n_pages, max_pages, page, dt);
    if (st != KDA_OK) return st;
    if (!cu && N != B) return KDA_ERR_INVALID_ARGUMENT;
    if ((long long)N * Hkv > kMaxRows / 8) return KDA_ERR_UNSUPPORTED;   // at most 16 threads each, and a workgroup more a head
    if (N == 0 || Hkv == 0) return KDA_OK;
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(pages, 4) || !aligned(cu, 4) || !aligned(start, 4))
        return KDA_ERR_INVALID_ARGUMENT;
    if ((n_pages > 0 && (!k_cache || !v_cache)) || ((long long)B * max_pages > 0 && !pages)) return KDA_ERR_INVALID_ARGUMENT;
    return KDA_OK;
}

// The most slots of keys that a call of attn_step can have, and how many its sequences are to share: four
// workgroups per compute unit where the lengths allow it, and one more for every sequence's last slot.
void step_plan(int N, int m, int H, int Hkv, int max_pages, int page, int* want, int* slots) {
    const long long units = (long long)Hkv * ((m * (long long)(H / Hkv) + 15) / 16);
    long long w = 4LL * cu_count() / units;
    if (w < 1) w = 1;
    const long long tiles = ((long long)max_pages * page + 127) / 128, most = (long long)N * (tiles > 1 ? tiles : 1);
    *want = (int)w;
    *slots = (int)(w + N < most ? w + N : most);
}

kda_status_t check_step_shape(int N, int m, int H, int Hkv, int d, int n_pages, int max_pages, int page, kda_dtype_t dt) {
    if (m < 0) return KDA_ERR_INVALID_ARGUMENT;
    kda_status_t st = check_heads(H, Hkv, d, dt);
    if (st == KDA_OK) st = check_cache(N, Hkv, d, n_pages, max_pages, page, dt);
    if (st != KDA_OK || H == 0 || N == 0 || m == 0) return st;
    const long long tiles = ((long long)max_pages * page + 127) / 128;
    long long rows = 0;
    if (!mul_ok((long long)N * m, H, &rows) || rows > 2 * kMaxUnits) return KDA_ERR_UNSUPPORTED;   // the join's workgroups of 256
    if ((long long)N * (tiles + 1) > kMaxRows) return KDA_ERR_UNSUPPORTED;
    int want = 0, slots = 0;
    step_plan(N, m, H, Hkv, max_pages, page, &want, &slots);
    if ((long long)slots * Hkv * ((m * (long long)(H / Hkv) + 15) / 16) > 2 * kMaxUnits) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

}  // namespace

extern "C" {

size_t kda_attn_prefill_workspace_bytes(int B, int Nq, int Nk, int H, int Hkv, int d, kda_dtype_t dt) {
    if (check_attn_shape(B, Nq, Nk, H, Hkv, d, dt) != KDA_OK || H == 0) return 0;
    int few = 0, ns = 1;
    attn_plan(B, Nq, Nk, H, Hkv, d, dt, &few, &ns);
    return ns > 1 ? parts_bytes((long long)Nq * H * ns, d) : 0;
}

kda_status_t kda_attn_prefill(const void* q, const void* k, const void* v, const int* cu_q, const int* cu_k, void* o, int B,
                              int Nq, int Nk, int H, int Hkv, int d, float scale, long long q_stride, long long k_stride,
                              long long v_stride, kda_dtype_t dt, void* workspace, size_t workspace_bytes, void* stream) {
    kda_status_t st = check_attn_shape(B, Nq, Nk, H, Hkv, d, dt);
    if (st == KDA_OK && !scale_ok(scale)) st = KDA_ERR_INVALID_ARGUMENT;
    if (st == KDA_OK && !cu_k && Nq != Nk) st = KDA_ERR_INVALID_ARGUMENT;
    if (st != KDA_OK || B == 0 || H == 0 || Nq == 0) return st;
    const size_t esz = elem_size(dt);
    if (!q || !o || !cu_q || (Nk > 0 && (!k || !v))) return KDA_ERR_INVALID_ARGUMENT;
    if (!wide_rows_ok(q, Nq, (long long)H * d, q_stride, esz) || !wide_rows_ok(k, Nk, (long long)Hkv * d, k_stride, esz) ||
        !wide_rows_ok(v, Nk, (long long)Hkv * d, v_stride, esz))
        return KDA_ERR_INVALID_ARGUMENT;
    if (!aligned(o, 16) || !aligned(cu_q, 4) || !aligned(cu_k, 4) || !aligned(workspace, 16)) return KDA_ERR_INVALID_ARGUMENT;
    kda::AttnArgs a;
    memset(&a, 0, sizeof(a));
    attn_plan(B, Nq, Nk, H, Hkv, d, dt, &a.few, &a.n_split);
    if (!workspace) a.n_split = 1;
    const size_t need = a.n_split > 1 ? parts_bytes((long long)Nq * H * a.n_split, d) : 0;
    if (workspace_bytes < need) return KDA_ERR_WORKSPACE;
    const Range ro = range_of(o, (size_t)Nq * H * d * esz), rw = range_of(workspace, need);
    const Range ins[] = {rows_range(q, Nq, (long long)H * d, q_stride, esz), rows_range(k, Nk, (long long)Hkv * d, k_stride, esz),
                         rows_range(v, Nk, (long long)Hkv * d, v_stride, esz), range_of(cu_q, ((size_t)B + 1) * 4),
                         range_of(cu_k, cu_k ? ((size_t)B + 1) * 4 : 0)};
    for (const Range& r : ins)
        if (overlap(ro, r) || overlap(rw, r)) return KDA_ERR_INVALID_ARGUMENT;
    if (overlap(ro, rw)) return KDA_ERR_INVALID_ARGUMENT;
    a.q = q;
    a.k = k;
    a.v = v;
    a.cu_q = cu_q;
    a.cu_k = cu_k ? cu_k : cu_q;
    a.o = o;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.B = B;
    a.Nq = Nq;
    a.Nk = Nk;
    a.H = H;
    a.Hkv = Hkv;
    a.scale = scale;
    if (need > 0) {
        a.ws_o = reinterpret_cast<float*>(workspace);
        a.ws_ml = a.ws_o + (size_t)Nq * H * a.n_split * d;
    }
    (void)hipGetLastError();
    if (kda::launch_attn_prefill(d, dt == KDA_F32, a, reinterpret_cast<hipStream_t>(stream)) != hipSuccess) return KDA_ERR_DEVICE;
    return KDA_OK;
}

kda_status_t kda_cache_write(const void* k, const void* v, void* k_cache, void* v_cache, const int* pages, const int* cu,
                             const int* start, int B, int N, int Hkv, int d, int n_pages, int max_pages, int page,
                             long long k_stride, long long v_stride, kda_dtype_t dt, void* stream) {
    kda_status_t st = check_cache_rows(k_cache, v_cache, pages, cu, start, B, N, Hkv, d, n_pages, max_pages, page, dt);
    if (st != KDA_OK || B == 0 || N == 0 || Hkv == 0) return st;
    const size_t esz = elem_size(dt);
    if (!k || !v || !wide_rows_ok(k, N, (long long)Hkv * d, k_stride, esz) || !wide_rows_ok(v, N, (long long)Hkv * d, v_stride, esz))
        return KDA_ERR_INVALID_ARGUMENT;
    const size_t pool = (size_t)n_pages * Hkv * (size_t)page_bytes(d, page);
    const Range rk = range_of(k_cache, pool), rv = range_of(v_cache, pool);
    const Range ins[] = {rows_range(k, N, (long long)Hkv * d, k_stride, esz), rows_range(v, N, (long long)Hkv * d, v_stride, esz),
                         range_of(pages, (size_t)B * max_pages * 4), range_of(cu, cu ? ((size_t)B + 1) * 4 : 0),
                         range_of(start, start ? (size_t)B * 4 : 0)};
    for (const Range& r : ins)
        if (overlap(rk, r) || overlap(rv, r)) return KDA_ERR_INVALID_ARGUMENT;
    if (overlap(rk, rv)) return KDA_ERR_INVALID_ARGUMENT;
    if (n_pages == 0 || max_pages == 0) return KDA_OK;   // no token has a place
    kda::CacheArgs a = cache_args(pages, cu, start, B, N, Hkv, d, n_pages, max_pages, page);
    a.k = k;
    a.v = v;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.k_cache = reinterpret_cast<uint8_t*>(k_cache);
    a.v_cache = reinterpret_cast<uint8_t*>(v_cache);
    (void)hipGetLastError();
    if (kda::launch_cache_rows(true, d, dt == KDA_F32, a, reinterpret_cast<hipStream_t>(stream)) != hipSuccess) return KDA_ERR_DEVICE;
    return KDA_OK;
}

kda_status_t kda_cache_read(const void* k_cache, const void* v_cache, const int* pages, const int* cu, const int* start, void* k,
                            void* v, int B, int N, int Hkv, int d, int n_pages, int max_pages, int page, kda_dtype_t dt,
                            void* stream) {
    kda_status_t st = check_cache_rows(k_cache, v_cache, pages, cu, start, B, N, Hkv, d, n_pages, max_pages, page, dt);
    if (st != KDA_OK || B == 0 || N == 0 || Hkv == 0) return st;
    if (!k || !v || !aligned(k, 16) || !aligned(v, 16)) return KDA_ERR_INVALID_ARGUMENT;
    const size_t pool = (size_t)n_pages * Hkv * (size_t)page_bytes(d, page), out = (size_t)N * Hkv * d * elem_size(dt);
    const Range rk = range_of(k, out), rv = range_of(v, out);
    const Range ins[] = {range_of(k_cache, pool), range_of(v_cache, pool), range_of(pages, (size_t)B * max_pages * 4),
                         range_of(cu, cu ? ((size_t)B + 1) * 4 : 0), range_of(start, start ? (size_t)B * 4 : 0)};
    for (const Range& r : ins)
        if (overlap(rk, r) || overlap(rv, r)) return KDA_ERR_INVALID_ARGUMENT;
    if (overlap(rk, rv)) return KDA_ERR_INVALID_ARGUMENT;
    kda::CacheArgs a = cache_args(pages, cu, start, B, N, Hkv, d, n_pages, max_pages, page);
    a.k_cache = const_cast<uint8_t*>(reinterpret_cast<const uint8_t*>(k_cache));
    a.v_cache = const_cast<uint8_t*>(reinterpret_cast<const uint8_t*>(v_cache));
    a.k_out = k;
    a.v_out = v;
    a.streamed = 2 * out >= kStreamedBytes ? 1 : 0;
    (void)hipGetLastError();
    if (kda::launch_cache_rows(false, d, dt == KDA_F32, a, reinterpret_cast<hipStream_t>(stream)) != hipSuccess) return KDA_ERR_DEVICE;
    return KDA_OK;
}

size_t kda_attn_step_workspace_bytes(int N, int m, int H, int Hkv, int d, int max_pages, int page, kda_dtype_t dt) {
    if (check_step_shape(N, m, H, Hkv, d, 0, max_pages, page, dt) != KDA_OK || N == 0 || m == 0 || H == 0) return 0;
    int want = 0, slots = 0;
    step_plan(N, m, H, Hkv, max_pages, page, &want, &slots);
    return slots > N ? parts_bytes((long long)slots * m * H, d) : 0;
}

kda_status_t kda_attn_step(const void* q, const void* k_cache, const void* v_cache, const int* pages, const int* lens, void* o,
                           int N, int m, int H, int Hkv, int d, int n_pages, int max_pages, int page, float scale,
                           long long q_stride, kda_dtype_t dt, void* workspace, size_t workspace_bytes, void* stream) {
    kda_status_t st = check_step_shape(N, m, H, Hkv, d, n_pages, max_pages, page, dt);
    if (st == KDA_OK && !scale_ok(scale)) st = KDA_ERR_INVALID_ARGUMENT;
    if (st != KDA_OK || N == 0 || m == 0 || H == 0) return st;
    const size_t esz = elem_size(dt);
    const long long rows = (long long)N * m;
    // (every tile reads something: a pool without pages has nothing that it could)
    if (!q || !o || !lens || !k_cache || !v_cache || n_pages == 0 || (max_pages > 0 && !pages)) return KDA_ERR_INVALID_ARGUMENT;
    if (!wide_rows_ok(q, rows, (long long)H * d, q_stride, esz)) return KDA_ERR_INVALID_ARGUMENT;
    if (!aligned(o, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(lens, 4) || !aligned(pages, 4) ||
        !aligned(workspace, 16))
        return KDA_ERR_INVALID_ARGUMENT;
    kda::AttnStepArgs a;
    memset(&a, 0, sizeof(a));
    step_plan(N, m, H, Hkv, max_pages, page, &a.want, &a.slots);
    const size_t need = a.slots > N ? parts_bytes((long long)a.slots * m * H, d) : 0;
    if (need > 0 && (!workspace || workspace_bytes < need)) return KDA_ERR_WORKSPACE;
    const size_t pool = (size_t)n_pages * Hkv * (size_t)page_bytes(d, page);
    const Range ro = range_of(o, (size_t)rows * H * d * esz), rw = range_of(workspace, need);
    const Range ins[] = {rows_range(q, rows, (long long)H * d, q_stride, esz), range_of(k_cache, pool), range_of(v_cache, pool),
                         range_of(pages, (size_t)N * max_pages * 4), range_of(lens, (size_t)N * 4)};
    for (const Range& r : ins)
        if (overlap(ro, r) || overlap(rw, r)) return KDA_ERR_INVALID_ARGUMENT;
    if (overlap(ro, rw)) return KDA_ERR_INVALID_ARGUMENT;
    a.q = q;
    a.k_cache = reinterpret_cast<const uint8_t*>(k_cache);
    a.v_cache = reinterpret_cast<const uint8_t*>(v_cache);
    a.pages = pages;
    a.lens = lens;
    a.o = o;
    a.q_stride = q_stride;
    a.N = N;
    a.m = m;
    a.H = H;
    a.Hkv = Hkv;
    a.n_pages = n_pages;
    a.max_pages = max_pages;
    a.page = page;
    a.page_shift = shift_of(page);
    a.page_bytes = page_bytes(d, page);
    a.scale = scale;
    if (need > 0) {
        a.ws_o = reinterpret_cast<float*>(workspace);
        a.ws_ml = a.ws_o + (size_t)a.slots * m * H * d;
    }
    (void)hipGetLastError();
    if (kda::launch_attn_step(d, dt == KDA_F32, a, reinterpret_cast<hipStream_t>(stream)) != hipSuccess) return KDA_ERR_DEVICE;
    return KDA_OK;
}

}  // extern "C"
