// Host side of the token mixers beside KDA: argument validation, launch plans and launches of the
// short convolution, the state space scan and the window attention.  Nothing here allocates
// memory or synchronises the host with the device.
#include <string.h>

#include <hip/hip_runtime.h>

#include "../../include/kda.h"
#include "kda_host.h"
#include "kda_mixers.h"

using kda::Range;
using kda::aligned;
using kda::mul_ok;
using kda::overlap;
using kda::range_of;

namespace {

constexpr long long kMaxGridYZ = 65535;   // blocks of a launch along y or z

size_t elem_size(kda_dtype_t dt) { return dt == KDA_BF16 ? 2 : 4; }

// The bytes spanned by `rows` rows of `width` elements whose starts lie `stride` elements apart.
Range rows_range(const void* p, long long rows, long long width, long long stride, size_t esz) {
    if (rows <= 0 || width <= 0 || !p) return range_of(p, 0);
    return range_of(p, ((size_t)(rows - 1) * (size_t)stride + (size_t)width) * esz);
}

// rows * stride elements stay far inside 63 bits, and a stride is at least a row's width.
bool stride_ok(long long rows, long long width, long long stride) {
    long long n = 0;
    if (rows <= 1) return stride >= 0;
    return stride >= width && mul_ok(rows, stride, &n) && n < (1LL << 58);
}

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
    // Long tiles re-read fewer rows (W - 1 per tile); short ones keep the GPU busy on short inputs.
    // Halve the tile until there are about 16 waves per compute unit of 256.
    const long long groups = (D + (vec ? (dt == KDA_BF16 ? 8 : 4) : 1) - 1) / (vec ? (dt == KDA_BF16 ? 8 : 4) : 1);
    int tile = 64;
    while (tile > 4 && groups * B * (((long long)T + tile - 1) / tile) < 64LL * 4096) tile >>= 1;
    while ((T + (long long)tile - 1) / tile > kMaxGridYZ) tile <<= 1;
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

}  // extern "C"
