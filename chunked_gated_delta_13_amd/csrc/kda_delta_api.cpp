// Host side of the gated delta rule: argument validation, launch plans and launches.  Nothing here allocates
// memory or synchronises the host with the device.
#include <string.h>

#include <hip/hip_runtime.h>

#include "../../include/kda.h"
#include "kda_host.h"
#include "kda_mixers.h"

using namespace kda::host;

namespace {

constexpr int kSegment = 64;   // segments are whole multiples of this many tokens

kda_status_t check_shape(int B, int T, int H, int Hk, int dk, int dv, kda_dtype_t dt) {
    if (B < 0 || T < 0 || H < 0 || Hk < 0 || dk <= 0 || dv <= 0) return KDA_ERR_INVALID_ARGUMENT;
    if (dt != KDA_BF16 && dt != KDA_F32) return KDA_ERR_INVALID_ARGUMENT;
    if ((dk != 64 && dk != 128) || (dv != 64 && dv != 128)) return KDA_ERR_UNSUPPORTED;
    if (H > 0 && (Hk == 0 || H % Hk != 0)) return KDA_ERR_INVALID_ARGUMENT;
    long long a = 0;
    if (!mul_ok((long long)B * T, (long long)H * dv, &a) || a >= (1LL << 58)) return KDA_ERR_INVALID_ARGUMENT;
    if ((long long)B * H > kMaxUnits / 4 || T > (1 << 30)) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

// State columns per workgroup: 128 where the sequences and heads alone fill the compute units, else 64.
int delta_width(long long units, int dv) { return dv == 128 && 2 * units > cu_count() ? 128 : 64; }

// The split's first pass takes 128 columns too where both the state's and the transition's allow it.
int first_width(long long units, int dk, int dv) { return dk == 128 && dv == 128 && 4 * units > cu_count() ? 128 : 64; }

// Microseconds of a chunk: outputs and states of bf16, by columns of a workgroup.
double chunk_us(int dk, int width, kda_dtype_t dt, bool out) {
    const double us = (width == 128 ? 6.2 : 5.0) * (out ? 1.0 : 0.84) * (dk == 128 ? 1.0 : 0.8);
    return dt == KDA_F32 ? 2.2 * us : us;
}

// Segments of seg_in tokens, or (seg_in 0) as many as take the least time: with fewer sequences and heads than
// compute units a split shortens the chain of chunks.  Its first pass runs all segments but the last from zero, and their
// transitions (dk columns more), the second all of them with outputs.  (Where decays leave nothing of a state over a
// segment, the first pass runs its end alone; the plan, which does not know them, counts whole segments.)
kda_status_t delta_plan(int B, int T, int H, int dk, int dv, kda_dtype_t dt, int seg_in, long long* seg_len, int* n_seg) {
    if (seg_in < 0 || seg_in % kSegment != 0) return KDA_ERR_INVALID_ARGUMENT;
    const long long chunks = ((long long)T + kSegment - 1) / kSegment, units = (long long)B * H;
    long long per = seg_in > 0 ? seg_in / kSegment : chunks;
    if (seg_in == 0 && units > 0) {
        const long long cus = cu_count();
        const auto rounds = [&](long long n) { return (double)((n + cus - 1) / cus); };
        const auto second = [&](long long ns) {
            const int w = delta_width(units * ns, dv);
            return rounds(units * ns * (dv / w)) * chunk_us(dk, w, dt, true);
        };
        const auto first = [&](long long ns) {
            const int w = first_width(units * (ns - 1), dk, dv);
            return rounds(units * (ns - 1) * ((dv + dk) / w)) * chunk_us(dk, w, dt, false);
        };
        double best = (double)chunks * second(1);
        if (2 * units <= cus) {
            for (long long ns = 2; ns <= cus / units && ns <= chunks; ++ns) {
                const long long c = (chunks + ns - 1) / ns;
                const double us = (double)c * (first(ns) + second(ns)) + 1.5 * (double)ns + 12.0;
                if (us < best) {
                    best = us;
                    per = c;
                }
            }
        }
    }
    if (per < 1) per = 1;
    const long long ns = chunks > 0 ? (chunks + per - 1) / per : 1;
    if (units * ns > kMaxUnits / 4) return KDA_ERR_UNSUPPORTED;
    *seg_len = per * kSegment;
    *n_seg = (int)ns;
    return KDA_OK;
}

// Workspace of a split: the segments' entry states [B * H, n_seg, dk, dv] and transitions [B * H, n_seg - 1, dk, dk], fp32, and
// which of the latter are dead, int32 [B * H, n_seg - 1], padded to 16 bytes.
size_t delta_workspace(int B, int H, int dk, int dv, int ns) {
    if (ns <= 1) return 0;
    const size_t bh = (size_t)B * H;
    return bh * sizeof(float) * ((size_t)ns * dk * dv + (size_t)(ns - 1) * dk * dk) + (bh * (ns - 1) * sizeof(int) + 15) / 16 * 16;
}

struct Inputs {
    const void *q, *k, *v;
    const float *g, *beta;
    const int* lens;
    long long q_stride, k_stride, v_stride;
};

// Pointer, stride and overlap checks shared by the prompt and the token form.  S_in is NULL where the state is updated in
// place; `need` bytes of the workspace are used.
kda_status_t check_ptrs(const Inputs& x, const float* S_in, const void* o, const float* S_out, const void* ws, size_t need, int B, int T,
                        int H, int Hk, int dk, int dv, kda_dtype_t dt) {
    const size_t esz = elem_size(dt);
    const long long rows = (long long)B * T;
    if (rows > 0 && (!x.q || !x.k || !x.v || !x.g || !x.beta || !o)) return KDA_ERR_INVALID_ARGUMENT;
    if (!wide_rows_ok(x.q, rows, (long long)Hk * dk, x.q_stride, esz) || !wide_rows_ok(x.k, rows, (long long)Hk * dk, x.k_stride, esz) ||
        !wide_rows_ok(x.v, rows, (long long)H * dv, x.v_stride, esz))
        return KDA_ERR_INVALID_ARGUMENT;
    // offsets inside a chunk are 32-bit: 64 rows of at most 2^22 elements
    const long long widest = 1LL << 22;
    if ((long long)H * dv > widest || (rows > 1 && (x.q_stride > widest || x.k_stride > widest || x.v_stride > widest)))
        return KDA_ERR_UNSUPPORTED;
    if (!aligned(x.g, 4) || !aligned(x.beta, 4) || !aligned(x.lens, 4) || !aligned(o, 16) || !aligned(S_in, 16) || !aligned(S_out, 16) ||
        !aligned(ws, 16))
        return KDA_ERR_INVALID_ARGUMENT;
    const size_t state = (size_t)B * H * dk * dv * sizeof(float);
    const Range outs[] = {range_of(o, (size_t)rows * H * dv * esz), range_of(S_out, S_out ? state : 0), range_of(ws, need)};
    const Range ri = range_of(S_in, S_in ? state : 0);
    const Range ins[] = {rows_range(x.q, rows, (long long)Hk * dk, x.q_stride, esz), rows_range(x.k, rows, (long long)Hk * dk, x.k_stride, esz),
                         rows_range(x.v, rows, (long long)H * dv, x.v_stride, esz), range_of(x.g, (size_t)rows * H * 4),
                         range_of(x.beta, (size_t)rows * H * 4), range_of(x.lens, x.lens ? (size_t)B * 4 : 0)};
    for (int i = 0; i < 3; ++i) {
        for (const Range& r : ins)
            if (overlap(outs[i], r)) return KDA_ERR_INVALID_ARGUMENT;
        for (int j = i + 1; j < 3; ++j)
            if (overlap(outs[i], outs[j])) return KDA_ERR_INVALID_ARGUMENT;
    }
    if (overlap(outs[0], ri) || overlap(outs[2], ri) || (S_in != S_out && overlap(outs[1], ri))) return KDA_ERR_INVALID_ARGUMENT;
    return KDA_OK;
}

kda::DeltaArgs delta_args(const Inputs& x, void* o, int B, int T, int H, int Hk, int dv) {
    kda::DeltaArgs a;
    memset(&a, 0, sizeof(a));
    a.q = x.q;
    a.k = x.k;
    a.v = x.v;
    a.g = x.g;
    a.beta = x.beta;
    a.lens = x.lens;
    a.o = o;
    a.q_stride = x.q_stride;
    a.k_stride = x.k_stride;
    a.v_stride = x.v_stride;
    a.T = T;
    a.BH = B * H;
    a.H = H;
    a.Hk = Hk;
    a.dv = dv;
    return a;
}

}  // namespace

extern "C" {

size_t kda_delta_prefill_workspace_bytes(int B, int T, int H, int Hk, int dk, int dv, kda_dtype_t dt, int seg_len) {
    long long sl = 0;
    int ns = 1;
    if (check_shape(B, T, H, Hk, dk, dv, dt) != KDA_OK || delta_plan(B, T, H, dk, dv, dt, seg_len, &sl, &ns) != KDA_OK) return 0;
    return delta_workspace(B, H, dk, dv, ns);
}

kda_status_t kda_delta_prefill(const void* q, const void* k, const void* v, const float* g, const float* beta, const float* S0,
                               const int* lens, void* o, float* S_T, int B, int T, int H, int Hk, int dk, int dv, long long q_stride,
                               long long k_stride, long long v_stride, kda_dtype_t dt, int seg_len, void* workspace,
                               size_t workspace_bytes, void* stream) {
    kda_status_t st = check_shape(B, T, H, Hk, dk, dv, dt);
    if (st != KDA_OK) return st;
    long long sl = 0;
    int ns = 1;
    st = delta_plan(B, T, H, dk, dv, dt, seg_len, &sl, &ns);
    if (st != KDA_OK || B == 0 || H == 0) return st;
    const Inputs x = {q, k, v, g, beta, lens, q_stride, k_stride, v_stride};
    const size_t need = delta_workspace(B, H, dk, dv, ns);
    st = check_ptrs(x, S0, o, S_T, workspace, need, B, T, H, Hk, dk, dv, dt);
    if (st != KDA_OK) return st;
    if (need > 0 && (!workspace || workspace_bytes < need)) return KDA_ERR_WORKSPACE;
    if (T == 0 && !S_T) return KDA_OK;
    const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const bool f32 = dt == KDA_F32;
    const long long state = (long long)dk * dv;
    kda::DeltaArgs a = delta_args(x, o, B, T, H, Hk, dv);
    a.seg_len = sl;
    a.S_in = S0;
    a.sin_bh = state;
    (void)hipGetLastError();
    if (ns > 1) {
        float* entry = reinterpret_cast<float*>(workspace);
        float* M = entry + (size_t)B * H * ns * state;
        kda::DeltaArgs p = a;
        p.S_in = nullptr;
        p.S_out = entry + state;   // a segment's state from zero lies where the next one's entry state will
        p.sout_bh = ns * state;
        p.sout_seg = state;
        p.out_seg = -1;
        p.M_out = M;
        p.dead = reinterpret_cast<int*>(M + (size_t)B * H * (ns - 1) * dk * dk);
        p.m_bh = ns - 1;
        p.n_seg_launch = ns - 1;
        if (kda::launch_delta_prefill(false, dk, f32, first_width((long long)B * H * (ns - 1), dk, dv), p, s) != hipSuccess) return KDA_ERR_DEVICE;
        if (kda::launch_delta_join(dk, dv, B * H, ns, M, p.dead, S0, entry, s) != hipSuccess) return KDA_ERR_DEVICE;
        a.S_in = entry;
        a.sin_bh = ns * state;
        a.sin_seg = state;
    }
    a.S_out = S_T;
    a.sout_bh = state;
    a.out_seg = ns - 1;
    a.n_seg_launch = ns;
    if (kda::launch_delta_prefill(true, dk, f32, delta_width((long long)B * H * ns, dv), a, s) != hipSuccess) return KDA_ERR_DEVICE;
    return KDA_OK;
}

kda_status_t kda_delta_step(const void* q, const void* k, const void* v, const float* g, const float* beta, float* S, void* o, int N, int H,
                            int Hk, int dk, int dv, long long q_stride, long long k_stride, long long v_stride, kda_dtype_t dt,
                            void* stream) {
    kda_status_t st = check_shape(N, 1, H, Hk, dk, dv, dt);
    if (st != KDA_OK || N == 0 || H == 0) return st;
    if (!S) return KDA_ERR_INVALID_ARGUMENT;
    const Inputs x = {q, k, v, g, beta, nullptr, q_stride, k_stride, v_stride};
    st = check_ptrs(x, nullptr, o, S, nullptr, 0, N, 1, H, Hk, dk, dv, dt);
    if (st != KDA_OK) return st;
    kda::DeltaArgs a = delta_args(x, o, N, 1, H, Hk, dv);
    a.S_out = S;
    a.n_units = (long long)N * H;
    (void)hipGetLastError();
    if (kda::launch_delta_step(dk, dt == KDA_F32, a, reinterpret_cast<hipStream_t>(stream)) != hipSuccess) return KDA_ERR_DEVICE;
    return KDA_OK;
}

}  // extern "C"
