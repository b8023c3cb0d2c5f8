// LDS tiles shared by the state space scan and the window attention (gfx950, wave64).
//
// A tile holds 64-bit (bf16) or 128-bit (fp32) chunks of four elements.  Chunk c of row r lies at
// chunk c ^ f(r) of the row, f(r) = 4 (r & 3) + ((r >> 2) & 3): the sixteen rows of a matrix
// operand, and the four rows by four chunks that one transposed read takes, then fall on different
// banks, with no padding between rows.  Rows hold a multiple of 64 elements.
#pragma once

#include "kda_device.h"

namespace kda {

typedef __attribute__((ext_vector_type(4))) short s16x4_t;

__device__ __forceinline__ int tile_f(int r) { return ((r & 3) << 2) | ((r >> 2) & 3); }

// Transposed read of bf16: within each 16-lane group, lane 4k + j names four elements of row k
// (columns 4j .. 4j + 3) and lane i receives column i of rows 0 .. 3.  (Not a template: see lds_dma16.)
__device__ __forceinline__ bf16x4_t lds_read_tr(const KDA_LDS __bf16* p) {
    const s16x4_t v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((KDA_LDS s16x4_t*)(p));
    return __builtin_bit_cast(bf16x4_t, v);
}

// Lane offsets (elements) into a tile of rows of WIDTH elements.
template <typename T, int WIDTH> struct TileLane {
    int row[4];   // row operand: row r, chunk (g ^ 4x) ^ f(r), x = 2 (block & 1) + half
    int tr[4];    // transposed operand: column tile t with t & 3 = x
    __device__ __forceinline__ void set(int lane) {
        const int g = lane >> 4, r = lane & 15, k = r >> 2, j = r & 3;
        const int q = g ^ tile_f(r);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            row[x] = r * WIDTH + ((q ^ (x << 2)) << 2);
            tr[x] = (4 * g + k) * WIDTH + ((((x << 2) | j) ^ ((k << 2) | g)) << 2);
        }
    }
};

// Row operand: rows 16 a .. 16 a + 15, contraction block kb of 32 columns.
template <typename T, int WIDTH>
__device__ __forceinline__ void tile_row_frag(Frag<T>& f, const KDA_LDS T* tile, const TileLane<T, WIDTH>& l, int a,
                                              int kb) {
    const KDA_LDS T* p = tile + 16 * a * WIDTH + (kb >> 1) * 64;
    const int x = (kb & 1) * 2;
    if constexpr (sizeof(T) == 2) {
        const bf16x4_t lo = *reinterpret_cast<const KDA_LDS bf16x4_t*>(p + l.row[x]);
        const bf16x4_t hi = *reinterpret_cast<const KDA_LDS bf16x4_t*>(p + l.row[x + 1]);
        f.v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    } else {
        const f32x4_t lo = *reinterpret_cast<const KDA_LDS f32x4_t*>(p + l.row[x]);
        const f32x4_t hi = *reinterpret_cast<const KDA_LDS f32x4_t*>(p + l.row[x + 1]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f.v[i] = lo[i];
            f.v[4 + i] = hi[i];
        }
    }
}

// The lower half of a row operand's block, the upper half zero.
template <typename T, int WIDTH>
__device__ __forceinline__ void tile_row_frag_lo(Frag<T>& f, const KDA_LDS T* tile, const TileLane<T, WIDTH>& l, int a,
                                                 int kb) {
    const KDA_LDS T* p = tile + 16 * a * WIDTH + (kb >> 1) * 64 + l.row[(kb & 1) * 2];
    if constexpr (sizeof(T) == 2) {
        const bf16x4_t lo = *reinterpret_cast<const KDA_LDS bf16x4_t*>(p);
        const bf16x4_t z = {(__bf16)0.0f, (__bf16)0.0f, (__bf16)0.0f, (__bf16)0.0f};
        f.v = __builtin_shufflevector(lo, z, 0, 1, 2, 3, 4, 5, 6, 7);
    } else {
        const f32x4_t lo = *reinterpret_cast<const KDA_LDS f32x4_t*>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f.v[i] = lo[i];
            f.v[4 + i] = 0.0f;
        }
    }
}

// Transposed operand: its row (or column) r is column 16 t + r of the tile, its contraction block the
// tile's rows 32 kb .. 32 kb + 31.
template <typename T, int WIDTH>
__device__ __forceinline__ void tile_tr_frag(Frag<T>& f, const KDA_LDS T* tile, const TileLane<T, WIDTH>& l, int t,
                                             int kb, int lane) {
    const KDA_LDS T* p = tile + 32 * kb * WIDTH + (t >> 2) * 64;
    if constexpr (sizeof(T) == 2) {
        const bf16x4_t lo = lds_read_tr(p + l.tr[t & 3]);
        const bf16x4_t hi = lds_read_tr(p + l.tr[t & 3] + 16 * WIDTH);
        f.v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    } else {
        const int g = lane >> 4, r = lane & 15;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = (((t & 3) ^ i) << 2) | ((r >> 2) ^ g);
            const KDA_LDS T* q = p + (4 * g + i) * WIDTH + (c << 2) + (r & 3);
            f.v[i] = q[0];
            f.v[4 + i] = q[16 * WIDTH];
        }
    }
}

// Sixteen bytes of a row (8 bf16 or 4 fp32, piece m of the row) into a tile.
__device__ __forceinline__ void tile_put(KDA_LDS __bf16* row, int m, int r, u32x4_t v) {
    const int f = tile_f(r);
    const bool swap = f & 1;
    const u32x4_t w = {swap ? v[2] : v[0], swap ? v[3] : v[1], swap ? v[0] : v[2], swap ? v[1] : v[3]};
    *reinterpret_cast<KDA_LDS u32x4_t*>(row + (((2 * m) ^ (f & ~1)) << 2)) = w;
}
__device__ __forceinline__ void tile_put(KDA_LDS float* row, int m, int r, u32x4_t v) {
    *reinterpret_cast<KDA_LDS u32x4_t*>(row + ((m ^ tile_f(r)) << 2)) = v;
}

}  // namespace kda
