// LDS tiles shared by the state space scan and the window attention (gfx950, wave64).
//
// A tile of ROWS rows is stored in blocks of 32 columns, row after row inside a block, in chunks of four
// elements (8 bytes of bf16, 16 of fp32).  Chunk c of row r lies at place c ^ f(r) of its 8.  One cycle
// reads 256 bytes from 64 banks (measured with the bank conflict counter): f spreads the 16 rows by two
// chunks (bf16) or the 16 rows of one chunk (fp32) that a cycle of a row read takes, and the eight rows
// by four chunks of a transposed read of bf16, over all banks without padding.  f is even for bf16, so 16
// bytes of a row stay together.
//
// A matrix operand's 32 contraction slots are two stacked 16-wide tiles, as in kda_device.h, but tiles
// half the contraction apart instead of neighbours: (a, a + n/2).  Both halves then lie a constant
// distance apart, in reach of one two-address read with an immediate offset, and arrive in adjacent
// registers; neighbours would differ by an exclusive-or of the lane's address.
#pragma once

#include "kda_device.h"

namespace kda {

typedef __attribute__((ext_vector_type(4))) short s16x4_t;

template <typename T> __device__ __forceinline__ int tile_f(int r);
template <> __device__ __forceinline__ int tile_f<__bf16>(int r) { return (r & 4) | ((r >> 2) & 2); }
template <> __device__ __forceinline__ int tile_f<float>(int r) { return (r >> 1) & 7; }

// Four elements as one vector.
template <typename T> struct Vec4 { typedef bf16x4_t type; };
template <> struct Vec4<float> { typedef f32x4_t type; };

// Transposed read of bf16: within each 16-lane group, lane 4k + j names four elements of row k
// (columns 4j .. 4j + 3) and lane i receives column i of rows 0 .. 3.  (Not a template: see lds_dma16.)
__device__ __forceinline__ bf16x4_t lds_read_tr(const KDA_LDS __bf16* p) {
    const s16x4_t v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((KDA_LDS s16x4_t*)(p));
    return __builtin_bit_cast(bf16x4_t, v);
}

__device__ __forceinline__ void frag_join(Frag<__bf16>& f, bf16x4_t lo, bf16x4_t hi) {
    f.v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}
__device__ __forceinline__ void frag_join(Frag<float>& f, f32x4_t lo, f32x4_t hi) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f.v[i] = lo[i];
        f.v[4 + i] = hi[i];
    }
}

// Offset (elements) of chunk c (of the whole row) of row r in a tile.
template <typename T, int ROWS> __device__ __forceinline__ int tile_at(int r, int c) {
    return (c >> 3) * (ROWS * 32) + r * 32 + (((c & 7) ^ tile_f<T>(r)) << 2);
}

// Row operand of a tile of WIDTH columns (a multiple of 64): a lane's addresses, pinned in registers, so
// that everything it reads lies at a constant offset from one of them.  `delta` arguments are constant
// element offsets, by which tiles of one shape share the addresses.  The two reads of an operand are
// volatile: each then stays with its operand.  (The compiler otherwise pairs reads of different operands
// into one two-address read and sorts their halves with register moves.)
template <typename T, int ROWS, int WIDTH> struct TileRows {
    typedef typename Vec4<T>::type vec4;
    KDA_LDS T* at[2];   // row r, chunk 4 x + g of a block
    __device__ __forceinline__ void set(KDA_LDS T* tile, int lane) {
        const int g = lane >> 4, r = lane & 15;
        at[0] = lds_pin(tile + tile_at<T, ROWS>(r, g));
        at[1] = lds_pin(tile + tile_at<T, ROWS>(r, 4 + g));
    }
    // the same lane's addresses `delta` elements (not a constant) further
    __device__ __forceinline__ TileRows at_delta(int delta) const {
        TileRows o;
        o.at[0] = lds_pin(at[0] + delta);
        o.at[1] = lds_pin(at[1] + delta);
        return o;
    }
    // rows 16 a .. 16 a + 15, contraction block q: columns of tiles q and q + WIDTH/32
    __device__ __forceinline__ void frag(Frag<T>& f, int delta, int a, int q) const {
        const KDA_LDS T* p = at[q & 1] + delta + 16 * 32 * a + (q >> 1) * (ROWS * 32);
        frag_join(f, *reinterpret_cast<const volatile KDA_LDS vec4*>(p),
                  *reinterpret_cast<const volatile KDA_LDS vec4*>(p + (WIDTH / 64) * (ROWS * 32)));
    }
    // the first tile of the block, the second one zero
    __device__ __forceinline__ void frag_lo(Frag<T>& f, int delta, int a, int q) const {
        const KDA_LDS T* p = at[q & 1] + delta + 16 * 32 * a + (q >> 1) * (ROWS * 32);
        const vec4 z = {(T)0.0f, (T)0.0f, (T)0.0f, (T)0.0f};
        frag_join(f, *reinterpret_cast<const KDA_LDS vec4*>(p), z);
    }
};

// Transposed operand: its row (or column) r is column 16 t + r of the tile, its contraction block q the
// tile's rows 16 q .. and 16 q + ROWS/2 ..
template <typename T, int ROWS> struct TileCols;

template <int ROWS> struct TileCols<__bf16, ROWS> {
    KDA_LDS __bf16* at[2];   // column tile t with t & 1 = x
    __device__ __forceinline__ KDA_LDS __bf16* of(KDA_LDS __bf16* tile, int lane, int t) const {
        return lds_pin(tile + tile_at<__bf16, ROWS>(4 * (lane >> 4) + ((lane & 15) >> 2), 4 * t + (lane & 3)));
    }
    __device__ __forceinline__ void set(KDA_LDS __bf16* tile, int lane) {
        at[0] = of(tile, lane, 0);
        at[1] = of(tile, lane, 1);
    }
    __device__ __forceinline__ TileCols at_delta(int delta) const {
        TileCols o;
        o.at[0] = lds_pin(at[0] + delta);
        o.at[1] = lds_pin(at[1] + delta);
        return o;
    }
    // addresses for column tile t only, which is then used as t = 0
    __device__ __forceinline__ void set_tile(KDA_LDS __bf16* tile, int lane, int t) { at[0] = of(tile, lane, t); }
    __device__ __forceinline__ void frag(Frag<__bf16>& f, int delta, int t, int q) const {
        KDA_LDS __bf16* p = at[t & 1] + delta + (t >> 1) * (ROWS * 32) + 16 * 32 * q;
        frag_join(f, lds_read_tr(p), lds_read_tr(p + (ROWS / 2) * 32));
    }
};

template <int ROWS> struct TileCols<float, ROWS> {
    KDA_LDS float* at[2][4];   // element r of column tile t with t & 1 = x, row 4 g + i
    __device__ __forceinline__ KDA_LDS float* of(KDA_LDS float* tile, int lane, int t, int i) const {
        const int g = lane >> 4, r = lane & 15;
        return lds_pin(tile + tile_at<float, ROWS>(4 * g + i, 4 * t + (r >> 2)) + (r & 3));
    }
    __device__ __forceinline__ void set(KDA_LDS float* tile, int lane) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            at[0][i] = of(tile, lane, 0, i);
            at[1][i] = of(tile, lane, 1, i);
        }
    }
    __device__ __forceinline__ TileCols at_delta(int delta) const {
        TileCols o;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            o.at[0][i] = lds_pin(at[0][i] + delta);
            o.at[1][i] = lds_pin(at[1][i] + delta);
        }
        return o;
    }
    __device__ __forceinline__ void set_tile(KDA_LDS float* tile, int lane, int t) {
#pragma unroll
        for (int i = 0; i < 4; ++i) at[0][i] = of(tile, lane, t, i);
    }
    __device__ __forceinline__ void frag(Frag<float>& f, int delta, int t, int q) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const KDA_LDS float* p = at[t & 1][i] + delta + (t >> 1) * (ROWS * 32) + 16 * 32 * q;
            f.v[i] = p[0];
            f.v[4 + i] = p[(ROWS / 2) * 32];
        }
    }
};

// How a wave moves rows into a tile: one step is 16 bytes per lane, 16 rows (bf16) or 8 rows (fp32) of
// one block of 32 columns.
template <typename T> struct TileStep {
    static constexpr int PIECES = 2 * (int)sizeof(T), ROWS = 64 / PIECES, ELEMS = 16 / (int)sizeof(T);
    static __device__ __forceinline__ int row(int lane) { return lane / PIECES; }
    static __device__ __forceinline__ int piece(int lane) { return lane % PIECES; }
};

// A lane's places for its steps from row group `group0` on (places repeat every 16 rows).
template <typename T, int ROWS> struct TilePut {
    typedef TileStep<T> S;
    static constexpr int PER16 = 16 / S::ROWS;
    KDA_LDS T* at[PER16];
    __device__ __forceinline__ void set(KDA_LDS T* tile, int group0, int lane) {
#pragma unroll
        for (int x = 0; x < PER16; ++x)
            at[x] = lds_pin(tile + tile_at<T, ROWS>((group0 + x) * S::ROWS + S::row(lane), S::piece(lane) * (S::ELEMS / 4)));
    }
    // `group` row groups and `block` blocks further (constants)
    __device__ __forceinline__ void put(int group, int block, u32x4_t v) const {
        *reinterpret_cast<KDA_LDS u32x4_t*>(at[group % PER16] + (group / PER16) * 16 * 32 + block * ROWS * 32) = v;
    }
};

// The 16-byte piece of its row that a lane fetches when a step goes straight from memory to LDS, lane by
// lane: the one whose place in the block is the lane's.
template <typename T> __device__ __forceinline__ int tile_dma_piece(int row, int lane) {
    constexpr int CH = TileStep<T>::ELEMS / 4;   // chunks per piece
    return ((TileStep<T>::piece(lane) * CH) ^ tile_f<T>(row)) / CH;
}

// The steps of NW waves over a tile of ROWS x WIDTH: a wave's steps i = 0 .. N - 1 cover blocks of 32
// columns of one row group, or whole row groups one after the other.
template <typename T, int ROWS, int WIDTH, int NW> struct TileSteps {
    static constexpr int NB = WIDTH / 32, TOTAL = NB * (ROWS / TileStep<T>::ROWS);
    static constexpr int N = TOTAL / NW;
    static_assert(TOTAL % NW == 0 && (N % NB == 0 || NB % N == 0), "waves share the steps evenly");
    static __device__ __forceinline__ int group0(int wave) { return N >= NB ? wave * (N / NB) : wave / (NB / N); }
    static __device__ __forceinline__ int block0(int wave) { return N >= NB ? 0 : (wave % (NB / N)) * N; }
    static constexpr int group(int i) { return N >= NB ? i / NB : 0; }   // beyond group0
    static constexpr int block(int i) { return N >= NB ? i % NB : i; }   // beyond block0
};

// A range of memory with bounds: loads past its end give zeros, stores past it are dropped.  The address
// is a lane offset plus a uniform one, in bytes.  (Not templates: see lds_dma16.)
typedef __amdgpu_buffer_rsrc_t buffer_t;
__device__ __forceinline__ buffer_t make_buffer(const void* p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, 0x00027000);
}
// `rows` rows of `width` bytes that start `step` bytes apart; no rows give an empty buffer.
__device__ __forceinline__ buffer_t make_rows(const void* p, int rows, uint32_t step, uint32_t width) {
    return make_buffer(p, rows > 0 ? (uint32_t)(rows - 1) * step + width : 0u);
}
__device__ __forceinline__ u32x4_t buffer_load16(buffer_t b, uint32_t lane_off, uint32_t off) {
    return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(b, (int)lane_off, (int)off, 0));
}
__device__ __forceinline__ u32x2_t buffer_load8(buffer_t b, uint32_t lane_off, uint32_t off) {
    return __builtin_bit_cast(u32x2_t, __builtin_amdgcn_raw_buffer_load_b64(b, (int)lane_off, (int)off, 0));
}
__device__ __forceinline__ void buffer_store16(buffer_t b, uint32_t lane_off, uint32_t off, u32x4_t v) {
    __builtin_amdgcn_raw_buffer_store_b128(v, b, (int)lane_off, (int)off, 0);
}
__device__ __forceinline__ void buffer_store8(buffer_t b, uint32_t lane_off, uint32_t off, u32x2_t v) {
    __builtin_amdgcn_raw_buffer_store_b64(v, b, (int)lane_off, (int)off, 0);
}
// One element, widened.
__device__ __forceinline__ float buffer_load1(const __bf16*, buffer_t b, uint32_t lane_off) {
    const unsigned short u = __builtin_amdgcn_raw_buffer_load_b16(b, (int)lane_off, 0, 0);
    return __uint_as_float((uint32_t)u << 16);
}
__device__ __forceinline__ float buffer_load1(const float*, buffer_t b, uint32_t lane_off) {
    return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(b, (int)lane_off, 0, 0));
}
// Four elements.
__device__ __forceinline__ void buffer_load4(bf16x4_t& v, buffer_t b, uint32_t lane_off, uint32_t off) {
    v = __builtin_bit_cast(bf16x4_t, buffer_load8(b, lane_off, off));
}
__device__ __forceinline__ void buffer_load4(f32x4_t& v, buffer_t b, uint32_t lane_off, uint32_t off) {
    v = __builtin_bit_cast(f32x4_t, buffer_load16(b, lane_off, off));
}
__device__ __forceinline__ void buffer_store4(bf16x4_t v, buffer_t b, uint32_t lane_off, uint32_t off) {
    buffer_store8(b, lane_off, off, __builtin_bit_cast(u32x2_t, v));
}
__device__ __forceinline__ void buffer_store4(f32x4_t v, buffer_t b, uint32_t lane_off, uint32_t off) {
    buffer_store16(b, lane_off, off, __builtin_bit_cast(u32x4_t, v));
}

}  // namespace kda
