// kda_tile.hpp -- matrix products, token tiles in LDS and transfers into them, shared by the chunked passes of
// linear attention and of the selective scan.
#pragma once

#include "kda_chunk_util.hpp"

namespace kda {
namespace {

// Segments of sequences.  A launch description L_t has cu (packed offsets or nullptr), T, n_seqs, seg (tokens of a
// segment) and n_seg (segments of a fixed-length sequence); slot numbers as its file defines them.
struct Where {
    int32_t n, s, n_seg;     // sequence, segment, segments of the sequence
    int64_t lo, hi;          // tokens of the segment
};
template <typename L_t>
__device__ __forceinline__ void seq_range(const L_t& L, int32_t n, int64_t& lo, int64_t& hi) {
    if (L.cu == nullptr) {
        lo = n * L.T;
        hi = lo + L.T;
    } else {
        const int64_t x = L.cu[n], y = L.cu[n + 1];
        lo = x < 0 ? 0 : (x > L.T ? L.T : x);
        hi = y < lo ? lo : (y > L.T ? L.T : y);
    }
}
template <typename L_t>
__device__ __forceinline__ int32_t first_slot(const L_t& L, int32_t n) {
    int64_t lo, hi;
    seq_range(L, n, lo, hi);
    return static_cast<int32_t>(static_cast<uint32_t>(lo) / static_cast<uint32_t>(L.seg)) + n;
}
template <typename L_t>
__device__ __forceinline__ int32_t segments(const L_t& L, int64_t len) {
    if (L.cu == nullptr) return L.n_seg;
    return len <= L.seg ? 1 : static_cast<int32_t>((static_cast<uint32_t>(len) - 1u) / static_cast<uint32_t>(L.seg)) + 1;
}
template <typename L_t>
__device__ __forceinline__ bool locate(const L_t& L, int32_t slot, Where& w) {
    int64_t lo, hi;
    if (L.cu == nullptr) {
        w.n = slot / L.n_seg;
        w.s = slot - w.n * L.n_seg;
        seq_range(L, w.n, lo, hi);
    } else {
        int32_t a = 0, b = L.n_seqs - 1;          // the last sequence whose first slot is <= slot
        while (a < b) {
            const int32_t m = (a + b + 1) / 2;
            if (first_slot(L, m) <= slot) a = m; else b = m - 1;
        }
        w.n = a;
        w.s = slot - first_slot(L, a);
        seq_range(L, a, lo, hi);
    }
    w.n_seg = segments(L, hi - lo);
    if (w.s < 0 || w.s >= w.n_seg) return false;
    w.lo = lo + static_cast<int64_t>(w.s) * L.seg;
    w.hi = w.s == w.n_seg - 1 ? hi : w.lo + L.seg;
    return true;
}

__device__ __forceinline__ f32x4 mfma_bf16(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                   0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma_f32(float a, float b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}
// Two floats as bf16 (nearest even), x in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float x, float y) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{x, y}, bf16x2));
}
__device__ __forceinline__ float lo_f32(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f32(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
// Three bf16 terms, each a truncation: 24 bits, exact.
__device__ __forceinline__ void split3(float x, float y, uint32_t& h, uint32_t& m, uint32_t& l) {
    const uint32_t ux = __float_as_uint(x), uy = __float_as_uint(y);
    h = __builtin_amdgcn_perm(uy, ux, 0x07060302u);
    const float x1 = x - hi_f32(ux), y1 = y - hi_f32(uy);
    const uint32_t ux1 = __float_as_uint(x1), uy1 = __float_as_uint(y1);
    m = __builtin_amdgcn_perm(uy1, ux1, 0x07060302u);
    const float x2 = x1 - hi_f32(ux1), y2 = y1 - hi_f32(uy1);
    l = __builtin_amdgcn_perm(__float_as_uint(y2), __float_as_uint(x2), 0x07060302u);
}

// x times f, with f as hi + lo: a state that goes from call to call would otherwise take the rounding of f
// along each time, the same way (10000 pieces of a prompt that each decay by 1e-3: the state off by 3.0e-4 of
// itself with f as one fp32 number, by 1.3e-6 so).
__device__ __forceinline__ f32x4 times(f32x4 x, double f) {
    const float hi = static_cast<float>(f), lo = static_cast<float>(f - static_cast<double>(hi));
#pragma unroll
    for (int r = 0; r < 4; ++r) x[r] = __builtin_fmaf(x[r], hi, x[r] * lo);
    return x;
}

template <typename T>
__device__ __forceinline__ T lds_get(const void* sm, uint32_t byte) {
    typedef T __attribute__((may_alias)) T_ma;
    return *reinterpret_cast<const T_ma*>(static_cast<const uint8_t*>(sm) + byte);
}
template <typename T>
__device__ __forceinline__ void lds_put(void* sm, uint32_t byte, T x) {
    typedef T __attribute__((may_alias)) T_ma;
    *reinterpret_cast<T_ma*>(static_cast<uint8_t*>(sm) + byte) = x;
}
// The transposing read gives lane i of each 16 channel i of the 4 tokens whose 8-byte pieces the lanes
// point at (lane 4 r + s: token r, channels 4 s .. 4 s + 3).
__device__ __forceinline__ u32x2 lds_transpose(const uint8_t* sm) {
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)sm));
}
// Workgroup barrier for LDS: this wave's LDS accesses are done; loads and stores may stay in flight (a
// __syncthreads would wait for them).
__device__ __forceinline__ void lds_barrier() {
    wave_fence();
    __builtin_amdgcn_s_waitcnt(0xC07F);              // lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    wave_fence();
}

// A tile of token rows in LDS.  A row's 16-byte units are XOR-ed with bits of the row inside groups of
// eight, and every 1 KB of rows (R of them) is followed by PAD bytes, such that
//   16 rows' equal units (operands along the channels) fill all 64 banks;
//   fp32: so do 4 neighbouring units of every fourth row (operands along the tokens);
//   16 bits: 8 rows' 4 neighbouring half units (transposing reads, half a wavefront at a time) fill half
//   of them, in two turns -- the halves of a unit cannot be told apart by a swizzle of whole units;
// while 16 tokens, and groups of eight units, stay a constant apart.
template <int DIM, int ES>
struct Tile {
    static constexpr int RB = DIM * ES, UPR = RB / 16, R = 1024 / RB;
    static constexpr int PAD = ES == 2 ? (R == 4 ? 128 : 0) : (R == 4 ? 64 : 32), PIECE = 1024 + PAD;
    static constexpr int ROWS16 = 16 / R * PIECE;
    static __device__ __forceinline__ int mix(int row) {
        if constexpr (ES == 2) return 2 * ((R == 4 ? row : row >> 1) & 3);
        else return row % R;
    }
    static __device__ __forceinline__ uint32_t at(int row, int unit) {
        return (row / R) * PIECE + (row % R) * RB + (unit & ~7) * 16 + ((unit & 7) ^ mix(row)) * 16;
    }
};

// 16 bytes per lane from a buffer to 1 KB of LDS.
__device__ __forceinline__ void transfer16(__amdgpu_buffer_rsrc_t r, uint32_t offset, uint8_t* sm) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)sm, 16, offset, 0, 0, 0);
}
// n rows, `row` bytes apart, straight into a tile, 1 KB per wave instruction; a lane's 16 bytes come from
// wherever the tile's layout wants them.  Rows past the n-th lie outside the buffer range and read as zeros
// (n = 0: all of them).
template <typename TT, int TOK, int WAVES>
__device__ __forceinline__ void fetch_rows(uint8_t* sm, const void* first, uint32_t row, int n, int wave, int lane) {
    const __amdgpu_buffer_rsrc_t r = make_rsrc_u(first, n > 0 ? (n - 1) * row + TT::RB : 0);
    const int r0 = wave * TT::R + lane / TT::UPR, un = lane % TT::UPR;     // WAVES R rows on: the same units
    const uint32_t at = r0 * row + ((un & ~7) | ((un & 7) ^ TT::mix(r0))) * 16;
#pragma unroll
    for (int i = 0; i < TOK / TT::R / WAVES; ++i)
        transfer16(r, at + WAVES * i * TT::R * row, sm + TT::PIECE * (WAVES * i + wave));
}

// The groups (token tile it, 32 tokens tg) of scores on the near side of the diagonal, 0 .. 5.
template <bool BACK>
__device__ __forceinline__ constexpr int score_group(int it, int tg) {
    if (BACK) return tg == 1 ? it : 4 + it;          // group 1: tiles 0 .. 3, group 0: tiles 0, 1
    return tg == 0 ? it : 2 + it;                    // group 0: tiles 0 .. 3, group 1: tiles 2, 3
}

}  // namespace
}  // namespace kda
