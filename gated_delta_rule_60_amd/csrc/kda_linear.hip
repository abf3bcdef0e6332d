// kda_linear.hip -- linear attention with one decay per head: prefill, gradients, decode step.
//
// Every output is one and the same pass over a sequence, with roles a (query), b (key), c (value) and
// a state M [DA, DC] (fp32):
//     forward in time:   M <- lam M + ub b_t c_t^T,  out_t = so M^T a_t
//     backward in time:  G = M + ub b_t c_t^T,       out_t = so G^T a_t,  M <- lam G
//   o  : a = q,  b = k,  c = v, forward,  so = scale, M from the initial state, to the final state
//   dq : a = do, b = v,  c = k, forward,  so = scale, M from the initial state transposed
//   dk : a = v,  b = do, c = q, backward, ub = scale, M from the final state's gradient transposed
//   dv : a = k,  b = q,  c = do, backward, ub = scale, M from the final state's gradient, to the
//        initial state's gradient
#include "kda_chunk_util.hpp"
#include "kda_linear.hpp"

#include <algorithm>
#include <type_traits>

namespace kda {
namespace {

struct Pass {
    const void *a, *b, *c;
    void* out;
    const float* m_in;       // [N, H, DA, DC], or [N, H, DC, DA] with m_transposed; nullptr = zeros
    float* m_out;            // [N, H, DA, DC] or nullptr
    float* seg_states;       // [slots, H, DA, DC] (or transposed); nullptr: whole sequences
    float so, ub;
    int32_t back;            // backward in time
    int32_t m_transposed;    // m_in and seg_states are
    int32_t exact;           // the segment states end in a state that is handed out
};
constexpr int MAX_PASSES = 3;

// A launch covers (sequence, segment) slots times heads times passes.  A segment is `seg` tokens.
// Fixed-length batches: n_seg slots per sequence; packed ones: slot floor(cu[n] / seg) + n + s for
// segment s of sequence n, which leaves unused slots between sequences.
struct Launch {
    Pass pass[MAX_PASSES];
    const float* g;
    const int32_t* cu;
    int64_t T;
    int32_t n_seqs, H, slots;
    int32_t seg;             // WHOLE: whole sequences
    int32_t n_seg;           // of a fixed-length sequence
    int32_t passes;
};
constexpr int32_t WHOLE = 0x7fffffff;

struct Where {
    int32_t n, s, n_seg;     // sequence, segment, segments of the sequence
    int64_t lo, hi;          // tokens of the segment
};
__device__ __forceinline__ void seq_range(const Launch& L, int32_t n, int64_t& lo, int64_t& hi) {
    if (L.cu == nullptr) {
        lo = n * L.T;
        hi = lo + L.T;
    } else {
        const int64_t x = L.cu[n], y = L.cu[n + 1];
        lo = x < 0 ? 0 : (x > L.T ? L.T : x);
        hi = y < lo ? lo : (y > L.T ? L.T : y);
    }
}
__device__ __forceinline__ int32_t first_slot(const Launch& L, int32_t n) {
    int64_t lo, hi;
    seq_range(L, n, lo, hi);
    return static_cast<int32_t>(static_cast<uint32_t>(lo) / static_cast<uint32_t>(L.seg)) + n;
}
__device__ __forceinline__ int32_t segments(const Launch& L, int64_t len) {
    if (L.cu == nullptr) return L.n_seg;
    return len <= L.seg ? 1 : static_cast<int32_t>((static_cast<uint32_t>(len) - 1u) / static_cast<uint32_t>(L.seg)) + 1;
}
__device__ __forceinline__ bool locate(const Launch& L, int32_t slot, Where& w) {
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
// A chunk's rows of one head (n tokens from tok0) straight into a tile, 1 KB per wave instruction; a
// lane's 16 bytes come from wherever the tile's layout wants them.  Rows past the n-th lie outside the
// buffer range and read as zeros.
template <typename TT, int TOK, int WAVES>
__device__ __forceinline__ void fetch_tile(uint8_t* sm, const void* base, int64_t tok0, int n, int32_t H, int32_t h,
                                           int wave, int lane) {
    const uint32_t row = static_cast<uint32_t>(H) * TT::RB;
    const __amdgpu_buffer_rsrc_t r = make_rsrc_u(static_cast<const uint8_t*>(base) + (tok0 * H + h) * TT::RB,
                                                 (n - 1) * row + TT::RB);
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

// The workgroup's LDS.
template <int DT, int DA, int DC, bool STATE_ONLY>
struct ChunkLds {
    static constexpr int ES = DT == KDA_BF16 ? 2 : 4, TOK = DT == KDA_BF16 ? 64 : 32;
    using TA = Tile<DA, ES>;
    using TC = Tile<DC, ES>;
    __align__(16) uint8_t b[TOK / TA::R * TA::PIECE];
    __align__(16) uint8_t c[TOK / TC::R * TC::PIECE];
    __align__(16) uint8_t a[STATE_ONLY ? 16 : TOK / TA::R * TA::PIECE];
    // scores: 16-bit hi and lo operands per group, or fp32 tiles
    __align__(16) uint8_t p[STATE_ONLY ? 16 : (ES == 2 ? 12 : 3) * 1024];
    __align__(16) float rd[TOK];                     // decays of the state's part and of the update
    __align__(16) float up[TOK];
    // so ub lam^(i-j) of a lane's scores: tile on the diagonal (masked), tile next to it
    f32x4 on_diag[STATE_ONLY ? 1 : 64], next[STATE_ONLY ? 1 : 64];
    double lam[TOK + 1];
    double lam_n_inv;                                // of the chunk's length
};

// The pass in chunks of TOK tokens; one workgroup per (segment, head), wave w with the output columns
// 16 w .. 16 w + 15.  With lam^p = e^(p g), i and j tokens of a chunk of n:
//     out_i = so lam^(i+1) M^T a_i + so ub sum_{j <= i} lam^(i-j) (b_j . a_i) c_j,
//     M    <- lam^n M + ub sum_j lam^(n-1-j) b_j c_j^T                         (forward; backward:
//     j >= i, lam^(j-i), lam^(n-1-i) for the state's part and lam^(j+1) for the update).
// All products are MFMAs computed transposed (out^T = M^T a^T, scores^T = b a^T), which makes every
// accumulator the next product's operand without a shuffle: an accumulator holds four neighbouring rows
// per lane, and an operand wants eight (fp32: one) values along the contraction per lane -- any, as
// long as both operands take the same ones.  So M's tiles feed out^T = M^T a^T from the registers that
// M = b^T c left them in, and the scores likewise (through LDS, since all waves need all scores).  The
// decays multiply accumulators (fp32) where they can; only the update's sits inside a contraction, on c.
//   16-bit inputs: M and the scores are read as two bf16 terms (2^-16); the decayed c as three (exact)
//   where M ends in a state that is handed out in fp32, as two where it only feeds 16-bit outputs.
//   fp32 inputs: 16x16x4 fp32 MFMAs throughout.
//   16-bit outputs leave through LDS as whole rows past the caches (4 x 4096 x 16 heads, the same inputs over
//   and over: 67 us for the pass, 73 us with each wave's 32-byte pieces stored as they are).
// One workgroup's transfers run under another's products.  16-bit inputs, on a CU: DA x DC = 128 x 128 two
// workgroups of eight waves (128 registers, 69 KB of LDS each), 64 x 128 two (49 KB), 64 x 64 four of four
// waves (39 KB), 128 x 64 two of four (59 KB, more than 128 registers).
// STATE_ONLY: just M from zero, the segment's own contribution.
template <int DT, int ODT, int DA, int DC, bool BACK, bool STATE_ONLY>
__device__ __forceinline__ void chunk_pass(const Launch& L, const Pass& p, int32_t slot, int32_t h,
                                           ChunkLds<DT, DA, DC, STATE_ONLY>& lds) {
    using Lds = ChunkLds<DT, DA, DC, STATE_ONLY>;
    using TA = typename Lds::TA;
    using TC = typename Lds::TC;
    constexpr bool BF = DT == KDA_BF16;
    constexpr int TOK = Lds::TOK, WAVES = DC / 16;
    constexpr int IT = TOK / 16, MT = DA / 16;       // token tiles, state row tiles
    constexpr int KK = DA / 32, JG = TOK / 32;       // 16 bits: contraction steps over channels, tokens
    constexpr int OS = ODT == KDA_BF16 ? 2 : 4;
    constexpr bool STAGED = BF && OS == 2 && !STATE_ONLY;

    Where w;
    if (!locate(L, slot, w)) return;
    if (STATE_ONLY && w.s == (BACK ? 0 : w.n_seg - 1)) return;    // nothing follows it
    const int t = threadIdx.x, lane = t & 63, q = lane >> 4, l16 = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int64_t len = w.hi - w.lo;
    const int n_chunks = static_cast<int>((len + TOK - 1) / TOK);
    const int64_t unit = static_cast<int64_t>(w.n) * L.H + h;

    auto load_ab = [&](int c) {
        const int64_t off = static_cast<int64_t>(BACK ? n_chunks - 1 - c : c) * TOK;
        const int n = static_cast<int>(len - off < TOK ? len - off : TOK);
        fetch_tile<TA, TOK, WAVES>(lds.b, p.b, w.lo + off, n, L.H, h, wave, lane);
        if constexpr (!STATE_ONLY) fetch_tile<TA, TOK, WAVES>(lds.a, p.a, w.lo + off, n, L.H, h, wave, lane);
    };
    auto load_c = [&](int c) {
        const int64_t off = static_cast<int64_t>(BACK ? n_chunks - 1 - c : c) * TOK;
        const int n = static_cast<int>(len - off < TOK ? len - off : TOK);
        fetch_tile<TC, TOK, WAVES>(lds.c, p.c, w.lo + off, n, L.H, h, wave, lane);
    };
    if (n_chunks > 0) {
        load_ab(0);
        load_c(0);
    }

    // ---- the state: tile mt, register r of lane (l16, q) holds row row(mt) + r, column 16 wave + l16
    auto row = [&](int mt) { return BF ? 32 * (mt >> 1) + 8 * q + 4 * (mt & 1) : 16 * mt + 4 * q; };
    const int col = 16 * wave + l16;
    f32x4 M[MT];
    {
        const float* src = nullptr;                  // none: an empty range, which reads as zeros
        if constexpr (!STATE_ONLY) {
            // (the first segment too: its initial state may be the final state the last one writes)
            if (w.n_seg > 1) src = p.seg_states + (static_cast<int64_t>(slot) * L.H + h) * (DA * DC);
            else if (p.m_in) src = p.m_in + unit * (DA * DC);
        }
        const __amdgpu_buffer_rsrc_t rs = make_rsrc_u(src, src ? DA * DC * 4 : 0);
        if (p.m_transposed) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
                M[mt] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, (col * DA + row(mt)) * 4, 0, 0));
        } else {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    M[mt][r] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, ((row(mt) + r) * DC + col) * 4, 0, 0));
        }
    }

    // ---- decays lam^p
    if (len > 0) {
        const double g = static_cast<double>(L.g[h]);
        if (t <= TOK) lds.lam[t] = t == 0 ? 1.0 : exp(t * g);
    }
    lds_barrier();
    if constexpr (!STATE_ONLY) {
        if (len > 0 && t < 64) {
            f32x4 d, e;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int x = BACK ? 4 * q + r - l16 : l16 - 4 * q - r;
                d[r] = x < 0 ? 0.f : p.so * p.ub * static_cast<float>(lds.lam[x < 0 ? 0 : x]);
                e[r] = p.so * p.ub * static_cast<float>(lds.lam[16 + x]);
            }
            lds.on_diag[lane] = d;
            lds.next[lane] = e;
        }
    }

    // ---- operands' byte offsets.  16 bits, along the channels: channels 32 kk + 8 q .. + 7 of token
    // 16 it + l16; along the tokens: tokens 32 tg + 4 q .. + 3 and 32 tg + 16 + 4 q .. + 3, of state row
    // tile mt's rows (channels 32 (mt / 2) + 8 s + 4 (mt % 2) .. + 3 in piece s) or of the wave's columns.
    uint32_t chan[2], tok[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        chan[x] = TA::at(l16, 4 * x + q);
        tok[x] = TA::at(4 * q + (l16 >> 2), 4 * x + (l16 & 3));
    }
    const uint32_t tok_c = TC::at(4 * q + (l16 >> 2), 2 * wave + ((l16 & 3) >> 1)) + 8 * (l16 & 1);
    auto channels = [&](const uint8_t* sm, int it, int kk) {
        return lds_get<u32x4>(sm, chan[kk & 1] + it * TA::ROWS16 + (kk >> 1) * 128);
    };
    auto tokens = [&](uint32_t at, const uint8_t* sm, int rows16) {
        const u32x2 x = lds_transpose(sm + at), y = lds_transpose(sm + at + rows16);
        return u32x4{x[0], x[1], y[0], y[1]};
    };

    // The state is held as f times the registers, so that most chunks need not multiply it; f and 1 / f
    // are fp64, and the registers take f over before it leaves [2^-12, 2^12] (rounded to fp32: not more often
    // than every eight e-foldings).
    double f = 1.0, f_inv = 1.0;
    const bool exact = STATE_ONLY ? p.exact != 0 : p.m_out && w.s == (BACK ? 0 : w.n_seg - 1);
    int table_n = -1;
    for (int c = 0; c < n_chunks; ++c) {
        const int64_t off = static_cast<int64_t>(BACK ? n_chunks - 1 - c : c) * TOK;
        const int64_t tok0 = w.lo + off;
        const int n = static_cast<int>(len - off < TOK ? len - off : TOK);
        if (n != table_n) {
            table_n = n;
            if (t == TOK) lds.lam_n_inv = 1.0 / lds.lam[n];
            if (t < TOK) {
                const int from_end = n - 1 - t;
                lds.rd[t] = p.so * static_cast<float>(lds.lam[BACK ? (from_end < 0 ? 0 : from_end) : t + 1]);
                lds.up[t] = p.ub * static_cast<float>(lds.lam[BACK ? t + 1 : (from_end < 0 ? 0 : from_end)]);
            }
        }
        __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
        lds_barrier();                               // the tiles are there

        f32x4 O[IT];
        if constexpr (!STATE_ONLY) {
            // ---- scores, shared out over the waves
            if constexpr (BF) {
                for (int grp = wave; grp < 6; grp += WAVES) {
                    // (it, tg) with score_group(it, tg) == grp
                    const int tg = BACK ? (grp < 4) : (grp >= 4), it = BACK ? (grp & 3) : (grp < 4 ? grp : grp - 2);
                    u32x4 hi, lo;
                    f32x4 P[2] = {zero4(), zero4()};
#pragma unroll
                    for (int kk = 0; kk < KK; ++kk) {
                        const u32x4 a = channels(lds.a, it, kk);
#pragma unroll
                        for (int hh = 0; hh < 2; ++hh) P[hh] = mfma_bf16(channels(lds.b, 2 * tg + hh, kk), a, P[hh]);
                    }
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
                        const int jt = 2 * tg + hh, dist = BACK ? jt - it : it - jt;
                        if (dist < 0) P[hh] = zero4();
                        else if (dist == 0) P[hh] *= lds.on_diag[lane];
                        else P[hh] *= lds.next[lane] * static_cast<float>(lds.lam[16 * (dist - 1)]);
                        uint32_t h0, o0, h1, o1;
                        split_pair(P[hh][0], P[hh][1], h0, o0);
                        split_pair(P[hh][2], P[hh][3], h1, o1);
                        hi[2 * hh] = h0; hi[2 * hh + 1] = h1;
                        lo[2 * hh] = o0; lo[2 * hh + 1] = o1;
                    }
                    lds_put(lds.p, grp * 2048 + lane * 16, hi);
                    lds_put(lds.p, grp * 2048 + 1024 + lane * 16, lo);
                }
            } else if (wave < 3) {
                // tiles (out, in): (0, 0), (1, 1) and (1, 0), backward (0, 1)
                const int it = BACK ? (wave == 1) : (wave > 0), jt = BACK ? (wave > 0) : (wave == 1);
                f32x4 P = zero4();
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    const f32x4 a = lds_get<f32x4>(lds.a, TA::at(16 * it + l16, 4 * mt + q));
                    const f32x4 b = lds_get<f32x4>(lds.b, TA::at(16 * jt + l16, 4 * mt + q));
#pragma unroll
                    for (int r = 0; r < 4; ++r) P = mfma_f32(b[r], a[r], P);
                }
                P *= wave < 2 ? lds.on_diag[lane] : lds.next[lane];
                lds_put(lds.p, wave * 1024 + lane * 16, P);
            }
            // ---- the state's part
#pragma unroll
            for (int it = 0; it < IT; ++it) O[it] = zero4();
            if constexpr (BF) {
#pragma unroll
                for (int kk = 0; kk < KK; ++kk) {
                    u32x4 hi, lo, a[IT];
#pragma unroll
                    for (int it = 0; it < IT; ++it) a[it] = channels(lds.a, it, kk);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const f32x4& m = M[2 * kk + (e >> 1)];
                        uint32_t x, y;
                        split_pair(m[2 * (e & 1)], m[2 * (e & 1) + 1], x, y);
                        hi[e] = x;
                        lo[e] = y;
                    }
#pragma unroll
                    for (int it = 0; it < IT; ++it) O[it] = mfma_bf16(hi, a[it], O[it]);
#pragma unroll
                    for (int it = 0; it < IT; ++it) O[it] = mfma_bf16(lo, a[it], O[it]);
                }
            } else {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int it = 0; it < IT; ++it) {
                        const f32x4 a = lds_get<f32x4>(lds.a, TA::at(16 * it + l16, 4 * mt + q));
#pragma unroll
                        for (int r = 0; r < 4; ++r) O[it] = mfma_f32(M[mt][r], a[r], O[it]);
                    }
            }
            const float ff = static_cast<float>(f);
#pragma unroll
            for (int it = 0; it < IT; ++it) O[it] *= lds.rd[16 * it + l16] * ff;
        }
        // ---- decay
        const double fn = f * lds.lam[n];
        if (fn >= 0x1p-12 && fn <= 0x1p12) {
            f = fn;
            f_inv *= lds.lam_n_inv;
        } else {
            const float x = static_cast<float>(fn);
            f = f_inv = 1.0;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) M[mt] *= x;
        }
        const float up_scale = static_cast<float>(f_inv);

        // ---- c along the tokens
        constexpr int CJ = BF ? JG : IT;
        u32x4 vf[CJ];
#pragma unroll
        for (int j = 0; j < CJ; ++j) {
            if constexpr (BF) vf[j] = tokens(tok_c + 2 * j * TC::ROWS16, lds.c, TC::ROWS16);
            else
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    vf[j][r] = lds_get<uint32_t>(lds.c, TC::at(16 * j + 4 * q + r, 4 * wave + (l16 >> 2)) + 4 * (l16 & 3));
        }
        if constexpr (!STATE_ONLY) {
            lds_barrier();                           // the scores are there
            if constexpr (BF) {
#pragma unroll
                for (int it = 0; it < IT; ++it)
#pragma unroll
                    for (int tg = 0; tg < JG; ++tg) {
                        if (BACK ? 2 * tg + 1 < it : 2 * tg > it) continue;
                        const uint32_t at = score_group<BACK>(it, tg) * 2048 + lane * 16;
                        O[it] = mfma_bf16(vf[tg], lds_get<u32x4>(lds.p, at), O[it]);
                        O[it] = mfma_bf16(vf[tg], lds_get<u32x4>(lds.p, at + 1024), O[it]);
                    }
            } else {
#pragma unroll
                for (int tile = 0; tile < 3; ++tile) {
                    const int it = BACK ? (tile == 1) : (tile > 0), jt = BACK ? (tile > 0) : (tile == 1);
                    const f32x4 P = lds_get<f32x4>(lds.p, tile * 1024 + lane * 16);
#pragma unroll
                    for (int r = 0; r < 4; ++r) O[it] = mfma_f32(__uint_as_float(vf[jt][r]), P[r], O[it]);
                }
            }
            // ---- out, through c's tile (which all waves have read by now): lane l16 holds token 16 it + l16,
            // four neighbouring columns
            if constexpr (STAGED) {
                int ll = l16;
                asm volatile("" : "+v"(ll));
#pragma unroll
                for (int it = 0; it < IT; ++it)
                    lds_put(lds.c, TC::at(16 * it + ll, 2 * wave + (q >> 1)) + 8 * (q & 1),
                            u32x2{pack_bf16(O[it][0], O[it][1]), pack_bf16(O[it][2], O[it][3])});
            } else {
                const uint32_t orow = static_cast<uint32_t>(L.H) * DC * OS;
                const __amdgpu_buffer_rsrc_t ro = make_rsrc_u(static_cast<uint8_t*>(p.out) + (tok0 * L.H + h) * DC * OS,
                                                              (n - 1) * orow + DC * OS);
#pragma unroll
                for (int it = 0; it < IT; ++it) {
                    const uint32_t at = (16 * it + l16) * orow + (16 * wave + 4 * q) * OS;
                    if constexpr (ODT == KDA_BF16)
                        __builtin_amdgcn_raw_buffer_store_b64(u32x2{pack_bf16(O[it][0], O[it][1]), pack_bf16(O[it][2], O[it][3])},
                                                              ro, at, 0, 0);
                    else __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, O[it]), ro, at, 0, 0);
                }
            }
        }
        // ---- update
        if constexpr (BF) {
            // the decayed c in three terms (exact) where the state leaves in fp32, else in two
            auto update = [&](auto three) {
                constexpr bool THREE = decltype(three)::value;
#pragma unroll
                for (int tg = 0; tg < JG; ++tg) {
                    const f32x4 w0 = lds_get<f32x4>(lds.up, 4 * (32 * tg + 4 * q)) * up_scale;
                    const f32x4 w1 = lds_get<f32x4>(lds.up, 4 * (32 * tg + 16 + 4 * q)) * up_scale;
                    u32x4 ch, cm, cl;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const f32x4& ww = e < 2 ? w0 : w1;
                        const float c0 = lo_f32(vf[tg][e]) * ww[2 * (e & 1)], c1 = hi_f32(vf[tg][e]) * ww[2 * (e & 1) + 1];
                        uint32_t x, y, z = 0;
                        if constexpr (THREE) split3(c0, c1, x, y, z);
                        else split_pair(c0, c1, x, y);
                        ch[e] = x;
                        cm[e] = y;
                        cl[e] = z;
                    }
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        const u32x4 kt = tokens(tok[(mt >> 1) & 1] + 2 * tg * TA::ROWS16 + (mt >> 2) * 128 + 8 * (mt & 1), lds.b,
                                                TA::ROWS16);
                        if constexpr (THREE) M[mt] = mfma_bf16(kt, cl, M[mt]);
                        M[mt] = mfma_bf16(kt, cm, M[mt]);
                        M[mt] = mfma_bf16(kt, ch, M[mt]);
                    }
                }
            };
            if (exact) update(std::true_type{});
            else update(std::false_type{});
        } else {
#pragma unroll
            for (int jt = 0; jt < IT; ++jt) {
                const f32x4 ww = lds_get<f32x4>(lds.up, 4 * (16 * jt + 4 * q)) * up_scale;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float cw = __uint_as_float(vf[jt][r]) * ww[r];
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
                        M[mt] = mfma_f32(lds_get<float>(lds.b, TA::at(16 * jt + 4 * q + r, 4 * mt + (l16 >> 2)) + 4 * (l16 & 3)),
                                         cw, M[mt]);
                }
            }
        }
        lds_barrier();                               // the tiles have been read, the output is there
        if (c + 1 < n_chunks) load_ab(c + 1);
        if constexpr (STAGED) {
            const uint32_t orow = static_cast<uint32_t>(L.H) * DC * OS;
            const __amdgpu_buffer_rsrc_t ro = make_rsrc_u(static_cast<uint8_t*>(p.out) + (tok0 * L.H + h) * DC * OS,
                                                          (n - 1) * orow + DC * OS);
            int tt = t;                              // formed anew in each chunk: no registers over the loop
            asm volatile("" : "+v"(tt));
#pragma unroll
            for (int i = 0; i < TOK * TC::UPR / (64 * WAVES); ++i) {
                const int u = tt + 64 * WAVES * i, r = u / TC::UPR, un = u % TC::UPR;
                __builtin_amdgcn_raw_buffer_store_b128(lds_get<u32x4>(lds.c, TC::at(r, un)), ro, r * orow + un * 16, 0, CP_NT);
            }
            lds_barrier();                           // the output has been read
        }
        if (c + 1 < n_chunks) load_c(c + 1);
    }

    float* dst = nullptr;
    if constexpr (STATE_ONLY) dst = p.seg_states + (static_cast<int64_t>(slot) * L.H + h) * (DA * DC);
    else if (p.m_out && w.s == (BACK ? 0 : w.n_seg - 1)) dst = p.m_out + unit * (DA * DC);
    if (dst) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const f32x4 x = times(M[mt], f);
#pragma unroll
            for (int r = 0; r < 4; ++r) dst[(row(mt) + r) * DC + col] = x[r];
        }
    }
}

// Workgroups are handed to the 8 XCDs in turn, and each XCD has an L2 whose channels interleave by a few
// hundred bytes -- about one head's row.  So an XCD takes a contiguous range of (slot, head) units, heads
// fastest, which spreads its rows over all its channels (heads dealt out to the XCDs one by one would
// leave each XCD the same few channels of every token).  All passes of a unit follow one another there and
// share the L2's copies of its rows.
template <int DT, int ODT, int DA, int DC, bool STATE_ONLY>
__global__ void __launch_bounds__(DC * 4, DA > DC ? 2 : 4) linear_chunk_kernel(Launch L) {
    __shared__ ChunkLds<DT, DA, DC, STATE_ONLY> lds;
    const uint32_t units = static_cast<uint32_t>(L.slots) * L.H, per_xcd = (units + 7) / 8;
    const uint32_t j = blockIdx.x / 8, x = blockIdx.x % 8 * per_xcd + j / L.passes;
    if (j / L.passes >= per_xcd || x >= units) return;
    const int32_t slot = static_cast<int32_t>(x / L.H), h = static_cast<int32_t>(x % L.H);
    const Pass& p = L.pass[j % L.passes];
    if (p.back) chunk_pass<DT, ODT, DA, DC, true, STATE_ONLY>(L, p, slot, h, lds);
    else chunk_pass<DT, ODT, DA, DC, false, STATE_ONLY>(L, p, slot, h, lds);
}

// Segment states: from each segment's own contribution to the state it starts from, in place.  Grid
// (sequence * H + head, element blocks of 1024, pass); each lane carries four elements along, eight
// segments' loads at a time: 10.4 us for 4 x 4096 x 16 heads (8 segments of 64 KB each; the same inputs over
// and over), 11.3 us with one load at a time.
__global__ void __launch_bounds__(256) linear_scan_kernel(Launch L, int32_t elems) {
    const Pass& p = L.pass[blockIdx.z];
    const int32_t n = blockIdx.x / L.H, h = blockIdx.x % L.H;
    const int32_t e = blockIdx.y * 1024 + threadIdx.x * 4;
    int64_t lo, hi;
    seq_range(L, n, lo, hi);
    const int64_t len = hi - lo;
    const int32_t n_seg = segments(L, len);
    if (n_seg == 1) return;
    const int32_t first = L.cu ? first_slot(L, n) : n * n_seg;
    const double g = static_cast<double>(L.g[h]);
    f32x4 x = zero4();
    if (p.m_in) x = *reinterpret_cast<const f32x4*>(p.m_in + (static_cast<int64_t>(n) * L.H + h) * elems + e);
    float* at = p.seg_states + (static_cast<int64_t>(first) * L.H + h) * elems + e;
    const int64_t step = static_cast<int64_t>(L.H) * elems;
    // decay over a segment as hi + lo: its rounding would act the same way segment after segment
    const int64_t part = len - static_cast<int64_t>(n_seg - 1) * L.seg;
    const double full = exp(static_cast<double>(L.seg) * g), last = exp(static_cast<double>(part) * g);
    auto slot = [&](int32_t i) { return reinterpret_cast<f32x4*>(at + (p.back ? n_seg - 1 - i : i) * step); };
    f32x4 ahead = *slot(0);                       // read before the batch before it writes its place
    *slot(0) = x;
    for (int32_t i0 = 0; i0 < n_seg - 1; i0 += 8) {
        f32x4 own[9];
        own[0] = ahead;
#pragma unroll
        for (int32_t j = 1; j < 9; ++j) own[j] = i0 + j < n_seg - 1 ? *slot(i0 + j) : zero4();
        ahead = own[8];
#pragma unroll
        for (int32_t j = 0; j < 8; ++j) {
            if (i0 + j >= n_seg - 1) break;
            const double l = p.back && i0 + j == 0 ? last : full;     // only the last segment may be shorter
            const float l_hi = static_cast<float>(l), l_lo = static_cast<float>(l - static_cast<double>(l_hi));
#pragma unroll
            for (int r = 0; r < 4; ++r) x[r] = __builtin_fmaf(x[r], l_hi, __builtin_fmaf(x[r], l_lo, own[j][r]));
            *slot(i0 + j + 1) = x;                // segment i's end is what segment i + 1 starts from
        }
    }
}

// ---------------------------------------------------------------- host side

// Tokens per segment, a multiple of 64 (figures: bf16, d = 128 unless said otherwise).
//   Whole sequences from 256 (sequence, head) units on: every CU has a workgroup.  Right for sequences of about
//   one length: 16 x 4096 tokens x 16 heads 348 us whole, 371 us in two segments each (gradients 763, 881);
//   packed 8 x 8192 x 32 heads 664 us, 1033 us in segments of 8192 by all tokens (gradients 1573, 2225).  Wrong
//   for a packed batch of that many units where one sequence holds most tokens -- the lengths are on the device:
//   8 sequences x 32 heads, one of 55702 of the 65536 tokens, 4028 us whole, 1418 us in segments of 8192
//   (gradients 8456, 2910); the same tokens as one sequence take 777 us.
//   Whole, too, below 1024 tokens (of a packed batch: in all).  A call is one launch then, and needs no
//   workspace, but from 500 tokens on (fp32: from fewer) it is slower than three launches: 500 x 8 heads 32.5 us
//   whole, 32.7 in segments, 1000 x 8 59.8 and 33.7, fp32 89 and 45, 174 and 47.  Gradients of 4 x 1000 x 16
//   gain (68.5 and 76.0, fp32 186 and 208).
//   Else segments for two workgroups a CU, in one round: 512 in all, a few fewer for a packed batch, whose
//   sequences each end in a short one (65536 tokens x 33 heads: 796 us, in 528 segments 1033 us).  No shorter
//   than 256 tokens (fp32, whose chunks take longer: 128), so that a segment's state, read and written about
//   four times, stays small against its rows (16384 x 4 heads, d = 64: 46 us with 256, 62 us with 128).
int32_t segment_tokens(int32_t n_seqs, int64_t total, int32_t H, int32_t in_dtype, bool packed) {
    const int64_t units = int64_t(n_seqs) * H, longest = packed ? total : total / n_seqs;
    if (units >= 256 || longest < 1024) return WHOLE;
    const int64_t shares = packed ? std::max<int64_t>(1, 512 / H - n_seqs / 2) : 512 / units;   // of `longest`
    const int64_t seg = std::max<int64_t>(((longest + shares - 1) / shares + 63) / 64 * 64, in_dtype == KDA_BF16 ? 256 : 128);
    return seg >= longest || seg >= WHOLE ? WHOLE : static_cast<int32_t>(seg);
}
int64_t segment_slots(int32_t n_seqs, int64_t total, int32_t seg, bool packed) {
    if (packed) return total / seg + n_seqs;
    return seg == WHOLE ? n_seqs : n_seqs * ((total / n_seqs + seg - 1) / seg);
}

template <int DT, int ODT, bool STATE_ONLY>
hipError_t launch_chunks(const Launch& L, int32_t da, int32_t dc, hipStream_t stream) {
    const int64_t groups = (int64_t(L.slots) * L.H + 7) / 8;
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(groups * 8 * L.passes)), dim3(dc * 4), 0, stream, L);
        return hipGetLastError();
    };
    if (da == 128 && dc == 128) return go(linear_chunk_kernel<DT, ODT, 128, 128, STATE_ONLY>);
    if (da == 128) return go(linear_chunk_kernel<DT, ODT, 128, 64, STATE_ONLY>);
    if (dc == 128) return go(linear_chunk_kernel<DT, ODT, 64, 128, STATE_ONLY>);
    return go(linear_chunk_kernel<DT, ODT, 64, 64, STATE_ONLY>);
}
hipError_t launch_scan(const Launch& L, int32_t elems, hipStream_t stream) {
    const dim3 grid(static_cast<unsigned>(L.n_seqs * L.H), static_cast<unsigned>(elems / 1024), static_cast<unsigned>(L.passes));
    hipLaunchKernelGGL(linear_scan_kernel, grid, dim3(256), 0, stream, L, elems);
    return hipGetLastError();
}

Launch base_launch(const LinearArgs& a) {
    Launch L{};
    const int64_t total = int64_t(a.B) * a.T;
    L.g = a.g; L.cu = a.cu; L.T = a.T; L.n_seqs = a.n_seqs; L.H = a.H;
    L.seg = segment_tokens(a.n_seqs, total, a.H, a.in_dtype, a.cu != nullptr);
    L.slots = static_cast<int32_t>(segment_slots(a.n_seqs, total, L.seg, a.cu != nullptr));
    L.n_seg = L.slots / a.n_seqs;
    return L;
}
Pass make_pass(const void* a, const void* b, const void* c, void* out, bool back, float so, float ub,
               const float* m_in, bool transposed, float* m_out) {
    Pass p{};
    p.a = a; p.b = b; p.c = c; p.out = out; p.back = back; p.so = so; p.ub = ub; p.m_in = m_in;
    p.m_transposed = transposed; p.m_out = m_out;
    return p;
}

template <int DT, int ODT>
hipError_t forward(const LinearArgs& a, hipStream_t stream) {
    Launch L = base_launch(a);
    L.passes = 1;
    L.pass[0] = make_pass(a.q, a.k, a.v, a.o, false, a.scale, 1.f, a.h0, false, a.hT);
    if (L.seg < WHOLE) {
        L.pass[0].seg_states = static_cast<float*>(a.workspace);
        L.pass[0].exact = a.hT != nullptr;
        hipError_t e = launch_chunks<DT, DT, true>(L, a.dk, a.dv, stream);
        if (e == hipSuccess) e = launch_scan(L, a.dk * a.dv, stream);
        if (e != hipSuccess) return e;
    }
    return launch_chunks<DT, ODT, false>(L, a.dk, a.dv, stream);
}

template <int DT>
hipError_t backward(const LinearArgs& a, hipStream_t stream) {
    const Launch base = base_launch(a);
    Pass q = make_pass(a.d_o, a.v, a.k, a.dq, false, a.scale, 1.f, a.h0, true, nullptr);
    Pass k = make_pass(a.v, a.d_o, a.q, a.dkk, true, 1.f, a.scale, a.dhT, true, nullptr);
    Pass v = make_pass(a.k, a.q, a.d_o, a.dvv, true, 1.f, a.scale, a.dhT, false, a.dh0);
    hipError_t e = hipSuccess;
    if (base.seg < WHOLE) {
        // the forward states (b = k, c = v) and their gradients (b = q, c = do)
        Launch L = base;
        L.passes = 2;
        L.pass[0] = make_pass(nullptr, a.k, a.v, nullptr, false, 1.f, 1.f, a.h0, false, nullptr);
        L.pass[1] = v;
        L.pass[1].exact = a.dh0 != nullptr;
        L.pass[0].seg_states = q.seg_states = static_cast<float*>(a.workspace);
        L.pass[1].seg_states = k.seg_states = v.seg_states =
            static_cast<float*>(a.workspace) + int64_t(L.slots) * a.H * a.dk * a.dv;
        e = launch_chunks<DT, DT, true>(L, a.dk, a.dv, stream);
        if (e == hipSuccess) e = launch_scan(L, a.dk * a.dv, stream);
    }
    Launch L = base;
    L.pass[0] = q; L.pass[1] = k; L.pass[2] = v;
    L.passes = a.dk == a.dv ? 3 : 2;
    if (e == hipSuccess) e = launch_chunks<DT, DT, false>(L, a.dv, a.dk, stream);
    if (a.dk != a.dv) {
        L.pass[0] = v;
        L.passes = 1;
        if (e == hipSuccess) e = launch_chunks<DT, DT, false>(L, a.dk, a.dv, stream);
    }
    return e;
}

}  // namespace

size_t linear_workspace_bytes(int32_t n_seqs, int64_t total, int32_t H, int32_t dk, int32_t dv,
                              int32_t in_dtype, bool backward) {
    // what a packed batch of these sizes needs, or fixed-length sequences: whichever is more
    int64_t slots = 0;
    for (const bool packed : {false, true}) {
        const int32_t seg = segment_tokens(n_seqs, total, H, in_dtype, packed);
        if (seg < WHOLE) slots = std::max(slots, segment_slots(n_seqs, total, seg, packed));
    }
    return static_cast<size_t>(slots) * H * dk * dv * 4 * (backward ? 2 : 1);
}

hipError_t launch_linear_fwd(const LinearArgs& a, hipStream_t stream) {
    if (a.in_dtype == KDA_BF16)
        return a.o_dtype == KDA_BF16 ? forward<KDA_BF16, KDA_BF16>(a, stream) : forward<KDA_BF16, KDA_F32>(a, stream);
    return a.o_dtype == KDA_BF16 ? forward<KDA_F32, KDA_BF16>(a, stream) : forward<KDA_F32, KDA_F32>(a, stream);
}

hipError_t launch_linear_bwd(const LinearArgs& a, hipStream_t stream) {
    return a.in_dtype == KDA_BF16 ? backward<KDA_BF16>(a, stream) : backward<KDA_F32>(a, stream);
}

// ---------------------------------------------------------------- decode step
namespace {

// One workgroup per (sequence, head): the state is read once, updated in registers and written once
// (non-temporal both ways: a step touches it once).  Lane t owns four columns of DK / RG rows.  Bound by
// HBM: 256 x 32 states of 128 x 128 in 176 us, 6.1 TB/s (a large copy reaches 4.92); one sequence of 32
// heads in 3.8 us.
template <int DT, int ODT, int DK, int DV>
__global__ void __launch_bounds__(256) linear_decode_kernel(const void* __restrict__ q, const void* __restrict__ k,
                                                            const void* __restrict__ v, const float* __restrict__ g,
                                                            float* __restrict__ state, void* __restrict__ o,
                                                            int32_t H, float scale) {
    constexpr int CG = DV / 4, RG = 256 / CG, RPT = DK / RG;
    __shared__ float sq[DK], sk[DK];
    __shared__ f32x4 red[RG][CG];
    const int64_t unit = blockIdx.x;
    const int t = threadIdx.x, cg = t % CG, rg = t / CG;
    float xq = 0.f, xk = 0.f;
    if (t < DK) {
        xq = load_as_f32<DT>(q, unit * DK + t);
        xk = load_as_f32<DT>(k, unit * DK + t);
    }
    const float4 vv = load4_as_f32<DT>(v, unit * DV + 4 * cg);
    const float gg = g[unit % H];
    float* S = state + unit * (DK * DV) + 4 * cg;
    f32x4 s[RPT];
#pragma unroll
    for (int i = 0; i < RPT; ++i)
        s[i] = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(S + (rg * RPT + i) * DV));
    if (t < DK) {
        sq[t] = xq;
        sk[t] = xk;
    }
    // e^g as hi + lo: its rounding to one fp32 number would act the same way token after token (up to 2^-25 of
    // the state each time: 3.0e-4 after 10000 tokens at g = -1.07e-3, 1.3e-6 with both).  0.2 us on a single
    // sequence, nothing on a batch.
    const double lam = exp(static_cast<double>(gg));
    const float lam_hi = static_cast<float>(lam), lam_lo = static_cast<float>(lam - static_cast<double>(lam_hi));
    __syncthreads();
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    const f32x4 c = {vv.x, vv.y, vv.z, vv.w};
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int r = rg * RPT + i;
        const float kr = sk[r], qr = sq[r];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            s[i][e] = __builtin_fmaf(lam_hi, s[i][e], __builtin_fmaf(kr, c[e], lam_lo * s[i][e]));
            acc[e] = __builtin_fmaf(qr, s[i][e], acc[e]);
        }
        __builtin_nontemporal_store(s[i], reinterpret_cast<f32x4*>(S + r * DV));
    }
    red[rg][cg] = acc;
    __syncthreads();
    if (rg == 0) {
        f32x4 sum = red[0][cg];
#pragma unroll
        for (int r = 1; r < RG; ++r) sum += red[r][cg];
        store4_from_f32<ODT>(o, unit * DV + 4 * cg,
                             make_float4(scale * sum[0], scale * sum[1], scale * sum[2], scale * sum[3]));
    }
}

}  // namespace

hipError_t launch_linear_decode(const void* q, const void* k, const void* v, int in_dtype, const float* g,
                                float* state, void* o, int o_dtype, int32_t N, int32_t H, int32_t dk,
                                int32_t dv, float scale, hipStream_t stream) {
    const dim3 grid(static_cast<unsigned>(N * H));
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, q, k, v, g, state, o, H, scale);
        return hipGetLastError();
    };
    auto by_size = [&](auto dt, auto odt) {
        constexpr int DT = decltype(dt)::value, ODT = decltype(odt)::value;
        if (dk == 128 && dv == 128) return go(linear_decode_kernel<DT, ODT, 128, 128>);
        if (dk == 128) return go(linear_decode_kernel<DT, ODT, 128, 64>);
        if (dv == 128) return go(linear_decode_kernel<DT, ODT, 64, 128>);
        return go(linear_decode_kernel<DT, ODT, 64, 64>);
    };
    using F = std::integral_constant<int, KDA_F32>;
    using Bf = std::integral_constant<int, KDA_BF16>;
    if (in_dtype == KDA_BF16) return o_dtype == KDA_BF16 ? by_size(Bf{}, Bf{}) : by_size(Bf{}, F{});
    return o_dtype == KDA_BF16 ? by_size(F{}, Bf{}) : by_size(F{}, F{});
}

}  // namespace kda
