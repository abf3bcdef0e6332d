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
#include "kda_common.hpp"
#include "kda_internal.hpp"

#include <algorithm>
#include <type_traits>

namespace kda {
namespace {

struct Pass {
    const void *a, *b, *c;
    void* out;
    const float* m_in;       // [N, H, DA, DC], or [N, H, DC, DA] with m_transposed; nullptr = zeros
    float* m_out;            // [N, H, DA, DC] or nullptr
    const float* g;
    const int32_t* cu;
    int64_t T;
    int32_t n_seqs, H;
    float so, ub;
    int32_t m_transposed;    // also of seg_states
    int64_t seg;             // tokens per segment (>= T: whole sequences)
    float* seg_states;       // [slots, H, DA, DC] (or transposed), segmented launches only
};

// A launch covers (sequence, segment) slots times heads.  Fixed-length batches: ceil(T / seg) slots per
// sequence; packed ones: slot floor(cu[n] / seg) + n + s for segment s of sequence n, which leaves
// unused slots between sequences.  seg >= T gives one slot per sequence.
struct Where {
    int32_t n, s, n_seg;     // sequence, segment, segments of the sequence
    int64_t lo, hi;          // tokens of the segment
};
__device__ __forceinline__ void seq_range(const Pass& p, int32_t n, int64_t& lo, int64_t& hi) {
    if (p.cu == nullptr) {
        lo = n * p.T;
        hi = lo + p.T;
    } else {
        const int64_t x = p.cu[n], y = p.cu[n + 1];
        lo = x < 0 ? 0 : (x > p.T ? p.T : x);
        hi = y < lo ? lo : (y > p.T ? p.T : y);
    }
}
__device__ __forceinline__ int32_t slot_base(const Pass& p, int32_t n) {
    int64_t lo, hi;
    seq_range(p, n, lo, hi);
    return static_cast<int32_t>(lo / p.seg) + n;
}
__device__ __forceinline__ int32_t segments(const Pass& p, int64_t len) {
    return len <= p.seg ? 1 : static_cast<int32_t>((len + p.seg - 1) / p.seg);
}
__device__ __forceinline__ bool locate(const Pass& p, int32_t slot, Where& w) {
    int32_t first;
    if (p.cu == nullptr) {
        const int32_t per = segments(p, p.T);
        w.n = slot / per;
        first = w.n * per;
    } else {
        int32_t a = 0, b = p.n_seqs - 1;          // the last sequence whose first slot is <= slot
        while (a < b) {
            const int32_t m = (a + b + 1) / 2;
            if (slot_base(p, m) <= slot) a = m; else b = m - 1;
        }
        w.n = a;
        first = slot_base(p, a);
    }
    int64_t lo, hi;
    seq_range(p, w.n, lo, hi);
    w.n_seg = segments(p, hi - lo);
    w.s = slot - first;
    if (w.s < 0 || w.s >= w.n_seg) return false;
    w.lo = lo + w.s * p.seg;
    w.hi = w.lo + p.seg < hi ? w.lo + p.seg : hi;
    return true;
}

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) uint8_t lds_u8;

__device__ __forceinline__ f32x4 mfma_bf16(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                   0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma_f32(float a, float b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}
// Two floats as bf16 (nearest even), x in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float x, float y) {
    const f32x2 v = {x, y};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}
__device__ __forceinline__ float lo_f32(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f32(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
// x, y as two bf16 terms each: hi + lo, off by at most 2^-16 of the value.
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
    hi = pack_bf16(x, y);
    lo = pack_bf16(x - lo_f32(hi), y - hi_f32(hi));
}
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

// A [TOK][DIM] tile in LDS, row-major in 16-byte units.  Units are XOR-ed with the row so that 16 rows'
// equal units (fragments along the channels) and 16 rows' neighbouring units (fragments along the
// tokens) both spread over all banks.
template <int DIM, int ES>
struct Tile {
    static constexpr int UPR = DIM * ES / 16;              // units per row
    static __device__ __forceinline__ uint32_t at(int row, int unit) {
        const int x = UPR >= 16 ? (row & 15) : ((row >> 1) & 7);
        return static_cast<uint32_t>((row * UPR + (unit ^ x)) * 16);
    }
};

// 4 tokens x 16 channels, transposed: lane i of each 16 gets channel i of the 4 tokens whose 8-byte
// pieces the lanes point at (lane 4 r + s: token r, piece s).
__device__ __forceinline__ u32x2 lds_tr(const lds_u8* p) {
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                         (__attribute__((address_space(3))) s16x4*)(p)));
}

// The pass in chunks of TOK tokens; one workgroup of four waves per (segment, head), wave w with the
// output columns [w DC / 4, (w + 1) DC / 4).  With lam^p = e^(p g), i and j tokens of a chunk of n:
//     out_i = so lam^(i+1) M^T a_i + so sum_{j <= i} lam^(i-j) (b_j . a_i) c_j,
//     M    <- lam^n M + ub sum_j lam^(n-1-j) b_j c_j^T                         (forward; backward:
//     j >= i, lam^(j-i), lam^(n-1-i) for the state's part and lam^(j+1) for the update).
// All three products are MFMAs computed transposed (out^T = M^T a^T, scores^T = b a^T), which makes
// every accumulator the next product's operand without a shuffle: an accumulator holds four
// neighbouring rows per lane, and an operand wants eight values along the contraction per lane -- any
// eight, as long as both operands take the same ones.  So M's tiles feed out^T = M^T a^T from the
// registers that M = b^T c left them in, and the scores likewise.  The decays multiply accumulators
// (fp32) wherever they can; only the update's sits inside a contraction, on c.
//   16-bit inputs: M and the scores are read as two bf16 terms, the decayed c as three (exact).
//   fp32 inputs: 16x16x4 fp32 MFMAs throughout.
// STATE_ONLY: just M from zero, the segment's own contribution.
template <int DT, int ODT, int DA, int DC, bool BACK, bool STATE_ONLY>
__global__ void __launch_bounds__(256) linear_chunk_kernel(Pass p) {
    constexpr bool BF = DT == KDA_BF16;
    constexpr int ES = BF ? 2 : 4;
    constexpr int TOK = BF ? 64 : 32;                // tokens per chunk
    constexpr int IT = TOK / 16;                     // token tiles
    constexpr int MT = DA / 16;                      // state row tiles
    constexpr int NT = DC / 64;                      // column tiles of a wave
    constexpr int UA = TOK * DA * ES / 16 / 256, UC = TOK * DC * ES / 16 / 256;   // units per lane
    using TA = Tile<DA, ES>;
    using TC = Tile<DC, ES>;
    constexpr int SA = TOK * DA * ES, SC = TOK * DC * ES;
    __shared__ __align__(16) uint8_t smem[(STATE_ONLY ? 0 : SA) + SA + SC];
    __shared__ float s_lam[TOK + 1], s_lam_lo[TOK + 1], s_rd[TOK];
    __shared__ __align__(16) float s_up[TOK];
    uint8_t* const smB = smem;
    uint8_t* const smC = smem + SA;
    uint8_t* const smA = smem + SA + SC;

    Where w;
    const int32_t h = static_cast<int32_t>(blockIdx.x % p.H);
    const int32_t slot = static_cast<int32_t>(blockIdx.x / p.H);
    if (!locate(p, slot, w)) return;
    if (STATE_ONLY && w.s == (BACK ? 0 : w.n_seg - 1)) return;    // nothing follows it
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6, q = lane >> 4, l16 = lane & 15;
    const int64_t len = w.hi - w.lo;
    const int n_chunks = static_cast<int>((len + TOK - 1) / TOK);

    // ---- decays
    if (t <= TOK && len > 0) {
        const double x = t == 0 ? 1.0 : exp(static_cast<double>(t) * static_cast<double>(p.g[h]));
        const float f = static_cast<float>(x);
        s_lam[t] = f;
        s_lam_lo[t] = f < 3.4e38f ? static_cast<float>(x - static_cast<double>(f)) : 0.f;
    }
    __syncthreads();

    // ---- the state: tile (mt, nt), register r holds row 16 mt + 4 q + r, column col(nt)
    const int wcol = wave * (DC / 4);
    auto col = [&](int nt) { return wcol + (NT == 2 ? 8 * (l16 >> 2) + (l16 & 3) + 4 * nt : l16); };
    const int64_t unit = static_cast<int64_t>(w.n) * p.H + h;
    f32x4 M[MT][NT];
    {
        const float* src = nullptr;
        if constexpr (!STATE_ONLY) {
            if (p.seg_states) src = p.seg_states + (static_cast<int64_t>(slot) * p.H + h) * (DA * DC);
            else if (p.m_in) src = p.m_in + unit * (DA * DC);
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int r0 = 16 * mt + 4 * q, c = col(nt);
                f32x4 x = {0.f, 0.f, 0.f, 0.f};
                if (src) {
                    if (p.m_transposed) x = *reinterpret_cast<const f32x4*>(src + c * DA + r0);
                    else
#pragma unroll
                        for (int r = 0; r < 4; ++r) x[r] = src[(r0 + r) * DC + c];
                }
                M[mt][nt] = x;
            }
    }

    // lam^(i-j) of the score tiles on the diagonal (masked) and of those next to it
    f32x4 Dd = {0.f, 0.f, 0.f, 0.f}, Dn = Dd;
    if constexpr (!STATE_ONLY) {
        if (len > 0)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int e = BACK ? 4 * q + r - l16 : l16 - 4 * q - r;
                Dd[r] = e < 0 ? 0.f : p.so * p.ub * s_lam[e < 0 ? 0 : e];
                Dn[r] = p.so * p.ub * s_lam[16 + e];
            }
    }

    // ---- tiles: global -> registers -> LDS
    u32x4 ra[UA], rb[UA], rc[UC];
    const int64_t row_a = static_cast<int64_t>(p.H) * DA * ES, row_c = static_cast<int64_t>(p.H) * DC * ES;
    auto fetch = [&](u32x4* reg, const void* base, auto dim, int64_t row_bytes, int64_t tok0, int n) {
        constexpr int DIM = decltype(dim)::value, UPR = DIM * ES / 16, U = TOK * UPR / 256;
        const uint8_t* src = static_cast<const uint8_t*>(base) + tok0 * row_bytes + static_cast<int64_t>(h) * DIM * ES;
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int u = t + 256 * i, row = u / UPR, un = u % UPR;
            u32x4 x = {0u, 0u, 0u, 0u};
            if (row < n) x = *reinterpret_cast<const u32x4*>(src + row * row_bytes + un * 16);
            reg[i] = x;
        }
    };
    auto chunk_range = [&](int c, int64_t& tok0, int& n) {
        const int64_t off = static_cast<int64_t>(BACK ? n_chunks - 1 - c : c) * TOK;
        tok0 = w.lo + off;
        n = static_cast<int>(len - off < TOK ? len - off : TOK);
    };
    using ic_a = std::integral_constant<int, DA>;
    using ic_c = std::integral_constant<int, DC>;
    auto fetch_all = [&](int c) {
        int64_t tok0;
        int n;
        chunk_range(c, tok0, n);
        fetch(rb, p.b, ic_a{}, row_a, tok0, n);
        fetch(rc, p.c, ic_c{}, row_c, tok0, n);
        if constexpr (!STATE_ONLY) fetch(ra, p.a, ic_a{}, row_a, tok0, n);
    };
    if (n_chunks > 0) fetch_all(0);

    int table_n = -1;
    for (int c = 0; c < n_chunks; ++c) {
        int64_t tok0;
        int n;
        chunk_range(c, tok0, n);
        if (c > 0) __syncthreads();                  // the last chunk's tiles have been read
#pragma unroll
        for (int i = 0; i < UA; ++i) {
            const int u = t + 256 * i, row = u / TA::UPR, un = u % TA::UPR;
            *reinterpret_cast<u32x4*>(smB + TA::at(row, un)) = rb[i];
            if constexpr (!STATE_ONLY) {
                if constexpr (BF) {
                    // a's channels in operand order: unit 4 G + q holds channels 32 G + 4 q .. + 3 and
                    // 32 G + 16 + 4 q .. + 3
                    const int d = (un & ~3) + 2 * (un & 1), half = (un >> 1) & 1;
                    *reinterpret_cast<u32x2*>(smA + TA::at(row, d) + 8 * half) = u32x2{ra[i][0], ra[i][1]};
                    *reinterpret_cast<u32x2*>(smA + TA::at(row, d + 1) + 8 * half) = u32x2{ra[i][2], ra[i][3]};
                } else {
                    *reinterpret_cast<u32x4*>(smA + TA::at(row, un)) = ra[i];
                }
            }
        }
#pragma unroll
        for (int i = 0; i < UC; ++i) {
            const int u = t + 256 * i, row = u / TC::UPR, un = u % TC::UPR;
            *reinterpret_cast<u32x4*>(smC + TC::at(row, un)) = rc[i];
        }
        if (n != table_n) {
            table_n = n;
            if (t < TOK) {
                const int from_end = n - 1 - t;
                s_rd[t] = p.so * s_lam[BACK ? (from_end < 0 ? 0 : from_end) : t + 1];
                s_up[t] = p.ub * s_lam[BACK ? t + 1 : (from_end < 0 ? 0 : from_end)];
            }
        }
        __syncthreads();
        if (c + 1 < n_chunks) fetch_all(c + 1);

        const float lam_n = s_lam[n], lam_n_lo = s_lam_lo[n];
        f32x4 O[IT][NT];
        if constexpr (!STATE_ONLY) {
            // ---- the state's part
#pragma unroll
            for (int it = 0; it < IT; ++it)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) O[it][nt] = f32x4{0.f, 0.f, 0.f, 0.f};
            if constexpr (BF) {
#pragma unroll
                for (int kk = 0; kk < DA / 32; ++kk) {
                    u32x4 hi[NT], lo[NT];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const f32x4& m = M[2 * kk + (e >> 1)][nt];
                            uint32_t x, y;
                            split2(m[2 * (e & 1)], m[2 * (e & 1) + 1], x, y);
                            hi[nt][e] = x;
                            lo[nt][e] = y;
                        }
#pragma unroll
                    for (int it = 0; it < IT; ++it) {
                        const u32x4 a = *reinterpret_cast<const u32x4*>(smA + TA::at(16 * it + l16, 4 * kk + q));
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            O[it][nt] = mfma_bf16(hi[nt], a, O[it][nt]);
                            O[it][nt] = mfma_bf16(lo[nt], a, O[it][nt]);
                        }
                    }
                }
            } else {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int it = 0; it < IT; ++it) {
                        const f32x4 a = *reinterpret_cast<const f32x4*>(smA + TA::at(16 * it + l16, 4 * mt + q));
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int r = 0; r < 4; ++r) O[it][nt] = mfma_f32(M[mt][nt][r], a[r], O[it][nt]);
                    }
            }
#pragma unroll
            for (int it = 0; it < IT; ++it) {
                const float rd = s_rd[16 * it + l16];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) O[it][nt] *= rd;
            }
        }
        // ---- decay (lam^n as hi + lo: its rounding would act the same way chunk after chunk)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    M[mt][nt][r] = __builtin_fmaf(M[mt][nt][r], lam_n_lo, M[mt][nt][r] * lam_n);

        if constexpr (BF) {
            constexpr int TG = TOK / 32;
            // c along the tokens: group tg, tokens 32 tg + 4 q .. + 3 and 32 tg + 16 + 4 q .. + 3
            u32x4 vf[TG][NT];
#pragma unroll
            for (int tg = 0; tg < TG; ++tg)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const int row = 32 * tg + 4 * q + (l16 >> 2), s = l16 & 3;
                    const int un = wcol / 8 + (NT == 2 ? s : s >> 1), half = NT == 2 ? nt : (s & 1);
                    const u32x2 x = lds_tr((const lds_u8*)(smC + TC::at(row, un) + 8 * half));
                    const u32x2 y = lds_tr((const lds_u8*)(smC + TC::at(row + 16, un) + 8 * half));
                    vf[tg][nt] = u32x4{x[0], x[1], y[0], y[1]};
                }
            // ---- scores and their part of the output
            if constexpr (!STATE_ONLY) {
                const float l16p = s_lam[16], l32p = s_lam[32];
#pragma unroll
                for (int it = 0; it < IT; ++it) {
                    u32x4 a[DA / 32];
#pragma unroll
                    for (int kk = 0; kk < DA / 32; ++kk)
                        a[kk] = *reinterpret_cast<const u32x4*>(smA + TA::at(16 * it + l16, 4 * kk + q));
#pragma unroll
                    for (int tg = 0; tg < TG; ++tg) {
                        if (BACK ? 2 * tg + 1 < it : 2 * tg > it) continue;
                        u32x4 hi = {0u, 0u, 0u, 0u}, lo = hi;
#pragma unroll
                        for (int hh = 0; hh < 2; ++hh) {
                            const int jt = 2 * tg + hh, dist = BACK ? jt - it : it - jt;
                            if (dist < 0) continue;
                            f32x4 P = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                            for (int kk = 0; kk < DA / 32; ++kk) {
                                const int row = 16 * jt + l16, un = 4 * kk + (q >> 1), half = 8 * (q & 1);
                                const u32x2 x = *reinterpret_cast<const u32x2*>(smB + TA::at(row, un) + half);
                                const u32x2 y = *reinterpret_cast<const u32x2*>(smB + TA::at(row, un + 2) + half);
                                P = mfma_bf16(u32x4{x[0], x[1], y[0], y[1]}, a[kk], P);
                            }
                            f32x4 D = dist == 0 ? Dd : Dn;
                            if (dist == 2) D *= l16p;
                            if (dist == 3) D *= l32p;
                            P *= D;
                            uint32_t h0, o0, h1, o1;
                            split2(P[0], P[1], h0, o0);
                            split2(P[2], P[3], h1, o1);
                            hi[2 * hh] = h0; hi[2 * hh + 1] = h1;
                            lo[2 * hh] = o0; lo[2 * hh + 1] = o1;
                        }
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            O[it][nt] = mfma_bf16(vf[tg][nt], hi, O[it][nt]);
                            O[it][nt] = mfma_bf16(vf[tg][nt], lo, O[it][nt]);
                        }
                    }
                }
            }
            // ---- update
#pragma unroll
            for (int tg = 0; tg < TG; ++tg) {
                const f32x4 w0 = *reinterpret_cast<const f32x4*>(s_up + 32 * tg + 4 * q);
                const f32x4 w1 = *reinterpret_cast<const f32x4*>(s_up + 32 * tg + 16 + 4 * q);
                u32x4 ch[NT], cm[NT], cl[NT];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const f32x4& ww = e < 2 ? w0 : w1;
                        uint32_t x, y, z;
                        split3(lo_f32(vf[tg][nt][e]) * ww[2 * (e & 1)], hi_f32(vf[tg][nt][e]) * ww[2 * (e & 1) + 1], x, y, z);
                        ch[nt][e] = x;
                        cm[nt][e] = y;
                        cl[nt][e] = z;
                    }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    const int row = 32 * tg + 4 * q + (l16 >> 2), s = l16 & 3;
                    const u32x2 x = lds_tr((const lds_u8*)(smB + TA::at(row, 2 * mt + (s >> 1)) + 8 * (s & 1)));
                    const u32x2 y = lds_tr((const lds_u8*)(smB + TA::at(row + 16, 2 * mt + (s >> 1)) + 8 * (s & 1)));
                    const u32x4 kt = {x[0], x[1], y[0], y[1]};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        M[mt][nt] = mfma_bf16(kt, cl[nt], M[mt][nt]);
                        M[mt][nt] = mfma_bf16(kt, cm[nt], M[mt][nt]);
                        M[mt][nt] = mfma_bf16(kt, ch[nt], M[mt][nt]);
                    }
                }
            }
        } else {
            auto element = [&](const uint8_t* sm, auto tile, int row, int ch) {
                using TT = decltype(tile);
                return *reinterpret_cast<const float*>(sm + TT::at(row, ch >> 2) + 4 * (ch & 3));
            };
            f32x4 vf[IT][NT];
#pragma unroll
            for (int jt = 0; jt < IT; ++jt)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int r = 0; r < 4; ++r) vf[jt][nt][r] = element(smC, TC{}, 16 * jt + 4 * q + r, col(nt));
            if constexpr (!STATE_ONLY) {
#pragma unroll
                for (int it = 0; it < IT; ++it)
#pragma unroll
                    for (int jt = 0; jt < IT; ++jt) {
                        const int dist = BACK ? jt - it : it - jt;
                        if (dist < 0) continue;
                        f32x4 P = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) {
                            const f32x4 a = *reinterpret_cast<const f32x4*>(smA + TA::at(16 * it + l16, 4 * mt + q));
                            const f32x4 b = *reinterpret_cast<const f32x4*>(smB + TA::at(16 * jt + l16, 4 * mt + q));
#pragma unroll
                            for (int r = 0; r < 4; ++r) P = mfma_f32(b[r], a[r], P);
                        }
                        P *= dist == 0 ? Dd : Dn;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int r = 0; r < 4; ++r) O[it][nt] = mfma_f32(vf[jt][nt][r], P[r], O[it][nt]);
                    }
            }
#pragma unroll
            for (int jt = 0; jt < IT; ++jt) {
                const f32x4 ww = *reinterpret_cast<const f32x4*>(s_up + 16 * jt + 4 * q);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) vf[jt][nt] *= ww;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float k = element(smB, TA{}, 16 * jt + 4 * q + r, 16 * mt + l16);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) M[mt][nt] = mfma_f32(k, vf[jt][nt][r], M[mt][nt]);
                    }
            }
        }
        // ---- out: lane l16 holds token 16 it + l16, four (eight) neighbouring columns
        if constexpr (!STATE_ONLY) {
            constexpr int OS = ODT == KDA_BF16 ? 2 : 4;
#pragma unroll
            for (int it = 0; it < IT; ++it) {
                const int i = 16 * it + l16;
                if (i < n) {
                    uint8_t* dst = static_cast<uint8_t*>(p.out) +
                                   (((tok0 + i) * p.H + h) * DC + wcol + 4 * NT * q) * OS;
                    if constexpr (ODT == KDA_BF16) {
                        uint32_t x[2 * NT];
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            x[2 * nt] = pack_bf16(O[it][nt][0], O[it][nt][1]);
                            x[2 * nt + 1] = pack_bf16(O[it][nt][2], O[it][nt][3]);
                        }
                        if constexpr (NT == 2) *reinterpret_cast<u32x4*>(dst) = u32x4{x[0], x[1], x[2], x[3]};
                        else *reinterpret_cast<u32x2*>(dst) = u32x2{x[0], x[1]};
                    } else {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) *reinterpret_cast<f32x4*>(dst + 16 * nt) = O[it][nt];
                    }
                }
            }
        }
    }

    float* dst = nullptr;
    if constexpr (STATE_ONLY) dst = p.seg_states + (static_cast<int64_t>(slot) * p.H + h) * (DA * DC);
    else if (p.m_out && w.s == (BACK ? 0 : w.n_seg - 1)) dst = p.m_out + unit * (DA * DC);
    if (dst)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int r = 0; r < 4; ++r) dst[(16 * mt + 4 * q + r) * DC + col(nt)] = M[mt][nt][r];
}

// Segment states: from each segment's own contribution to the state it starts from, in place.
// Grid (sequence * H + head, element blocks of 1024); each lane carries four elements along.
template <bool BACK>
__device__ __forceinline__ void scan_states(const Pass& p, int32_t elems) {
    const int32_t n = blockIdx.x / p.H, h = blockIdx.x % p.H;
    const int32_t e = blockIdx.y * 1024 + threadIdx.x * 4;
    int64_t lo, hi;
    seq_range(p, n, lo, hi);
    const int64_t len = hi - lo;
    const int32_t n_seg = segments(p, len);
    const int32_t first = p.cu ? slot_base(p, n) : n * n_seg;
    const double g = len > 0 ? static_cast<double>(p.g[h]) : 0.0;
    f32x4 x = {0.f, 0.f, 0.f, 0.f};
    if (p.m_in) x = *reinterpret_cast<const f32x4*>(p.m_in + (static_cast<int64_t>(n) * p.H + h) * elems + e);
    float* at = p.seg_states + (static_cast<int64_t>(first) * p.H + h) * elems + e;
    const int64_t step = static_cast<int64_t>(p.H) * elems;
    const double full = exp(static_cast<double>(p.seg) * g);
    const double part = exp(static_cast<double>(len - (n_seg - 1) * p.seg) * g);
    for (int32_t i = 0; i < n_seg; ++i) {
        const int32_t s = BACK ? n_seg - 1 - i : i;
        f32x4* slot = reinterpret_cast<f32x4*>(at + s * step);
        f32x4 own = {0.f, 0.f, 0.f, 0.f};
        if (i < n_seg - 1) own = *slot;
        *slot = x;
        const double l = s == n_seg - 1 ? part : full;
        const float l_hi = static_cast<float>(l), l_lo = static_cast<float>(l - static_cast<double>(l_hi));
#pragma unroll
        for (int r = 0; r < 4; ++r) x[r] = __builtin_fmaf(x[r], l_hi, __builtin_fmaf(x[r], l_lo, own[r]));
    }
}
__global__ void __launch_bounds__(256) linear_scan_kernel(Pass f, Pass b, int32_t elems) {
    if (blockIdx.z == 0) scan_states<false>(f, elems);
    else scan_states<true>(b, elems);
}

// ---------------------------------------------------------------- host side

// Tokens per segment: whole sequences where (sequence, head) units alone give every CU two workgroups,
// else so that all segments together do, but no shorter than 512 tokens.
int64_t segment_tokens(int32_t n_seqs, int64_t total, int32_t H) {
    const int64_t units = int64_t(n_seqs) * H;
    if (units >= 512) return int64_t(1) << 40;
    const int64_t want = (total * H + 511) / 512;                     // tokens of one of 512 equal shares
    const int64_t seg = std::max<int64_t>(512, (want + 63) / 64 * 64);
    return seg * n_seqs >= total ? int64_t(1) << 40 : seg;
}
int64_t segment_slots(int32_t n_seqs, int64_t total, int64_t seg, bool packed) {
    if (packed) return total / seg + n_seqs;
    const int64_t T = total / n_seqs;
    return n_seqs * std::max<int64_t>(1, (T + seg - 1) / seg);
}

template <int DT, int ODT, bool BACK, bool STATE_ONLY>
hipError_t launch_pass(const Pass& p, int64_t slots, int32_t da, int32_t dc, hipStream_t stream) {
    const dim3 grid(static_cast<unsigned>(slots * p.H));
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, p);
        return hipGetLastError();
    };
    if (da == 128 && dc == 128) return go(linear_chunk_kernel<DT, ODT, 128, 128, BACK, STATE_ONLY>);
    if (da == 128) return go(linear_chunk_kernel<DT, ODT, 128, 64, BACK, STATE_ONLY>);
    if (dc == 128) return go(linear_chunk_kernel<DT, ODT, 64, 128, BACK, STATE_ONLY>);
    return go(linear_chunk_kernel<DT, ODT, 64, 64, BACK, STATE_ONLY>);
}

Pass base_pass(const LinearArgs& a, int64_t seg) {
    Pass p{};
    p.g = a.g; p.cu = a.cu; p.T = a.T; p.n_seqs = a.n_seqs; p.H = a.H; p.so = 1.f; p.ub = 1.f; p.seg = seg;
    return p;
}

hipError_t launch_scan(const Pass& f, const Pass& b, int passes, int32_t elems, hipStream_t stream) {
    const dim3 grid(static_cast<unsigned>(f.n_seqs * f.H), static_cast<unsigned>(elems / 1024), static_cast<unsigned>(passes));
    hipLaunchKernelGGL(linear_scan_kernel, grid, dim3(256), 0, stream, f, b, elems);
    return hipGetLastError();
}

constexpr int64_t kWhole = int64_t(1) << 40;

template <int DT, int ODT>
hipError_t forward(const LinearArgs& a, hipStream_t stream) {
    const int64_t total = int64_t(a.B) * a.T, seg = segment_tokens(a.n_seqs, total, a.H);
    const int64_t slots = segment_slots(a.n_seqs, total, seg, a.cu != nullptr);
    Pass p = base_pass(a, seg);
    p.a = a.q; p.b = a.k; p.c = a.v; p.out = a.o; p.so = a.scale; p.m_in = a.h0; p.m_out = a.hT;
    if (seg < kWhole) {
        p.seg_states = static_cast<float*>(a.workspace);
        hipError_t e = launch_pass<DT, ODT, false, true>(p, slots, a.dk, a.dv, stream);
        if (e == hipSuccess) e = launch_scan(p, p, 1, a.dk * a.dv, stream);
        if (e != hipSuccess) return e;
    }
    return launch_pass<DT, ODT, false, false>(p, slots, a.dk, a.dv, stream);
}

template <int DT>
hipError_t backward(const LinearArgs& a, hipStream_t stream) {
    const int64_t total = int64_t(a.B) * a.T, seg = segment_tokens(a.n_seqs, total, a.H);
    const int64_t slots = segment_slots(a.n_seqs, total, seg, a.cu != nullptr);
    Pass q = base_pass(a, seg), k = q, v = q;
    q.a = a.d_o; q.b = a.v; q.c = a.k; q.out = a.dq; q.so = a.scale; q.m_in = a.h0; q.m_transposed = 1;
    k.a = a.v; k.b = a.d_o; k.c = a.q; k.out = a.dkk; k.ub = a.scale; k.m_in = a.dhT; k.m_transposed = 1;
    v.a = a.k; v.b = a.q; v.c = a.d_o; v.out = a.dvv; v.ub = a.scale; v.m_in = a.dhT; v.m_out = a.dh0;
    hipError_t e = hipSuccess;
    if (seg < kWhole) {
        // the forward states S (b = k, c = v) and their gradients G (b = q, c = do)
        Pass s = q, g = v;
        s.b = a.k; s.c = a.v; s.m_transposed = 0;
        s.seg_states = q.seg_states = static_cast<float*>(a.workspace);
        g.seg_states = k.seg_states = v.seg_states = s.seg_states + slots * a.H * a.dk * a.dv;
        e = launch_pass<DT, DT, false, true>(s, slots, a.dk, a.dv, stream);
        if (e == hipSuccess) e = launch_pass<DT, DT, true, true>(g, slots, a.dk, a.dv, stream);
        if (e == hipSuccess) e = launch_scan(s, g, 2, a.dk * a.dv, stream);
    }
    if (e == hipSuccess) e = launch_pass<DT, DT, false, false>(q, slots, a.dv, a.dk, stream);
    if (e == hipSuccess) e = launch_pass<DT, DT, true, false>(k, slots, a.dv, a.dk, stream);
    if (e == hipSuccess) e = launch_pass<DT, DT, true, false>(v, slots, a.dk, a.dv, stream);
    return e;
}

}  // namespace

size_t linear_workspace_bytes(int32_t n_seqs, int64_t total, int32_t H, int32_t dk, int32_t dv, int32_t, bool backward) {
    const int64_t seg = segment_tokens(n_seqs, total, H);
    if (seg >= kWhole) return 0;
    // packed batches may use one slot more per sequence than fixed-length ones
    return static_cast<size_t>(segment_slots(n_seqs, total, seg, true)) * H * dk * dv * 4 * (backward ? 2 : 1);
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
// (non-temporal both ways: a step touches it once).  Lane t owns four columns of DK / RG rows.
template <int DT, int ODT, int DK, int DV>
__global__ void __launch_bounds__(256) linear_decode_kernel(const void* __restrict__ q, const void* __restrict__ k,
                                                            const void* __restrict__ v, const float* __restrict__ g,
                                                            float* __restrict__ state, void* __restrict__ o,
                                                            int32_t H, float scale) {
    typedef float f32x4_t __attribute__((ext_vector_type(4)));
    constexpr int CG = DV / 4, RG = 256 / CG, RPT = DK / RG;
    __shared__ float sq[DK], sk[DK];
    __shared__ f32x4_t red[RG][CG];
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
    f32x4_t s[RPT];
#pragma unroll
    for (int i = 0; i < RPT; ++i)
        s[i] = __builtin_nontemporal_load(reinterpret_cast<const f32x4_t*>(S + (rg * RPT + i) * DV));
    if (t < DK) {
        sq[t] = xq;
        sk[t] = xk;
    }
    const float lam = expf(gg);
    __syncthreads();
    f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
    const f32x4_t c = {vv.x, vv.y, vv.z, vv.w};
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int r = rg * RPT + i;
        const float kr = sk[r], qr = sq[r];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            s[i][e] = __builtin_fmaf(kr, c[e], lam * s[i][e]);
            acc[e] = __builtin_fmaf(qr, s[i][e], acc[e]);
        }
        __builtin_nontemporal_store(s[i], reinterpret_cast<f32x4_t*>(S + r * DV));
    }
    red[rg][cg] = acc;
    __syncthreads();
    if (rg == 0) {
        f32x4_t sum = red[0][cg];
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
