// kda_scan.hip -- selective state space scan: prefill, gradients, single-token step.
//
// With delta_t = softplus(dt_t + bias), g_t = delta_t A (A <= 0) and B, C shared by the H / G heads of a group,
//     S_t = e^g_t S_{t-1} + delta_t B_t x_t^T,   y_t = S_t^T C_t + D x_t.
// In chunks of n tokens, c_i = g_1 + .. + g_i, S the state before the chunk and G the gradient of the one after:
//     y_i   = e^c_i S^T C_i + sum_{j <= i} e^(c_i - c_j) delta_j (B_j . C_i) x_j + D x_i
//     dC_i  = e^c_i S dy_i + sum_{j <= i} e^(c_i - c_j) delta_j (x_j . dy_i) B_j                  (sum over heads)
//     u_i   = e^(c_n - c_i) G^T B_i + sum_{j >= i} e^(c_j - c_i) (C_j . B_i) dy_j,   dx_i = delta_i u_i + D dy_i
//     dB_i  = delta_i (e^(c_n - c_i) G x_i + sum_{j >= i} e^(c_j - c_i) (dy_j . x_i) C_j)         (sum over heads)
//     S    <- e^c_n S + sum_j e^(c_n - c_j) delta_j B_j x_j^T,   G <- e^c_n G + sum_j e^c_j C_j dy_j^T.
// y and dx are one pass (value_pass: a state of d_k rows by a head's d_v columns), dC and dB another
// (shared_pass: its transpose, for several heads of a group whose outputs are added up in registers).
//
// The gradient dg_t = e^g_t <G_t, S_{t-1}> of a token's log-decay adds up all ways from a token before it (or the
// chunk's first state) to an output from it on (or the chunk's last state).  With
//     z_ij = e^(c_i - c_j) delta_j (C_i . B_j) (x_j . dy_i), j < i,
//     p_i  = e^c_i dy_i . S^T C_i,  r_j = delta_j e^(c_n - c_j) x_j . G^T B_j,  thr = e^c_n <G, S>
// it is  thr + sum_{i >= t} (sum_j z_ij - sum_{j > i} z_ji + p_i) + sum_{j < t} r_j,  and with S_n the state after the chunk
// <G, S_n> = thr + sum r, while the chunk before ends with thr + sum p.  So thr runs over a segment from <G, S> at its
// end, formed directly.  What one token adds and another takes off has to agree to fp32's accuracy, or the difference
// would stay in many tokens: both sums of z are over the same numbers, and the states behind p and r are updated with, and
// read as, three bf16 terms (exact).  Sums sum_t w_t dg_t over the tokens (dA: w = delta; dbias: w = A slope) are
// formed from the ways themselves, W the running sum of w in the chunk:
//     sum z_ij (W_i - W_j) + sum p_i W_i + sum r_j (W_n - W_j) + thr W_n.
// (Sums of dg as it comes out, from two terms: dA off by 5e-4 of itself on 63 tokens; from three: 1e-4 on 16384.)
//
// All decays between two tokens are 2^(difference of fp64 sums): a difference of fp32 sums would lose a weak decay
// behind a strong one.
#include "kda_ssm.hpp"
#include "kda_tile.hpp"

#include <algorithm>
#include <type_traits>

namespace kda {
namespace {

struct In {
    const uint8_t* p;
    int64_t ld;              // bytes from token to token
};
struct Out {
    uint8_t* p;
    int64_t ld;
};

struct Scan {
    In x, dt, B, C, dy;
    Out out[2];              // value pass: y or dx; shared passes: dC, dB
    const float *A, *bias, *D;
    const int32_t* cu;
    int64_t T, total;
    int32_t n_seqs, H, G, slots, seg, n_seg;
    const float* m_in[2];    // S: initial states; G: gradients of the final states; or nullptr
    float* m_out[2];         // S: final states; G: gradients of the initial states; or nullptr
    float* seg_states[2];    // [slots, H, dk, dv]: a segment's S before its first token, G behind its last one
    double* seg_log[2];      // [slots, H] log2 of a segment's decay
    float* S_last;           // [N, H, dk, dv] states behind the sequences, where E needs them
    float* part[2];          // [head blocks of a group, tokens, G, dk] dC, dB per block; nullptr: one block
    // [H, tokens]: sum_j z_tj - sum_i z_it; p_t; x_t . u_t from this chunk's outputs, and from later ones (r_t / delta_t)
    float *zz, *pp, *xz, *xr;
    float *zA, *zb;          // [slots, H]: sums of z_ij (W_i - W_j) for W of delta and of the slopes
    float *E, *dDp;          // [slots, H]: <G, S> at the segment's end, sums of x . dy
    Out ddt;
    float *dAp, *dbp;        // [slots, H]
    float *dA, *dD, *dbias;  // [H]
    int32_t exact[2];        // the segment states end in one that is handed out
    int32_t blocks;          // head blocks of a group
};
enum { S_STATE = 0, G_STATE = 1 };
enum Mode { Y, DX, S_ONLY, G_ONLY };
constexpr int32_t WHOLE = 0x7fffffff;
constexpr double LOG2E = 1.4426950408889634074;

// ---------------------------------------------------------------- decays

// softplus of dt + bias.  The sum's rounding error is carried along: for a strongly negative argument it would be
// a relative error of the result.
struct Strength {
    float delta, slope;      // softplus, its derivative
};
__device__ __forceinline__ Strength strength(float dt, float bias) {
#pragma clang fp contract(off)
    const float p = dt + bias, b1 = p - dt;
    const float rest = (dt - (p - b1)) + (bias - b1);              // two-sum: p + rest = dt + bias
    const float e = expf(-__builtin_fabsf(p)), s = 1.f / (1.f + e);
    const float slope = p >= 0.f ? s : e * s;
    const float plus = (p > 0.f ? p : 0.f) + log1pf(e);
    const float more = rest * slope;
    return {more == more ? plus + more : plus, slope};             // (an infinite p has no rest)
}

template <int CTRL, int ROWS>
__device__ __forceinline__ double add_dpp(double x) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const int lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(u), CTRL, ROWS, 0xf, false);
    const int hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(u >> 32), CTRL, ROWS, 0xf, false);
    return x + __builtin_bit_cast(double, (static_cast<uint64_t>(static_cast<uint32_t>(hi)) << 32) | static_cast<uint32_t>(lo));
}
// Sums over the lanes up to this one: inside rows of 16, then the rows' last lanes over to the rows behind.
__device__ __forceinline__ double prefix_sum(double x) {
    x = add_dpp<0x111, 0xf>(x);                      // row_shr:1
    x = add_dpp<0x112, 0xf>(x);
    x = add_dpp<0x114, 0xf>(x);
    x = add_dpp<0x118, 0xf>(x);
    x = add_dpp<0x142, 0xa>(x);                      // row_bcast:15 to rows 1 and 3
    return add_dpp<0x143, 0xc>(x);                   // row_bcast:31 to rows 2 and 3
}
__device__ __forceinline__ double lane_value(double x, int lane) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(u), lane), hi = __builtin_amdgcn_readlane(static_cast<int>(u >> 32), lane);
    return __builtin_bit_cast(double, (static_cast<uint64_t>(hi) << 32) | lo);
}
__device__ __forceinline__ double shuffle(double x, int lane) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __shfl(static_cast<int>(u), lane, 64), hi = __shfl(static_cast<int>(u >> 32), lane, 64);
    return __builtin_bit_cast(double, (static_cast<uint64_t>(hi) << 32) | lo);
}
// 2^x, x <= 0 where A <= 0.
__device__ __forceinline__ float pow2(double x) { return __builtin_amdgcn_exp2f(static_cast<float>(x)); }

// The states in registers change sign from chunk to chunk: chunk k works on (-1)^k S.  The MFMAs' sums lose what they
// drop towards minus infinity, which over all of a state's elements, against inputs that are positive on average (behind
// a SiLU), adds up: with the signs, dA of 4096 tokens was off by 6e-6 of itself, the same way in every head.
__device__ __forceinline__ float chunk_sign(int k) { return k & 1 ? -1.f : 1.f; }

// Per chunk and head: c (log2), delta, the update's weights and the chunk's decay as hi + lo (a state's decay goes
// the same way chunk after chunk, and so would its rounding), these two with the sign that takes the state to the next
// chunk's.  Two chunks' worth: one is made while the other is used.
// Forward also the running sums of delta and of its slope.
template <int TOK, int HB, bool BACK>
struct Decays {
    double cum[2][HB][TOK], dsum[BACK ? 1 : 2][HB][BACK ? 1 : TOK], ssum[BACK ? 1 : 2][HB][BACK ? 1 : TOK];
    float del[2][HB][TOK], up[2][HB][TOK];
    f32x2 over[2][HB];
};
template <int DT>
__device__ __forceinline__ float load_dt(const Scan& L, int64_t tok0, int n, int32_t h, int lane) {
    if (lane >= n) return 0.f;
    return load_as_f32<DT>(L.dt.p + (tok0 + lane) * L.dt.ld, h);
}
// One wave makes head hb's table: dt its token's value (lane), n tokens.
template <int TOK, int HB, bool BACK>
__device__ __forceinline__ void make_decays(Decays<TOK, HB, BACK>& t, int k, int hb, float dt, float bias, float A, int n, int lane) {
    const int buf = k & 1;
    const Strength s = lane < n ? strength(dt, bias) : Strength{0.f, 0.f};
    const double d = prefix_sum(static_cast<double>(s.delta)), o = BACK ? 0.0 : prefix_sum(static_cast<double>(s.slope));
    const double c = d * (static_cast<double>(A) * LOG2E), all = lane_value(c, TOK - 1), over = -exp2(all);
    const float hi = static_cast<float>(over), sign = chunk_sign(k + 1);
    if (lane < TOK) {
        t.cum[buf][hb][lane] = c;
        if constexpr (!BACK) {
            t.dsum[buf][hb][lane] = d;
            t.ssum[buf][hb][lane] = o;
        }
        t.del[buf][hb][lane] = s.delta;
        t.up[buf][hb][lane] = sign * (BACK ? pow2(c) : s.delta * pow2(all - c));
        if (lane == 0) t.over[buf][hb] = f32x2{hi, static_cast<float>(over - static_cast<double>(hi))};
    }
}

// What a lane's four scores of a tile (tokens i = 16 it + l16, j = 16 jt + 4 q + r) are multiplied by: the decay from the
// earlier of the two to the later, 0 where j lies on the wrong side; WEIGH_J: times delta_j; WEIGH_I: times delta_i.
template <bool BACK, bool WEIGH_J, bool WEIGH_I>
__device__ __forceinline__ f32x4 score_weights(const double* cum, const float* del, int it, int jt, int q, int l16) {
    const double ci = cum[16 * it + l16];
    f32x4 dj;
    if constexpr (WEIGH_J) dj = lds_get<f32x4>(del, 4 * (16 * jt + 4 * q));
    const float di = WEIGH_I ? del[16 * it + l16] : 1.f;
    f32x4 w;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int i = 16 * it + l16, j = 16 * jt + 4 * q + r;
        const double cj = cum[j];
        const bool seen = BACK ? j >= i : j <= i;
        float e = pow2(seen ? (BACK ? cj - ci : ci - cj) : 0.0);
        if constexpr (WEIGH_J) e *= dj[r];
        if constexpr (WEIGH_I) e *= di;
        w[r] = seen ? e : 0.f;
    }
    return w;
}

// M <- over M.
template <int MT>
__device__ __forceinline__ void decay_state(f32x4 (&M)[MT], f32x2 over) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int r = 0; r < 4; ++r) M[mt][r] = __builtin_fmaf(M[mt][r], over[0], M[mt][r] * over[1]);
}

// ---------------------------------------------------------------- y, dx and the segments' states

template <int DT, int DK, int DV, int HB, int MODE>
struct ValueLds {
    static constexpr bool STATE = MODE == S_ONLY || MODE == G_ONLY;
    static constexpr int ES = DT == KDA_BF16 ? 2 : 4, TOK = DT == KDA_BF16 ? 64 : 32, WAVES = HB * DV / 16;
    using TA = Tile<DK, ES>;
    using TC = Tile<DV, ES>;
    static constexpr int C_BYTES = TOK / TC::R * TC::PIECE, P_BYTES = (ES == 2 ? 12 : 3) * 1024;
    __align__(16) uint8_t b[TOK / TA::R * TA::PIECE];
    __align__(16) uint8_t c[HB * C_BYTES];
    __align__(16) uint8_t a[STATE ? 16 : TOK / TA::R * TA::PIECE];
    __align__(16) uint8_t p[STATE ? 16 : HB * P_BYTES];              // scores per head
    __align__(16) double cum[2][HB][TOK];
    __align__(16) float del[2][HB][TOK], up[STATE ? 2 : 1][HB][TOK];
    f32x2 over[2][HB];
    __align__(16) float red[MODE == DX ? WAVES * TOK : 1];   // r / delta by waves
};

// One workgroup per (segment, HB heads of a group): a and b rows are shared, wave w has 16 columns of head
// w / (DV / 16).  The products are those of linear attention's pass (transposed, so that an accumulator is the next
// product's operand): M and the scores are read as two bf16 terms (2^-16), the decayed c as three (exact) where M ends
// in a state that is handed out in fp32; fp32 inputs use fp32 MFMAs.  The raw scores b a^T are formed once for
// all HB heads, the last HB waves make the next chunk's decays meanwhile.
template <int DT, int ODT, int DK, int DV, int HB, int MODE>
__device__ __forceinline__ void value_pass(const Scan& L, int32_t slot, int32_t block, ValueLds<DT, DK, DV, HB, MODE>& lds) {
    using Lds = ValueLds<DT, DK, DV, HB, MODE>;
    using TA = typename Lds::TA;
    using TC = typename Lds::TC;
    constexpr bool BF = DT == KDA_BF16, STATE = Lds::STATE, BACK = MODE == DX || MODE == G_ONLY;
    constexpr int ES = Lds::ES, TOK = Lds::TOK, WAVES = Lds::WAVES, WPH = DV / 16;
    constexpr int IT = TOK / 16, MT = DK / 16, KK = DK / 32, JG = TOK / 32;
    constexpr int OS = ODT == KDA_BF16 ? 2 : 4;
    constexpr bool STAGED = BF && OS == 2 && !STATE;
    constexpr int ST = BACK ? G_STATE : S_STATE;

    Where w;
    if (!locate(L, slot, w)) return;
    // nothing follows the last segment's own contribution, but the state behind the sequence
    if (STATE && w.s == (BACK ? 0 : w.n_seg - 1) && !(MODE == S_ONLY && L.S_last)) return;
    const int t = threadIdx.x, lane = t & 63, q = lane >> 4, l16 = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int hb = wave / WPH, wc = wave % WPH;
    const int32_t rep = L.H / L.G, per_group = (rep + HB - 1) / HB, g = block / per_group;
    const int32_t h0 = g * rep + block % per_group * HB, h_end = (g + 1) * rep;
    const int32_t h = h0 + hb < h_end ? h0 + hb : h_end - 1;
    const bool live = h0 + hb < h_end;               // (a group's last block may have fewer than HB heads)
    const int64_t len = w.hi - w.lo;
    const int n_chunks = static_cast<int>((len + TOK - 1) / TOK);
    const int64_t unit = static_cast<int64_t>(w.n) * L.H + h, seg_unit = static_cast<int64_t>(slot) * L.H + h;

    const In &ra = BACK ? L.B : L.C, &rb = BACK ? L.C : L.B, &rc = BACK ? L.dy : L.x;
    auto chunk_at = [&](int c) { return static_cast<int64_t>(BACK ? n_chunks - 1 - c : c) * TOK; };
    auto chunk_n = [&](int64_t off) { return static_cast<int>(len - off < TOK ? len - off : TOK); };
    auto load_a = [&](int c) {
        const int64_t off = chunk_at(c);
        fetch_rows<TA, TOK, WAVES>(lds.a, ra.p + (w.lo + off) * ra.ld + g * TA::RB, static_cast<uint32_t>(ra.ld), chunk_n(off), wave, lane);
    };
    auto load_b = [&](int c) {
        const int64_t off = chunk_at(c);
        fetch_rows<TA, TOK, WAVES>(lds.b, rb.p + (w.lo + off) * rb.ld + g * TA::RB, static_cast<uint32_t>(rb.ld), chunk_n(off), wave, lane);
    };
    auto load_c = [&](int c) {
        const int64_t off = chunk_at(c);
#pragma unroll
        for (int i = 0; i < HB; ++i)
            fetch_rows<TC, TOK, WAVES>(lds.c + i * Lds::C_BYTES, rc.p + (w.lo + off) * rc.ld + (h0 + i) * TC::RB,
                                       static_cast<uint32_t>(rc.ld), h0 + i < h_end ? chunk_n(off) : 0, wave, lane);
    };
    // the wave that makes a head's decays
    const int table = wave - (WAVES - HB);
    const int32_t th = h0 + table < h_end ? h0 + (table < 0 ? 0 : table) : h_end - 1;
    const float A = L.A[th], bias = L.bias ? L.bias[th] : 0.f;
    auto dt_of = [&](int c) {
        const int64_t off = chunk_at(c);
        return load_dt<DT>(L, w.lo + off, chunk_n(off), th, lane);
    };
    double log_sum = 0.0;
    auto decays = [&](int c, float dt) {
        const int buf = c & 1, n = chunk_n(chunk_at(c));
        const float delta = lane < n ? strength(dt, bias).delta : 0.f;
        const double cum = prefix_sum(static_cast<double>(delta) * (static_cast<double>(A) * LOG2E));
        const double all = lane_value(cum, TOK - 1), over = -exp2(all);
        const float hi = static_cast<float>(over);
        log_sum += all;
        if (lane < TOK) {
            lds.cum[buf][table][lane] = cum;
            lds.del[buf][table][lane] = delta;
            if (STATE) lds.up[STATE ? buf : 0][table][lane] = chunk_sign(c + 1) * (BACK ? pow2(cum) : delta * pow2(all - cum));
            if (lane == 0) lds.over[buf][table] = f32x2{hi, static_cast<float>(over - static_cast<double>(hi))};
        }
    };

    if (n_chunks > 0) {
        load_b(0);
        if constexpr (!STATE) load_a(0);
        load_c(0);
        if (table >= 0) decays(0, dt_of(0));
    }

    // ---- the state: tile mt, register r of lane (l16, q) holds row row(mt) + r, column 16 wc + l16
    auto row = [&](int mt) { return BF ? 32 * (mt >> 1) + 8 * q + 4 * (mt & 1) : 16 * mt + 4 * q; };
    const int col = 16 * wc + l16;
    f32x4 M[MT];
    auto load_state = [&](const float* src) {        // nullptr: an empty range, which reads as zeros
        const __amdgpu_buffer_rsrc_t rs = make_rsrc_u(src, src ? DK * DV * 4 : 0);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                M[mt][r] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, ((row(mt) + r) * DV + col) * 4, 0, 0));
    };
    if constexpr (STATE) {
        load_state(nullptr);
    } else {
        if constexpr (MODE == DX) {                  // <G, S> at the segment's end
            const float* after = w.s < w.n_seg - 1 ? L.seg_states[S_STATE] + (seg_unit + L.H) * (DK * DV)
                                 : L.S_last        ? L.S_last + unit * (DK * DV)
                                                   : nullptr;
            load_state(after);
            const float* grad = w.n_seg > 1 ? L.seg_states[G_STATE] + seg_unit * (DK * DV)
                                : L.m_in[G_STATE] ? L.m_in[G_STATE] + unit * (DK * DV)
                                                  : nullptr;
            const __amdgpu_buffer_rsrc_t rs = make_rsrc_u(grad, grad ? DK * DV * 4 : 0);
            float sum = 0.f;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float x = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, ((row(mt) + r) * DV + col) * 4, 0, 0));
                    sum = __builtin_fmaf(M[mt][r], x, sum);
                    M[mt][r] = x;
                }
#pragma unroll
            for (int off = 1; off < 64; off <<= 1) sum += __shfl_xor(sum, off, 64);
            if (lane == 0) lds_put(lds.p, 4 * wave, sum);
            lds_barrier();
            if (wc == 0 && lane == 0 && live) {
                float all = 0.f;
                for (int i = 0; i < WPH; ++i) all += lds_get<float>(lds.p, 4 * (wave + i));
                L.E[seg_unit] = all;
            }
        } else {
            load_state(w.n_seg > 1 ? L.seg_states[ST] + seg_unit * (DK * DV) : L.m_in[ST] ? L.m_in[ST] + unit * (DK * DV) : nullptr);
        }
    }

    // ---- operands' byte offsets, as in linear attention's pass.  16 bits, along the channels: channels
    // 32 kk + 8 q .. + 7 of token 16 it + l16; along the tokens: tokens 32 tg + 4 q .. + 3 and 32 tg + 16 + 4 q .. + 3,
    // of state row tile mt's rows or of the wave's columns.
    uint32_t chan[2], tok[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        chan[x] = TA::at(l16, 4 * x + q);
        tok[x] = TA::at(4 * q + (l16 >> 2), 4 * x + (l16 & 3));
    }
    uint8_t* const lds_c = lds.c + hb * Lds::C_BYTES;
    uint8_t* const lds_p = lds.p + (STATE ? 0 : hb * Lds::P_BYTES);
    const uint32_t tok_c = TC::at(4 * q + (l16 >> 2), 2 * wc + ((l16 & 3) >> 1)) + 8 * (l16 & 1);
    auto channels = [&](const uint8_t* sm, int it, int kk) {
        return lds_get<u32x4>(sm, chan[kk & 1] + it * TA::ROWS16 + (kk >> 1) * 128);
    };
    auto tokens = [&](uint32_t at, const uint8_t* sm, int rows16) {
        const u32x2 x = lds_transpose(sm + at), y = lds_transpose(sm + at + rows16);
        return u32x4{x[0], x[1], y[0], y[1]};
    };
    // where a lane's four columns of a token's row of c (and of the output) stand
    auto own_at = [&](int it) {
        return BF ? TC::at(16 * it + l16, 2 * wc + (q >> 1)) + 8 * (q & 1) : TC::at(16 * it + l16, 4 * wc + q);
    };
    auto widen = [&](const uint8_t* sm, uint32_t at) {
        if constexpr (BF) {
            const u32x2 x = lds_get<u32x2>(sm, at);
            return f32x4{lo_f32(x[0]), hi_f32(x[0]), lo_f32(x[1]), hi_f32(x[1])};
        } else {
            return lds_get<f32x4>(sm, at);
        }
    };
    const float D = (MODE == Y || MODE == DX) && L.D ? L.D[h] : 0.f;
    float dD = 0.f;

    const bool exact = MODE == DX || (STATE ? L.exact[ST] != 0 : L.m_out[ST] && w.s == (BACK ? 0 : w.n_seg - 1));
    for (int c = 0; c < n_chunks; ++c) {
        const int64_t off = chunk_at(c), tok0 = w.lo + off;
        const int n = chunk_n(off), buf = c & 1;
        __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
        lds_barrier();                               // the tiles and the decays are there
        float dt_next = 0.f;
        if (table >= 0 && c + 1 < n_chunks) dt_next = dt_of(c + 1);
        const double* cum = lds.cum[buf][hb];
        const float* del = lds.del[buf][hb];

        f32x4 O[IT];
        u32x2 xr[MODE == DX && BF ? IT : 1];
        f32x4 xf[MODE == DX ? IT : 1];
        if constexpr (MODE == DX) {                  // x of the lane's tokens and columns
            const uint32_t ld = static_cast<uint32_t>(L.x.ld);
            const __amdgpu_buffer_rsrc_t rx = make_rsrc_u(L.x.p + tok0 * L.x.ld + h * TC::RB, (n - 1) * ld + TC::RB);
#pragma unroll
            for (int it = 0; it < IT; ++it) {
                const uint32_t at = (16 * it + l16) * ld + (16 * wc + 4 * q) * ES;
                if constexpr (BF) xr[it] = __builtin_amdgcn_raw_buffer_load_b64(rx, at, 0, 0);
                else xf[it] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rx, at, 0, 0));
            }
        }
        if constexpr (!STATE) {
            if (table >= 0 && lane < TOK) {          // the update's weights, read behind the next barrier
                const double ct = lds.cum[buf][table][lane], all = lds.cum[buf][table][TOK - 1];
                lds.up[0][table][lane] = chunk_sign(c + 1) * (BACK ? pow2(ct) : lds.del[buf][table][lane] * pow2(all - ct));
            }
            // ---- scores, shared out over the waves, weighted for every head
            if constexpr (BF) {
                for (int grp = wave; grp < 6; grp += WAVES) {
                    // (it, tg) with score_group(it, tg) == grp
                    const int tg = BACK ? (grp < 4) : (grp >= 4), it = BACK ? (grp & 3) : (grp < 4 ? grp : grp - 2);
                    f32x4 P[2] = {zero4(), zero4()};
#pragma unroll
                    for (int kk = 0; kk < KK; ++kk) {
                        const u32x4 a = channels(lds.a, it, kk);
#pragma unroll
                        for (int hh = 0; hh < 2; ++hh) P[hh] = mfma_bf16(channels(lds.b, 2 * tg + hh, kk), a, P[hh]);
                    }
#pragma unroll
                    for (int i = 0; i < HB; ++i) {
                        u32x4 hi, lo;
#pragma unroll
                        for (int hh = 0; hh < 2; ++hh) {
                            const f32x4 x = P[hh] * score_weights<BACK, !BACK, false>(lds.cum[buf][i], lds.del[buf][i], it, 2 * tg + hh, q, l16);
                            uint32_t h0_, o0, h1, o1;
                            split_pair(x[0], x[1], h0_, o0);
                            split_pair(x[2], x[3], h1, o1);
                            hi[2 * hh] = h0_; hi[2 * hh + 1] = h1;
                            lo[2 * hh] = o0; lo[2 * hh + 1] = o1;
                        }
                        lds_put(lds.p + i * Lds::P_BYTES, grp * 2048 + lane * 16, hi);
                        lds_put(lds.p + i * Lds::P_BYTES, grp * 2048 + 1024 + lane * 16, lo);
                    }
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
#pragma unroll
                for (int i = 0; i < HB; ++i)
                    lds_put(lds.p + i * Lds::P_BYTES, wave * 1024 + lane * 16,
                            P * score_weights<BACK, !BACK, false>(lds.cum[buf][i], lds.del[buf][i], it, jt, q, l16));
            }
            // ---- the state's part
#pragma unroll
            for (int it = 0; it < IT; ++it) O[it] = zero4();
            if constexpr (BF) {
#pragma unroll
                for (int kk = 0; kk < KK; ++kk) {
                    u32x4 hi, mid, lo, a[IT];
#pragma unroll
                    for (int it = 0; it < IT; ++it) a[it] = channels(lds.a, it, kk);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const f32x4& m = M[2 * kk + (e >> 1)];
                        uint32_t x, y, z = 0;
                        if constexpr (MODE == DX) split3(m[2 * (e & 1)], m[2 * (e & 1) + 1], x, y, z);
                        else split_pair(m[2 * (e & 1)], m[2 * (e & 1) + 1], x, y);
                        hi[e] = x;
                        mid[e] = y;
                        lo[e] = z;
                    }
#pragma unroll
                    for (int it = 0; it < IT; ++it) O[it] = mfma_bf16(hi, a[it], O[it]);
#pragma unroll
                    for (int it = 0; it < IT; ++it) O[it] = mfma_bf16(mid, a[it], O[it]);
                    if constexpr (MODE == DX)
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
            const double all = cum[TOK - 1];
#pragma unroll
            for (int it = 0; it < IT; ++it) {
                const double ci = cum[16 * it + l16];
                O[it] *= chunk_sign(c) * pow2(BACK ? all - ci : ci);
                if constexpr (MODE == DX) {          // r / delta
                    if constexpr (BF) xf[it] = f32x4{lo_f32(xr[it][0]), hi_f32(xr[it][0]), lo_f32(xr[it][1]), hi_f32(xr[it][1])};
                    float s = 0.f;
#pragma unroll
                    for (int r = 0; r < 4; ++r) s = __builtin_fmaf(xf[it][r], O[it][r], s);
                    s += __shfl_xor(s, 16, 64);
                    s += __shfl_xor(s, 32, 64);
                    if (q == 0) lds.red[wave * TOK + 16 * it + l16] = s;
                }
            }
        }
        if (table >= 0 && c + 1 < n_chunks) decays(c + 1, dt_next);
        decay_state(M, lds.over[buf][hb]);

        // ---- c along the tokens
        constexpr int CJ = BF ? JG : IT;
        u32x4 vf[CJ];
#pragma unroll
        for (int j = 0; j < CJ; ++j) {
            if constexpr (BF) vf[j] = tokens(tok_c + 2 * j * TC::ROWS16, lds_c, TC::ROWS16);
            else
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    vf[j][r] = lds_get<uint32_t>(lds_c, TC::at(16 * j + 4 * q + r, 4 * wc + (l16 >> 2)) + 4 * (l16 & 3));
        }
        if constexpr (!STATE) {
            lds_barrier();                           // the scores and the update's weights are there
            if constexpr (BF) {
#pragma unroll
                for (int it = 0; it < IT; ++it)
#pragma unroll
                    for (int tg = 0; tg < JG; ++tg) {
                        if (BACK ? 2 * tg + 1 < it : 2 * tg > it) continue;
                        const uint32_t at = score_group<BACK>(it, tg) * 2048 + lane * 16;
                        O[it] = mfma_bf16(vf[tg], lds_get<u32x4>(lds_p, at), O[it]);
                        O[it] = mfma_bf16(vf[tg], lds_get<u32x4>(lds_p, at + 1024), O[it]);
                    }
            } else {
#pragma unroll
                for (int tile = 0; tile < 3; ++tile) {
                    const int it = BACK ? (tile == 1) : (tile > 0), jt = BACK ? (tile > 0) : (tile == 1);
                    const f32x4 P = lds_get<f32x4>(lds_p, tile * 1024 + lane * 16);
#pragma unroll
                    for (int r = 0; r < 4; ++r) O[it] = mfma_f32(__uint_as_float(vf[jt][r]), P[r], O[it]);
                }
            }
            // ---- lane l16 holds token 16 it + l16, four neighbouring columns: D's part, and x . u
#pragma unroll
            for (int it = 0; it < IT; ++it) {
                const f32x4 own = widen(lds_c, own_at(it));
                if constexpr (MODE == Y) {
                    if (L.D) O[it] += D * own;
                } else {
                    f32x4 x;
                    if constexpr (BF) x = f32x4{lo_f32(xr[it][0]), hi_f32(xr[it][0]), lo_f32(xr[it][1]), hi_f32(xr[it][1])};
                    else x = xf[it];
#pragma unroll
                    for (int r = 0; r < 4; ++r) dD = __builtin_fmaf(x[r], own[r], dD);
                    const float di = del[16 * it + l16];
                    O[it] = O[it] * di + D * own;
                }
            }
            // ---- out, through c's tile (which all waves have read by now)
            if constexpr (STAGED) {
                int ll = l16;
                asm volatile("" : "+v"(ll));
#pragma unroll
                for (int it = 0; it < IT; ++it)
                    lds_put(lds_c, TC::at(16 * it + ll, 2 * wc + (q >> 1)) + 8 * (q & 1),
                            u32x2{pack_bf16(O[it][0], O[it][1]), pack_bf16(O[it][2], O[it][3])});
            } else {
                const uint32_t orow = static_cast<uint32_t>(L.out[0].ld);
                const __amdgpu_buffer_rsrc_t ro = make_rsrc_u(L.out[0].p + tok0 * L.out[0].ld + h * DV * OS,
                                                              live ? (n - 1) * orow + DV * OS : 0);
#pragma unroll
                for (int it = 0; it < IT; ++it) {
                    const uint32_t at = (16 * it + l16) * orow + (16 * wc + 4 * q) * OS;
                    if constexpr (ODT == KDA_BF16)
                        __builtin_amdgcn_raw_buffer_store_b64(u32x2{pack_bf16(O[it][0], O[it][1]), pack_bf16(O[it][2], O[it][3])},
                                                              ro, at, 0, 0);
                    else __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, O[it]), ro, at, 0, 0);
                }
            }
        }
        // ---- update
        const float* up = lds.up[STATE ? buf : 0][hb];
        if constexpr (BF) {
            auto update = [&](auto three) {
                constexpr bool THREE = decltype(three)::value;
#pragma unroll
                for (int tg = 0; tg < JG; ++tg) {
                    const f32x4 w0 = lds_get<f32x4>(up, 4 * (32 * tg + 4 * q));
                    const f32x4 w1 = lds_get<f32x4>(up, 4 * (32 * tg + 16 + 4 * q));
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
                const f32x4 ww = lds_get<f32x4>(up, 4 * (16 * jt + 4 * q));
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
        if (c + 1 < n_chunks) load_b(c + 1);
        if constexpr (!STATE)
            if (c + 1 < n_chunks) load_a(c + 1);
        if constexpr (MODE == DX) {
            for (int e = t; e < HB * TOK; e += WAVES * 64) {
                const int i = e / TOK, at = e % TOK;
                float r = 0.f;
#pragma unroll
                for (int x = 0; x < WPH; ++x) r += lds.red[(i * WPH + x) * TOK + at];
                if (at < n && h0 + i < h_end) L.xr[(h0 + i) * L.total + tok0 + at] = r;
            }
        }
        if constexpr (STAGED) {
            const uint32_t orow = static_cast<uint32_t>(L.out[0].ld);
            int tt = t;                              // formed anew in each chunk: no registers over the loop
            asm volatile("" : "+v"(tt));
#pragma unroll
            for (int i = 0; i < HB; ++i) {
                const __amdgpu_buffer_rsrc_t ro = make_rsrc_u(L.out[0].p + tok0 * L.out[0].ld + (h0 + i) * DV * OS,
                                                              h0 + i < h_end ? (n - 1) * orow + DV * OS : 0);
#pragma unroll
                for (int j = 0; j < TOK * TC::UPR / (64 * WAVES); ++j) {
                    const int u = tt + 64 * WAVES * j, r = u / TC::UPR, un = u % TC::UPR;
                    __builtin_amdgcn_raw_buffer_store_b128(lds_get<u32x4>(lds.c + i * Lds::C_BYTES, TC::at(r, un)), ro,
                                                           r * orow + un * 16, 0, CP_NT);
                }
            }
        }
        if constexpr (STAGED) lds_barrier();         // the output has been read
        if (c + 1 < n_chunks) load_c(c + 1);
    }

    float* dst = nullptr;
    if constexpr (STATE) dst = L.seg_states[ST] + seg_unit * (DK * DV);
    else if (L.m_out[ST] && w.s == (BACK ? 0 : w.n_seg - 1)) dst = L.m_out[ST] + unit * (DK * DV);
    if (dst && live) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int r = 0; r < 4; ++r) dst[(row(mt) + r) * DV + col] = chunk_sign(n_chunks) * M[mt][r];
    }
    if constexpr (STATE) {
        if (table >= 0 && h0 + table < h_end && lane == 0) L.seg_log[ST][static_cast<int64_t>(slot) * L.H + h0 + table] = log_sum;
    }
    if constexpr (MODE == DX) {
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) dD += __shfl_xor(dD, off, 64);
        lds_barrier();                               // (the first chunk's E may still be read)
        if (lane == 0) lds_put(lds.p, 4 * wave, dD);
        lds_barrier();
        if (wc == 0 && lane == 0 && live) {
            float all = 0.f;
            for (int i = 0; i < WPH; ++i) all += lds_get<float>(lds.p, 4 * (wave + i));
            L.dDp[seg_unit] = all;
        }
    }
}

// An XCD takes a contiguous range of (slot, head block) units, as in linear attention's pass.
__device__ __forceinline__ bool unit_of(uint32_t units, int32_t passes, uint32_t& unit, int32_t& pass) {
    const uint32_t per_xcd = (units + 7) / 8, j = blockIdx.x / 8;
    unit = blockIdx.x % 8 * per_xcd + j / passes;
    pass = static_cast<int32_t>(j % passes);
    return j / passes < per_xcd && unit < units;
}

template <int DT, int ODT, int DK, int DV, int HB, int MODE>
__global__ void __launch_bounds__(HB * DV * 4, HB * DV == 128 && MODE != DX ? 4 : 2) value_kernel(Scan L) {
    __shared__ ValueLds<DT, DK, DV, HB, MODE> lds;
    uint32_t unit;
    int32_t pass;
    if (!unit_of(static_cast<uint32_t>(L.slots) * L.blocks * L.G, 1, unit, pass)) return;
    const uint32_t blocks = static_cast<uint32_t>(L.blocks) * L.G;
    value_pass<DT, ODT, DK, DV, HB, MODE>(L, unit / blocks, unit % blocks, lds);
}
// The segments' states: S, or G, or both.
template <int DT, int DK, int DV, int HB>
__global__ void __launch_bounds__(HB * DV * 4, HB * DV == 128 ? 4 : 2) state_kernel(Scan L, int32_t first, int32_t passes) {
    __shared__ union {
        ValueLds<DT, DK, DV, HB, S_ONLY> s;
        ValueLds<DT, DK, DV, HB, G_ONLY> g;
    } lds;
    uint32_t unit;
    int32_t pass;
    if (!unit_of(static_cast<uint32_t>(L.slots) * L.blocks * L.G, passes, unit, pass)) return;
    const uint32_t blocks = static_cast<uint32_t>(L.blocks) * L.G;
    if (first + pass == S_STATE) value_pass<DT, DT, DK, DV, HB, S_ONLY>(L, unit / blocks, unit % blocks, lds.s);
    else value_pass<DT, DT, DK, DV, HB, G_ONLY>(L, unit / blocks, unit % blocks, lds.g);
}

// Segment states: from each segment's own contribution to the state it starts from (S) or that follows it (G), in
// place.  Grid (sequence * H + head, element blocks of 1024, pass); eight segments' loads at a time.
__global__ void __launch_bounds__(256) scan_kernel(Scan L, int32_t elems, int32_t first) {
    const int ST = first + blockIdx.z;
    const bool back = ST == G_STATE;
    const int32_t n = blockIdx.x / L.H, h = blockIdx.x % L.H;
    const int32_t e = blockIdx.y * 1024 + threadIdx.x * 4;
    int64_t lo, hi;
    seq_range(L, n, lo, hi);
    const int32_t n_seg = segments(L, hi - lo);
    float* last = back ? nullptr : L.S_last;
    if (n_seg == 1 && !last) return;
    const int64_t slot0 = L.cu ? first_slot(L, n) : static_cast<int64_t>(n) * n_seg;
    const int64_t unit = static_cast<int64_t>(n) * L.H + h;
    f32x4 x = zero4();
    if (L.m_in[ST]) x = *reinterpret_cast<const f32x4*>(L.m_in[ST] + unit * elems + e);
    auto index = [&](int32_t i) { return (slot0 + (back ? n_seg - 1 - i : i)) * L.H + h; };
    auto slot = [&](int32_t i) { return reinterpret_cast<f32x4*>(L.seg_states[ST] + index(i) * elems + e); };
    const int32_t steps = last ? n_seg : n_seg - 1;  // segments whose own contribution is taken in
    f32x4 ahead = *slot(0);                          // read before the batch before it writes its place
    *slot(0) = x;
    for (int32_t i0 = 0; i0 < steps; i0 += 8) {
        f32x4 own[9];
        double lg[8];
        own[0] = ahead;
#pragma unroll
        for (int32_t j = 1; j < 9; ++j) own[j] = i0 + j < steps ? *slot(i0 + j) : zero4();
#pragma unroll
        for (int32_t j = 0; j < 8; ++j) lg[j] = i0 + j < steps ? L.seg_log[ST][index(i0 + j)] : 0.0;
        ahead = own[8];
#pragma unroll
        for (int32_t j = 0; j < 8; ++j) {
            if (i0 + j >= steps) break;
            const double l = exp2(lg[j]);
            const float l_hi = static_cast<float>(l), l_lo = static_cast<float>(l - static_cast<double>(l_hi));
#pragma unroll
            for (int r = 0; r < 4; ++r) x[r] = __builtin_fmaf(x[r], l_hi, __builtin_fmaf(x[r], l_lo, own[j][r]));
            if (i0 + j + 1 < n_seg) *slot(i0 + j + 1) = x;
        }
    }
    if (last) *reinterpret_cast<f32x4*>(last + unit * elems + e) = x;
}

// ---------------------------------------------------------------- dC and dB

template <int DT, int DK, int DV, int HB, bool BACK>
struct SharedLds {
    static constexpr int ES = DT == KDA_BF16 ? 2 : 4, TOK = DT == KDA_BF16 ? 64 : 32, WAVES = DK / 16;
    using TA = Tile<DV, ES>;
    using TC = Tile<DK, ES>;
    static constexpr int A_BYTES = TOK / TA::R * TA::PIECE;
    __align__(16) uint8_t b[2 * A_BYTES];            // this head's and the next one's
    __align__(16) uint8_t a[2 * A_BYTES];
    __align__(16) uint8_t c[TOK / TC::R * TC::PIECE];
    __align__(16) uint8_t p[(ES == 2 ? 12 : 3) * 1024];    // scores, summed over the heads
    Decays<TOK, HB, BACK> t;
    // dC: p by waves, sums of z over j by 32 tokens j (fp32: 16), of z / delta over i by 16 tokens i, z_jj / delta_j
    static constexpr int RED = BACK ? 1 : WAVES + 2 + TOK / 16 + 1;
    float red[BACK ? 1 : HB][RED][BACK ? 1 : TOK];
};

// The sum over a row of 16 lanes, in its last one.
__device__ __forceinline__ float row_sum(float x) {
    auto add = [](float y, auto ctrl) {
        return y + __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(y), decltype(ctrl)::value, 0xf, 0xf, false));
    };
    x = add(x, std::integral_constant<int, 0x111>{});              // row_shr:1, :2, :4, :8
    x = add(x, std::integral_constant<int, 0x112>{});
    x = add(x, std::integral_constant<int, 0x114>{});
    return add(x, std::integral_constant<int, 0x118>{});
}

// One workgroup per (segment, up to HB heads of a group); wave w has the output columns 16 w .. 16 w + 15 and their
// states (rows d_v) of all its heads.  The heads' rows come one head after the other, the next one's under this one's
// products.  The output's sum over the heads is formed in registers, and since c is the group's, its product with
// the scores is formed once, with their sum.
template <int DT, int DK, int DV, int HB, bool BACK>
__device__ __forceinline__ void shared_pass(const Scan& L, int32_t slot, int32_t block, SharedLds<DT, DK, DV, HB, BACK>& lds) {
    using Lds = SharedLds<DT, DK, DV, HB, BACK>;
    using TA = typename Lds::TA;
    using TC = typename Lds::TC;
    constexpr bool BF = DT == KDA_BF16;
    constexpr int ES = Lds::ES, TOK = Lds::TOK, WAVES = Lds::WAVES;
    constexpr int IT = TOK / 16, MT = DV / 16, KK = DV / 32, JG = TOK / 32;
    constexpr int ST = BACK ? G_STATE : S_STATE;

    Where w;
    if (!locate(L, slot, w)) return;
    const int t = threadIdx.x, lane = t & 63, q = lane >> 4, l16 = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int32_t rep = L.H / L.G, g = block / L.blocks, blk = block % L.blocks;
    const int32_t h0 = g * rep + blk * HB, left = (g + 1) * rep - h0, heads = left < HB ? left : HB;
    const int64_t len = w.hi - w.lo;
    const int n_chunks = static_cast<int>((len + TOK - 1) / TOK);
    if (n_chunks == 0) return;

    const In &ra = BACK ? L.x : L.dy, &rb = BACK ? L.dy : L.x, &rc = BACK ? L.C : L.B;
    auto chunk_at = [&](int c) { return static_cast<int64_t>(BACK ? n_chunks - 1 - c : c) * TOK; };
    auto chunk_n = [&](int64_t off) { return static_cast<int>(len - off < TOK ? len - off : TOK); };
    auto load_ab = [&](int c, int hb, int buf) {
        const int64_t off = chunk_at(c);
        const int n = chunk_n(off);
        fetch_rows<TA, TOK, WAVES>(lds.a + buf * Lds::A_BYTES, ra.p + (w.lo + off) * ra.ld + (h0 + hb) * TA::RB, static_cast<uint32_t>(ra.ld), n, wave, lane);
        fetch_rows<TA, TOK, WAVES>(lds.b + buf * Lds::A_BYTES, rb.p + (w.lo + off) * rb.ld + (h0 + hb) * TA::RB, static_cast<uint32_t>(rb.ld), n, wave, lane);
    };
    auto load_c = [&](int c) {
        const int64_t off = chunk_at(c);
        fetch_rows<TC, TOK, WAVES>(lds.c, rc.p + (w.lo + off) * rc.ld + g * TC::RB, static_cast<uint32_t>(rc.ld), chunk_n(off), wave, lane);
    };
    auto dt_of = [&](int c, int hb) {
        const int64_t off = chunk_at(c);
        return load_dt<DT>(L, w.lo + off, chunk_n(off), h0 + hb, lane);
    };
    auto decays = [&](int c, int hb, float dt) {
        make_decays<TOK, HB, BACK>(lds.t, c, hb, dt, L.bias ? L.bias[h0 + hb] : 0.f, L.A[h0 + hb], chunk_n(chunk_at(c)), lane);
    };
    load_ab(0, 0, 0);
    load_c(0);
    for (int hb = wave; hb < heads; hb += WAVES) decays(0, hb, dt_of(0, hb));

    // ---- the states, transposed: row row(mt) + r of d_v, column 16 wave + l16 of d_k
    auto row = [&](int mt) { return BF ? 32 * (mt >> 1) + 8 * q + 4 * (mt & 1) : 16 * mt + 4 * q; };
    const int col = 16 * wave + l16;
    f32x4 M[HB][MT];
#pragma unroll
    for (int hb = 0; hb < HB; ++hb) {
        const float* src = nullptr;
        if (hb < heads) {
            if (w.n_seg > 1) src = L.seg_states[ST] + (static_cast<int64_t>(slot) * L.H + h0 + hb) * (DK * DV);
            else if (L.m_in[ST]) src = L.m_in[ST] + (static_cast<int64_t>(w.n) * L.H + h0 + hb) * (DK * DV);
        }
        const __amdgpu_buffer_rsrc_t rs = make_rsrc_u(src, src ? DK * DV * 4 : 0);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
            M[hb][mt] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, (col * DV + row(mt)) * 4, 0, 0));
    }

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
    auto channels_c = [&](int it, int kk) {          // of c's tile
        return lds_get<u32x4>(lds.c, TC::at(l16, (4 * kk + q) & 7) + it * TC::ROWS16 + (kk >> 1) * 128);
    };
    auto tokens = [&](uint32_t at, const uint8_t* sm, int rows16) {
        const u32x2 x = lds_transpose(sm + at), y = lds_transpose(sm + at + rows16);
        return u32x4{x[0], x[1], y[0], y[1]};
    };
    // the scores this wave makes: 16 bits: group wave, of tiles (it, 2 tg) and (it, 2 tg + 1); fp32: tile (it, jt)
    constexpr int GROUPS = BF ? 6 : 3, ROUNDS = (GROUPS + WAVES - 1) / WAVES, TILES = BF ? 2 : 1;
    auto tile_of = [&](int grp, int hh, int& it, int& jt) {
        if constexpr (BF) {
            const int tg = BACK ? (grp < 4) : (grp >= 4);
            it = BACK ? (grp & 3) : (grp < 4 ? grp : grp - 2);
            jt = 2 * tg + hh;
        } else {
            it = BACK ? (grp == 1) : (grp > 0);
            jt = BACK ? (grp > 0) : (grp == 1);
        }
    };

    int step = 0;
    float zA[BACK ? 1 : HB], zb[BACK ? 1 : HB];      // sums of z_ij (W_i - W_j)
#pragma unroll
    for (int hb = 0; hb < (BACK ? 1 : HB); ++hb) zA[hb] = zb[hb] = 0.f;
    for (int c = 0; c < n_chunks; ++c) {
        const int64_t off = chunk_at(c), tok0 = w.lo + off;
        const int n = chunk_n(off), buf = c & 1;
        f32x4 O[IT], P[ROUNDS][TILES], CB[BACK ? 1 : ROUNDS][TILES];
        u32x2 cr[!BACK && BF ? IT : 1];
        f32x4 cf[!BACK && !BF ? IT : 1];
#pragma unroll
        for (int it = 0; it < IT; ++it) O[it] = zero4();
#pragma unroll
        for (int i = 0; i < ROUNDS; ++i)
#pragma unroll
            for (int hh = 0; hh < TILES; ++hh) P[i][hh] = zero4();
        constexpr int CJ = BF ? JG : IT;
        u32x4 vf[CJ];
#pragma unroll
        for (int hb = 0; hb < HB; ++hb) {
            if (hb >= heads) break;
            __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
            lds_barrier();                           // this head's rows are there
            const uint8_t *sa = lds.a + (step & 1) * Lds::A_BYTES, *sb = lds.b + (step & 1) * Lds::A_BYTES;
            ++step;
            const bool more = c + 1 < n_chunks;
            if (hb + 1 < heads) load_ab(c, hb + 1, step & 1);
            else if (more) load_ab(c + 1, 0, step & 1);
            float dt_next = 0.f;
            if (wave == WAVES - 1 && more) dt_next = dt_of(c + 1, hb);
            if (hb == 0) {                           // what the chunk's heads share
#pragma unroll
                for (int j = 0; j < CJ; ++j) {
                    if constexpr (BF) vf[j] = tokens(tok_c + 2 * j * TC::ROWS16, lds.c, TC::ROWS16);
                    else
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            vf[j][r] = lds_get<uint32_t>(lds.c, TC::at(16 * j + 4 * q + r, 4 * wave + (l16 >> 2)) + 4 * (l16 & 3));
                }
                if constexpr (!BACK) {               // C . B of the wave's scores, C of its tokens and columns
                    const uint32_t ld = static_cast<uint32_t>(L.C.ld);
                    const __amdgpu_buffer_rsrc_t rC = make_rsrc_u(L.C.p + tok0 * L.C.ld + g * TC::RB, (n - 1) * ld + TC::RB);
#pragma unroll
                    for (int it = 0; it < IT; ++it) {
                        const uint32_t at = (16 * it + l16) * ld + (16 * wave + 4 * q) * ES;
                        if constexpr (BF) cr[it] = __builtin_amdgcn_raw_buffer_load_b64(rC, at, 0, 0);
                        else cf[it] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rC, at, 0, 0));
                    }
#pragma unroll
                    for (int i = 0; i < ROUNDS; ++i) {
                        const int grp = wave + i * WAVES;
#pragma unroll
                        for (int hh = 0; hh < TILES; ++hh) CB[i][hh] = zero4();
                        if (grp >= GROUPS) continue;
                        int it, jt;
                        tile_of(grp, 0, it, jt);
                        if constexpr (BF) {
#pragma unroll
                            for (int kk = 0; kk < DK / 32; ++kk) {
                                const u32x4 a = __builtin_amdgcn_raw_buffer_load_b128(rC, (16 * it + l16) * ld + (32 * kk + 8 * q) * 2, 0, 0);
#pragma unroll
                                for (int hh = 0; hh < 2; ++hh) CB[i][hh] = mfma_bf16(channels_c(jt + hh, kk), a, CB[i][hh]);
                            }
                        } else {
#pragma unroll
                            for (int mt = 0; mt < DK / 16; ++mt) {
                                const f32x4 a = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rC, (16 * it + l16) * ld + (16 * mt + 4 * q) * 4, 0, 0));
                                const f32x4 b = lds_get<f32x4>(lds.c, TC::at(16 * jt + l16, 4 * mt + q));
#pragma unroll
                                for (int r = 0; r < 4; ++r) CB[i][0] = mfma_f32(b[r], a[r], CB[i][0]);
                            }
                        }
                    }
                }
            }
            const double* cum = lds.t.cum[buf][hb];
            const float* del = lds.t.del[buf][hb];
            // ---- scores
#pragma unroll
            for (int i = 0; i < ROUNDS; ++i) {
                const int grp = wave + i * WAVES;
                if (grp >= GROUPS) continue;
                f32x4 X[TILES];
                int it, jt;
                tile_of(grp, 0, it, jt);
#pragma unroll
                for (int hh = 0; hh < TILES; ++hh) X[hh] = zero4();
                if constexpr (BF) {
#pragma unroll
                    for (int kk = 0; kk < KK; ++kk) {
                        const u32x4 a = channels(sa, it, kk);
#pragma unroll
                        for (int hh = 0; hh < 2; ++hh) X[hh] = mfma_bf16(channels(sb, jt + hh, kk), a, X[hh]);
                    }
                } else {
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        const f32x4 a = lds_get<f32x4>(sa, TA::at(16 * it + l16, 4 * mt + q));
                        const f32x4 b = lds_get<f32x4>(sb, TA::at(16 * jt + l16, 4 * mt + q));
#pragma unroll
                        for (int r = 0; r < 4; ++r) X[0] = mfma_f32(b[r], a[r], X[0]);
                    }
                }
                if constexpr (BACK) {
#pragma unroll
                    for (int hh = 0; hh < TILES; ++hh) P[i][hh] += X[hh] * score_weights<true, false, true>(cum, del, it, jt + hh, q, l16);
                } else {
                    float rows = 0.f, diag = 0.f;
                    const int ti = 16 * it + l16;
                    const double di = lds.t.dsum[buf][hb][ti], si = lds.t.ssum[buf][hb][ti];
#pragma unroll
                    for (int hh = 0; hh < TILES; ++hh) {
                        const int tj = 16 * (jt + hh) + 4 * q;
                        const f32x4 dj = lds_get<f32x4>(del, 4 * tj), x = X[hh] * score_weights<false, false, false>(cum, del, it, jt + hh, q, l16);
                        P[i][hh] += x * dj;
                        f32x4 cols;
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const float y = x[r] * CB[i][hh][r], below = tj + r < ti ? y : 0.f, z = below * dj[r];
                            if (tj + r == ti) diag += y;
                            rows += z;
                            zA[hb] = __builtin_fmaf(z, static_cast<float>(di - lds.t.dsum[buf][hb][tj + r]), zA[hb]);
                            zb[hb] = __builtin_fmaf(z, static_cast<float>(si - lds.t.ssum[buf][hb][tj + r]), zb[hb]);
                            cols[r] = row_sum(below);
                        }
                        if (l16 == 15) *reinterpret_cast<f32x4*>(&lds.red[hb][WAVES + 2 + it][tj]) = cols;
                    }
                    rows += __shfl_xor(rows, 16, 64);
                    rows += __shfl_xor(rows, 32, 64);
                    if (q == 0) lds.red[hb][WAVES + (BF ? jt / 2 : jt)][ti] = rows;
                    if (BF ? it / 2 == jt / 2 : it == jt) {        // the group of the tile's own tokens
                        diag += __shfl_xor(diag, 16, 64);
                        diag += __shfl_xor(diag, 32, 64);
                        if (q == 0) lds.red[hb][Lds::RED - 1][ti] = diag;
                    }
                }
            }
            // ---- the state's part
            f32x4 own[IT];
#pragma unroll
            for (int it = 0; it < IT; ++it) own[it] = zero4();
            if constexpr (BF) {
#pragma unroll
                for (int kk = 0; kk < KK; ++kk) {
                    u32x4 hi, mid, lo, a[IT];
#pragma unroll
                    for (int it = 0; it < IT; ++it) a[it] = channels(sa, it, kk);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const f32x4& m = M[hb][2 * kk + (e >> 1)];
                        uint32_t x, y, z = 0;
                        if constexpr (!BACK) split3(m[2 * (e & 1)], m[2 * (e & 1) + 1], x, y, z);
                        else split_pair(m[2 * (e & 1)], m[2 * (e & 1) + 1], x, y);
                        hi[e] = x;
                        mid[e] = y;
                        lo[e] = z;
                    }
#pragma unroll
                    for (int it = 0; it < IT; ++it) own[it] = mfma_bf16(hi, a[it], own[it]);
#pragma unroll
                    for (int it = 0; it < IT; ++it) own[it] = mfma_bf16(mid, a[it], own[it]);
                    if constexpr (!BACK)
#pragma unroll
                        for (int it = 0; it < IT; ++it) own[it] = mfma_bf16(lo, a[it], own[it]);
                }
            } else {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int it = 0; it < IT; ++it) {
                        const f32x4 a = lds_get<f32x4>(sa, TA::at(16 * it + l16, 4 * mt + q));
#pragma unroll
                        for (int r = 0; r < 4; ++r) own[it] = mfma_f32(M[hb][mt][r], a[r], own[it]);
                    }
            }
            const double all = cum[TOK - 1];
#pragma unroll
            for (int it = 0; it < IT; ++it) {
                const double ci = cum[16 * it + l16];
                own[it] *= chunk_sign(c) * (BACK ? del[16 * it + l16] * pow2(all - ci) : pow2(ci));
                O[it] += own[it];
                if constexpr (!BACK) {
                    f32x4 cc;
                    if constexpr (BF) cc = f32x4{lo_f32(cr[it][0]), hi_f32(cr[it][0]), lo_f32(cr[it][1]), hi_f32(cr[it][1])};
                    else cc = cf[it];
                    float s = 0.f;
#pragma unroll
                    for (int r = 0; r < 4; ++r) s = __builtin_fmaf(cc[r], own[it][r], s);
                    s += __shfl_xor(s, 16, 64);
                    s += __shfl_xor(s, 32, 64);
                    if (q == 0) lds.red[hb][wave][16 * it + l16] = s;
                }
            }
            // ---- update
            decay_state(M[hb], lds.t.over[buf][hb]);
            const float* up = lds.t.up[buf][hb];
            if constexpr (BF) {
#pragma unroll
                for (int tg = 0; tg < JG; ++tg) {
                    const f32x4 w0 = lds_get<f32x4>(up, 4 * (32 * tg + 4 * q));
                    const f32x4 w1 = lds_get<f32x4>(up, 4 * (32 * tg + 16 + 4 * q));
                    u32x4 ch, cm, cl;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const f32x4& ww = e < 2 ? w0 : w1;
                        const float c0 = lo_f32(vf[tg][e]) * ww[2 * (e & 1)], c1 = hi_f32(vf[tg][e]) * ww[2 * (e & 1) + 1];
                        uint32_t x, y, z = 0;
                        if constexpr (!BACK) split3(c0, c1, x, y, z);
                        else split_pair(c0, c1, x, y);
                        ch[e] = x;
                        cm[e] = y;
                        cl[e] = z;
                    }
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        const u32x4 kt = tokens(tok[(mt >> 1) & 1] + 2 * tg * TA::ROWS16 + (mt >> 2) * 128 + 8 * (mt & 1), sb,
                                                TA::ROWS16);
                        if constexpr (!BACK) M[hb][mt] = mfma_bf16(kt, cl, M[hb][mt]);
                        M[hb][mt] = mfma_bf16(kt, cm, M[hb][mt]);
                        M[hb][mt] = mfma_bf16(kt, ch, M[hb][mt]);
                    }
                }
            } else {
#pragma unroll
                for (int jt = 0; jt < IT; ++jt) {
                    const f32x4 ww = lds_get<f32x4>(up, 4 * (16 * jt + 4 * q));
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float cw = __uint_as_float(vf[jt][r]) * ww[r];
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt)
                            M[hb][mt] = mfma_f32(lds_get<float>(sb, TA::at(16 * jt + 4 * q + r, 4 * mt + (l16 >> 2)) + 4 * (l16 & 3)),
                                                 cw, M[hb][mt]);
                    }
                }
            }
            if (wave == WAVES - 1 && more) decays(c + 1, hb, dt_next);
        }
        // ---- the scores, summed over the heads
#pragma unroll
        for (int i = 0; i < ROUNDS; ++i) {
            const int grp = wave + i * WAVES;
            if (grp >= GROUPS) continue;
            if constexpr (BF) {
                u32x4 hi, lo;
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    uint32_t x0, y0, x1, y1;
                    split_pair(P[i][hh][0], P[i][hh][1], x0, y0);
                    split_pair(P[i][hh][2], P[i][hh][3], x1, y1);
                    hi[2 * hh] = x0; hi[2 * hh + 1] = x1;
                    lo[2 * hh] = y0; lo[2 * hh + 1] = y1;
                }
                lds_put(lds.p, grp * 2048 + lane * 16, hi);
                lds_put(lds.p, grp * 2048 + 1024 + lane * 16, lo);
            } else {
                lds_put(lds.p, grp * 1024 + lane * 16, P[i][0]);
            }
        }
        lds_barrier();                               // the scores and the sums are there, c has been read
        if (c + 1 < n_chunks) load_c(c + 1);
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
                const f32x4 X = lds_get<f32x4>(lds.p, tile * 1024 + lane * 16);
#pragma unroll
                for (int r = 0; r < 4; ++r) O[it] = mfma_f32(__uint_as_float(vf[jt][r]), X[r], O[it]);
            }
        }
        if constexpr (!BACK) {
            for (int e = t; e < heads * TOK; e += WAVES * 64) {
                const int hb = e / TOK, at = e % TOK;
                // 64 (32) tokens: the second half's z also reach to the first half, and are reached from it
                float rows = lds.red[hb][WAVES][at], cols = 0.f, p = 0.f;
                if (at >= TOK / 2) rows += lds.red[hb][WAVES + 1][at];
                for (int x = at / (TOK / 2) * (IT / 2); x < IT; ++x) cols += lds.red[hb][WAVES + 2 + x][at];
#pragma unroll
                for (int x = 0; x < WAVES; ++x) p += lds.red[hb][x][at];
                if (at < n) {
                    const int64_t i = (h0 + hb) * L.total + tok0 + at;
                    L.zz[i] = rows - lds.t.del[buf][hb][at] * cols;
                    L.xz[i] = cols + lds.red[hb][Lds::RED - 1][at];
                    L.pp[i] = p;
                }
            }
        }
        // ---- out: lane l16 holds token 16 it + l16, four neighbouring columns
        if (L.part[ST]) {
            const uint32_t orow = static_cast<uint32_t>(L.G) * DK * 4;
            const __amdgpu_buffer_rsrc_t ro = make_rsrc_u(L.part[ST] + ((blk * L.total + tok0) * L.G + g) * DK, (n - 1) * orow + DK * 4);
#pragma unroll
            for (int it = 0; it < IT; ++it)
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, O[it]), ro,
                                                       (16 * it + l16) * orow + (16 * wave + 4 * q) * 4, 0, 0);
        } else {
            const Out& out = L.out[ST];
            const uint32_t orow = static_cast<uint32_t>(out.ld);
            const __amdgpu_buffer_rsrc_t ro = make_rsrc_u(out.p + tok0 * out.ld + g * TC::RB, (n - 1) * orow + TC::RB);
#pragma unroll
            for (int it = 0; it < IT; ++it) {
                const uint32_t at = (16 * it + l16) * orow + (16 * wave + 4 * q) * ES;
                if constexpr (BF)
                    __builtin_amdgcn_raw_buffer_store_b64(u32x2{pack_bf16(O[it][0], O[it][1]), pack_bf16(O[it][2], O[it][3])}, ro, at, 0, 0);
                else __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, O[it]), ro, at, 0, 0);
            }
        }
    }
    if constexpr (!BACK) {
        lds_barrier();                               // the last chunk's sums have been read
#pragma unroll
        for (int hb = 0; hb < HB; ++hb) {
#pragma unroll
            for (int off = 1; off < 64; off <<= 1) {
                zA[hb] += __shfl_xor(zA[hb], off, 64);
                zb[hb] += __shfl_xor(zb[hb], off, 64);
            }
            if (lane == 0) {
                lds.red[hb][0][wave] = zA[hb];
                lds.red[hb][1][wave] = zb[hb];
            }
        }
        lds_barrier();
        if (t < 2 * heads) {
            float sum = 0.f;
            for (int x = 0; x < WAVES; ++x) sum += lds.red[t >> 1][t & 1][x];
            (t & 1 ? L.zb : L.zA)[static_cast<int64_t>(slot) * L.H + h0 + (t >> 1)] = sum;
        }
    }
}

template <int DT, int DK, int DV, int HB>
__global__ void __launch_bounds__(DK * 4, DK == 128 ? 2 : 1) shared_kernel(Scan L) {
    __shared__ union {
        SharedLds<DT, DK, DV, HB, false> c;
        SharedLds<DT, DK, DV, HB, true> b;
    } lds;
    uint32_t unit;
    int32_t pass;
    const uint32_t blocks = static_cast<uint32_t>(L.blocks) * L.G;
    if (!unit_of(L.slots * blocks, 2, unit, pass)) return;
    if (pass == 0) shared_pass<DT, DK, DV, HB, false>(L, unit / blocks, unit % blocks, lds.c);
    else shared_pass<DT, DK, DV, HB, true>(L, unit / blocks, unit % blocks, lds.b);
}

// ---------------------------------------------------------------- ddt, dA, dbias; sums over blocks and segments

// One wave per (segment, head): from its last chunk to its first, lane l has the token l before the chunk's last.
template <int DT>
__global__ void __launch_bounds__(256) decay_grad_kernel(Scan L) {
    const int64_t u = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    if (u >= static_cast<int64_t>(L.slots) * L.H) return;
    const int32_t slot = static_cast<int32_t>(u / L.H), h = static_cast<int32_t>(u % L.H);
    Where w;
    if (!locate(L, slot, w) || w.hi == w.lo) {       // no such segment, or an empty one: nothing to add up
        if (lane == 0) L.dAp[u] = L.dbp[u] = L.dDp[u] = 0.f;
        return;
    }
    const double A = static_cast<double>(L.A[h]);
    const float bias = L.bias ? L.bias[h] : 0.f;
    double end = static_cast<double>(L.E[u]);        // <G, S> behind the tokens in hand
    double dA = 0.0, db = 0.0, own = 0.0;            // a lane's part of sum delta dg, sum slope dg, sum slope x . u
    const int64_t row = h * L.total;
    constexpr int TOK = DT == KDA_BF16 ? 64 : 32;
    for (int64_t lo = w.lo + (w.hi - w.lo - 1) / TOK * TOK; lo >= w.lo; lo -= TOK) {
        const int64_t hi = lo + TOK < w.hi ? lo + TOK : w.hi, tok = hi - 1 - lane;
        const bool in = tok >= lo;
        double x = 0.0, z = 0.0, p = 0.0, r = 0.0;
        Strength s = {0.f, 0.f};
        if (in) {
            s = strength(load_as_f32<DT>(L.dt.p + tok * L.dt.ld, h), bias);
            const float later = L.xr[row + tok];
            x = static_cast<double>(L.xz[row + tok]) + later;
            z = static_cast<double>(L.zz[row + tok]);
            p = static_cast<double>(L.pp[row + tok]);
            r = static_cast<double>(s.delta) * later;
        }
        const double delta = static_cast<double>(s.delta), slope = static_cast<double>(s.slope);
        // sums over the tokens from a lane's own to the last
        const double zs = prefix_sum(z + p), ps = prefix_sum(p), rs = prefix_sum(r), ds = prefix_sum(delta), ss = prefix_sum(slope);
        const double r_all = lane_value(rs, 63), d_all = lane_value(ds, 63), s_all = lane_value(ss, 63);
        // Where a chunk or a token decays by more than e^-14, what goes through it is below the difference's rounding
        // (about 2^-20 of <G, S>, which W would multiply): it is taken as zero, and the sums start anew before it.
        const double through = d_all * A < -14.0 ? 0.0 : end - r_all;
        const uint64_t cuts = __ballot(in && delta * A < -14.0), seen = cuts & (~uint64_t(0) >> (63 - lane));
        const int cut = seen ? 63 - __builtin_clzll(seen) : -1;
        const double from = shuffle(zs - rs, cut < 0 ? 0 : cut);
        const double g = cut == lane ? 0.0 : (zs - rs) + (cut < 0 ? through + r_all : -from);
        end = through + lane_value(ps, 63);
        if (in) store_from_f32<DT>(L.ddt.p + tok * L.ddt.ld, h, static_cast<float>((x + A * g) * slope));
        // W_i = all - (from i on) + w_i, W_n - W_j = (from j on) - w_j
        dA += p * (d_all - ds + delta) + r * (ds - delta);
        db += p * (s_all - ss + slope) + r * (ss - slope);
        own += slope * x;
        if (lane == 0) {
            dA += through * d_all;
            db += through * s_all;
        }
    }
    if (lane == 0) {
        dA += static_cast<double>(L.zA[u]);
        db += static_cast<double>(L.zb[u]);
    }
    db = own + A * db;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        dA += __shfl_xor(dA, off, 64);
        db += __shfl_xor(db, off, 64);
    }
    if (lane == 0) {
        L.dAp[u] = static_cast<float>(dA);
        L.dbp[u] = static_cast<float>(db);
    }
}

// dB and dC: sums of the head blocks' parts, four channels a lane; only the tokens that belong to a sequence.
template <int DT>
__global__ void __launch_bounds__(256) part_sum_kernel(Scan L, int32_t row, int64_t quads) {
    const int64_t e = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4;
    if (e >= quads * 4) return;
    const int64_t tok = e / row;
    if (L.cu) {
        const int64_t from = L.cu[0], to = L.cu[L.n_seqs];
        if (tok < from || tok >= to) return;
    }
    const float* p = L.part[blockIdx.y];
    f32x4 s = *reinterpret_cast<const f32x4*>(p + e);
    for (int32_t b = 1; b < L.blocks; ++b) s += *reinterpret_cast<const f32x4*>(p + b * L.total * row + e);
    const Out& out = L.out[blockIdx.y];
    store4_from_f32<DT>(out.p + tok * out.ld, e % row, make_float4(s[0], s[1], s[2], s[3]));
}

// dA, dbias and dD of head blockIdx.x: sums over the segments.
__global__ void __launch_bounds__(256) head_sum_kernel(Scan L) {
    __shared__ double red[3][4];
    const int32_t h = blockIdx.x;
    double s[3] = {};
    for (int32_t i = threadIdx.x; i < L.slots; i += 256) {
        const int64_t u = static_cast<int64_t>(i) * L.H + h;
        s[0] += L.dAp[u];
        s[1] += L.dbp[u];
        s[2] += L.dDp[u];
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) {
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) s[k] += __shfl_xor(s[k], off, 64);
        if ((threadIdx.x & 63) == 0) red[k][threadIdx.x >> 6] = s[k];
    }
    __syncthreads();
    if (threadIdx.x < 3) {
        const int k = threadIdx.x;
        float* out = k == 0 ? L.dA : k == 1 ? L.dbias : L.dD;
        if (out) out[h] = static_cast<float>((red[k][0] + red[k][1]) + (red[k][2] + red[k][3]));
    }
}

// ---------------------------------------------------------------- host side

int32_t head_blocks(int32_t H, int32_t G, int HB) { return (H / G + HB - 1) / HB; }
int value_heads(int32_t H, int32_t G, int32_t dv) { return dv == 64 && H / G > 1 ? 2 : 1; }
int shared_heads(int32_t H, int32_t G, int32_t dv) {
    const int32_t rep = H / G;
    return rep == 1 ? 1 : (rep == 2 || dv == 128 ? 2 : 4);
}

// Tokens per segment, a multiple of 64.
int32_t forward_segment(int32_t n_seqs, int64_t total, int32_t blocks, int32_t in_dtype, bool packed) {
    const int64_t units = int64_t(n_seqs) * blocks, longest = packed ? total : total / n_seqs;
    if (units >= 256 || longest < 1024) return WHOLE;
    const int64_t shares = packed ? std::max<int64_t>(1, 512 / blocks - n_seqs / 2) : 512 / units;
    const int64_t seg = std::max<int64_t>(((longest + shares - 1) / shares + 63) / 64 * 64, in_dtype == KDA_BF16 ? 256 : 128);
    return seg >= longest || seg >= WHOLE ? WHOLE : static_cast<int32_t>(seg);
}
int32_t backward_segment(int32_t, int64_t, int32_t, int32_t, bool) { return 512; }

int64_t segment_slots(int32_t n_seqs, int64_t total, int32_t seg, bool packed) {
    if (packed) return total / seg + n_seqs;
    return n_seqs * std::max<int64_t>(1, (total / n_seqs + seg - 1) / seg);
}

// The workspace's parts, each on a 256-byte border.
struct Carver {
    uint8_t* base;
    size_t used = 0;
    template <typename T>
    T* take(int64_t count) {
        T* p = reinterpret_cast<T*>(base + used);
        used += (static_cast<size_t>(count) * sizeof(T) + 255) / 256 * 256;
        return p;
    }
};

void carve_forward(Scan& L, Carver& ws, int64_t elems) {
    if (L.seg == WHOLE) return;
    L.seg_states[S_STATE] = ws.take<float>(int64_t(L.slots) * L.H * elems);
    L.seg_log[S_STATE] = ws.take<double>(int64_t(L.slots) * L.H);
}
void carve_backward(Scan& L, Carver& ws, int64_t elems, int32_t dk, bool last) {
    const int64_t su = int64_t(L.slots) * L.H;
    for (int st : {S_STATE, G_STATE}) {
        L.seg_states[st] = ws.take<float>(su * elems);
        L.seg_log[st] = ws.take<double>(su);
    }
    float* S_last = ws.take<float>(int64_t(L.n_seqs) * L.H * elems);
    L.S_last = last ? S_last : nullptr;
    if (L.blocks > 1)
        for (int st : {S_STATE, G_STATE}) L.part[st] = ws.take<float>(L.total * L.G * dk * L.blocks);
    for (float** p : {&L.zz, &L.pp, &L.xz, &L.xr}) *p = ws.take<float>(L.H * L.total);
    for (float** p : {&L.zA, &L.zb, &L.E, &L.dDp, &L.dAp, &L.dbp}) *p = ws.take<float>(su);
}

void set_segments(Scan& L, bool backward, int32_t dv, int32_t in_dtype, bool packed) {
    const int32_t vb = head_blocks(L.H, L.G, value_heads(L.H, L.G, dv)) * L.G;
    L.seg = (backward ? backward_segment : forward_segment)(L.n_seqs, L.total, vb, in_dtype, packed);
    L.slots = static_cast<int32_t>(segment_slots(L.n_seqs, L.total, L.seg, packed));
    L.n_seg = L.slots / L.n_seqs;
}

Scan base(const ScanArgs& a) {
    const int64_t es = a.in_dtype == KDA_BF16 ? 2 : 4;
    auto in = [&](const RowsIn& r) { return In{static_cast<const uint8_t*>(r.p), r.ld * es}; };
    Scan L{};
    L.x = in(a.x); L.dt = in(a.dt); L.B = in(a.B); L.C = in(a.C); L.dy = in(a.dy);
    L.A = a.A; L.bias = a.bias; L.D = a.D; L.cu = a.cu; L.T = a.T; L.total = int64_t(a.batch) * a.T;
    L.n_seqs = a.n_seqs; L.H = a.H; L.G = a.G;
    L.m_in[S_STATE] = a.h0; L.m_in[G_STATE] = a.dhT;
    return L;
}

template <int V>
using Int = std::integral_constant<int, V>;
template <typename F>
hipError_t by_sizes(int32_t dk, int32_t dv, F go) {
    if (dk == 128) return dv == 128 ? go(Int<128>{}, Int<128>{}) : go(Int<128>{}, Int<64>{});
    return dv == 128 ? go(Int<64>{}, Int<128>{}) : go(Int<64>{}, Int<64>{});
}
unsigned xcd_grid(int64_t units, int32_t passes) { return static_cast<unsigned>((units + 7) / 8 * 8 * passes); }

template <int DT, int ODT, int MODE>
hipError_t launch_value(Scan L, int32_t dk, int32_t dv, hipStream_t stream) {
    return by_sizes(dk, dv, [&](auto k, auto v) {
        constexpr int DK = decltype(k)::value, DV = decltype(v)::value;
        auto go = [&](auto heads) {
            constexpr int HB = decltype(heads)::value;
            L.blocks = head_blocks(L.H, L.G, HB);
            hipLaunchKernelGGL((value_kernel<DT, ODT, DK, DV, HB, MODE>), dim3(xcd_grid(int64_t(L.slots) * L.blocks * L.G, 1)),
                               dim3(HB * DV * 4), 0, stream, L);
            return hipGetLastError();
        };
        if constexpr (DV == 64)
            if (value_heads(L.H, L.G, dv) == 2) return go(Int<2>{});
        return go(Int<1>{});
    });
}
template <int DT>
hipError_t launch_states(Scan L, int32_t dk, int32_t dv, int32_t first, int32_t passes, hipStream_t stream) {
    const hipError_t e = by_sizes(dk, dv, [&](auto k, auto v) {
        constexpr int DK = decltype(k)::value, DV = decltype(v)::value;
        auto go = [&](auto heads) {
            constexpr int HB = decltype(heads)::value;
            L.blocks = head_blocks(L.H, L.G, HB);
            hipLaunchKernelGGL((state_kernel<DT, DK, DV, HB>), dim3(xcd_grid(int64_t(L.slots) * L.blocks * L.G, passes)),
                               dim3(HB * DV * 4), 0, stream, L, first, passes);
            return hipGetLastError();
        };
        if constexpr (DV == 64)
            if (value_heads(L.H, L.G, dv) == 2) return go(Int<2>{});
        return go(Int<1>{});
    });
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(scan_kernel, dim3(static_cast<unsigned>(L.n_seqs * L.H), static_cast<unsigned>(dk * dv / 1024), passes),
                       dim3(256), 0, stream, L, dk * dv, first);
    return hipGetLastError();
}

template <int DT, int ODT>
hipError_t forward(const ScanArgs& a, hipStream_t stream) {
    Scan L = base(a);
    set_segments(L, false, a.dv, a.in_dtype, a.cu != nullptr);
    Carver ws{static_cast<uint8_t*>(a.workspace)};
    carve_forward(L, ws, int64_t(a.dk) * a.dv);
    L.m_out[S_STATE] = a.hT;
    L.exact[S_STATE] = a.hT != nullptr;
    L.out[0] = Out{static_cast<uint8_t*>(a.y.p), a.y.ld * (ODT == KDA_BF16 ? 2 : 4)};
    if (L.seg < WHOLE) {
        const hipError_t e = launch_states<DT>(L, a.dk, a.dv, S_STATE, 1, stream);
        if (e != hipSuccess) return e;
    }
    return launch_value<DT, ODT, Y>(L, a.dk, a.dv, stream);
}

template <int DT>
hipError_t backward(const ScanArgs& a, hipStream_t stream) {
    const int64_t es = DT == KDA_BF16 ? 2 : 4;
    auto out = [&](const RowsOut& r) { return Out{static_cast<uint8_t*>(r.p), r.ld * es}; };
    Scan L = base(a);
    set_segments(L, true, a.dv, a.in_dtype, a.cu != nullptr);
    const int HB = shared_heads(a.H, a.G, a.dv);
    L.blocks = head_blocks(a.H, a.G, HB);
    Carver ws{static_cast<uint8_t*>(a.workspace)};
    carve_backward(L, ws, int64_t(a.dk) * a.dv, a.dk, a.dhT != nullptr);
    L.m_out[G_STATE] = a.dh0;
    L.exact[S_STATE] = L.exact[G_STATE] = 1;
    L.ddt = out(a.ddt);
    L.dA = a.dA; L.dD = a.dD; L.dbias = a.dbias;
    hipError_t e = hipSuccess;
    // one segment a sequence and no gradient behind it: all states are known
    if (L.cu || L.n_seg > 1 || L.S_last) e = launch_states<DT>(L, a.dk, a.dv, S_STATE, 2, stream);
    if (e != hipSuccess) return e;
    L.out[S_STATE] = out(a.dC);
    L.out[G_STATE] = out(a.dB);
    e = by_sizes(a.dk, a.dv, [&](auto k, auto v) {
        constexpr int DK = decltype(k)::value, DV = decltype(v)::value;
        auto go = [&](auto heads) {
            hipLaunchKernelGGL((shared_kernel<DT, DK, DV, decltype(heads)::value>),
                               dim3(xcd_grid(int64_t(L.slots) * L.blocks * L.G, 2)), dim3(DK * 4), 0, stream, L);
            return hipGetLastError();
        };
        if (HB == 1) return go(Int<1>{});
        if constexpr (DV == 64)
            if (HB == 4) return go(Int<4>{});
        return go(Int<2>{});
    });
    if (e != hipSuccess) return e;
    if (L.blocks > 1 && L.total > 0) {
        const int32_t row = a.G * a.dk;
        const int64_t quads = L.total * row / 4;
        hipLaunchKernelGGL(part_sum_kernel<DT>, dim3(static_cast<unsigned>((quads + 255) / 256), 2), dim3(256), 0, stream, L, row, quads);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    L.out[0] = out(a.dx);
    e = launch_value<DT, DT, DX>(L, a.dk, a.dv, stream);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(decay_grad_kernel<DT>, dim3(static_cast<unsigned>((int64_t(L.slots) * L.H + 3) / 4)), dim3(256), 0, stream, L);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(head_sum_kernel, dim3(L.H), dim3(256), 0, stream, L);
    return hipGetLastError();
}

}  // namespace

size_t scan_workspace_bytes(int32_t n_seqs, int64_t total, int32_t H, int32_t G, int32_t dk, int32_t dv,
                            int32_t in_dtype, bool backward) {
    // what a packed batch of these sizes needs, or fixed-length sequences: whichever is more
    size_t most = 0;
    for (const bool packed : {false, true}) {
        Scan L{};
        L.n_seqs = n_seqs; L.total = total; L.H = H; L.G = G;
        set_segments(L, backward, dv, in_dtype, packed);
        Carver ws{nullptr};
        if (backward) {
            L.blocks = head_blocks(H, G, shared_heads(H, G, dv));
            carve_backward(L, ws, int64_t(dk) * dv, dk, true);
        } else {
            carve_forward(L, ws, int64_t(dk) * dv);
        }
        most = std::max(most, ws.used);
    }
    return most;
}

hipError_t launch_scan_fwd(const ScanArgs& a, hipStream_t stream) {
    if (a.in_dtype == KDA_BF16)
        return a.y_dtype == KDA_BF16 ? forward<KDA_BF16, KDA_BF16>(a, stream) : forward<KDA_BF16, KDA_F32>(a, stream);
    return a.y_dtype == KDA_BF16 ? forward<KDA_F32, KDA_BF16>(a, stream) : forward<KDA_F32, KDA_F32>(a, stream);
}

hipError_t launch_scan_bwd(const ScanArgs& a, hipStream_t stream) {
    return a.in_dtype == KDA_BF16 ? backward<KDA_BF16>(a, stream) : backward<KDA_F32>(a, stream);
}

// ---------------------------------------------------------------- one token
namespace {

// One workgroup per (sequence, head): the state is read once, updated in registers and written once (non-temporal
// both ways).  Lane t owns four columns of DK / RG rows.
template <int DT, int ODT, int DK, int DV>
__global__ void __launch_bounds__(256) step_kernel(Scan L, float* __restrict__ states, const int32_t* __restrict__ slots,
                                                   int32_t N, int32_t n_slots) {
    constexpr int CG = DV / 4, RG = 256 / CG, RPT = DK / RG;
    __shared__ float sb[DK], sc[DK];
    __shared__ f32x4 red[RG][CG];
    const int32_t n = blockIdx.x / L.H, h = blockIdx.x % L.H, g = h / (L.H / L.G);
    const int t = threadIdx.x, cg = t % CG, rg = t / CG;
    const int32_t slot = slots ? slots[n] : n;
    uint8_t* out = L.out[0].p + n * L.out[0].ld;
    bool live = slot >= 0 && slot < n_slots;
    float* S = states + (static_cast<int64_t>(live ? slot : 0) * L.H + h) * (DK * DV) + 4 * cg;
    f32x4 s[RPT];
    if (live) {
#pragma unroll
        for (int i = 0; i < RPT; ++i) s[i] = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(S + (rg * RPT + i) * DV));
    }
    if (t < DK) {
        sb[t] = load_as_f32<DT>(L.B.p + n * L.B.ld, g * DK + t);
        sc[t] = load_as_f32<DT>(L.C.p + n * L.C.ld, g * DK + t);
    }
    const float4 xx = load4_as_f32<DT>(L.x.p + n * L.x.ld, h * DV + 4 * cg);
    const Strength st = strength(load_as_f32<DT>(L.dt.p + n * L.dt.ld, h), L.bias ? L.bias[h] : 0.f);
    const double a = exp(static_cast<double>(st.delta) * static_cast<double>(L.A[h]));
    const float a_hi = static_cast<float>(a), a_lo = static_cast<float>(a - static_cast<double>(a_hi));
    const float D = L.D ? L.D[h] : 0.f;
    bool later = false;                              // a later sequence with the same slot takes it
    if (slots && live)
        for (int32_t m = n + 1 + t; m < N; m += 256) later |= slots[m] == slot;
    if (__syncthreads_or(later)) live = false;
    if (!live) {
        if (rg == 0) store4_from_f32<ODT>(out, h * DV + 4 * cg, make_float4(0.f, 0.f, 0.f, 0.f));
        return;
    }
    const f32x4 x = {xx.x, xx.y, xx.z, xx.w};
    f32x4 acc = zero4();
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int r = rg * RPT + i;
        const float br = sb[r] * st.delta, cr = sc[r];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            s[i][e] = __builtin_fmaf(a_hi, s[i][e], __builtin_fmaf(br, x[e], a_lo * s[i][e]));
            acc[e] = __builtin_fmaf(cr, s[i][e], acc[e]);
        }
        __builtin_nontemporal_store(s[i], reinterpret_cast<f32x4*>(S + r * DV));
    }
    red[rg][cg] = acc;
    __syncthreads();
    if (rg == 0) {
        f32x4 sum = red[0][cg];
#pragma unroll
        for (int r = 1; r < RG; ++r) sum += red[r][cg];
        sum += D * x;
        store4_from_f32<ODT>(out, h * DV + 4 * cg, make_float4(sum[0], sum[1], sum[2], sum[3]));
    }
}

}  // namespace

hipError_t launch_scan_step(const ScanArgs& a, float* states, const int32_t* slots, int32_t N, int32_t n_slots,
                            hipStream_t stream) {
    Scan L = base(a);
    L.out[0] = Out{static_cast<uint8_t*>(a.y.p), a.y.ld * (a.y_dtype == KDA_BF16 ? 2 : 4)};
    auto with = [&](auto dt, auto odt) {
        return by_sizes(a.dk, a.dv, [&](auto k, auto v) {
            hipLaunchKernelGGL((step_kernel<decltype(dt)::value, decltype(odt)::value, decltype(k)::value, decltype(v)::value>),
                               dim3(static_cast<unsigned>(int64_t(N) * a.H)), dim3(256), 0, stream, L, states, slots, N, n_slots);
            return hipGetLastError();
        });
    };
    using Bf = Int<KDA_BF16>;
    using F = Int<KDA_F32>;
    if (a.in_dtype == KDA_BF16) return a.y_dtype == KDA_BF16 ? with(Bf{}, Bf{}) : with(Bf{}, F{});
    return a.y_dtype == KDA_BF16 ? with(F{}, Bf{}) : with(F{}, F{});
}

}  // namespace kda
