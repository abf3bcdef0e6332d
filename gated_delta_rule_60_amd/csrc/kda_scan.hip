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
// y and dx are one pass along the tokens (value_pass: a state of d_k rows by a head's d_v columns in registers).  For the
// gradients the same pass writes the states before, and the gradients behind, every chunk; dC, dB and the decays'
// gradients then come from all chunks at once (grad_kernel), with the sums over the heads in registers.
//
// The gradient dg_t = e^g_t <G_t, S_{t-1}> of a token's log-decay adds up all ways from a token before it (or the
// chunk's first state) to an output from it on (or the chunk's last state).  With
//     z_ij = e^(c_i - c_j) delta_j (C_i . B_j) (x_j . dy_i), j < i,
//     p_i  = e^c_i dy_i . S^T C_i,  r_j = delta_j e^(c_n - c_j) x_j . G^T B_j,  thr = e^c_n <G, S>
// it is  thr + sum_{i >= t} (sum_j z_ij - sum_{j > i} z_ji + p_i) + sum_{j < t} r_j.  Sums sum_t w_t dg_t over the tokens (dA:
// w = delta; dbias: w = A slope) are formed from the ways themselves, W the running sum of w in the chunk:
//     sum z_ij (W_i - W_j) + sum p_i W_i + sum r_j (W_n - W_j) + thr W_n.
// (The sum of C . dC - B . dB over the tokens behind t is dg_t, too, and needs no chunk's states; but what it adds at one
// token and takes off at another only cancels to rounding: dA was off by 1e-4 of itself on 16384 tokens.)
//
// All decays between two tokens are 2^(difference of fp64 sums): a difference of fp32 sums would lose a weak decay
// behind a strong one.
//
// Measured, one group, bf16, d_k x d_v = 128 x 64, 32 heads: prompt of 65536 tokens 420 us (in a trace: state pass
// 148, scan 14, y 273), 4 x 4096 tokens 118; gradients of 4 x 4096 tokens 450 us (in a trace: chunks' states 183, grad 169,
// dx 80, decays and sums 25); fp32: 304 and 1009 us.  128 x 128, 16 heads: 125 and 539 us (chunks' states 217, grad 228, dx
// 76, decays and sums 18).
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
    f32x2* seg_decay[2];     // [slots, H] a segment's decay as a sum of two
    float* chunk_states[2];  // [c_slots, H, dk, dv]: S before a chunk, G behind it
    float* part[2];          // [head blocks of a group, tokens, G, dk] dC, dB per block; nullptr: one block
    uint8_t* cards;          // [c_slots, H] Card of a chunk's decays
    // [H, tokens]: sum_j z_tj - sum_i z_it; p_t; x_t . u_t from this chunk's outputs, and from later ones (r_t / delta_t)
    // (fp32: each is a sum inside a chunk, rounded once; what is formed from them over a chunk or a sequence is fp64)
    float *zz, *pp, *xz, *xr;
    // [c_slots, H]: sums of z_ij (W_i - W_j) for W of delta and of the slopes, of x . dy, <G, S>
    float *zA, *zb, *dDp, *thr;
    float *dAp, *dbp;        // [c_slots, H]
    Out ddt;
    float *dA, *dD, *dbias;  // [H]
    int32_t ct, c_slots, c_per_seq;      // tokens of a chunk, chunks in all, chunks of a fixed-length sequence
    int32_t heads;           // of a block of the gradients
    int32_t exact[2];        // the segment states end in one that is handed out
    int32_t blocks;          // head blocks of a group
};
enum { S_STATE = 0, G_STATE = 1 };
// Passes along the tokens: y, dx, a segment's own contribution to the states, and the states of every chunk.
enum Mode { Y, DX, S_ONLY, G_ONLY, S_CHUNKS, G_CHUNKS };
constexpr int32_t WHOLE = 0x7fffffff;

template <int DT>
constexpr int CHUNK = DT == KDA_BF16 ? 64 : 32;      // tokens

// What a chunk's decays of one head come to, made once for all kernels of the backward pass.  D_i is the running sum of
// delta in the chunk, e the last token of a token's tile of 16, s the last one before that tile.
template <int CT>
struct Card {
    double dsum[CT], ssum[CT];                       // D_i, running sums of delta's slope
    float del[CT];
    float d_end[CT], s_end[CT];                      // D_e - D_j, and the slopes' sums
    float w_end[CT], w_start[CT];                    // delta_j e^(A (D_e - D_j)), e^(A (D_i - D_s))
    float before[CT], after[CT];                     // e^(A D_i), e^(A (D_n - D_i))
    f32x2 over, pad;         // -e^(A D_n) as a sum of two
};
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

// 2^x to 2^-47, x <= 0: what a state is multiplied by, chunk after chunk, so that errors of 2^-24 would add up.  Taylor's
// series of e^y for |y| <= ln 2 / 2.  The coefficients are formed where they are used: hoisted out of a loop over the
// chunks they take 20 registers a lane, which the loops do not have (each then came from scratch memory, behind all loads
// under way: a third of the forward pass).
template <typename T>
__device__ __forceinline__ T here(T c) {
    asm volatile("" : "+s"(c));
    return c;
}
__device__ __forceinline__ double pow2_wide(double x) {
    x = x < -1100.0 ? -1100.0 : x;
    const double n = __builtin_rint(x), y = (x - n) * here(0.69314718055994530942);
    constexpr double over_factorial[12] = {1.0, 1.0, 1.0 / 2, 1.0 / 6, 1.0 / 24, 1.0 / 120, 1.0 / 720, 1.0 / 5040, 1.0 / 40320,
                                           1.0 / 362880, 1.0 / 3628800, 1.0 / 39916800};
    double p = over_factorial[11];
#pragma unroll
    for (int k = 10; k >= 0; --k) {
        p = __builtin_fma(p, y, here(over_factorial[k]));
    }
    return __builtin_ldexp(p, static_cast<int>(n));
}
// The states in registers change sign from chunk to chunk: chunk k works on (-1)^k S.  The MFMAs' sums lose what they
// drop towards minus infinity, which over all of a state's elements, against inputs that are positive on average (behind
// a SiLU), adds up: with the signs, dA of 4096 tokens was off by 6e-6 of itself, the same way in every head.
__device__ __forceinline__ float chunk_sign(int k) { return k & 1 ? -1.f : 1.f; }

// A chunk's dt of one head, one token a lane, as it comes: to be opened where it is used, a chunk later.
template <int DT>
__device__ __forceinline__ uint32_t load_dt(const Scan& L, int64_t tok0, int n, int32_t h, int lane) {
    constexpr uint32_t ES = DT == KDA_BF16 ? 2 : 4;
    const uint32_t ld = static_cast<uint32_t>(L.dt.ld);
    const __amdgpu_buffer_rsrc_t r = make_rsrc_u(L.dt.p + tok0 * L.dt.ld + h * ES, (n - 1) * ld + ES);
    if constexpr (DT == KDA_BF16) return __builtin_amdgcn_raw_buffer_load_b16(r, lane * ld, 0, 0);
    else return __builtin_amdgcn_raw_buffer_load_b32(r, lane * ld, 0, 0);
}
template <int DT>
__device__ __forceinline__ float open_dt(uint32_t x) { return __uint_as_float(DT == KDA_BF16 ? x << 16 : x); }

// What a lane's four scores of a tile (tokens i = 16 it + l16, j = 16 jt + 4 q + r) are multiplied by: the decay from the
// earlier of the two to the later, 0 where j lies on the wrong side; forward: times delta_j.
template <bool BACK>
__device__ __forceinline__ f32x4 score_weights(const double* cum, const float* del, int it, int jt, int q, int l16) {
    const double ci = cum[16 * it + l16];
    f32x4 dj;
    if constexpr (!BACK) dj = lds_get<f32x4>(del, 4 * (16 * jt + 4 * q));
    f32x4 w;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int i = 16 * it + l16, j = 16 * jt + 4 * q + r;
        const double cj = cum[j];
        const bool seen = BACK ? j >= i : j <= i;
        float e = pow2(seen ? (BACK ? cj - ci : ci - cj) : 0.0);
        if constexpr (!BACK) e *= dj[r];
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
    static constexpr bool STATE = MODE >= S_ONLY;
    static constexpr int ES = DT == KDA_BF16 ? 2 : 4, TOK = CHUNK<DT>, WAVES = HB * DV / 16;
    using TA = Tile<DK, ES>;
    using TC = Tile<DV, ES>;
    static constexpr int C_BYTES = TOK / TC::R * TC::PIECE, P_BYTES = (ES == 2 ? 12 : 3) * 1024;
    // STATE: this chunk's rows and the next one's
    static constexpr int B_BYTES = TOK / TA::R * TA::PIECE, BUFS = STATE ? 2 : 1;
    __align__(16) uint8_t b[BUFS * B_BYTES];
    __align__(16) uint8_t c[BUFS * HB * C_BYTES];
    __align__(16) uint8_t a[STATE ? 16 : TOK / TA::R * TA::PIECE];
    __align__(16) uint8_t p[STATE ? 16 : HB * P_BYTES];              // scores per head
    static constexpr bool OWN = MODE == S_ONLY || MODE == G_ONLY;
    __align__(16) double cum[STATE ? 1 : 2][HB][STATE ? 4 : TOK];  // STATE: the makers' sums of log2 e^g
    __align__(16) float del[STATE ? 1 : 2][HB][STATE ? 4 : TOK], up[OWN ? 8 : STATE ? 2 : 1][HB][TOK];
    f32x2 over[OWN ? 8 : 2][HB];
};

// One workgroup per (segment, HB heads of a group): a and b rows are shared, wave w has 16 columns of head
// w / (DV / 16).  The products are those of linear attention's pass (transposed, so that an accumulator is the next
// product's operand): M and the scores are read as two bf16 terms (2^-17 each), the decayed c as three (exact) where M ends
// in a state that is handed out in fp32, else as two; fp32 inputs use fp32 MFMAs.  (Two, whatever y's type: beside inputs of
// 8 bits an fp32 y is off by 1.2e-6 of its size, a third term would be half as many MFMAs and splits again.  The states
// between segments count as handed out where a final state is.)  The raw scores b a^T are formed once for all HB heads,
// the last HB waves make the next chunk's decays meanwhile.
//
// y and dx are bound by instruction issue: 630 VALU instructions (splits of the state and of c, weights of the scores)
// and 82 MFMAs a wave and chunk, four waves a SIMD at 128 registers; the rows' transfers are only hidden by the CU's
// other workgroup.  (A transfer issued before the update's transposing reads would be waited for in front of them.)
// 65536 x 32: 2.0 TB/s of rows.  Bf16 inputs at 128 x 128, or with an fp32 y, are 4 to 8 registers over 128 (5 to 9 reloads
// from scratch memory).  The states of all chunks are bound by writing them: 2.9 TB/s for 4 x 4096 x 32; without the
// stores the pass takes 110 us of 183, without the rows 127.
template <int DT, int ODT, int DK, int DV, int HB, int MODE>
__device__ __forceinline__ void value_pass(const Scan& L, int32_t slot, int32_t block, ValueLds<DT, DK, DV, HB, MODE>& lds) {
    using Lds = ValueLds<DT, DK, DV, HB, MODE>;
    using TA = typename Lds::TA;
    using TC = typename Lds::TC;
    constexpr bool BF = DT == KDA_BF16, STATE = Lds::STATE, BACK = MODE == DX || MODE == G_ONLY || MODE == G_CHUNKS;
    constexpr bool OWN = MODE == S_ONLY || MODE == G_ONLY, CHUNKS = MODE == S_CHUNKS || MODE == G_CHUNKS;
    constexpr bool CARDS = CHUNKS || MODE == DX;
    constexpr int TOK = Lds::TOK, WAVES = Lds::WAVES, WPH = DV / 16;
    constexpr int IT = TOK / 16, MT = DK / 16, KK = DK / 32, JG = TOK / 32;
    constexpr int OS = ODT == KDA_BF16 ? 2 : 4;
    constexpr bool STAGED = BF && OS == 2 && !STATE;
    constexpr int ST = BACK ? G_STATE : S_STATE;

    Where w;
    if (!locate(L, slot, w)) return;
    if (OWN && w.s == (BACK ? 0 : w.n_seg - 1)) return;            // nothing follows it
    if (MODE == DX && w.hi == w.lo) return;
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
    auto state = [&](auto* all, int64_t u) { return all + u * (DK * DV); };

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
    // STATE: rows come by way of registers (a transfer to LDS under way would be waited for at the next transposing read)
    constexpr int NB = TOK / TA::R / WAVES, NC = TOK / TC::R / WAVES;
    struct Rows {
        u32x4 b[STATE ? NB : 1], c[STATE ? NC : 1];
    };
    auto take = [&](auto tile, u32x4* to, const In& from, int64_t unit_bytes, int c) {
        using TT = decltype(tile);
        const int64_t off = chunk_at(c);
        const uint32_t ld = static_cast<uint32_t>(from.ld);
        const __amdgpu_buffer_rsrc_t r = make_rsrc_u(from.p + (w.lo + off) * from.ld + unit_bytes, (chunk_n(off) - 1) * ld + TT::RB);
        int ln = lane;
        asm volatile("" : "+v"(ln));
        const int r0 = wave * TT::R + ln / TT::UPR, un = ln % TT::UPR;
        const uint32_t at = r0 * ld + ((un & ~7) | ((un & 7) ^ TT::mix(r0))) * 16;
#pragma unroll
        for (int i = 0; i < TOK / TT::R / WAVES; ++i) to[i] = __builtin_amdgcn_raw_buffer_load_b128(r, at + WAVES * i * TT::R * ld, 0, 0);
    };
    auto take_rows = [&](Rows& x, int c) {
        take(TA{}, x.b, rb, g * TA::RB, c);
        take(TC{}, x.c, rc, h0 * TC::RB, c);
    };
    auto put_rows = [&](const Rows& x, int c) {
#pragma unroll
        for (int i = 0; i < NB; ++i) lds_put(lds.b + (STATE ? c & 1 : 0) * Lds::B_BYTES, TA::PIECE * (WAVES * i + wave) + lane * 16, x.b[i]);
#pragma unroll
        for (int i = 0; i < NC; ++i) lds_put(lds.c + (STATE ? c & 1 : 0) * Lds::C_BYTES, TC::PIECE * (WAVES * i + wave) + lane * 16, x.c[i]);
    };
    // The wave that makes a head's decays of the next chunk.  OWN: four waves, each those of one of the next four chunks, all
    // at a time (one wave alone holds up the others for half the chunk's time).
    const int table = OWN ? (wave < 4 ? 0 : -1) : wave - (WAVES - HB);
    auto ring = [](int c) { return OWN ? c & 7 : c & 1; };
    const int32_t th = h0 + table < h_end ? h0 + (table < 0 ? 0 : table) : h_end - 1;
    const float A = L.A[th], bias = L.bias ? L.bias[th] : 0.f;
    // a chunk's place among those of all sequences: of the chunk that token w.lo + off belongs to
    const int64_t first = w.lo - static_cast<int64_t>(w.s) * L.seg;
    const int64_t chunk0 = (L.cu ? first / TOK + w.n : static_cast<int64_t>(w.n) * L.c_per_seq);
    auto chunk_unit = [&](int64_t off, int32_t head) { return (chunk0 + (w.lo - first + off) / TOK) * L.H + head; };
    // what the decays are made of, a lane's token; fetched a chunk ahead of its use
    struct Ahead {
        uint32_t dt;
        double dsum;
        float del, w;
        f32x2 over;
    };
    auto ahead_of = [&](int c) {
        const int64_t off = chunk_at(c);
        Ahead a{};
        if constexpr (CARDS) {
            using Cd = Card<TOK>;
            const uint32_t l = lane % TOK;
            const __amdgpu_buffer_rsrc_t r = make_rsrc_u(L.cards + chunk_unit(off, th) * sizeof(Cd), sizeof(Cd));
            auto word = [&](uint32_t at) { return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, at + 4 * l, 0, 0)); };
            if constexpr (MODE != G_CHUNKS) a.del = word(offsetof(Cd, del));
            if constexpr (MODE == DX) a.dsum = __builtin_bit_cast(double, __builtin_amdgcn_raw_buffer_load_b64(r, 8 * l, 0, 0));
            else a.w = word(BACK ? offsetof(Cd, before) : offsetof(Cd, after));
            a.over = __builtin_bit_cast(f32x2, __builtin_amdgcn_raw_buffer_load_b64(r, offsetof(Cd, over), 0, 0));
        } else {
            a.dt = load_dt<DT>(L, w.lo + off, chunk_n(off), th, lane);
        }
        return a;
    };
    double log_sum = 0.0;
    auto decays = [&](int c, const Ahead& a) {
        const int buf = ring(c), n = chunk_n(chunk_at(c));
        if constexpr (CARDS) {
            if (lane < TOK) {
                if constexpr (MODE == DX) {
                    lds.cum[buf][table][lane] = a.dsum * (static_cast<double>(A) * LOG2E);
                    lds.del[buf][table][lane] = a.del;
                } else {
                    lds.up[STATE ? buf : 0][table][lane] = chunk_sign(c + 1) * (BACK ? a.w : a.del * a.w);
                }
                if (lane == 0) lds.over[buf][table] = a.over;
            }
            return;
        }
        const float delta = lane < n ? strength(open_dt<DT>(a.dt), bias).delta : 0.f;
        const double cum = prefix_sum(static_cast<double>(delta) * (static_cast<double>(here(__uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(A))))) * here(LOG2E)));
        const double all = lane_value(cum, TOK - 1), over = -pow2_wide(all);
        const float hi = static_cast<float>(over);
        log_sum += all;
        if (lane < TOK) {
            if constexpr (!STATE) {
                lds.cum[buf][table][lane] = cum;
                lds.del[buf][table][lane] = delta;
            }
            if (STATE) lds.up[STATE ? buf : 0][table][lane] = chunk_sign(c + 1) * (BACK ? pow2(cum) : delta * pow2(all - cum));
            if (lane == 0) lds.over[buf][table] = f32x2{hi, static_cast<float>(over - static_cast<double>(hi))};
        }
    };

    Rows even{}, odd{};                              // rows under way: of the next chunk and of the one after it
    if (n_chunks > 0) {
        if constexpr (STATE) {
            take_rows(even, 0);
            if (n_chunks > 1) take_rows(odd, 1);
        } else {
            load_b(0);
            load_a(0);
            load_c(0);
        }
        if (table >= 0 && (!OWN || wave < n_chunks)) decays(OWN ? wave : 0, ahead_of(OWN ? wave : 0));
    }
    Ahead ahead{};
    const int first_ahead = OWN ? 4 + wave : 1;
    if (table >= 0 && first_ahead < n_chunks) ahead = ahead_of(first_ahead);

    // ---- the state, tile mt of 16 rows.  Y and DX: register r of lane (l16, q) holds row row(mt) + r, column 16 wc + l16;
    // STATE: row 16 mt + l16, column 16 wc + 4 q + r, so that a lane's four lie side by side.  The states of the chunks
    // are kept as those tiles, 1 KB each.
    auto row = [&](int mt) { return BF ? 32 * (mt >> 1) + 8 * q + 4 * (mt & 1) : 16 * mt + 4 * q; };
    const int col = 16 * wc + l16;
    f32x4 M[MT];
    auto state_at = [&](bool tiles) {                // of tile 0; tile mt stands 64 DV mt bytes behind it
        uint32_t at = tiles ? (wc * 64 + lane) * 16 : (l16 * DV + 16 * wc + 4 * q) * 4;
        asm volatile("" : "+v"(at));                 // formed anew, not kept over the loop
        return at;
    };
    auto store_state = [&](float* dst, float sign, bool tiles) {
        const __amdgpu_buffer_rsrc_t rs = make_rsrc_u(dst, DK * DV * 4);
        if constexpr (STATE) {
            const uint32_t at = state_at(tiles);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, sign * M[mt]), rs, at + 64 * DV * mt, 0, 0);
        } else {
            uint32_t at = (row(0) * DV + col) * 4;
            asm volatile("" : "+v"(at));             // formed anew, not kept over the loop
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(sign * M[mt][r]), rs,
                                                          at + ((BF ? 32 * (mt >> 1) + 4 * (mt & 1) : 16 * mt) + r) * DV * 4, 0, 0);
        }
    };
    auto load_state = [&](const float* src, bool tiles) {          // nullptr: an empty range, which reads as zeros
        const __amdgpu_buffer_rsrc_t rs = make_rsrc_u(src, src ? DK * DV * 4 : 0);
        if constexpr (STATE) {
            const uint32_t at = state_at(tiles);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
                M[mt] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, at + 64 * DV * mt, 0, 0));
        } else {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int k = row(mt) + r;
                    const uint32_t at = tiles ? k / 16 * (DV * 64) + wc * 1024 + (l16 >> 2) * 256 + k % 16 * 16 + (l16 & 3) * 4
                                              : (k * DV + col) * 4;
                    M[mt][r] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, at, 0, 0));
                }
        }
    };
    if constexpr (OWN) load_state(nullptr, false);
    else if constexpr (MODE == DX) load_state(state(L.chunk_states[ST], chunk_unit(len - 1, h)), true);
    else load_state(w.n_seg > 1 ? state(L.seg_states[ST], seg_unit) : L.m_in[ST] ? state(L.m_in[ST], unit) : nullptr, false);

    // ---- operands' byte offsets, as in linear attention's pass.  16 bits, along the channels: channels
    // 32 kk + 8 q .. + 7 of token 16 it + l16; along the tokens: tokens 32 tg + 4 q .. + 3 and 32 tg + 16 + 4 q .. + 3,
    // of state row tile mt's rows or of the wave's columns.  (STATE: tile mt has 16 neighbouring rows; the layout's
    // swizzle is an exclusive or on the units' number, so tile mt's offset is tile 0's with one of its own.)
    uint32_t chan[2], tok[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        chan[x] = TA::at(l16, 4 * x + q);
        tok[x] = TA::at(4 * q + (l16 >> 2), 4 * x + (l16 & 3));
    }
    const uint32_t tok_b = TA::at(4 * q + (l16 >> 2), (l16 & 3) >> 1) + 8 * (l16 & 1);
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
    const bool exact = STATE ? L.exact[ST] != 0 : MODE == Y && L.m_out[ST] && w.s == w.n_seg - 1;
    if constexpr (STATE)
        if (n_chunks > 0) put_rows(even, 0);
    auto chunk = [&](int c, Rows& far, const Rows& near) __attribute__((always_inline)) {
        const int64_t off = chunk_at(c), tok0 = w.lo + off;
        const int n = chunk_n(off), buf = c & 1, at_ring = ring(c);
        const uint8_t* const lds_b = lds.b + (STATE ? buf : 0) * Lds::B_BYTES;
        uint8_t* const lds_c = lds.c + ((STATE ? buf : 0) * HB + hb) * Lds::C_BYTES;
        if constexpr (!STATE) __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
        lds_barrier();                               // the tiles and the decays are there
        if constexpr (STATE)
            if (c + 2 < n_chunks) take_rows(far, c + 2);
        const Ahead next = ahead;
        const bool makes = table >= 0 && (!OWN || c % 4 == 0);
        const int made = c + first_ahead, far_made = made + (OWN ? 4 : 1);
        if (makes && far_made < n_chunks) ahead = ahead_of(far_made);
        const double* cum = lds.cum[STATE ? 0 : buf][hb];
        const float* del = lds.del[STATE ? 0 : buf][hb];

        f32x4 O[IT];
        if constexpr (CHUNKS) {
            if (live) store_state(state(L.chunk_states[ST], chunk_unit(off, h)), chunk_sign(c), true);
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
                            const f32x4 x = P[hh] * score_weights<BACK>(lds.cum[buf][i], lds.del[buf][i], it, 2 * tg + hh, q, l16);
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
                            P * score_weights<BACK>(lds.cum[buf][i], lds.del[buf][i], it, jt, q, l16));
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
            const double all = cum[TOK - 1];
#pragma unroll
            for (int it = 0; it < IT; ++it) {
                const double ci = cum[16 * it + l16];
                O[it] *= chunk_sign(c) * pow2(BACK ? all - ci : ci);
            }
        }
        if (makes && made < n_chunks) decays(made, next);
        decay_state(M, lds.over[at_ring][hb]);

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
            // ---- lane l16 holds token 16 it + l16, four neighbouring columns
#pragma unroll
            for (int it = 0; it < IT; ++it) {
                if constexpr (MODE == DX) O[it] *= del[16 * it + l16];
                if (L.D) O[it] += D * widen(lds_c, own_at(it));
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
        const float* up = lds.up[STATE ? at_ring : 0][hb];
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
                    auto add = [&](int mt, const u32x4& kt, const u32x4& cw) {
                        M[mt] = STATE ? mfma_bf16(cw, kt, M[mt]) : mfma_bf16(kt, cw, M[mt]);
                    };
                    constexpr int NM = STATE ? MT : 1;             // tiles at a time: products that do not wait for each other
#pragma unroll
                    for (int m0 = 0; m0 < MT; m0 += NM) {
                        u32x4 kt[NM];
#pragma unroll
                        for (int m = 0; m < NM; ++m) {
                            const int mt = m0 + m;
                            const uint32_t at = STATE ? (tok_b ^ (32 * (mt & 3))) + (mt >> 2) * 128
                                                      : tok[(mt >> 1) & 1] + (mt >> 2) * 128 + 8 * (mt & 1);
                            kt[m] = tokens(at + 2 * tg * TA::ROWS16, lds_b, TA::ROWS16);
                        }
                        if constexpr (THREE)
#pragma unroll
                            for (int m = 0; m < NM; ++m) add(m0 + m, kt[m], cl);
#pragma unroll
                        for (int m = 0; m < NM; ++m) add(m0 + m, kt[m], cm);
#pragma unroll
                        for (int m = 0; m < NM; ++m) add(m0 + m, kt[m], ch);
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
                    for (int mt = 0; mt < MT; ++mt) {
                        const float b = lds_get<float>(lds_b, TA::at(16 * jt + 4 * q + r, 4 * mt + (l16 >> 2)) + 4 * (l16 & 3));
                        M[mt] = STATE ? mfma_f32(cw, b, M[mt]) : mfma_f32(b, cw, M[mt]);
                    }
                }
            }
        }
        if constexpr (STATE) {
            if (c + 1 < n_chunks) put_rows(near, c + 1);           // (all have left the tiles before them)
            return;
        }
        lds_barrier();                               // the tiles have been read, the output is there
        if (c + 1 < n_chunks) {
            load_b(c + 1);
            load_a(c + 1);
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
    };
    if constexpr (STATE) {
        for (int c = 0; c < n_chunks; c += 2) {
            chunk(c, even, odd);
            if (c + 1 < n_chunks) chunk(c + 1, odd, even);
        }
    } else {
        for (int c = 0; c < n_chunks; ++c) chunk(c, even, odd);
    }

    float* dst = nullptr;
    if constexpr (OWN) dst = state(L.seg_states[ST], seg_unit);
    else if (MODE != DX && L.m_out[ST] && w.s == (BACK ? 0 : w.n_seg - 1)) dst = state(L.m_out[ST], unit);
    if (dst && live) store_state(dst, chunk_sign(n_chunks), false);
    if constexpr (OWN) {
        if (table >= 0 && lane == 0) lds.cum[0][0][wave] = log_sum;
        lds_barrier();
        if (t == 0) {
            const double all = pow2_wide((lds.cum[0][0][0] + lds.cum[0][0][1]) + (lds.cum[0][0][2] + lds.cum[0][0][3]));
            const float hi = static_cast<float>(all);
            L.seg_decay[ST][seg_unit] = f32x2{hi, static_cast<float>(all - static_cast<double>(hi))};
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
__global__ void __launch_bounds__(HB * DV * 4, HB * DV == 128 ? 4 : 2) value_kernel(Scan L) {
    __shared__ ValueLds<DT, DK, DV, HB, MODE> lds;
    uint32_t unit;
    int32_t pass;
    if (!unit_of(static_cast<uint32_t>(L.slots) * L.blocks * L.G, 1, unit, pass)) return;
    const uint32_t blocks = static_cast<uint32_t>(L.blocks) * L.G;
    value_pass<DT, ODT, DK, DV, HB, MODE>(L, unit / blocks, unit % blocks, lds);
}
// The segments' own contributions to S, or G, or both; or the states of all chunks.  One head a workgroup: with two, for
// d_v = 64, half the CUs had none, and what they saved in rows of B and C was not missed.
template <int DT, int DK, int DV, bool CHUNKS>
__global__ void __launch_bounds__(DV * 4, 2) state_kernel(Scan L, int32_t passes) {
    constexpr int SM = CHUNKS ? S_CHUNKS : S_ONLY, GM = CHUNKS ? G_CHUNKS : G_ONLY;
    __shared__ union {
        ValueLds<DT, DK, DV, 1, SM> s;
        ValueLds<DT, DK, DV, 1, GM> g;
    } lds;
    uint32_t unit;
    int32_t pass;
    if (!unit_of(static_cast<uint32_t>(L.slots) * L.H, passes, unit, pass)) return;
    if (pass == S_STATE) value_pass<DT, DT, DK, DV, 1, SM>(L, unit / L.H, unit % L.H, lds.s);
    else value_pass<DT, DT, DK, DV, 1, GM>(L, unit / L.H, unit % L.H, lds.g);
}

// Segment states: from each segment's own contribution to the state it starts from (S) or that follows it (G), in
// place.  Grid (sequence * H + head, element blocks of 1024, pass); sixteen segments' loads at a time (eight: 16.4 us for the
// packed 16455 tokens of 8 heads, five round trips to memory for the longest sequence).
__global__ void __launch_bounds__(256) scan_kernel(Scan L, int32_t elems) {
    const int ST = blockIdx.z;
    const bool back = ST == G_STATE;
    const int32_t n = blockIdx.x / L.H, h = blockIdx.x % L.H;
    const int32_t e = blockIdx.y * 1024 + threadIdx.x * 4;
    int64_t lo, hi;
    seq_range(L, n, lo, hi);
    const int32_t n_seg = segments(L, hi - lo);
    if (n_seg == 1) return;
    const int64_t slot0 = L.cu ? first_slot(L, n) : static_cast<int64_t>(n) * n_seg;
    f32x4 x = zero4();
    if (L.m_in[ST]) x = *reinterpret_cast<const f32x4*>(L.m_in[ST] + (static_cast<int64_t>(n) * L.H + h) * elems + e);
    auto index = [&](int32_t i) { return (slot0 + (back ? n_seg - 1 - i : i)) * L.H + h; };
    auto slot = [&](int32_t i) { return reinterpret_cast<f32x4*>(L.seg_states[ST] + index(i) * elems + e); };
    f32x4 ahead = *slot(0);                          // read before the batch before it writes its place
    *slot(0) = x;
    constexpr int AT = 16;
    for (int32_t i0 = 0; i0 < n_seg - 1; i0 += AT) {
        f32x4 own[AT + 1];
        f32x2 decay[AT];
        own[0] = ahead;
#pragma unroll
        for (int32_t j = 1; j <= AT; ++j) own[j] = i0 + j < n_seg - 1 ? *slot(i0 + j) : zero4();
#pragma unroll
        for (int32_t j = 0; j < AT; ++j) decay[j] = L.seg_decay[ST][index(i0 + j < n_seg - 1 ? i0 + j : n_seg - 2)];
        ahead = own[AT];
#pragma unroll
        for (int32_t j = 0; j < AT; ++j) {
            if (i0 + j >= n_seg - 1) break;
#pragma unroll
            for (int r = 0; r < 4; ++r) x[r] = __builtin_fmaf(x[r], decay[j][0], __builtin_fmaf(x[r], decay[j][1], own[j][r]));
            *slot(i0 + j + 1) = x;                   // segment i's end is what segment i + 1 starts from
        }
    }
}

// ---------------------------------------------------------------- dC, dB and the ways between tokens

// A chunk's decays, one wave per (chunk, head), a token a lane.
template <int DT>
__global__ void __launch_bounds__(256) card_kernel(Scan L) {
    constexpr int CT = CHUNK<DT>;
    const int64_t u = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    if (u >= static_cast<int64_t>(L.c_slots) * L.H) return;
    const int32_t slot = static_cast<int32_t>(u / L.H), h = static_cast<int32_t>(u % L.H);
    Where w;
    if (!locate(L, slot, w)) return;
    const double A2 = static_cast<double>(L.A[h]) * LOG2E;
    Strength s = {0.f, 0.f};
    if (lane < w.hi - w.lo) s = strength(load_as_f32<DT>(L.dt.p + (w.lo + lane) * L.dt.ld, h), L.bias ? L.bias[h] : 0.f);
    const double d = prefix_sum(static_cast<double>(s.delta)), o = prefix_sum(static_cast<double>(s.slope));
    const int e = lane | 15, start = (lane & ~15) - 1;
    const double de = shuffle(d, e), oe = shuffle(o, e), ds = shuffle(d, start < 0 ? 0 : start), all = lane_value(d, CT - 1);
    if (lane >= CT) return;
    Card<CT>& c = reinterpret_cast<Card<CT>*>(L.cards)[u];
    c.dsum[lane] = d;
    c.del[lane] = s.delta;
    c.ssum[lane] = o;
    c.d_end[lane] = static_cast<float>(de - d);
    c.s_end[lane] = static_cast<float>(oe - o);
    c.w_end[lane] = s.delta * pow2(A2 * (de - d));
    c.w_start[lane] = pow2(A2 * (start < 0 ? d : d - ds));
    c.before[lane] = pow2(A2 * d);
    c.after[lane] = pow2(A2 * (all - d));
    if (lane == 0) {
        const double over = -pow2_wide(A2 * all);
        const float hi = static_cast<float>(over);
        c.over = f32x2{hi, static_cast<float>(over - static_cast<double>(hi))};
    }
}

template <int DT, int DK, int DV>
struct GradLds {
    static constexpr int ES = DT == KDA_BF16 ? 2 : 4, CT = CHUNK<DT>, WAVES = DK / 16;    // of either kind
    using TA = Tile<DV, ES>;
    using TC = Tile<DK, ES>;
    static constexpr int A_BYTES = CT / TA::R * TA::PIECE, C_BYTES = CT / TC::R * TC::PIECE;
    // scores are made in groups: a tile of 16 tokens by 32 (fp32: 16) others on its near side
    static constexpr int IT = CT / 16, TG = DT == KDA_BF16 ? CT / 32 : IT;
    static constexpr int GROUPS = DT == KDA_BF16 ? TG * (TG + 1) : IT * (IT + 1) / 2, G_BYTES = DT == KDA_BF16 ? 2048 : 1024;
    static constexpr int TILES = DT == KDA_BF16 ? 2 : 1;           // of a group
    __align__(16) uint8_t B[C_BYTES];
    __align__(16) uint8_t C[C_BYTES];
    // x and dy of a head and of the next one; in the end the scores, summed over the heads, one direction at a time
    __align__(16) uint8_t xy[4 * A_BYTES];
    static_assert(GROUPS * G_BYTES <= 4 * A_BYTES, "the scores take the place of the rows");
    static constexpr int CARD = (sizeof(Card<CT>) + 1023) / 1024;  // KB
    static_assert(CARD <= WAVES, "a wave per KB");
    __align__(16) uint8_t card[2][CARD * 1024];
    // p and r / delta by waves, sums of z over j and of z / delta over i by groups, z_jj / delta_j
    static constexpr int P = 0, R = WAVES, ROWS = 2 * WAVES, COLS = ROWS + TG, DIAG = COLS + TG;
    float red[DIAG + 1][CT];
    float sums[4][WAVES];
    // a wave's rows of the next head's states (16 bits; both states of more would not fit, and of fewer would cost the
    // CU's second workgroup its place)
    static constexpr bool AHEAD = DT == KDA_BF16 && DK == 128 && DV == 64;
    static constexpr int S_BYTES = 16 * DV * 4;
    __align__(16) uint8_t states[AHEAD ? WAVES * 2 * S_BYTES : 16];
    // direction 0: outputs i by groups of j <= i; direction 1: outputs j by groups of i >= j, mirrored.  Group number of
    // (output tile, group of others), and back.
    static __host__ __device__ constexpr int number(int dir, int out, int tg) {
        const int o = dir ? IT - 1 - out : out, g = dir ? TG - 1 - tg : tg;
        return g * IT - (TILES == 2 ? g * (g - 1) : g * (g - 1) / 2) + o - TILES * g;
    }
    static __device__ __forceinline__ void group(int dir, int k, int& out, int& tg) {
        int g = 0;
        for (int n = IT; k >= n; n -= TILES) {
            k -= n;
            ++g;
        }
        out = dir ? IT - 1 - (TILES * g + k) : TILES * g + k;
        tg = dir ? TG - 1 - g : g;
    }
    static __host__ __device__ constexpr bool near(int dir, int out, int tg) {
        return dir ? TILES * tg + TILES - 1 >= out : TILES * tg <= out;
    }
};

// The sum of a value over the four lanes of one l16, in all of them: rows of 16 lanes and halves of the wave swapped.
__device__ __forceinline__ float sum_q(float x) {
    const uint32_t u = __float_as_uint(x);
    const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    const float y = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    const uint32_t v = __float_as_uint(y);
    const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}
__device__ __forceinline__ float sum_wave(float x) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {                    // rows of 16 lanes, turned by 8, 4, 2, 1
        const int u = static_cast<int>(__float_as_uint(x));
        const int v = k == 0   ? __builtin_amdgcn_update_dpp(0, u, 0x128, 0xf, 0xf, false)
                      : k == 1 ? __builtin_amdgcn_update_dpp(0, u, 0x124, 0xf, 0xf, false)
                      : k == 2 ? __builtin_amdgcn_update_dpp(0, u, 0x122, 0xf, 0xf, false)
                               : __builtin_amdgcn_update_dpp(0, u, 0x121, 0xf, 0xf, false);
        x += __uint_as_float(static_cast<uint32_t>(v));
    }
    return sum_q(x);
}

// 2^(A d / ln 2) for a sum d of delta between two tokens, A / ln 2 as hi + lo.
struct Decay {
    double A2;
    float hi, lo;
    __device__ __forceinline__ explicit Decay(float A)
        : A2(static_cast<double>(A) * LOG2E), hi(static_cast<float>(A2)), lo(static_cast<float>(A2 - static_cast<double>(hi))) {}
    __device__ __forceinline__ float operator()(float d) const { return __builtin_amdgcn_exp2f(__builtin_fmaf(d, hi, d * lo)); }
};

// Bound by instruction issue and by the states' reads (537 MB, 3.2 TB/s for 4 x 4096 x 32, 169 us).  At 128 x 128 in bf16 a
// lane's rows of both states are 34 registers more than it has: 28 reloads from scratch memory, 228 us for 16 heads.
// One workgroup per (chunk, block of a group's heads), of two kinds of waves: wave w of the first kind has the output
// channels 16 w .. 16 w + 15 of dC and dB and forms the states' parts, those of the second share the groups of scores of
// both directions and move the rows.  (One kind for both needs 300 registers a lane; what does not fit waits for the rows
// under way: 743 us for 4 x 4096 x 32.)  B and C are read once, the heads' rows come one head after the other, the next
// one's under this one's products.  The scores' products with B and C are formed once, from their sums over the heads (two
// bf16 terms, 2^-17 each: they only feed 16-bit outputs).  The states are read as three (exact), for p, r and what comes of
// them is handed out in fp32.
template <int DT, int DK, int DV>
__device__ __forceinline__ void grad_pass(const Scan& L, int32_t slot, int32_t block, GradLds<DT, DK, DV>& lds) {
    using Lds = GradLds<DT, DK, DV>;
    using TA = typename Lds::TA;
    using TC = typename Lds::TC;
    constexpr bool BF = DT == KDA_BF16;
    constexpr int ES = Lds::ES, CT = Lds::CT, WAVES = Lds::WAVES, IT = Lds::IT, TG = Lds::TG, TILES = Lds::TILES;
    constexpr int KV = DV / 32, KC = DK / 32, NS = DV / 16;
    constexpr int ROUNDS = (2 * Lds::GROUPS + WAVES - 1) / WAVES;

    Where w;
    if (!locate(L, slot, w) || w.hi == w.lo) return;
    const int t = threadIdx.x, lane = t & 63;
    const int wave_all = __builtin_amdgcn_readfirstlane(t >> 6), wave = wave_all % WAVES;
    const bool scores = wave_all >= WAVES;           // the second kind
    const int32_t rep = L.H / L.G, g = block / L.blocks, blk = block % L.blocks;
    const int32_t h0 = g * rep + blk * L.heads, left = (g + 1) * rep - h0, heads = left < L.heads ? left : L.heads;
    const int n = static_cast<int>(w.hi - w.lo);
    const int64_t units = static_cast<int64_t>(slot) * L.H + h0;   // of the block's first head

    auto load_head = [&](int k, int buf) {
        fetch_rows<TA, CT, WAVES>(lds.xy + buf * 2 * Lds::A_BYTES, L.x.p + w.lo * L.x.ld + (h0 + k) * TA::RB, static_cast<uint32_t>(L.x.ld), n, wave, lane);
        fetch_rows<TA, CT, WAVES>(lds.xy + (buf * 2 + 1) * Lds::A_BYTES, L.dy.p + w.lo * L.dy.ld + (h0 + k) * TA::RB, static_cast<uint32_t>(L.dy.ld), n, wave, lane);
        if (wave < Lds::CARD)
            transfer16(make_rsrc_u(L.cards + (units + k) * sizeof(Card<CT>), sizeof(Card<CT>)), wave * 1024 + lane * 16, lds.card[buf] + wave * 1024);
    };
    // row 16 wave + l16 of the states, d_v along the contraction: of tile `wave` of 16 rows, as the state pass leaves it
    auto state_of = [&](int st, int k) { return L.chunk_states[st] + (units + k) * (DK * DV) + 16 * DV * wave; };
    auto tile_at = [&](int i) {                      // (16 bits: channels 32 (i >> 1) + 8 q + 4 (i & 1) ..)
        const int q = lane >> 4, l16 = lane & 15;
        return BF ? (2 * (i >> 1) + (q >> 1)) * 1024 + (2 * (q & 1) + (i & 1)) * 256 + l16 * 16 : i * 1024 + lane * 16;
    };
    auto request_states = [&](int st, int k) {
        const __amdgpu_buffer_rsrc_t r = make_rsrc_u(state_of(st, k), Lds::S_BYTES);
#pragma unroll
        for (int i = 0; i < NS; ++i)
            transfer16(r, i * 1024 + lane * 16, lds.states + (2 * wave + st) * Lds::S_BYTES + i * 1024);
    };
    auto load_state = [&](f32x4 (&X)[NS], int st, int k) {
#pragma unroll
        for (int i = 0; i < NS; ++i)
            if constexpr (Lds::AHEAD) X[i] = lds_get<f32x4>(lds.states + (2 * wave + st) * Lds::S_BYTES, tile_at(i));
            else X[i] = *reinterpret_cast<const f32x4*>(reinterpret_cast<const uint8_t*>(state_of(st, k)) + tile_at(i));
    };
    const int ts = t - WAVES * 64;                   // the second kind's lanes
    if (scores) {
        fetch_rows<TC, CT, WAVES>(lds.C, L.C.p + w.lo * L.C.ld + g * TC::RB, static_cast<uint32_t>(L.C.ld), n, wave, lane);
        load_head(0, 0);
    } else {
        fetch_rows<TC, CT, WAVES>(lds.B, L.B.p + w.lo * L.B.ld + g * TC::RB, static_cast<uint32_t>(L.B.ld), n, wave, lane);
    }

    // A lane's place in the tiles, formed anew for every head: what comes of it would else be kept in registers over the
    // loop, more of them than there are.
    struct Place {
        int q, l16;
        uint32_t chan[2], chan_c[2], own;
    };
    auto place = [&]() {
        int ln = lane;
        asm volatile("" : "+v"(ln));
        Place a;
        a.q = ln >> 4;
        a.l16 = ln & 15;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            a.chan[x] = TA::at(a.l16, 4 * x + a.q);
            a.chan_c[x] = TC::at(a.l16, 4 * x + a.q);
        }
        a.own = BF ? TC::at(a.l16, 2 * wave + (a.q >> 1)) + 8 * (a.q & 1) : TC::at(a.l16, 4 * wave + a.q);
        return a;
    };
    // 16 rows' dot products with 16 others, channels along the contraction
    auto dots = [&](const Place& a, const uint8_t* rows, const uint8_t* cols, int rt, int ct, auto wide, f32x4 acc) {
        constexpr bool WIDE = decltype(wide)::value;               // B and C, or x and dy
        using TT = std::conditional_t<WIDE, TC, TA>;
        rows += rt * TT::ROWS16;
        cols += ct * TT::ROWS16;
        if constexpr (BF) {
#pragma unroll
            for (int kk = 0; kk < (WIDE ? KC : KV); ++kk) {
                const uint32_t at = (WIDE ? a.chan_c : a.chan)[kk & 1] + (kk >> 1) * 128;
                acc = mfma_bf16(lds_get<u32x4>(rows, at), lds_get<u32x4>(cols, at), acc);
            }
        } else {
#pragma unroll
            for (int mt = 0; mt < (WIDE ? DK : DV) / 16; ++mt) {
                const uint32_t at = TT::at(a.l16, 4 * mt + a.q);
                const f32x4 x = lds_get<f32x4>(rows, at), y = lds_get<f32x4>(cols, at);
#pragma unroll
                for (int r = 0; r < 4; ++r) acc = mfma_f32(x[r], y[r], acc);
            }
        }
        return acc;
    };
    auto own = [&](const Place& a, const uint8_t* sm, int it) {    // token 16 it + l16's channels 16 wave + 4 q .. + 3
        if constexpr (BF) {
            const u32x2 x = lds_get<u32x2>(sm, a.own + it * TC::ROWS16);
            return f32x4{lo_f32(x[0]), hi_f32(x[0]), lo_f32(x[1]), hi_f32(x[1])};
        } else {
            return lds_get<f32x4>(sm, a.own + it * TC::ROWS16);
        }
    };

    // Both kinds meet at the same barriers: one in front, two a head, three behind.
    if (scores) {
        f32x4 P[ROUNDS][TILES], CB[ROUNDS][TILES];
        __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
        lds_barrier();                               // B and C and the first head's rows are there
        {
            const Place a = place();
#pragma unroll
            for (int i = 0; i < ROUNDS; ++i) {
                const int grp = wave + i * WAVES, dir = grp >= Lds::GROUPS;
#pragma unroll
                for (int hh = 0; hh < TILES; ++hh) P[i][hh] = CB[i][hh] = zero4();
                if (grp >= 2 * Lds::GROUPS) continue;
                int out, tg;
                Lds::group(dir, grp - dir * Lds::GROUPS, out, tg);
#pragma unroll
                for (int hh = 0; hh < TILES; ++hh)
                    CB[i][hh] = dots(a, dir ? lds.C : lds.B, dir ? lds.B : lds.C, TILES * tg + hh, out, std::true_type{}, CB[i][hh]);
            }
        }
        for (int k = 0; k < heads; ++k) {
            const int buf = k & 1;
            const Place a = place();
            const int q = a.q, l16 = a.l16;
            const uint8_t *x = lds.xy + buf * 2 * Lds::A_BYTES, *dy = x + Lds::A_BYTES;
            const Card<CT>& card = *reinterpret_cast<const Card<CT>*>(lds.card[buf]);
            const double* dsum = card.dsum;
            const Decay decay(L.A[h0 + k]);
            if (k + 1 < heads) load_head(k + 1, buf ^ 1);          // (all have left the last head's)
            // rows 16 rt + 4 q + r, column 16 out + l16; direction 0: rows j, column i, direction 1: rows i, column j
            float zA = 0.f, zb = 0.f, dD = 0.f;
#pragma unroll
            for (int i = 0; i < ROUNDS; ++i) {
                const int grp = wave + i * WAVES, dir = grp >= Lds::GROUPS;
                if (grp >= 2 * Lds::GROUPS) continue;
                int out, tg;
                Lds::group(dir, grp - dir * Lds::GROUPS, out, tg);
                const int col = 16 * out + l16;
                const double dcol = dsum[col];
                const double scol = card.ssum[col];
                const float dc = card.del[col];
                float sum = 0.f, diag = 0.f;
#pragma unroll
                for (int hh = 0; hh < TILES; ++hh) {
                    const int rt = TILES * tg + hh, row = 16 * rt + 4 * q;
                    if (dir ? rt < out : rt > out) continue;       // (a group's tile on the diagonal's far side)
                    const f32x4 X = dots(a, dir ? dy : x, dir ? x : dy, rt, out, std::false_type{}, zero4());
                    const f32x4 cb = CB[i][hh];
                    if (rt != out) {
                        // the decay by way of the border of the earlier tile: a factor of the row, one of the column
                        const double border = dsum[16 * (dir ? rt : rt + 1) - 1];
                        const float d = static_cast<float>(dir ? border - dcol : dcol - border), f = decay(d);
                        float part = 0.f;
                        if (dir == 0) {
                            const f32x4 we = lds_get<f32x4>(card.w_end, 4 * row), de = lds_get<f32x4>(card.d_end, 4 * row),
                                        se = lds_get<f32x4>(card.s_end, 4 * row);
#pragma unroll
                            for (int r = 0; r < 4; ++r) {
                                const float v = X[r] * f * we[r], z = v * cb[r];
                                P[i][hh][r] += v;
                                part += z;
                                zA = __builtin_fmaf(z, de[r], zA);
                                zb = __builtin_fmaf(z, se[r], zb);
                            }
                            zA = __builtin_fmaf(part, d, zA);
                            zb = __builtin_fmaf(part, static_cast<float>(scol - card.ssum[16 * rt + 15]), zb);
                            sum += part;
                        } else {
                            const f32x4 ws = lds_get<f32x4>(card.w_start, 4 * row);
                            const float fd = f * dc;
#pragma unroll
                            for (int r = 0; r < 4; ++r) {
                                const float v = X[r] * ws[r];
                                P[i][hh][r] = __builtin_fmaf(v, fd, P[i][hh][r]);
                                part = __builtin_fmaf(v, cb[r], part);
                            }
                            sum = __builtin_fmaf(part, f, sum);
                        }
                    } else if (dir == 0) {
                        const f32x4 dr = lds_get<f32x4>(card.del, 4 * row);
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const int j = row + r;
                            const float d = static_cast<float>(dcol - dsum[j]), e = j <= col ? decay(d) * X[r] : 0.f, y = e * cb[r];
                            const float z = j < col ? y * dr[r] : 0.f;
                            P[i][hh][r] = __builtin_fmaf(e, dr[r], P[i][hh][r]);
                            sum += z;
                            zA = __builtin_fmaf(z, d, zA);
                            zb = __builtin_fmaf(z, static_cast<float>(scol - card.ssum[j]), zb);
                            if (j == col) {
                                diag = y;
                                dD += X[r];
                            }
                        }
                    } else {
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const int j = row + r;
                            const float e = j >= col ? decay(static_cast<float>(dsum[j] - dcol)) * X[r] : 0.f;
                            P[i][hh][r] = __builtin_fmaf(e, dc, P[i][hh][r]);
                            sum += j > col ? e * cb[r] : 0.f;
                        }
                    }
                }
                sum = sum_q(sum);
                if (q == 0) lds.red[(dir ? Lds::COLS : Lds::ROWS) + tg][col] = sum;
                if (dir == 0 && out / TILES == tg) { // the group that holds the tile's own tokens
                    diag = sum_q(diag);
                    if (q == 0) lds.red[Lds::DIAG][col] = diag;
                }
            }
            zA = sum_wave(zA);
            zb = sum_wave(zb);
            dD = sum_wave(dD);
            if (lane == 0) {
                lds.sums[0][wave] = zA;
                lds.sums[1][wave] = zb;
                lds.sums[2][wave] = dD;
            }
            __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
            lds_barrier();                           // the sums and the next head's rows are there
            if (ts < 4) {
                float sum = 0.f;
#pragma unroll
                for (int v = 0; v < WAVES; ++v) sum += lds.sums[ts][v];
                if (ts == 3) sum = -(sum * card.over[0] + sum * card.over[1]);
                (ts == 0 ? L.zA : ts == 1 ? L.zb : ts == 2 ? L.dDp : L.thr)[units + k] = sum;
            }
            lds_barrier();                           // the sums have been read
        }
#pragma unroll
        for (int dir = 0; dir < 2; ++dir) {
            if (dir == 1) lds_barrier();             // direction 0's scores have been read
#pragma unroll
            for (int i = 0; i < ROUNDS; ++i) {
                const int grp = wave + i * WAVES - dir * Lds::GROUPS;
                if (grp < 0 || grp >= Lds::GROUPS) continue;
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
                    lds_put(lds.xy, grp * 2048 + lane * 16, hi);
                    lds_put(lds.xy, grp * 2048 + 1024 + lane * 16, lo);
                } else {
                    lds_put(lds.xy, grp * 1024 + lane * 16, P[i][0]);
                }
            }
            lds_barrier();
        }
        return;
    }

    f32x4 dC[IT], dB[IT];
#pragma unroll
    for (int it = 0; it < IT; ++it) dC[it] = dB[it] = zero4();
    if constexpr (Lds::AHEAD) {
        request_states(S_STATE, 0);
        request_states(G_STATE, 0);
    }
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
    lds_barrier();
    for (int k = 0; k < heads; ++k) {
        const int buf = k & 1;
        const Place a = place();
        const int q = a.q, l16 = a.l16;
        const uint8_t *x = lds.xy + buf * 2 * Lds::A_BYTES, *dy = x + Lds::A_BYTES;
        const Card<CT>& card = *reinterpret_cast<const Card<CT>*>(lds.card[buf]);
        f32x4 S[NS], G[NS];
        if constexpr (Lds::AHEAD) {                  // the states are there; wave 0's four stores behind them may be under way
            if (wave == 0 && k > 0) __builtin_amdgcn_s_waitcnt(vmcnt_imm(4));
            else __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
            wave_fence();
        }
        load_state(S, S_STATE, k);
        load_state(G, G_STATE, k);
        if constexpr (Lds::AHEAD) {
            __builtin_amdgcn_s_waitcnt(0xC07F);      // they are in registers: lgkmcnt(0)
            wave_fence();
            if (k + 1 < heads) {
                request_states(S_STATE, k + 1);
                request_states(G_STATE, k + 1);
            }
        }
        float thr = 0.f;
#pragma unroll
        for (int i = 0; i < NS; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) thr = __builtin_fmaf(S[i][r], G[i][r], thr);
        thr = sum_wave(thr);
        if (lane == 0) lds.sums[3][wave] = thr;
        auto state_part = [&](const f32x4 (&X)[NS], const uint8_t* rows, auto back) {
            constexpr bool BACK = decltype(back)::value;
            u32x4 hi[BF ? KV : 1], mid[BF ? KV : 1], lo[BF ? KV : 1];
            if constexpr (BF) {
#pragma unroll
                for (int kk = 0; kk < KV; ++kk)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const f32x4& m = X[2 * kk + (e >> 1)];
                        uint32_t u, v, w3;
                        split3(m[2 * (e & 1)], m[2 * (e & 1) + 1], u, v, w3);
                        hi[kk][e] = u;
                        mid[kk][e] = v;
                        lo[kk][e] = w3;
                    }
            }
#pragma unroll
            for (int it = 0; it < IT; ++it) {
                if (it % 2 == 0) __builtin_amdgcn_sched_barrier(0);    // (few loads at a time: registers)
                f32x4 O = zero4();
                if constexpr (BF) {
#pragma unroll
                    for (int kk = 0; kk < KV; ++kk) {
                        const u32x4 v = lds_get<u32x4>(rows, a.chan[kk & 1] + it * TA::ROWS16 + (kk >> 1) * 128);
                        O = mfma_bf16(lo[kk], v, O);
                        O = mfma_bf16(mid[kk], v, O);
                        O = mfma_bf16(hi[kk], v, O);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < NS; ++i) {
                        const f32x4 v = lds_get<f32x4>(rows, TA::at(l16, 4 * i + q) + it * TA::ROWS16);
#pragma unroll
                        for (int r = 0; r < 4; ++r) O = mfma_f32(X[i][r], v[r], O);
                    }
                }
                O *= (BACK ? card.after : card.before)[16 * it + l16];
                const f32x4 o = own(a, BACK ? lds.B : lds.C, it);
                if constexpr (BACK) dB[it] += O * card.del[16 * it + l16];
                else dC[it] += O;
                const float s = sum_q(__builtin_fmaf(o[3], O[3], __builtin_fmaf(o[2], O[2], __builtin_fmaf(o[1], O[1], o[0] * O[0]))));
                if (q == 0) lds.red[(BACK ? Lds::R : Lds::P) + wave][16 * it + l16] = s;
            }
        };
        state_part(S, dy, std::false_type{});
        state_part(G, x, std::true_type{});
        lds_barrier();                               // the sums are there
        static_assert(CT <= 64, "wave 0 alone stores");
        if (t < n) {
            float p = 0.f, r = 0.f, rows = 0.f, cols = 0.f;
#pragma unroll
            for (int i = 0; i < WAVES; ++i) {
                p += lds.red[Lds::P + i][t];
                r += lds.red[Lds::R + i][t];
            }
            const int tile = t / 16;
#pragma unroll
            for (int tg = 0; tg < TG; ++tg) {
                if (Lds::near(0, tile, tg)) rows += lds.red[Lds::ROWS + tg][t];
                if (Lds::near(1, tile, tg)) cols += lds.red[Lds::COLS + tg][t];
            }
            // (builtins, so that they are four: see the wait)
            auto put = [&](float* all, float x) {
                __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(x), make_rsrc_u(all + (h0 + k) * L.total + w.lo, n * 4), t * 4, 0, 0);
            };
            put(L.zz, rows - card.del[t] * cols);
            put(L.xz, cols + lds.red[Lds::DIAG][t]);
            put(L.pp, p);
            put(L.xr, r);
        }
        lds_barrier();                               // the sums have been read
    }
    const int q = lane >> 4, l16 = lane & 15;
    const uint32_t tok_c = TC::at(4 * q + (l16 >> 2), 2 * wave + ((l16 & 3) >> 1)) + 8 * (l16 & 1);
    auto tokens = [&](const uint8_t* sm, int tg) {   // the wave's channels of B or C, 32 tokens along the contraction
        const u32x2 x = lds_transpose(sm + tok_c + 2 * tg * TC::ROWS16), y = lds_transpose(sm + tok_c + (2 * tg + 1) * TC::ROWS16);
        return u32x4{x[0], x[1], y[0], y[1]};
    };
#pragma unroll
    for (int dir = 0; dir < 2; ++dir) {
        lds_barrier();                               // the scores are there
        f32x4(&O)[IT] = dir ? dB : dC;
        const uint8_t* sm = dir ? lds.C : lds.B;
#pragma unroll
        for (int tg = 0; tg < TG; ++tg) {
            u32x4 v;
            if constexpr (BF) v = tokens(sm, tg);
            else
#pragma unroll
                for (int r = 0; r < 4; ++r) v[r] = lds_get<uint32_t>(sm, TC::at(16 * tg + 4 * q + r, 4 * wave + (l16 >> 2)) + 4 * (l16 & 3));
#pragma unroll
            for (int it = 0; it < IT; ++it) {
                if (!Lds::near(dir, it, tg)) continue;
                const uint32_t at = Lds::number(dir, it, tg) * Lds::G_BYTES + lane * 16;
                if constexpr (BF) {
                    O[it] = mfma_bf16(v, lds_get<u32x4>(lds.xy, at), O[it]);
                    O[it] = mfma_bf16(v, lds_get<u32x4>(lds.xy, at + 1024), O[it]);
                } else {
                    const f32x4 X = lds_get<f32x4>(lds.xy, at);
#pragma unroll
                    for (int r = 0; r < 4; ++r) O[it] = mfma_f32(__uint_as_float(v[r]), X[r], O[it]);
                }
            }
        }
        if (dir == 0) lds_barrier();                 // direction 0's scores have been read
        // ---- out: lane l16 holds token 16 it + l16, four neighbouring channels
        if (L.part[dir]) {
            const uint32_t orow = static_cast<uint32_t>(L.G) * DK * 4;
            const __amdgpu_buffer_rsrc_t ro = make_rsrc_u(L.part[dir] + ((blk * L.total + w.lo) * L.G + g) * DK, (n - 1) * orow + DK * 4);
#pragma unroll
            for (int it = 0; it < IT; ++it)
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, O[it]), ro,
                                                       (16 * it + l16) * orow + (16 * wave + 4 * q) * 4, 0, 0);
        } else {
            const Out& out = L.out[dir];
            const uint32_t orow = static_cast<uint32_t>(out.ld);
            const __amdgpu_buffer_rsrc_t ro = make_rsrc_u(out.p + w.lo * out.ld + g * TC::RB, (n - 1) * orow + TC::RB);
#pragma unroll
            for (int it = 0; it < IT; ++it) {
                const uint32_t at = (16 * it + l16) * orow + (16 * wave + 4 * q) * ES;
                if constexpr (BF)
                    __builtin_amdgcn_raw_buffer_store_b64(u32x2{pack_bf16(O[it][0], O[it][1]), pack_bf16(O[it][2], O[it][3])}, ro, at, 0, 0);
                else __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, O[it]), ro, at, 0, 0);
            }
        }
    }
}

template <int DT, int DK, int DV>
__global__ void __launch_bounds__(DK * 8, DK / 32) grad_kernel(Scan L) {
    __shared__ GradLds<DT, DK, DV> lds;
    uint32_t unit;
    int32_t pass;
    const uint32_t blocks = static_cast<uint32_t>(L.blocks) * L.G;
    if (!unit_of(L.slots * blocks, 1, unit, pass)) return;
    grad_pass<DT, DK, DV>(L, unit / blocks, unit % blocks, lds);
}

// ---------------------------------------------------------------- ddt, dA, dbias; sums over blocks and chunks

// One wave per (chunk, head), a token a lane.
template <int DT>
__global__ void __launch_bounds__(256) decay_grad_kernel(Scan L) {
    constexpr int CT = CHUNK<DT>;
    const int64_t u = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    if (u >= static_cast<int64_t>(L.c_slots) * L.H) return;
    const int32_t slot = static_cast<int32_t>(u / L.H), h = static_cast<int32_t>(u % L.H);
    Where w;
    if (!locate(L, slot, w) || w.hi == w.lo) {       // no such chunk, or an empty one: nothing to add up
        if (lane == 0) L.dAp[u] = L.dbp[u] = L.dDp[u] = 0.f;
        return;
    }
    const double A = static_cast<double>(L.A[h]), thr = static_cast<double>(L.thr[u]);
    const Card<CT>& card = reinterpret_cast<const Card<CT>*>(L.cards)[u];
    const int64_t at = h * L.total + w.lo + lane;
    const bool live = lane < w.hi - w.lo;
    double x = 0.0, zp = 0.0, p = 0.0, r = 0.0, slope = 0.0, ds = 0.0, ss = 0.0;
    if (live) {
        const Strength s = strength(load_as_f32<DT>(L.dt.p + (w.lo + lane) * L.dt.ld, h), L.bias ? L.bias[h] : 0.f);
        const float later = L.xr[at];
        x = static_cast<double>(L.xz[at]) + later;
        p = static_cast<double>(L.pp[at]);
        zp = static_cast<double>(L.zz[at]) + p;
        r = static_cast<double>(s.delta) * later;
        slope = static_cast<double>(s.slope);
        ds = card.dsum[lane];
        ss = card.ssum[lane];
    }
    const double zs = prefix_sum(zp), rs = prefix_sum(r);
    const double d_all = card.dsum[CT - 1], s_all = card.ssum[CT - 1];
    const double dg = thr + (lane_value(zs, 63) - zs + zp) + (rs - r);
    // a lane's part of sum delta dg, sum slope dg, sum slope x . u
    double dA = p * ds + r * (d_all - ds), db = p * ss + r * (s_all - ss), own = slope * x;
    if (live) store_from_f32<DT>(L.ddt.p + (w.lo + lane) * L.ddt.ld, h, static_cast<float>((x + A * dg) * slope));
    if (lane == 0) {
        dA += static_cast<double>(L.zA[u]) + thr * d_all;
        db += static_cast<double>(L.zb[u]) + thr * s_all;
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

// dA, dbias and dD of head blockIdx.x: sums over the chunks.
__global__ void __launch_bounds__(256) head_sum_kernel(Scan L) {
    __shared__ double red[3][4];
    const int32_t h = blockIdx.x;
    double s[3] = {};
    for (int32_t i = threadIdx.x; i < L.c_slots; i += 256) {
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
// Heads of a workgroup of y and dx: two share the rows of B and C and the raw scores (24 sequences of 2048 tokens, 32 heads:
// 249 us; one head: 307.  Few heads would rather have more workgroups: 1000 tokens of 8 heads whole 76 and 62 us, but they
// run in segments, 36).
int value_heads(int32_t H, int32_t G, int32_t dv) { return dv == 64 && H / G > 1 ? 2 : 1; }

template <int V>
using Int = std::integral_constant<int, V>;
template <typename F>
auto by_sizes(int32_t dk, int32_t dv, F go) {
    if (dk == 128) return dv == 128 ? go(Int<128>{}, Int<128>{}) : go(Int<128>{}, Int<64>{});
    return dv == 128 ? go(Int<64>{}, Int<128>{}) : go(Int<64>{}, Int<64>{});
}
// Tokens per segment of the forward pass, a multiple of 128, for `units` (sequence, head block) pairs: two workgroups a CU,
// or one where those would have fewer than six chunks (packed 1 .. 8209, 16455 tokens, 8 heads: 71 us with two, 64 with
// one; one sequence of 65536 tokens, 32 heads: 409 us with two, 494 with one, 433 with four).  256 pairs fill the CUs
// by themselves.  Short sequences run whole: 520 tokens of 4 heads in bf16 take 44 us whole and 35 in segments, in fp32
// 111 and 45, but 16 of 600 tokens of 16 heads 55 and 63.
int32_t forward_segment(int64_t units, int32_t n_seqs, int64_t total, int32_t in_dtype, bool packed) {
    const int64_t longest = packed ? total : total / n_seqs, blocks = units / n_seqs, least = in_dtype == KDA_BF16 ? 256 : 128;
    if (units >= 256 || longest < 2 * least * std::max<int64_t>(1, units / 64)) return WHOLE;
    auto for_workgroups = [&](int64_t n) {
        const int64_t shares = packed ? std::max<int64_t>(1, n / blocks - n_seqs / 2) : std::max<int64_t>(1, n / units);
        return ((longest + shares - 1) / shares + 127) / 128 * 128;
    };
    int64_t seg = for_workgroups(512);
    if (2 * seg < 3 * least) seg = std::max(for_workgroups(256), least);
    return seg >= longest || seg >= WHOLE ? WHOLE : static_cast<int32_t>(seg);
}
// Of the pass that writes the states of all chunks: it has a workgroup per head and direction, and what segments add (the
// segments' own states, their scan) must pay.  Gradients of 32 heads: 4 x 4096 tokens 451 us whole, 516 in four segments;
// 2 x 4096 300 and 295, 1 x 4096 199 and 148 (1024 tokens, the shortest that run so, 76 and 85).
int32_t state_segment(int64_t units, int32_t n_seqs, int64_t total, int32_t in_dtype, bool packed) {
    const int64_t longest = packed ? total : total / n_seqs, blocks = units / n_seqs;
    if (units >= 64 || longest < 1024) return WHOLE;
    const int64_t shares = packed ? std::max<int64_t>(1, 256 / blocks - n_seqs / 2) : 256 / units;
    const int64_t seg = std::max<int64_t>(((longest + shares - 1) / shares + 127) / 128 * 128, 512);
    return seg >= longest || seg >= WHOLE ? WHOLE : static_cast<int32_t>(seg);
}
// dx starts from the states of a chunk, so its segments cost a state's read only: short ones, for four workgroups a CU.
int32_t dx_segment(int64_t units, int32_t n_seqs, int64_t total, int32_t in_dtype, bool packed) {
    const int64_t longest = packed ? total : total / n_seqs, blocks = units / n_seqs;
    const int64_t shares = packed ? std::max<int64_t>(1, 1024 / blocks) : std::max<int64_t>(1, 1024 / units);
    const int64_t seg = std::max<int64_t>(((longest + shares - 1) / shares + 63) / 64 * 64, 64);
    return seg >= longest || seg >= WHOLE ? WHOLE : static_cast<int32_t>(seg);
}

// The rules' segments jump as the sizes grow, and a workspace that is kept for the largest batch must serve every smaller
// one.  So the workspace's size is formed from the most segments that n_seqs sequences of `total` tokens or fewer of
// either have, `blocks` head blocks a sequence (n of the sequences that still run in segments):
//   a segment has `least` tokens or more: total / least + n;
//   fixed lengths: at most n (W / (n blocks)) for W workgroups; packed: W / blocks - n / 2 and one more a sequence.
int64_t most_segments(int64_t blocks, int32_t n_seqs, int64_t total, int64_t whole, int64_t workgroups, int64_t shortest, int64_t least) {
    if (blocks >= whole || total < shortest) return 0;
    const int64_t n = std::min<int64_t>(n_seqs, (whole - 1) / blocks);
    return std::min(total / least + n, workgroups / blocks + (n + 1) / 2);
}
int64_t most_forward_segments(int64_t blocks, int32_t n_seqs, int64_t total, int32_t in_dtype) {
    const int64_t least = in_dtype == KDA_BF16 ? 256 : 128;
    return most_segments(blocks, n_seqs, total, 256, 512, 2 * least, least);
}
int64_t most_state_segments(int64_t blocks, int32_t n_seqs, int64_t total) {
    return most_segments(blocks, n_seqs, total, 64, 256, 1024, 512);
}

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

void set_segments(Scan& L, int32_t (*rule)(int64_t, int32_t, int64_t, int32_t, bool), int32_t dv, int32_t in_dtype, bool packed) {
    const int64_t units = int64_t(L.n_seqs) * head_blocks(L.H, L.G, value_heads(L.H, L.G, dv)) * L.G;
    L.seg = rule(units, L.n_seqs, L.total, in_dtype, packed);
    L.slots = static_cast<int32_t>(segment_slots(L.n_seqs, L.total, L.seg, packed));
    L.n_seg = L.slots / L.n_seqs;
}
// Chunks of the gradients and blocks of heads: as few as leave every CU a workgroup.
void set_chunks(Scan& L, int32_t in_dtype, bool packed) {
    L.ct = in_dtype == KDA_BF16 ? CHUNK<KDA_BF16> : CHUNK<KDA_F32>;
    L.c_slots = static_cast<int32_t>(segment_slots(L.n_seqs, L.total, L.ct, packed));
    L.c_per_seq = L.c_slots / L.n_seqs;
    L.heads = L.H / L.G;
    while (L.heads > 1 && int64_t(L.c_slots) * L.G * head_blocks(L.H, L.G, L.heads) < 256) L.heads = (L.heads + 1) / 2;
    L.blocks = head_blocks(L.H, L.G, L.heads);
}

// Rows of d_k that the head blocks of the gradients leave to be added up (where there is more than one block).
int64_t block_parts(const Scan& L) { return L.total * L.G * L.blocks; }
// The most of them, for L.total tokens or fewer.  set_chunks halves the heads of a block, and so doubles the blocks at
// most, while c chunks of ct tokens have c G blocks < 256: fewer than 512 / (c G) blocks, of c ct tokens or fewer.
int64_t most_block_parts(const Scan& L) { return std::min(L.total * L.H, int64_t(510) * L.ct); }

// Called with a call's own segments and chunks, and with the most that smaller sizes have.
void carve_segments(Scan& L, Carver& ws, int64_t elems, int passes) {
    if (L.seg == WHOLE || L.slots == 0) return;
    for (int st = 0; st < passes; ++st) {
        L.seg_states[st] = ws.take<float>(int64_t(L.slots) * L.H * elems);
        L.seg_decay[st] = ws.take<f32x2>(int64_t(L.slots) * L.H);
    }
}
void carve_forward(Scan& L, Carver& ws, int64_t elems) { carve_segments(L, ws, elems, 1); }
void carve_backward(Scan& L, Carver& ws, int32_t dk, int32_t dv, int64_t parts) {
    const int64_t cu = int64_t(L.c_slots) * L.H;
    carve_segments(L, ws, int64_t(dk) * dv, 2);
    for (float*& p : L.chunk_states) p = ws.take<float>(cu * dk * dv);
    if (L.blocks > 1)
        for (float*& p : L.part) p = ws.take<float>(parts * dk);
    L.cards = ws.take<uint8_t>(cu * (L.ct == CHUNK<KDA_BF16> ? sizeof(Card<CHUNK<KDA_BF16>>) : sizeof(Card<CHUNK<KDA_F32>>)));
    for (float** p : {&L.zz, &L.pp, &L.xz, &L.xr}) *p = ws.take<float>(L.H * L.total);
    for (float** p : {&L.zA, &L.zb, &L.dDp, &L.thr, &L.dAp, &L.dbp}) *p = ws.take<float>(cu);
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
template <int DT, bool CHUNKS>
hipError_t launch_states(Scan L, int32_t dk, int32_t dv, int32_t passes, hipStream_t stream) {
    L.blocks = L.H / L.G;
    return by_sizes(dk, dv, [&](auto k, auto v) {
        hipLaunchKernelGGL((state_kernel<DT, decltype(k)::value, decltype(v)::value, CHUNKS>), dim3(xcd_grid(int64_t(L.slots) * L.H, passes)),
                           dim3(decltype(v)::value * 4), 0, stream, L, passes);
        return hipGetLastError();
    });
}
// The states that the segments start from (S), or that follow them (G).
template <int DT>
hipError_t launch_segments(const Scan& L, int32_t dk, int32_t dv, int32_t passes, hipStream_t stream) {
    const hipError_t e = launch_states<DT, false>(L, dk, dv, passes, stream);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(scan_kernel, dim3(static_cast<unsigned>(L.n_seqs * L.H), static_cast<unsigned>(dk * dv / 1024), passes),
                       dim3(256), 0, stream, L, dk * dv);
    return hipGetLastError();
}

template <int DT, int ODT>
hipError_t forward(const ScanArgs& a, hipStream_t stream) {
    Scan L = base(a);
    set_segments(L, forward_segment, a.dv, a.in_dtype, a.cu != nullptr);
    Carver ws{static_cast<uint8_t*>(a.workspace)};
    carve_forward(L, ws, int64_t(a.dk) * a.dv);
    L.m_out[S_STATE] = a.hT;
    L.exact[S_STATE] = a.hT != nullptr;
    L.out[0] = Out{static_cast<uint8_t*>(a.y.p), a.y.ld * (ODT == KDA_BF16 ? 2 : 4)};
    if (L.seg < WHOLE) {
        const hipError_t e = launch_segments<DT>(L, a.dk, a.dv, 1, stream);
        if (e != hipSuccess) return e;
    }
    return launch_value<DT, ODT, Y>(L, a.dk, a.dv, stream);
}

template <int DT>
hipError_t backward(const ScanArgs& a, hipStream_t stream) {
    const int64_t es = DT == KDA_BF16 ? 2 : 4;
    auto out = [&](const RowsOut& r) { return Out{static_cast<uint8_t*>(r.p), r.ld * es}; };
    const bool packed = a.cu != nullptr;
    Scan L = base(a);
    set_chunks(L, a.in_dtype, packed);
    set_segments(L, state_segment, a.dv, a.in_dtype, packed);
    Carver ws{static_cast<uint8_t*>(a.workspace)};
    carve_backward(L, ws, a.dk, a.dv, block_parts(L));
    L.m_out[G_STATE] = a.dh0;
    L.exact[S_STATE] = L.exact[G_STATE] = 1;
    L.ddt = out(a.ddt);
    L.dA = a.dA; L.dD = a.dD; L.dbias = a.dbias;
    // the decays, chunk by chunk
    Scan K = L;
    K.seg = L.ct;
    K.slots = L.c_slots;
    K.n_seg = L.c_per_seq;
    const unsigned waves = static_cast<unsigned>((int64_t(L.c_slots) * L.H + 3) / 4);
    hipLaunchKernelGGL((card_kernel<DT>), dim3(waves), dim3(256), 0, stream, K);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    // the states of every chunk
    if (L.seg < WHOLE) e = launch_segments<DT>(L, a.dk, a.dv, 2, stream);
    if (e == hipSuccess) e = launch_states<DT, true>(L, a.dk, a.dv, 2, stream);
    if (e != hipSuccess) return e;
    // dx from them, in segments of its own
    Scan X = L;
    set_segments(X, dx_segment, a.dv, a.in_dtype, packed);
    X.out[0] = out(a.dx);
    e = launch_value<DT, DT, DX>(X, a.dk, a.dv, stream);
    if (e != hipSuccess) return e;
    // the other gradients, chunk by chunk
    K.out[S_STATE] = out(a.dC);
    K.out[G_STATE] = out(a.dB);
    e = by_sizes(a.dk, a.dv, [&](auto k, auto v) {
        constexpr int DK = decltype(k)::value, DV = decltype(v)::value;
        hipLaunchKernelGGL((grad_kernel<DT, DK, DV>), dim3(xcd_grid(int64_t(K.slots) * K.blocks * K.G, 1)), dim3(DK * 8), 0, stream, K);
        return hipGetLastError();
    });
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((decay_grad_kernel<DT>), dim3(waves), dim3(256), 0, stream, K);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (L.blocks > 1 && L.total > 0) {
        const int32_t row = a.G * a.dk;
        const int64_t quads = K.total * row / 4;
        hipLaunchKernelGGL(part_sum_kernel<DT>, dim3(static_cast<unsigned>((quads + 255) / 256), 2), dim3(256), 0, stream, K, row, quads);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(head_sum_kernel, dim3(K.H), dim3(256), 0, stream, K);
    return hipGetLastError();
}

}  // namespace

size_t scan_workspace_bytes(int32_t n_seqs, int64_t total, int32_t H, int32_t G, int32_t dk, int32_t dv,
                            int32_t in_dtype, bool backward) {
    // what sizes up to these may need, which is never less than what these do as fixed lengths or packed
    size_t most = 0;
    const int64_t blocks = int64_t(head_blocks(H, G, value_heads(H, G, dv))) * G;
    for (const int kind : {0, 1, 2}) {               // fixed lengths, packed, the most of all
        Scan L{};
        L.n_seqs = n_seqs; L.total = total; L.H = H; L.G = G;
        Carver ws{nullptr};
        if (backward) {
            set_chunks(L, in_dtype, kind >= 1);      // (a packed batch has the more chunks)
            set_segments(L, state_segment, dv, in_dtype, kind == 1);
            if (kind == 2) {
                L.blocks = H / G;
                L.seg = 0;
                L.slots = static_cast<int32_t>(most_state_segments(blocks, n_seqs, total));
            }
            carve_backward(L, ws, dk, dv, kind == 2 ? most_block_parts(L) : block_parts(L));
        } else {
            set_segments(L, forward_segment, dv, in_dtype, kind == 1);
            if (kind == 2) {
                L.seg = 0;
                L.slots = static_cast<int32_t>(most_forward_segments(blocks, n_seqs, total, in_dtype));
            }
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
// both ways).  Lane t owns four columns of DK / RG rows.  Bound by HBM: 256 sequences, 32 heads of 128 x 64 in 100 to
// 104 us, 5.2 TB/s; one sequence in 4.7 us.
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
