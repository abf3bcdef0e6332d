// kda_api_ssm.cpp -- the extern "C" boundary of the short convolution, the selective scan and the slot pools:
// argument validation, dispatch, status.  Declarations and error behaviour are documented in include/kda.h.
#include <cstdint>
#include <initializer_list>

#include "kda_api_util.hpp"
#include "kda_ssm.hpp"

namespace {

// Bytes from token to token.  The kernels' offsets into a run of 128 tokens, with up to 3 on either side, are unsigned 32-bit
// numbers: 134 rows span less than 2^32 bytes (though more than 2^31).
constexpr int64_t kMaxRow = int64_t(1) << 24;
constexpr int64_t kMaxTokens = (int64_t(1) << 31) - 1;

// `rows` rows of `bytes` each, `ld` bytes apart.
struct Strided {
    uintptr_t lo;
    int64_t rows, bytes, ld;
};
Strided strided(const void* p, int64_t rows, int64_t bytes, int64_t ld) {
    return Strided{reinterpret_cast<uintptr_t>(p), p ? rows : 0, bytes, ld};
}
Strided flat(const void* p, int64_t bytes) { return strided(p, bytes > 0 ? 1 : 0, bytes, bytes); }
// Rows of one stride may lie side by side in a wider row (x, B and C of one buffer).
bool overlap(const Strided& a, const Strided& b) {
    if (a.rows == 0 || b.rows == 0) return false;
    const uintptr_t a_hi = a.lo + (a.rows - 1) * a.ld + a.bytes, b_hi = b.lo + (b.rows - 1) * b.ld + b.bytes;
    if (a_hi <= b.lo || b_hi <= a.lo) return false;
    if (a.ld != b.ld || a.rows == 1 || b.rows == 1) return true;
    const int64_t ld = a.ld, d = static_cast<int64_t>(b.lo >= a.lo ? (b.lo - a.lo) % ld : (ld - (a.lo - b.lo) % ld) % ld);
    return d < a.bytes || ld - d < b.bytes;
}
bool disjoint(std::initializer_list<Strided> outs, std::initializer_list<Strided> ins) {
    for (const Strided* a = outs.begin(); a != outs.end(); ++a) {
        for (const Strided* b = a + 1; b != outs.end(); ++b)
            if (overlap(*a, *b)) return false;
        for (const Strided& b : ins)
            if (overlap(*a, b)) return false;
    }
    return true;
}
bool aligned(std::initializer_list<const void*> ps, int64_t bytes) {
    for (const void* p : ps)
        if (reinterpret_cast<uintptr_t>(p) % bytes != 0) return false;
    return true;
}

// ---- convolution

int conv_sizes(int dtype, const int32_t* cu, int32_t B, int64_t T, int32_t n_seqs, int32_t C, int32_t W) {
    if (!valid_dtype(dtype) || B < 1 || T < 0 || n_seqs < 1 || C < 1 || W < 1) return KDA_ERR_INVALID_ARGUMENT;
    if (cu ? (B != 1) : (n_seqs != B)) return KDA_ERR_INVALID_ARGUMENT;
    if (W < 2 || W > 4) return KDA_ERR_UNSUPPORTED;
    if (T > kMaxTokens / B || int64_t(C) * esize(dtype) > kMaxRow) return KDA_ERR_UNSUPPORTED;
    // grids of 256-lane workgroups (128 tokens by at least 32 channels, 256 elements of the final windows) must stay
    // within 2^32 lanes
    const int64_t blocks = (int64_t(B) * T / 128 + n_seqs) * (C / 32 + 1), windows = int64_t(n_seqs) * 3 * C / 256;
    if (blocks + windows > (int64_t(1) << 24) - 2) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}
int row_stride(int64_t ld, int64_t row, int64_t es) {
    if (ld < row) return KDA_ERR_INVALID_ARGUMENT;
    return ld > kMaxRow / es ? KDA_ERR_UNSUPPORTED : KDA_OK;
}
int check_cu(const int32_t* cu, int32_t n_seqs, int64_t ntok, void* stream) {
    return cu ? linear_debug(nullptr, cu, n_seqs, ntok, 0, stream) : KDA_OK;
}

// ---- scan

struct ScanShape {
    int32_t B;
    int64_t T;
    int32_t n_seqs, H, G, dk, dv;
};
int scan_sizes(int in_dtype, const int32_t* cu, const ScanShape& s) {
    if (!valid_dtype(in_dtype) || s.B < 1 || s.T < 0 || s.n_seqs < 1 || s.H < 1 || s.G < 1 || s.dk < 1 || s.dv < 1)
        return KDA_ERR_INVALID_ARGUMENT;
    if (s.H % s.G != 0 || (cu ? (s.B != 1) : (s.n_seqs != s.B))) return KDA_ERR_INVALID_ARGUMENT;
    if (!supported_d(s.dk) || !supported_d(s.dv)) return KDA_ERR_UNSUPPORTED;
    if (s.T > kMaxTokens / s.B) return KDA_ERR_UNSUPPORTED;
    const int64_t ntok = s.B * s.T;
    // grids of up to 1024 lanes per (segment of at least 128 tokens, head) must stay within 2^32 lanes, and so must
    // one lane per four channels of B
    if (s.H > 32768 || (ntok / 128 + s.n_seqs) > (int64_t(1) << 21) / s.H) return KDA_ERR_UNSUPPORTED;
    if (ntok * s.G > (int64_t(1) << 33) / s.dk) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}
// Workgroups of 1024 lanes per (chunk of the gradients, head) must stay within 2^32 lanes, rounded up to the XCDs.
bool chunks_fit(int in_dtype, int64_t ntok, int64_t n_seqs, int32_t H) {
    return ntok / (in_dtype == KDA_BF16 ? 64 : 32) + n_seqs <= ((int64_t(1) << 22) - 8) / H;
}
// Row strides of x, dt, B, C and the like: at least a row, 16-byte steps but for dt.
struct Ld {
    int64_t ld, row;
    bool wide;
};
int strides_ok(std::initializer_list<Ld> lds, int64_t es) {
    for (const Ld& l : lds) {
        const int st = row_stride(l.ld, l.row, es);
        if (st != KDA_OK) return st;
    }
    for (const Ld& l : lds)
        if (l.wide && l.ld * es % 16 != 0) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

// ---- slots

constexpr int32_t kMaxSlots = 1 << 20;

int planes_ok(const void* const* a, const void* const* b, const int64_t* bytes, int32_t n, int64_t pairs,
              kda::Planes* p) {
    if (n < 1 || !a || !b || !bytes) return KDA_ERR_INVALID_ARGUMENT;
    if (n > kda::MAX_PLANES) return KDA_ERR_UNSUPPORTED;
    int64_t parts = 0;
    for (int32_t i = 0; i < n; ++i) {
        if (!a[i] || !b[i] || bytes[i] < 1) return KDA_ERR_INVALID_ARGUMENT;
        if (!aligned16({a[i], b[i]}) || bytes[i] > (int64_t(1) << 40)) return KDA_ERR_UNSUPPORTED;
        p->src[i] = static_cast<const uint8_t*>(a[i]);
        p->dst[i] = static_cast<uint8_t*>(const_cast<void*>(b[i]));
        p->bytes[i] = bytes[i];
        parts += (bytes[i] + 32767) / 32768;
    }
    p->n = n;
    // a grid of 256-lane workgroups, one per 32 KB of a pair, must stay within 2^32 lanes
    if (parts > ((int64_t(1) << 24) - 1) / (pairs > 0 ? pairs : 1)) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}
// No plane overlaps another or one of the arrays, and no two arrays overlap.
bool planes_disjoint(const kda::Planes& p, int64_t n_slots, std::initializer_list<Strided> arrays) {
    for (int32_t i = 0; i < p.n; ++i) {
        const Strided a = flat(p.dst[i], p.bytes[i] * n_slots);
        for (int32_t j = i + 1; j < p.n; ++j)
            if (overlap(a, flat(p.dst[j], p.bytes[j] * n_slots))) return false;
        for (const Strided& b : arrays)
            if (overlap(a, b)) return false;
    }
    return disjoint(arrays, {});
}

}  // namespace

extern "C" {

size_t kda_conv_bwd_workspace_size(int32_t n_seqs, int64_t total_tokens, int32_t C, int32_t W) {
    if (n_seqs < 1 || total_tokens < 0 || total_tokens > kMaxTokens || C < 1 || C > kMaxRow / 2 || W < 2 || W > 4) return 0;
    return kda::conv_workspace_bytes(n_seqs, total_tokens, C, W);
}

int kda_conv_fwd(const void* x, int64_t ldx, int dtype, const float* weight, const float* bias,
                 const void* initial_state, void* final_state, const int32_t* cu_seqlens, void* y, int64_t ldy,
                 int32_t B, int64_t T, int32_t n_seqs, int32_t C, int32_t W, int silu, void* stream) {
    int st = conv_sizes(dtype, cu_seqlens, B, T, n_seqs, C, W);
    if (st != KDA_OK) return st;
    const int64_t es = esize(dtype), ntok = B * T, window = int64_t(n_seqs) * (W - 1) * C * es;
    if ((st = row_stride(ldx, C, es)) != KDA_OK || (st = row_stride(ldy, C, es)) != KDA_OK) return st;
    if (!weight || (ntok > 0 && (!x || !y))) return KDA_ERR_INVALID_ARGUMENT;
    if (!aligned({x, y, initial_state, final_state}, es) || !aligned4({weight, bias, cu_seqlens})) return KDA_ERR_UNSUPPORTED;
    if (!disjoint({strided(y, ntok, C * es, ldy * es), flat(final_state, window)},
                  {strided(x, ntok, C * es, ldx * es), flat(initial_state, window), flat(weight, int64_t(C) * W * 4),
                   flat(bias, int64_t(C) * 4), flat(cu_seqlens, int64_t(n_seqs + 1) * 4)}))
        return KDA_ERR_INVALID_ARGUMENT;
    if ((st = check_cu(cu_seqlens, n_seqs, ntok, stream)) != KDA_OK) return st;
    kda::ConvArgs a{};
    a.x = {x, ldx}; a.dy = {nullptr, ldx}; a.out = {y, ldy}; a.weight = weight; a.bias = bias; a.h0 = initial_state;
    a.hT = final_state; a.cu = cu_seqlens; a.dtype = dtype; a.silu = silu != 0; a.B = B; a.T = T; a.n_seqs = n_seqs;
    a.C = C; a.W = W;
    return from_hip(kda::launch_conv_fwd(a, static_cast<hipStream_t>(stream)));
}

int kda_conv_bwd(const void* x, int64_t ldx, int dtype, const float* weight, const float* bias,
                 const void* initial_state, const int32_t* cu_seqlens, const void* dy, int64_t lddy,
                 const void* d_final_state, void* dx, int64_t lddx, float* d_weight, float* d_bias,
                 void* d_initial_state, int32_t B, int64_t T, int32_t n_seqs, int32_t C, int32_t W, int silu,
                 void* workspace, size_t workspace_bytes, void* stream) {
    int st = conv_sizes(dtype, cu_seqlens, B, T, n_seqs, C, W);
    if (st != KDA_OK) return st;
    const int64_t es = esize(dtype), ntok = B * T, window = int64_t(n_seqs) * (W - 1) * C * es;
    for (int64_t ld : {ldx, lddy, lddx})
        if ((st = row_stride(ld, C, es)) != KDA_OK) return st;
    if (!weight || !d_weight || (ntok > 0 && (!x || !dy || !dx))) return KDA_ERR_INVALID_ARGUMENT;
    if (!aligned({x, dy, dx, initial_state, d_final_state, d_initial_state}, es) ||
        !aligned4({weight, bias, d_weight, d_bias, cu_seqlens}) || !aligned16({workspace}))
        return KDA_ERR_UNSUPPORTED;
    const size_t need = kda::conv_workspace_bytes(n_seqs, ntok, C, W);
    if (workspace_bytes < need || !workspace) return KDA_ERR_WORKSPACE;
    if (!disjoint({strided(dx, ntok, C * es, lddx * es), flat(d_weight, int64_t(C) * W * 4), flat(d_bias, int64_t(C) * 4),
                   flat(d_initial_state, window), flat(workspace, static_cast<int64_t>(workspace_bytes))},
                  {strided(x, ntok, C * es, ldx * es), strided(dy, ntok, C * es, lddy * es), flat(initial_state, window),
                   flat(d_final_state, window), flat(weight, int64_t(C) * W * 4), flat(bias, int64_t(C) * 4),
                   flat(cu_seqlens, int64_t(n_seqs + 1) * 4)}))
        return KDA_ERR_INVALID_ARGUMENT;
    if ((st = check_cu(cu_seqlens, n_seqs, ntok, stream)) != KDA_OK) return st;
    kda::ConvArgs a{};
    a.x = {x, ldx}; a.dy = {dy, lddy}; a.out = {dx, lddx}; a.weight = weight; a.bias = bias; a.h0 = initial_state;
    a.dhT = d_final_state; a.dh0 = d_initial_state; a.dw = d_weight; a.db = d_bias; a.cu = cu_seqlens; a.dtype = dtype;
    a.silu = silu != 0; a.B = B; a.T = T; a.n_seqs = n_seqs; a.C = C; a.W = W; a.workspace = workspace;
    return from_hip(kda::launch_conv_bwd(a, static_cast<hipStream_t>(stream)));
}

int kda_conv_step(const void* x, int64_t ldx, int dtype, const float* weight, const float* bias, void* windows,
                  const int32_t* slots, void* y, int64_t ldy, int32_t N, int32_t n_slots, int32_t C, int32_t W,
                  int silu, void* stream) {
    if (!valid_dtype(dtype) || N < 0 || n_slots < 1 || C < 1 || W < 1) return KDA_ERR_INVALID_ARGUMENT;
    if (W < 2 || W > 4 || int64_t(C) * esize(dtype) > kMaxRow) return KDA_ERR_UNSUPPORTED;
    if (!slots && N > n_slots) return KDA_ERR_INVALID_ARGUMENT;
    const int64_t es = esize(dtype);
    int st;
    if ((st = row_stride(ldx, C, es)) != KDA_OK || (st = row_stride(ldy, C, es)) != KDA_OK) return st;
    if (N == 0) return KDA_OK;
    if (!x || !weight || !windows || !y) return KDA_ERR_INVALID_ARGUMENT;
    if (!aligned({x, y, windows}, es) || !aligned4({weight, bias, slots})) return KDA_ERR_UNSUPPORTED;
    // a grid of 256-lane workgroups must stay within 2^32 lanes
    if (int64_t(N) * (C / 256 + 1) > (int64_t(1) << 24) - 1) return KDA_ERR_UNSUPPORTED;
    if (!disjoint({strided(y, N, C * es, ldy * es), flat(windows, int64_t(n_slots) * (W - 1) * C * es)},
                  {strided(x, N, C * es, ldx * es), flat(weight, int64_t(C) * W * 4), flat(bias, int64_t(C) * 4),
                   flat(slots, int64_t(N) * 4)}))
        return KDA_ERR_INVALID_ARGUMENT;
    kda::ConvArgs a{};
    a.x = {x, ldx}; a.dy = {nullptr, ldx}; a.out = {y, ldy}; a.weight = weight; a.bias = bias; a.dtype = dtype;
    a.silu = silu != 0; a.C = C; a.W = W;
    return from_hip(kda::launch_conv_step(a, windows, slots, N, n_slots, static_cast<hipStream_t>(stream)));
}

size_t kda_ssm_chunk_workspace_size(int32_t n_seqs, int64_t total_tokens, int32_t H, int32_t G, int32_t dk,
                                    int32_t dv, int in_dtype, int backward) {
    if (n_seqs < 1 || total_tokens < 0 || total_tokens > kMaxTokens || H < 1 || G < 1 || H % G != 0 ||
        !supported_d(dk) || !supported_d(dv) || !valid_dtype(in_dtype))
        return 0;
    if (H > 32768 || (total_tokens / 128 + n_seqs) > (int64_t(1) << 21) / H) return 0;
    if (backward && !chunks_fit(in_dtype, total_tokens, n_seqs, H)) return 0;
    return kda::scan_workspace_bytes(n_seqs, total_tokens, H, G, dk, dv, in_dtype, backward != 0);
}

int kda_ssm_chunk_fwd(const void* x, int64_t ldx, const void* dt, int64_t lddt, const void* Bm, int64_t ldb,
                      const void* Cm, int64_t ldc, int in_dtype, const float* A, const float* dt_bias, const float* D,
                      const float* initial_state, float* final_state, const int32_t* cu_seqlens, void* y, int64_t ldy,
                      int y_dtype, int32_t B, int64_t T, int32_t n_seqs, int32_t H, int32_t G, int32_t dk, int32_t dv,
                      void* workspace, size_t workspace_bytes, void* stream) {
    if (!valid_dtype(y_dtype)) return KDA_ERR_INVALID_ARGUMENT;
    int st = scan_sizes(in_dtype, cu_seqlens, {B, T, n_seqs, H, G, dk, dv});
    if (st != KDA_OK) return st;
    const int64_t es = esize(in_dtype), os = esize(y_dtype), ntok = B * T, rv = int64_t(H) * dv, rk = int64_t(G) * dk;
    if ((st = strides_ok({{ldx, rv, true}, {lddt, H, false}, {ldb, rk, true}, {ldc, rk, true}}, es)) != KDA_OK) return st;
    if ((st = strides_ok({{ldy, rv, true}}, os)) != KDA_OK) return st;
    if (!A || (ntok > 0 && (!x || !dt || !Bm || !Cm || !y))) return KDA_ERR_INVALID_ARGUMENT;
    if (!aligned16({x, Bm, Cm, y, initial_state, final_state, workspace}) || !aligned({dt}, es) ||
        !aligned4({A, dt_bias, D, cu_seqlens}))
        return KDA_ERR_UNSUPPORTED;
    const size_t need = kda::scan_workspace_bytes(n_seqs, ntok, H, G, dk, dv, in_dtype, false);
    if (workspace_bytes < need || (need > 0 && !workspace)) return KDA_ERR_WORKSPACE;
    const int64_t states = int64_t(n_seqs) * H * dk * dv * 4;
    const Strided r_y = strided(y, ntok, rv * os, ldy * os), r_hT = flat(final_state, states), r_h0 = flat(initial_state, states);
    const Strided r_ws = flat(workspace, static_cast<int64_t>(workspace_bytes));
    if (!disjoint({r_y, r_hT, r_ws},
                  {strided(x, ntok, rv * es, ldx * es), strided(dt, ntok, H * es, lddt * es),
                   strided(Bm, ntok, rk * es, ldb * es), strided(Cm, ntok, rk * es, ldc * es), flat(A, int64_t(H) * 4),
                   flat(dt_bias, int64_t(H) * 4), flat(D, int64_t(H) * 4), flat(cu_seqlens, int64_t(n_seqs + 1) * 4)}) ||
        overlap(r_y, r_h0) || overlap(r_ws, r_h0))
        return KDA_ERR_INVALID_ARGUMENT;
    // the final state may be the initial state itself, but must not partly overlap it
    if (initial_state != final_state && overlap(r_h0, r_hT)) return KDA_ERR_INVALID_ARGUMENT;
    if ((st = linear_debug(A, cu_seqlens, n_seqs, ntok, H, stream)) != KDA_OK) return st;
    kda::ScanArgs a{};
    a.x = {x, ldx}; a.dt = {dt, lddt}; a.B = {Bm, ldb}; a.C = {Cm, ldc}; a.A = A; a.bias = dt_bias; a.D = D;
    a.h0 = initial_state; a.hT = final_state; a.cu = cu_seqlens; a.y = {y, ldy}; a.in_dtype = in_dtype;
    a.y_dtype = y_dtype; a.batch = B; a.T = T; a.n_seqs = n_seqs; a.H = H; a.G = G; a.dk = dk; a.dv = dv;
    a.workspace = workspace;
    return from_hip(kda::launch_scan_fwd(a, static_cast<hipStream_t>(stream)));
}

int kda_ssm_chunk_bwd(const void* x, int64_t ldx, const void* dt, int64_t lddt, const void* Bm, int64_t ldb,
                      const void* Cm, int64_t ldc, int in_dtype, const float* A, const float* dt_bias, const float* D,
                      const float* initial_state, const int32_t* cu_seqlens, const void* dy, int64_t lddy,
                      const float* d_final_state, void* dx, int64_t lddx, void* ddt, int64_t ldddt, void* dBm,
                      int64_t lddb, void* dCm, int64_t lddc, float* dA, float* dD, float* d_dt_bias,
                      float* d_initial_state, int32_t B, int64_t T, int32_t n_seqs, int32_t H, int32_t G, int32_t dk,
                      int32_t dv, void* workspace, size_t workspace_bytes, void* stream) {
    int st = scan_sizes(in_dtype, cu_seqlens, {B, T, n_seqs, H, G, dk, dv});
    if (st != KDA_OK) return st;
    const int64_t es = esize(in_dtype), ntok = B * T, rv = int64_t(H) * dv, rk = int64_t(G) * dk;
    if (!chunks_fit(in_dtype, ntok, n_seqs, H)) return KDA_ERR_UNSUPPORTED;
    if ((st = strides_ok({{ldx, rv, true}, {lddt, H, false}, {ldb, rk, true}, {ldc, rk, true}, {lddy, rv, true},
                          {lddx, rv, true}, {ldddt, H, false}, {lddb, rk, true}, {lddc, rk, true}}, es)) != KDA_OK)
        return st;
    if (!A || !dA || (ntok > 0 && (!x || !dt || !Bm || !Cm || !dy || !dx || !ddt || !dBm || !dCm)))
        return KDA_ERR_INVALID_ARGUMENT;
    if (!aligned16({x, Bm, Cm, dy, dx, dBm, dCm, initial_state, d_final_state, d_initial_state, workspace}) ||
        !aligned({dt, ddt}, es) || !aligned4({A, dt_bias, D, dA, dD, d_dt_bias, cu_seqlens}))
        return KDA_ERR_UNSUPPORTED;
    const size_t need = kda::scan_workspace_bytes(n_seqs, ntok, H, G, dk, dv, in_dtype, true);
    if (workspace_bytes < need || !workspace) return KDA_ERR_WORKSPACE;
    const int64_t states = int64_t(n_seqs) * H * dk * dv * 4, per_head = int64_t(H) * 4;
    if (!disjoint({strided(dx, ntok, rv * es, lddx * es), strided(ddt, ntok, H * es, ldddt * es),
                   strided(dBm, ntok, rk * es, lddb * es), strided(dCm, ntok, rk * es, lddc * es), flat(dA, per_head),
                   flat(dD, per_head), flat(d_dt_bias, per_head), flat(d_initial_state, states),
                   flat(workspace, static_cast<int64_t>(workspace_bytes))},
                  {strided(x, ntok, rv * es, ldx * es), strided(dt, ntok, H * es, lddt * es),
                   strided(Bm, ntok, rk * es, ldb * es), strided(Cm, ntok, rk * es, ldc * es),
                   strided(dy, ntok, rv * es, lddy * es), flat(A, per_head), flat(dt_bias, per_head), flat(D, per_head),
                   flat(initial_state, states), flat(d_final_state, states), flat(cu_seqlens, int64_t(n_seqs + 1) * 4)}))
        return KDA_ERR_INVALID_ARGUMENT;
    if ((st = linear_debug(A, cu_seqlens, n_seqs, ntok, H, stream)) != KDA_OK) return st;
    kda::ScanArgs a{};
    a.x = {x, ldx}; a.dt = {dt, lddt}; a.B = {Bm, ldb}; a.C = {Cm, ldc}; a.dy = {dy, lddy}; a.A = A; a.bias = dt_bias;
    a.D = D; a.h0 = initial_state; a.dhT = d_final_state; a.dh0 = d_initial_state; a.cu = cu_seqlens;
    a.dx = {dx, lddx}; a.ddt = {ddt, ldddt}; a.dB = {dBm, lddb}; a.dC = {dCm, lddc}; a.dA = dA; a.dD = dD;
    a.dbias = d_dt_bias; a.in_dtype = in_dtype; a.y_dtype = in_dtype; a.batch = B; a.T = T; a.n_seqs = n_seqs; a.H = H;
    a.G = G; a.dk = dk; a.dv = dv; a.workspace = workspace;
    return from_hip(kda::launch_scan_bwd(a, static_cast<hipStream_t>(stream)));
}

int kda_ssm_decode_step(const void* x, int64_t ldx, const void* dt, int64_t lddt, const void* Bm, int64_t ldb,
                        const void* Cm, int64_t ldc, int in_dtype, const float* A, const float* dt_bias, const float* D,
                        float* state, const int32_t* slots, void* y, int64_t ldy, int y_dtype, int32_t N,
                        int32_t n_slots, int32_t H, int32_t G, int32_t dk, int32_t dv, void* stream) {
    if (!valid_dtype(in_dtype) || !valid_dtype(y_dtype)) return KDA_ERR_INVALID_ARGUMENT;
    if (N < 0 || n_slots < 1 || H < 1 || G < 1 || dk < 1 || dv < 1 || H % G != 0) return KDA_ERR_INVALID_ARGUMENT;
    if (!supported_d(dk) || !supported_d(dv)) return KDA_ERR_UNSUPPORTED;
    if (!slots && N > n_slots) return KDA_ERR_INVALID_ARGUMENT;
    const int64_t es = esize(in_dtype), os = esize(y_dtype), rv = int64_t(H) * dv, rk = int64_t(G) * dk;
    int st;
    if ((st = strides_ok({{ldx, rv, true}, {lddt, H, false}, {ldb, rk, true}, {ldc, rk, true}}, es)) != KDA_OK) return st;
    if ((st = strides_ok({{ldy, rv, true}}, os)) != KDA_OK) return st;
    if (N == 0) return KDA_OK;
    if (!x || !dt || !Bm || !Cm || !A || !state || !y) return KDA_ERR_INVALID_ARGUMENT;
    if (!aligned16({x, Bm, Cm, state, y}) || !aligned({dt}, es) || !aligned4({A, dt_bias, D, slots}))
        return KDA_ERR_UNSUPPORTED;
    // a grid of 256-lane workgroups must stay within 2^32 lanes
    if (int64_t(N) * H > (int64_t(1) << 24) - 1) return KDA_ERR_UNSUPPORTED;
    if (!disjoint({strided(y, N, rv * os, ldy * os), flat(state, int64_t(n_slots) * H * dk * dv * 4)},
                  {strided(x, N, rv * es, ldx * es), strided(dt, N, H * es, lddt * es), strided(Bm, N, rk * es, ldb * es),
                   strided(Cm, N, rk * es, ldc * es), flat(A, int64_t(H) * 4), flat(dt_bias, int64_t(H) * 4),
                   flat(D, int64_t(H) * 4), flat(slots, int64_t(N) * 4)}))
        return KDA_ERR_INVALID_ARGUMENT;
    if ((st = linear_debug(A, nullptr, 0, 1, H, stream)) != KDA_OK) return st;
    kda::ScanArgs a{};
    a.x = {x, ldx}; a.dt = {dt, lddt}; a.B = {Bm, ldb}; a.C = {Cm, ldc}; a.A = A; a.bias = dt_bias; a.D = D;
    a.y = {y, ldy}; a.in_dtype = in_dtype; a.y_dtype = y_dtype; a.batch = 1; a.T = N; a.n_seqs = N; a.H = H; a.G = G;
    a.dk = dk; a.dv = dv;
    return from_hip(kda::launch_scan_step(a, state, slots, N, n_slots, static_cast<hipStream_t>(stream)));
}

// ---- slot pools

size_t kda_slots_workspace_size(int32_t n_slots, int32_t N) {
    if (n_slots < 1 || n_slots > kMaxSlots || N < 0) return 0;
    return kda::slots_workspace_bytes(n_slots, N);
}

int kda_slots_copy(const void* const* src, void* const* dst, const int64_t* slot_bytes, int32_t n_planes,
                   const int32_t* src_slots, const int32_t* dst_slots, int32_t N, int32_t n_src, int32_t n_dst,
                   void* stream) {
    if (N < 0 || n_src < 1 || n_dst < 1) return KDA_ERR_INVALID_ARGUMENT;
    if ((!src_slots && N > n_src) || (!dst_slots && N > n_dst)) return KDA_ERR_INVALID_ARGUMENT;
    kda::Planes p{};
    const int st = planes_ok(src, const_cast<const void* const*>(dst), slot_bytes, n_planes, N, &p);
    if (st != KDA_OK) return st;
    if (N == 0) return KDA_OK;
    if (!aligned4({src_slots, dst_slots})) return KDA_ERR_UNSUPPORTED;
    const Strided r_s = flat(src_slots, int64_t(N) * 4), r_d = flat(dst_slots, int64_t(N) * 4);
    for (int32_t i = 0; i < n_planes; ++i) {
        const Strided d = flat(dst[i], p.bytes[i] * n_dst);
        if (overlap(d, r_s) || overlap(d, r_d)) return KDA_ERR_INVALID_ARGUMENT;
        for (int32_t j = 0; j < n_planes; ++j)
            if (overlap(d, flat(src[j], p.bytes[j] * n_src)) || (j > i && overlap(d, flat(dst[j], p.bytes[j] * n_dst))))
                return KDA_ERR_INVALID_ARGUMENT;
    }
    return from_hip(kda::launch_slots_copy(p, src_slots, dst_slots, N, n_src, n_dst, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

namespace {

int slots_count(int32_t* refs, const int32_t* slots, int32_t N, int32_t n_slots, bool up, void* stream) {
    if (N < 0 || n_slots < 1) return KDA_ERR_INVALID_ARGUMENT;
    if (N == 0) return KDA_OK;
    if (!refs || !slots) return KDA_ERR_INVALID_ARGUMENT;
    if (!aligned4({refs, slots}) || n_slots > kMaxSlots) return KDA_ERR_UNSUPPORTED;
    if (overlap(flat(refs, int64_t(n_slots) * 4), flat(slots, int64_t(N) * 4))) return KDA_ERR_INVALID_ARGUMENT;
    return from_hip(kda::launch_slots_count(refs, slots, N, n_slots, up, static_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

int kda_slots_retain(int32_t* refs, const int32_t* slots, int32_t N, int32_t n_slots, void* stream) {
    return slots_count(refs, slots, N, n_slots, true, stream);
}

int kda_slots_release(int32_t* refs, const int32_t* slots, int32_t N, int32_t n_slots, void* stream) {
    return slots_count(refs, slots, N, n_slots, false, stream);
}

int kda_slots_fork(void* const* planes, const int64_t* slot_bytes, int32_t n_planes, int32_t* refs,
                   const int32_t* parents, int32_t* children, int32_t N, int32_t n_slots, void* workspace,
                   size_t workspace_bytes, void* stream) {
    if (N < 0 || n_slots < 1) return KDA_ERR_INVALID_ARGUMENT;
    if (n_slots > kMaxSlots) return KDA_ERR_UNSUPPORTED;
    kda::Planes p{};
    const void* const* q = const_cast<const void* const*>(planes);
    const int st = planes_ok(q, q, slot_bytes, n_planes, 0, &p);
    if (st != KDA_OK) return st;
    if (N == 0) return KDA_OK;
    if (!refs || !children) return KDA_ERR_INVALID_ARGUMENT;
    if (!aligned4({refs, parents, children}) || !aligned16({workspace})) return KDA_ERR_UNSUPPORTED;
    if (workspace_bytes < kda::slots_workspace_bytes(n_slots, N) || !workspace) return KDA_ERR_WORKSPACE;
    if (!planes_disjoint(p, n_slots, {flat(refs, int64_t(n_slots) * 4), flat(parents, int64_t(N) * 4),
                                      flat(children, int64_t(N) * 4), flat(workspace, static_cast<int64_t>(workspace_bytes))}))
        return KDA_ERR_INVALID_ARGUMENT;
    return from_hip(kda::launch_slots_fork(p, refs, parents, children, N, n_slots, workspace, static_cast<hipStream_t>(stream)));
}

int kda_slots_compact(void* const* planes, const int64_t* slot_bytes, int32_t n_planes, int32_t* refs, int32_t* table,
                      int64_t n_table, int32_t* used, int32_t n_slots, void* workspace, size_t workspace_bytes,
                      void* stream) {
    if (n_slots < 1 || n_table < 0) return KDA_ERR_INVALID_ARGUMENT;
    if (n_slots > kMaxSlots || n_table > (int64_t(1) << 31)) return KDA_ERR_UNSUPPORTED;
    kda::Planes p{};
    const void* const* q = const_cast<const void* const*>(planes);
    const int st = planes_ok(q, q, slot_bytes, n_planes, 0, &p);
    if (st != KDA_OK) return st;
    if (!refs || !used || (n_table > 0 && !table)) return KDA_ERR_INVALID_ARGUMENT;
    if (!aligned4({refs, table, used}) || !aligned16({workspace})) return KDA_ERR_UNSUPPORTED;
    if (workspace_bytes < kda::slots_workspace_bytes(n_slots, 0) || !workspace) return KDA_ERR_WORKSPACE;
    if (!planes_disjoint(p, n_slots, {flat(refs, int64_t(n_slots) * 4), flat(table, n_table * 4), flat(used, 4),
                                      flat(workspace, static_cast<int64_t>(workspace_bytes))}))
        return KDA_ERR_INVALID_ARGUMENT;
    return from_hip(kda::launch_slots_compact(p, refs, table, n_table, used, n_slots, workspace, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
