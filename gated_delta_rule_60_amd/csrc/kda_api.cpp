// kda_api.cpp -- the extern "C" boundary of libkda.so: argument validation, dispatch, status.
// Declarations, layouts and error behaviour are documented in include/kda.h.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <initializer_list>
#include <mutex>

#include "../../include/kda.h"
#include "kda_api_util.hpp"
#include "kda_internal.hpp"
#include "kda_linear.hpp"

namespace {

constexpr int kVersion = 300;  // 0.3.0

// ---- the prefill workspace of kda_chunk_fwd_gated_noalloc: a static device array ------------
// Each GPU the library runs on holds its own copy from the first use on that device until the
// process ends.  In host code `scratch` names a host-side stand-in, not device memory: the
// device address comes from hipGetSymbolAddress, taken once per device with that device
// current, and only that address is ever handed to kernels.
__device__ __align__(256) uint8_t scratch[KDA_NOALLOC_SCRATCH_BYTES];

constexpr int kMaxDevices = 64;
std::mutex g_scratch_mu;
void* g_scratch_ptr[kMaxDevices] = {};

// Device address of `scratch` on the device `stream` belongs to.
hipError_t scratch_address(hipStream_t stream, void** out) {
    int dev = 0, cur = 0;
    hipError_t e = hipGetDevice(&cur);
    if (e != hipSuccess) return e;
    dev = cur;
    if (stream != nullptr) {
        e = hipStreamGetDevice(stream, &dev);
        if (e != hipSuccess) return e;
    }
    if (dev < 0 || dev >= kMaxDevices) return hipErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(g_scratch_mu);
    if (g_scratch_ptr[dev] == nullptr) {
        if (dev != cur && (e = hipSetDevice(dev)) != hipSuccess) return e;
        void* p = nullptr;
        e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
        if (dev != cur) {
            const hipError_t r = hipSetDevice(cur);
            if (e == hipSuccess) e = r;
        }
        if (e != hipSuccess) return e;
        if (p == nullptr) return hipErrorInvalidSymbol;
        g_scratch_ptr[dev] = p;
    }
    *out = g_scratch_ptr[dev];
    return hipSuccess;
}

}  // namespace

extern "C" {

const char* kda_status_string(int status) {
    switch (status) {
        case KDA_OK: return "KDA_OK";
        case KDA_ERR_INVALID_ARGUMENT: return "KDA_ERR_INVALID_ARGUMENT";
        case KDA_ERR_UNSUPPORTED: return "KDA_ERR_UNSUPPORTED";
        case KDA_ERR_WORKSPACE: return "KDA_ERR_WORKSPACE";
        case KDA_ERR_HIP: return "KDA_ERR_HIP";
        default: return "KDA_UNKNOWN_STATUS";
    }
}

int kda_version(void) { return kVersion; }

int kda_gate(const float* A, const void* z, int z_dtype, void* g, int g_dtype, int64_t n_tokens,
             int32_t H, int32_t dk, float g_min, void* stream) {
    if (!valid_dtype(z_dtype) || !valid_dtype(g_dtype) || n_tokens < 0 || H < 1 || dk < 1)
        return KDA_ERR_INVALID_ARGUMENT;
    if (!std::isfinite(g_min) || !(g_min >= -5.0f && g_min < 0.0f)) return KDA_ERR_UNSUPPORTED;
    if (n_tokens == 0) return KDA_OK;
    if (!A || !z || !g) return KDA_ERR_INVALID_ARGUMENT;
    const int64_t n = n_tokens * H * dk;
    const Range rg = range(g, n * esize(g_dtype));
    if (overlap(rg, range(z, n * esize(z_dtype))) || overlap(rg, range(A, int64_t(H) * dk * 4)))
        return KDA_ERR_INVALID_ARGUMENT;
    return from_hip(kda::launch_gate(A, z, z_dtype, g, g_dtype, n_tokens, H, dk, g_min,
                                     static_cast<hipStream_t>(stream)));
}

size_t kda_chunk_fwd_workspace_size(int32_t n_seqs, int64_t total_tokens, int32_t H, int32_t dk,
                                    int32_t dv, int32_t chunk, int in_dtype) {
    if (n_seqs < 1 || total_tokens < 0 || H < 1 || !supported_d(dk) || !supported_d(dv) ||
        chunk != 64 || !valid_dtype(in_dtype))
        return 0;
    return kda::chunk_workspace_bytes(n_seqs, total_tokens, H, dk, dv, in_dtype);
}

}  // extern "C"

namespace {

// Validation and dispatch shared by kda_chunk_fwd (g given) and kda_chunk_fwd_gated (A, z given:
// gate_A != nullptr, g = z, g_dtype = z's dtype).
int chunk_fwd_impl(const void* q, const void* k, const void* v, const void* beta, int in_dtype,
                   const void* g, int g_dtype, const float* gate_A, float g_min,
                   const float* initial_state, float* final_state, const int32_t* cu_seqlens,
                   void* o, int o_dtype, int32_t B, int64_t T, int32_t n_seqs, int32_t H,
                   int32_t dk, int32_t dv, int32_t chunk, float scale, void* workspace,
                   size_t workspace_bytes, void* stream, bool gated, float* ckpt = nullptr,
                   int32_t ckpt_every = 0, int64_t ckpt_slots = 0, bool single_stream = false) {
    if (!valid_dtype(in_dtype) || !valid_dtype(g_dtype) || !valid_dtype(o_dtype))
        return KDA_ERR_INVALID_ARGUMENT;
    if (B < 1 || T < 0 || n_seqs < 1 || H < 1 || dk < 1 || dv < 1 || !std::isfinite(scale))
        return KDA_ERR_INVALID_ARGUMENT;
    if (cu_seqlens ? (B != 1) : (n_seqs != B)) return KDA_ERR_INVALID_ARGUMENT;
    if (!supported_d(dk) || !supported_d(dv) || chunk != 64) return KDA_ERR_UNSUPPORTED;
    if (gated && (!std::isfinite(g_min) || !(g_min >= -5.0f && g_min < 0.0f)))
        return KDA_ERR_UNSUPPORTED;
    const int64_t ntok = int64_t(B) * T;
    if (ntok > 0 && (!q || !k || !v || !beta || !g || !o || (gated && !gate_A)))
        return KDA_ERR_INVALID_ARGUMENT;
    const size_t need = kda::chunk_workspace_bytes(n_seqs, ntok, H, dk, dv, in_dtype);
    if (workspace_bytes < need || (need > 0 && !workspace)) return KDA_ERR_WORKSPACE;

    const int64_t state_bytes = int64_t(n_seqs) * H * dk * dv * 4;
    const Range r_q = range(q, ntok * H * dk * esize(in_dtype));
    const Range r_k = range(k, ntok * H * dk * esize(in_dtype));
    const Range r_v = range(v, ntok * H * dv * esize(in_dtype));
    const Range r_b = range(beta, ntok * H * esize(in_dtype));
    const Range r_g = range(g, ntok * H * dk * esize(g_dtype));
    const Range r_a = range(gate_A, gated && ntok > 0 ? int64_t(H) * dk * 4 : 0);
    const Range r_o = range(o, ntok * H * dv * esize(o_dtype));
    const Range r_h0 = range(initial_state, initial_state ? state_bytes : 0);
    const Range r_hT = range(final_state, final_state ? state_bytes : 0);
    const Range r_cu = range(cu_seqlens, cu_seqlens ? int64_t(n_seqs + 1) * 4 : 0);
    const Range r_ws = range(workspace, int64_t(workspace_bytes));
    const Range r_ck = range(ckpt, ckpt ? ckpt_slots * H * dk * dv * 4 : 0);
    for (const Range& x : {r_q, r_k, r_v, r_b, r_g, r_a, r_h0, r_hT, r_cu, r_ws, r_ck})
        if (overlap(r_o, x)) return KDA_ERR_INVALID_ARGUMENT;
    for (const Range& x : {r_q, r_k, r_v, r_b, r_g, r_a, r_h0, r_hT, r_cu, r_ws})
        if (overlap(r_ck, x)) return KDA_ERR_INVALID_ARGUMENT;
    // the final state may be the initial state itself, but must not partly overlap it
    if (initial_state && final_state && initial_state != final_state && overlap(r_h0, r_hT))
        return KDA_ERR_INVALID_ARGUMENT;
    for (const Range& x : {r_q, r_k, r_v, r_b, r_g, r_a, r_cu, r_ws})
        if (overlap(r_hT, x)) return KDA_ERR_INVALID_ARGUMENT;
    for (const Range& x : {r_q, r_k, r_v, r_b, r_g, r_a, r_h0, r_cu})
        if (overlap(r_ws, x)) return KDA_ERR_INVALID_ARGUMENT;

    if (kda::debug_validation_enabled() && ntok > 0) {
        bool ok = true;
        const hipError_t e = kda::debug_validate(gated ? nullptr : g, g_dtype, ntok * H * dk, cu_seqlens,
                                                 n_seqs, ntok, static_cast<hipStream_t>(stream), &ok);
        if (e != hipSuccess) return KDA_ERR_HIP;
        if (!ok) return KDA_ERR_INVALID_ARGUMENT;
    }

    kda::ChunkArgs a{};
    a.q = q; a.k = k; a.v = v; a.beta = beta; a.g = g;
    a.gate_A = gated ? gate_A : nullptr; a.g_min = g_min;
    a.h0 = initial_state; a.hT = final_state; a.cu = cu_seqlens; a.o = o;
    a.in_dtype = in_dtype; a.g_dtype = g_dtype; a.o_dtype = o_dtype;
    a.B = B; a.T = T; a.n_seqs = n_seqs; a.H = H; a.dk = dk; a.dv = dv;
    a.head0 = 0; a.heads = H; a.single_stream = single_stream ? 1 : 0;
    a.scale = scale; a.workspace = workspace; a.workspace_bytes = workspace_bytes;
    a.ckpt = ckpt; a.ckpt_every = ckpt_every; a.ckpt_slots = ckpt_slots;
    return from_hip(kda::launch_chunk(a, static_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

int kda_chunk_fwd(const void* q, const void* k, const void* v, const void* beta, int in_dtype,
                  const void* g, int g_dtype, const float* initial_state, float* final_state,
                  const int32_t* cu_seqlens, void* o, int o_dtype, int32_t B, int64_t T,
                  int32_t n_seqs, int32_t H, int32_t dk, int32_t dv, int32_t chunk, float scale,
                  void* workspace, size_t workspace_bytes, void* stream) {
    return chunk_fwd_impl(q, k, v, beta, in_dtype, g, g_dtype, nullptr, 0.0f, initial_state,
                          final_state, cu_seqlens, o, o_dtype, B, T, n_seqs, H, dk, dv, chunk,
                          scale, workspace, workspace_bytes, stream, false);
}

int kda_chunk_fwd_gated(const void* q, const void* k, const void* v, const void* beta,
                        int in_dtype, const float* A, const void* z, int z_dtype, float g_min,
                        const float* initial_state, float* final_state, const int32_t* cu_seqlens,
                        void* o, int o_dtype, int32_t B, int64_t T, int32_t n_seqs, int32_t H,
                        int32_t dk, int32_t dv, int32_t chunk, float scale, void* workspace,
                        size_t workspace_bytes, void* stream) {
    return chunk_fwd_impl(q, k, v, beta, in_dtype, z, z_dtype, A, g_min, initial_state,
                          final_state, cu_seqlens, o, o_dtype, B, T, n_seqs, H, dk, dv, chunk,
                          scale, workspace, workspace_bytes, stream, true);
}

int kda_chunk_fwd_gated_noalloc(const void* q, const void* k, const void* v, const void* beta,
                                int in_dtype, const float* A, const void* z, int z_dtype,
                                float g_min, const float* initial_state, float* final_state,
                                const int32_t* cu_seqlens, void* o, int o_dtype, int32_t B,
                                int64_t T, int32_t n_seqs, int32_t H, int32_t dk, int32_t dv,
                                int32_t chunk, float scale, void* stream) {
    // sizes first: a call whose workspace would not fit is refused before any device work
    if (B < 1 || T < 0 || n_seqs < 1 || H < 1 || !valid_dtype(in_dtype))
        return KDA_ERR_INVALID_ARGUMENT;
    if (!supported_d(dk) || !supported_d(dv) || chunk != 64) return KDA_ERR_UNSUPPORTED;
    const size_t need = kda::chunk_workspace_bytes(n_seqs, int64_t(B) * T, H, dk, dv, in_dtype);
    if (need > KDA_NOALLOC_SCRATCH_BYTES) return KDA_ERR_WORKSPACE;
    void* ws = nullptr;
    if (need > 0) {
        const hipError_t e = scratch_address(static_cast<hipStream_t>(stream), &ws);
        if (e != hipSuccess) return KDA_ERR_HIP;
    }
    return chunk_fwd_impl(q, k, v, beta, in_dtype, z, z_dtype, A, g_min, initial_state,
                          final_state, cu_seqlens, o, o_dtype, B, T, n_seqs, H, dk, dv, chunk,
                          scale, ws, need > 0 ? size_t(KDA_NOALLOC_SCRATCH_BYTES) : 0, stream,
                          true, nullptr, 0, 0, /*single_stream=*/true);
}

int kda_chunk_fwd_checkpointed(const void* q, const void* k, const void* v, const void* beta,
                               int in_dtype, const float* A, const void* g_or_z, int gz_dtype,
                               float g_min, const float* initial_state, float* final_state,
                               const int32_t* cu_seqlens, void* o, int o_dtype, int32_t B,
                               int64_t T, int32_t n_seqs, int32_t H, int32_t dk, int32_t dv,
                               int32_t chunk, float scale, float* checkpoints,
                               int32_t checkpoint_every, int64_t max_checkpoints, void* workspace,
                               size_t workspace_bytes, void* stream) {
    if (!checkpoints || checkpoint_every < 64 || checkpoint_every % 64 != 0 || max_checkpoints < 0)
        return KDA_ERR_INVALID_ARGUMENT;
    if (B < 1 || T < 0 || n_seqs < 1) return KDA_ERR_INVALID_ARGUMENT;
    // slots the layout can reach: B * floor(T / every), or floor(T / every) + n_seqs when packed
    const int64_t need = cu_seqlens ? T / checkpoint_every + n_seqs : int64_t(B) * (T / checkpoint_every);
    if (max_checkpoints < need) return KDA_ERR_INVALID_ARGUMENT;
    return chunk_fwd_impl(q, k, v, beta, in_dtype, g_or_z, gz_dtype, A, A ? g_min : 0.0f,
                          initial_state, final_state, cu_seqlens, o, o_dtype, B, T, n_seqs, H, dk,
                          dv, chunk, scale, workspace, workspace_bytes, stream, A != nullptr,
                          checkpoints, checkpoint_every, max_checkpoints);
}

int kda_decode_step(const void* q, const void* k, const void* v, const void* beta, int in_dtype,
                    const void* g, int g_dtype, float* state, void* o, int o_dtype, int32_t N,
                    int32_t H, int32_t dk, int32_t dv, float scale, void* stream) {
    if (!valid_dtype(in_dtype) || !valid_dtype(g_dtype) || !valid_dtype(o_dtype))
        return KDA_ERR_INVALID_ARGUMENT;
    if (N < 0 || H < 1 || dk < 1 || dv < 1 || !std::isfinite(scale)) return KDA_ERR_INVALID_ARGUMENT;
    if (!supported_d(dk) || !supported_d(dv)) return KDA_ERR_UNSUPPORTED;
    if (N == 0) return KDA_OK;
    if (!q || !k || !v || !beta || !g || !state || !o) return KDA_ERR_INVALID_ARGUMENT;
    const int64_t units = int64_t(N) * H;
    const Range r_o = range(o, units * dv * esize(o_dtype));
    const Range r_s = range(state, units * dk * dv * 4);
    const Range ins[] = {range(q, units * dk * esize(in_dtype)), range(k, units * dk * esize(in_dtype)),
                         range(v, units * dv * esize(in_dtype)), range(beta, units * esize(in_dtype)),
                         range(g, units * dk * esize(g_dtype))};
    for (const Range& x : ins)
        if (overlap(r_o, x) || overlap(r_s, x)) return KDA_ERR_INVALID_ARGUMENT;
    if (overlap(r_o, r_s)) return KDA_ERR_INVALID_ARGUMENT;
    if (kda::debug_validation_enabled()) {
        bool ok = true;
        if (kda::debug_validate(g, g_dtype, int64_t(N) * H * dk, nullptr, 0, 0, static_cast<hipStream_t>(stream), &ok) !=
            hipSuccess)
            return KDA_ERR_HIP;
        if (!ok) return KDA_ERR_INVALID_ARGUMENT;
    }
    return from_hip(kda::launch_decode(q, k, v, beta, in_dtype, g, g_dtype, state, o, o_dtype, N,
                                       H, dk, dv, scale, static_cast<hipStream_t>(stream)));
}

int kda_decode_verify(const void* q, const void* k, const void* v, const void* beta, int in_dtype,
                      const void* g, int g_dtype, const float* state, void* o, int o_dtype,
                      int32_t N, int32_t K, int32_t H, int32_t dk, int32_t dv, float scale,
                      void* stream) {
    if (!valid_dtype(in_dtype) || !valid_dtype(g_dtype) || !valid_dtype(o_dtype))
        return KDA_ERR_INVALID_ARGUMENT;
    if (N < 0 || K < 1 || H < 1 || dk < 1 || dv < 1 || !std::isfinite(scale))
        return KDA_ERR_INVALID_ARGUMENT;
    if (!supported_d(dk) || !supported_d(dv)) return KDA_ERR_UNSUPPORTED;
    if (N == 0) return KDA_OK;
    if (!q || !k || !v || !beta || !g || !state || !o) return KDA_ERR_INVALID_ARGUMENT;
    const int64_t rows = int64_t(N) * K * H;
    const Range r_o = range(o, rows * dv * esize(o_dtype));
    const Range others[] = {range(q, rows * dk * esize(in_dtype)), range(k, rows * dk * esize(in_dtype)),
                            range(v, rows * dv * esize(in_dtype)), range(beta, rows * esize(in_dtype)),
                            range(g, rows * dk * esize(g_dtype)), range(state, int64_t(N) * H * dk * dv * 4)};
    for (const Range& x : others)
        if (overlap(r_o, x)) return KDA_ERR_INVALID_ARGUMENT;
    if (kda::debug_validation_enabled()) {
        bool ok = true;
        if (kda::debug_validate(g, g_dtype, int64_t(N) * K * H * dk, nullptr, 0, 0, static_cast<hipStream_t>(stream), &ok) !=
            hipSuccess)
            return KDA_ERR_HIP;
        if (!ok) return KDA_ERR_INVALID_ARGUMENT;
    }
    return from_hip(kda::launch_decode_verify(q, k, v, beta, in_dtype, g, g_dtype, state, o, o_dtype,
                                              N, K, H, dk, dv, scale, static_cast<hipStream_t>(stream)));
}

int kda_decode_commit(const void* q, const void* k, const void* v, const void* beta, int in_dtype,
                      const void* g, int g_dtype, float* state, const int32_t* accepted, int32_t N,
                      int32_t K, int32_t H, int32_t dk, int32_t dv, void* stream) {
    if (!valid_dtype(in_dtype) || !valid_dtype(g_dtype)) return KDA_ERR_INVALID_ARGUMENT;
    if (N < 0 || K < 1 || H < 1 || dk < 1 || dv < 1) return KDA_ERR_INVALID_ARGUMENT;
    if (!supported_d(dk) || !supported_d(dv)) return KDA_ERR_UNSUPPORTED;
    if (N == 0) return KDA_OK;
    if (!q || !k || !v || !beta || !g || !state || !accepted) return KDA_ERR_INVALID_ARGUMENT;
    const int64_t rows = int64_t(N) * K * H;
    const Range r_s = range(state, int64_t(N) * H * dk * dv * 4);
    const Range others[] = {range(q, rows * dk * esize(in_dtype)), range(k, rows * dk * esize(in_dtype)),
                            range(v, rows * dv * esize(in_dtype)), range(beta, rows * esize(in_dtype)),
                            range(g, rows * dk * esize(g_dtype)), range(accepted, int64_t(N) * 4)};
    for (const Range& x : others)
        if (overlap(r_s, x)) return KDA_ERR_INVALID_ARGUMENT;
    if (kda::debug_validation_enabled()) {
        bool ok = true;
        if (kda::debug_validate(g, g_dtype, int64_t(N) * K * H * dk, nullptr, 0, 0, static_cast<hipStream_t>(stream), &ok) !=
            hipSuccess)
            return KDA_ERR_HIP;
        if (!ok) return KDA_ERR_INVALID_ARGUMENT;
    }
    return from_hip(kda::launch_decode_commit(q, k, v, beta, in_dtype, g, g_dtype, state, accepted,
                                              N, K, H, dk, dv, static_cast<hipStream_t>(stream)));
}

// ---- linear attention with one decay per head ------------------------------------------------

size_t kda_linear_chunk_workspace_size(int32_t n_seqs, int64_t total_tokens, int32_t H, int32_t dk,
                                       int32_t dv, int in_dtype, int backward) {
    if (n_seqs < 1 || total_tokens < 0 || H < 1 || !supported_d(dk) || !supported_d(dv) ||
        !valid_dtype(in_dtype))
        return 0;
    return kda::linear_workspace_bytes(n_seqs, total_tokens, H, dk, dv, in_dtype, backward != 0);
}

}  // extern "C"

namespace {

// Checks the forward and the backward share; KDA_OK, or the status to return.
int linear_sizes(int in_dtype, const int32_t* cu, int32_t B, int64_t T, int32_t n_seqs, int32_t H,
                 int32_t dk, int32_t dv, float scale) {
    if (!valid_dtype(in_dtype)) return KDA_ERR_INVALID_ARGUMENT;
    if (B < 1 || T < 0 || n_seqs < 1 || H < 1 || dk < 1 || dv < 1 || !std::isfinite(scale))
        return KDA_ERR_INVALID_ARGUMENT;
    if (cu ? (B != 1) : (n_seqs != B)) return KDA_ERR_INVALID_ARGUMENT;
    if (!supported_d(dk) || !supported_d(dv)) return KDA_ERR_UNSUPPORTED;
    // 64 token rows of all heads must stay within a 2 GiB buffer range (a token row of all heads:
    // H * 512 bytes at most)
    if (H > 32768) return KDA_ERR_UNSUPPORTED;
    // a grid of 256-lane workgroups (up to six per (sequence, head)) must stay within 2^32 lanes
    if (int64_t(n_seqs) * H > (int64_t(1) << 21)) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

int state_cache_check(const float* states, const int32_t* slots, const void* codes, int code,
                      const float* scales, int32_t N, int32_t n_slots, int32_t H, int32_t dk, int32_t dv,
                      int32_t group, bool store, kda::StateCacheArgs* a) {
    if ((code != KDA_CODE_I8 && code != KDA_CODE_E4M3) || N < 0 || n_slots < 1 || H < 1 || dk < 1 || dv < 1 ||
        group < 1)
        return KDA_ERR_INVALID_ARGUMENT;
    if (!supported_d(dk) || !supported_d(dv) || (group != 32 && group != 64 && group != 128) || group > dv)
        return KDA_ERR_UNSUPPORTED;
    if (!slots && N > n_slots) return KDA_ERR_INVALID_ARGUMENT;
    if (N == 0) return KDA_OK;
    if (!states || !codes || !scales) return KDA_ERR_INVALID_ARGUMENT;
    if (!aligned16({states, codes}) || !aligned4({scales, slots})) return KDA_ERR_UNSUPPORTED;
    const int64_t per_seq = int64_t(H) * dk * dv;
    // a grid of 256-lane workgroups must stay within 2^32 lanes (4096 elements a workgroup)
    if (per_seq / 4096 * N > (int64_t(1) << 24) - 1) return KDA_ERR_UNSUPPORTED;
    const Range r_st = range(states, N * per_seq * 4), r_sl = range(slots, slots ? int64_t(N) * 4 : 0);
    const Range r_c = range(codes, n_slots * per_seq), r_sc = range(scales, n_slots * (per_seq / group) * 4);
    if (store ? !disjoint({r_c, r_sc}, {r_st, r_sl}) : !disjoint({r_st}, {r_c, r_sc, r_sl}))
        return KDA_ERR_INVALID_ARGUMENT;
    a->codes = const_cast<void*>(codes); a->scales = const_cast<float*>(scales); a->slots = slots;
    a->code = code; a->N = N; a->n_slots = n_slots; a->H = H; a->dk = dk; a->dv = dv; a->group = group;
    return KDA_OK;
}

}  // namespace

extern "C" {

int kda_linear_chunk_fwd(const void* q, const void* k, const void* v, int in_dtype, const float* g,
                         const float* initial_state, float* final_state, const int32_t* cu_seqlens,
                         void* o, int o_dtype, int32_t B, int64_t T, int32_t n_seqs, int32_t H,
                         int32_t dk, int32_t dv, float scale, void* workspace,
                         size_t workspace_bytes, void* stream) {
    if (!valid_dtype(o_dtype)) return KDA_ERR_INVALID_ARGUMENT;
    const int st = linear_sizes(in_dtype, cu_seqlens, B, T, n_seqs, H, dk, dv, scale);
    if (st != KDA_OK) return st;
    const int64_t ntok = int64_t(B) * T, rows = ntok * H;
    if (ntok > 0 && (!q || !k || !v || !g || !o)) return KDA_ERR_INVALID_ARGUMENT;
    if (!aligned16({q, k, v, o, initial_state, final_state, workspace}) || !aligned4({g, cu_seqlens}))
        return KDA_ERR_UNSUPPORTED;
    const size_t need = kda::linear_workspace_bytes(n_seqs, ntok, H, dk, dv, in_dtype, false);
    if (workspace_bytes < need || (need > 0 && !workspace)) return KDA_ERR_WORKSPACE;
    const int64_t es = esize(in_dtype), state_bytes = int64_t(n_seqs) * H * dk * dv * 4;
    const Range r_h0 = range(initial_state, initial_state ? state_bytes : 0);
    const Range r_hT = range(final_state, final_state ? state_bytes : 0);
    const Range r_q = range(q, rows * dk * es), r_k = range(k, rows * dk * es), r_v = range(v, rows * dv * es);
    const Range r_g = range(g, ntok > 0 ? int64_t(H) * 4 : 0), r_o = range(o, rows * dv * esize(o_dtype));
    const Range r_cu = range(cu_seqlens, cu_seqlens ? int64_t(n_seqs + 1) * 4 : 0);
    const Range r_ws = range(workspace, workspace ? int64_t(workspace_bytes) : 0);
    if (!disjoint({r_o, r_hT, r_ws}, {r_q, r_k, r_v, r_g, r_cu}) || overlap(r_o, r_h0) || overlap(r_ws, r_h0))
        return KDA_ERR_INVALID_ARGUMENT;
    // the final state may be the initial state itself, but must not partly overlap it
    if (initial_state != final_state && overlap(r_h0, r_hT)) return KDA_ERR_INVALID_ARGUMENT;
    const int dbg = linear_debug(g, cu_seqlens, n_seqs, ntok, H, stream);
    if (dbg != KDA_OK) return dbg;
    kda::LinearArgs a{};
    a.q = q; a.k = k; a.v = v; a.g = g; a.h0 = initial_state; a.hT = final_state; a.cu = cu_seqlens; a.o = o;
    a.in_dtype = in_dtype; a.o_dtype = o_dtype; a.B = B; a.T = T; a.n_seqs = n_seqs; a.H = H; a.dk = dk;
    a.dv = dv; a.scale = scale; a.workspace = workspace;
    return from_hip(kda::launch_linear_fwd(a, static_cast<hipStream_t>(stream)));
}

int kda_linear_chunk_bwd(const void* q, const void* k, const void* v, int in_dtype, const float* g,
                         const float* initial_state, const int32_t* cu_seqlens, const void* d_o,
                         const float* d_final_state, void* dq, void* dk_out, void* dv_out,
                         float* d_initial_state, int32_t B, int64_t T, int32_t n_seqs, int32_t H,
                         int32_t dk, int32_t dv, float scale, void* workspace,
                         size_t workspace_bytes, void* stream) {
    const int st = linear_sizes(in_dtype, cu_seqlens, B, T, n_seqs, H, dk, dv, scale);
    if (st != KDA_OK) return st;
    const int64_t ntok = int64_t(B) * T, rows = ntok * H;
    if (ntok > 0 && (!q || !k || !v || !g || !d_o || !dq || !dk_out || !dv_out)) return KDA_ERR_INVALID_ARGUMENT;
    if (!aligned16({q, k, v, d_o, dq, dk_out, dv_out, initial_state, d_final_state, d_initial_state, workspace}) ||
        !aligned4({g, cu_seqlens}))
        return KDA_ERR_UNSUPPORTED;
    const size_t need = kda::linear_workspace_bytes(n_seqs, ntok, H, dk, dv, in_dtype, true);
    if (workspace_bytes < need || (need > 0 && !workspace)) return KDA_ERR_WORKSPACE;
    const int64_t es = esize(in_dtype), state_bytes = int64_t(n_seqs) * H * dk * dv * 4;
    const int64_t kb = rows * dk * es, vb = rows * dv * es;
    if (!disjoint({range(dq, kb), range(dk_out, kb), range(dv_out, vb),
                   range(d_initial_state, d_initial_state ? state_bytes : 0),
                   range(workspace, workspace ? int64_t(workspace_bytes) : 0)},
                  {range(q, kb), range(k, kb), range(v, vb), range(d_o, vb), range(g, ntok > 0 ? int64_t(H) * 4 : 0),
                   range(initial_state, initial_state ? state_bytes : 0),
                   range(d_final_state, d_final_state ? state_bytes : 0),
                   range(cu_seqlens, cu_seqlens ? int64_t(n_seqs + 1) * 4 : 0)}))
        return KDA_ERR_INVALID_ARGUMENT;
    const int dbg = linear_debug(g, cu_seqlens, n_seqs, ntok, H, stream);
    if (dbg != KDA_OK) return dbg;
    kda::LinearArgs a{};
    a.q = q; a.k = k; a.v = v; a.d_o = d_o; a.g = g; a.h0 = initial_state; a.dhT = d_final_state;
    a.dh0 = d_initial_state; a.cu = cu_seqlens; a.dq = dq; a.dkk = dk_out; a.dvv = dv_out;
    a.in_dtype = in_dtype; a.o_dtype = in_dtype; a.B = B; a.T = T; a.n_seqs = n_seqs; a.H = H; a.dk = dk;
    a.dv = dv; a.scale = scale; a.workspace = workspace;
    return from_hip(kda::launch_linear_bwd(a, static_cast<hipStream_t>(stream)));
}

int kda_linear_decode_step(const void* q, const void* k, const void* v, int in_dtype,
                           const float* g, float* state, void* o, int o_dtype, int32_t N, int32_t H,
                           int32_t dk, int32_t dv, float scale, void* stream) {
    if (!valid_dtype(in_dtype) || !valid_dtype(o_dtype)) return KDA_ERR_INVALID_ARGUMENT;
    if (N < 0 || H < 1 || dk < 1 || dv < 1 || !std::isfinite(scale)) return KDA_ERR_INVALID_ARGUMENT;
    if (!supported_d(dk) || !supported_d(dv)) return KDA_ERR_UNSUPPORTED;
    if (N == 0) return KDA_OK;
    if (!q || !k || !v || !g || !state || !o) return KDA_ERR_INVALID_ARGUMENT;
    if (!aligned16({q, k, v, state, o}) || !aligned4({g})) return KDA_ERR_UNSUPPORTED;
    const int64_t units = int64_t(N) * H, es = esize(in_dtype);
    // a grid of 256-lane workgroups must stay within 2^32 lanes
    if (units > (int64_t(1) << 24) - 1) return KDA_ERR_UNSUPPORTED;
    if (!disjoint({range(o, units * dv * esize(o_dtype)), range(state, units * dk * dv * 4)},
                  {range(q, units * dk * es), range(k, units * dk * es), range(v, units * dv * es),
                   range(g, int64_t(H) * 4)}))
        return KDA_ERR_INVALID_ARGUMENT;
    const int dbg = linear_debug(g, nullptr, 0, 1, H, stream);
    if (dbg != KDA_OK) return dbg;
    return from_hip(kda::launch_linear_decode(q, k, v, in_dtype, g, state, o, o_dtype, N, H, dk, dv, scale,
                                              static_cast<hipStream_t>(stream)));
}

// ---- 8-bit state cache -----------------------------------------------------------------------

int kda_state_store(const float* states, const int32_t* slots, void* codes, int code, float* scales,
                    int32_t N, int32_t n_slots, int32_t H, int32_t dk, int32_t dv, int32_t group,
                    void* stream) {
    kda::StateCacheArgs a{};
    const int st = state_cache_check(states, slots, codes, code, scales, N, n_slots, H, dk, dv, group, true, &a);
    if (st != KDA_OK || N == 0) return st;
    return from_hip(kda::launch_state_store(a, states, static_cast<hipStream_t>(stream)));
}

int kda_state_load(const void* codes, int code, const float* scales, const int32_t* slots,
                   float* states, int32_t N, int32_t n_slots, int32_t H, int32_t dk, int32_t dv,
                   int32_t group, void* stream) {
    kda::StateCacheArgs a{};
    const int st = state_cache_check(states, slots, codes, code, scales, N, n_slots, H, dk, dv, group, false, &a);
    if (st != KDA_OK || N == 0) return st;
    return from_hip(kda::launch_state_load(a, states, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
