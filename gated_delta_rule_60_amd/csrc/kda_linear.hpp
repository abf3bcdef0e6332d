// kda_linear.hpp -- launchers of linear attention and of the state cache, which the C ABI layer calls after
// it has validated the arguments.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace kda {

// Linear attention with one decay per head (kda_linear.hip).
struct LinearArgs {
    const void *q, *k, *v, *d_o;     // d_o: backward only
    const float* g;                  // [H]
    const float* h0;                 // initial state or nullptr
    float* hT;                       // final state or nullptr (forward)
    const float* dhT;                // its gradient or nullptr (backward)
    float* dh0;                      // the initial state's gradient or nullptr (backward)
    const int32_t* cu;               // device cu_seqlens or nullptr
    void* o;                         // forward
    void *dq, *dkk, *dvv;            // backward: gradients of q, k, v
    int in_dtype, o_dtype;
    int32_t B;
    int64_t T;
    int32_t n_seqs, H, dk, dv;
    float scale;
    void* workspace;
};
size_t linear_workspace_bytes(int32_t n_seqs, int64_t total_tokens, int32_t H, int32_t dk, int32_t dv,
                              int32_t in_dtype, bool backward);
hipError_t launch_linear_fwd(const LinearArgs& a, hipStream_t stream);
hipError_t launch_linear_bwd(const LinearArgs& a, hipStream_t stream);
hipError_t launch_linear_decode(const void* q, const void* k, const void* v, int in_dtype, const float* g,
                                float* state, void* o, int o_dtype, int32_t N, int32_t H, int32_t dk,
                                int32_t dv, float scale, hipStream_t stream);

// 8-bit state cache (kda_state_cache.hip).
struct StateCacheArgs {
    void* codes;                     // read only by launch_state_load
    float* scales;
    const int32_t* slots;            // [N] or nullptr (sequence n in slot n)
    int32_t code, N, n_slots, H, dk, dv, group;
};
hipError_t launch_state_store(const StateCacheArgs& a, const float* states, hipStream_t stream);
hipError_t launch_state_load(const StateCacheArgs& a, float* states, hipStream_t stream);

// debug_validate with a lower bound of g other than -5.
hipError_t debug_validate_from(float g_lo, const void* g, int g_dtype, int64_t g_elems, const int32_t* cu,
                               int32_t n_seqs, int64_t total, hipStream_t stream, bool* ok);

}  // namespace kda
