// kda_ssm.hpp -- launchers of the short convolution, the selective scan and the slot pools, which the C ABI
// layer calls after it has validated the arguments.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace kda {

// Rows of tokens: `ld` elements from one token to the next.
struct RowsIn {
    const void* p;
    int64_t ld;
};
struct RowsOut {
    void* p;
    int64_t ld;
};

// Short causal convolution (kda_conv.hip).
struct ConvArgs {
    RowsIn x, dy;                    // dy: backward only
    RowsOut out;                     // y, or dx
    const float *weight, *bias;      // [C, W]; [C] or nullptr
    const void* h0;                  // [N, W - 1, C] or nullptr
    void* hT;                        // forward: final windows or nullptr
    const void* dhT;                 // backward: their gradient or nullptr
    void* dh0;                       // backward: the initial windows' gradient or nullptr
    float *dw, *db;                  // backward
    const int32_t* cu;
    int dtype, silu;
    int32_t B;
    int64_t T;
    int32_t n_seqs, C, W;
    void* workspace;
};
size_t conv_workspace_bytes(int32_t n_seqs, int64_t total_tokens, int32_t C, int32_t W);
hipError_t launch_conv_fwd(const ConvArgs& a, hipStream_t stream);
hipError_t launch_conv_bwd(const ConvArgs& a, hipStream_t stream);
// a.x and a.out: [N, C] rows; windows [n_slots, W - 1, C] updated in place; slots [N] or nullptr.
hipError_t launch_conv_step(const ConvArgs& a, void* windows, const int32_t* slots, int32_t N, int32_t n_slots,
                            hipStream_t stream);

// Selective scan (kda_scan.hip).
struct ScanArgs {
    RowsIn x, dt, B, C, dy;          // dy: backward only
    const float *A, *bias, *D;       // [H]; bias, D: or nullptr
    const float* h0;                 // [N, H, dk, dv] or nullptr
    float* hT;                       // forward: final states or nullptr
    const float* dhT;                // backward: their gradient or nullptr
    float* dh0;                      // backward: the initial states' gradient or nullptr
    const int32_t* cu;
    RowsOut y;                       // forward
    RowsOut dx, ddt, dB, dC;         // backward
    float *dA, *dD, *dbias;          // backward; dD, dbias: or nullptr
    int in_dtype, y_dtype;
    int32_t batch;
    int64_t T;
    int32_t n_seqs, H, G, dk, dv;
    void* workspace;
};
size_t scan_workspace_bytes(int32_t n_seqs, int64_t total_tokens, int32_t H, int32_t G, int32_t dk, int32_t dv,
                            int32_t in_dtype, bool backward);
hipError_t launch_scan_fwd(const ScanArgs& a, hipStream_t stream);
hipError_t launch_scan_bwd(const ScanArgs& a, hipStream_t stream);
// One token: rows of N sequences; states [n_slots, H, dk, dv] updated in place; slots [N] or nullptr.
hipError_t launch_scan_step(const ScanArgs& a, float* states, const int32_t* slots, int32_t N, int32_t n_slots,
                            hipStream_t stream);

// Slot pools (kda_slots.hip): up to MAX_PLANES arrays of n_slots slots.
constexpr int MAX_PLANES = 4;
struct Planes {
    const uint8_t* src[MAX_PLANES];
    uint8_t* dst[MAX_PLANES];
    int64_t bytes[MAX_PLANES];       // of a slot
    int32_t n;
};
size_t slots_workspace_bytes(int32_t n_slots, int32_t N);
hipError_t launch_slots_copy(const Planes& p, const int32_t* src_slots, const int32_t* dst_slots, int32_t N,
                             int32_t n_src, int32_t n_dst, hipStream_t stream);
hipError_t launch_slots_count(int32_t* refs, const int32_t* slots, int32_t N, int32_t n_slots, bool up,
                              hipStream_t stream);
hipError_t launch_slots_fork(const Planes& p, int32_t* refs, const int32_t* parents, int32_t* children, int32_t N,
                             int32_t n_slots, void* workspace, hipStream_t stream);
hipError_t launch_slots_compact(const Planes& p, int32_t* refs, int32_t* table, int64_t n_table, int32_t* used,
                                int32_t n_slots, void* workspace, hipStream_t stream);

}  // namespace kda
