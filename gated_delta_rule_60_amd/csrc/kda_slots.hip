// kda_slots.hip -- slots of pools of recurrent states: copying between pools, users' counts, forking and
// compacting.
//
// A pool is up to four planes (arrays of n_slots slots: states, 8-bit codes and scales, convolution windows)
// and refs, the number of users of each slot (0: free).  Forking and compacting are two launches: one workgroup
// plans, i.e. ranks free or used slots by prefix sums over refs, and a grid copies.  The copies are bound by
// HBM: 406 slots of 1.06 MB forked and moved in 175 us (4.9 TB/s read and written).  They stream past the
// caches, each byte is touched once.
#include "kda_chunk_util.hpp"
#include "kda_ssm.hpp"

#include <algorithm>

namespace kda {
namespace {

constexpr int THREADS = 256, DEEP = 8;
constexpr int64_t PART = int64_t(THREADS) * DEEP * 16;       // bytes of a slot that a workgroup takes at a time
constexpr int PLAN = 1024;                                   // lanes of the planning workgroup

// The workgroup copies part `part` of a slot (of all planes' parts in turn) from slot src (none if negative:
// zeros) to slot dst.
__device__ __forceinline__ void copy_part(const Planes& p, int64_t part, int64_t src, int64_t dst) {
    const uint8_t* s = p.src[0];
    uint8_t* d = p.dst[0];
    int64_t bytes = p.bytes[0];
#pragma unroll
    for (int i = 1; i < MAX_PLANES; ++i) {           // the plane that the part falls into
        const int64_t before = (bytes + PART - 1) / PART;
        if (i < p.n && part >= before) {
            part -= before;
            s = p.src[i];
            d = p.dst[i];
            bytes = p.bytes[i];
        } else {
            break;
        }
    }
    const int64_t at = part * PART, n = bytes - at < PART ? bytes - at : PART;
    const __amdgpu_buffer_rsrc_t rs = make_rsrc_u(s + (src < 0 ? 0 : src) * bytes + at, src < 0 ? 0 : static_cast<uint32_t>(n));
    const __amdgpu_buffer_rsrc_t rd = make_rsrc_u(d + dst * bytes + at, static_cast<uint32_t>(n));
    const uint32_t t = threadIdx.x;
    if ((bytes & 15) == 0) {                         // whole units; the planes start on 16-byte borders
        u32x4 x[DEEP];
#pragma unroll
        for (int j = 0; j < DEEP; ++j) x[j] = __builtin_amdgcn_raw_buffer_load_b128(rs, (t + j * THREADS) * 16, 0, CP_NT);
#pragma unroll
        for (int j = 0; j < DEEP; ++j) __builtin_amdgcn_raw_buffer_store_b128(x[j], rd, (t + j * THREADS) * 16, 0, CP_NT);
    } else if ((bytes & 3) == 0) {
#pragma unroll 8
        for (uint32_t e = t * 4; e < n; e += THREADS * 4)
            __builtin_amdgcn_raw_buffer_store_b32(__builtin_amdgcn_raw_buffer_load_b32(rs, e, 0, 0), rd, e, 0, 0);
    } else {
#pragma unroll 8
        for (uint32_t e = t; e < n; e += THREADS)
            __builtin_amdgcn_raw_buffer_store_b8(__builtin_amdgcn_raw_buffer_load_b8(rs, e, 0, 0), rd, e, 0, 0);
    }
}

// Pair n of a copy between pools, part blockIdx.x % parts.
__global__ void __launch_bounds__(THREADS, 8) pair_kernel(Planes p, const int32_t* __restrict__ src_slots,
                                                       const int32_t* __restrict__ dst_slots, int32_t N, int32_t n_src,
                                                       int32_t n_dst, int32_t parts) {
    const int32_t n = blockIdx.x / parts, part = blockIdx.x % parts;
    const int32_t dst = dst_slots ? dst_slots[n] : n, src = src_slots ? src_slots[n] : n;
    if (dst < 0 || dst >= n_dst) return;
    if (dst_slots) {                                 // a later pair with the same destination takes it
        bool later = false;
        for (int32_t m = n + 1 + static_cast<int32_t>(threadIdx.x); m < N; m += THREADS) later |= dst_slots[m] == dst;
        if (__syncthreads_or(later)) return;
    }
    copy_part(p, part, src < 0 || src >= n_src ? -1 : src, dst);
}

// The pairs (src[i], dst[i]) of a plan, src negative: zeros, dst negative: nothing to do; *count of them, or N.
__global__ void __launch_bounds__(THREADS, 8) plan_copy_kernel(Planes p, const int32_t* __restrict__ src,
                                                            const int32_t* __restrict__ dst,
                                                            const int32_t* __restrict__ count, int32_t N, int32_t parts) {
    const int64_t n = count ? *count : N;
    for (int64_t u = blockIdx.x; u < n * parts; u += gridDim.x) {
        const int64_t i = u / parts;
        const int32_t to = dst[i];
        if (to >= 0) copy_part(p, u % parts, src[i], to);
    }
}

__global__ void __launch_bounds__(THREADS) count_kernel(int32_t* refs, const int32_t* __restrict__ slots, int32_t N,
                                                        int32_t n_slots, int32_t up) {
    const int32_t n = blockIdx.x * THREADS + threadIdx.x;
    if (n >= N) return;
    const int32_t slot = slots[n];
    if (slot < 0 || slot >= n_slots) return;
    // a free slot stays free; the order of the changes does not matter
    int32_t old = __hip_atomic_load(refs + slot, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    while (old > 0 && !__hip_atomic_compare_exchange_weak(refs + slot, &old, old + (up ? 1 : -1), __ATOMIC_RELAXED,
                                                          __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)) {
    }
}

// How many lanes of the planning workgroup before this one have the flag set, and in all.
__device__ __forceinline__ int rank_of(bool flag, int32_t* waves, int& total) {
    const uint64_t mask = __ballot(flag);
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    if (lane == 0) waves[wave] = __popcll(mask);
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < PLAN / 64; ++w) {
        before += w < wave ? waves[w] : 0;
        all += waves[w];
    }
    __syncthreads();
    total = all;
    return before + __popcll(mask & ((uint64_t(1) << lane) - 1));
}

// children[i] = the i-th free slot from below (-1: none left), in use once from now on; from[i] = the slot whose
// contents it gets, -1 for zeros.
__global__ void __launch_bounds__(PLAN) fork_plan_kernel(int32_t* refs, const int32_t* __restrict__ parents,
                                                         int32_t* __restrict__ children, int32_t* __restrict__ from,
                                                         int32_t N, int32_t n_slots) {
    __shared__ int32_t waves[PLAN / 64];
    const int t = threadIdx.x;
    for (int32_t i = t; i < N; i += PLAN) {          // before any slot is taken
        const int32_t parent = parents ? parents[i] : -1;
        from[i] = parent >= 0 && parent < n_slots && refs[parent] > 0 ? parent : -1;
    }
    __syncthreads();
    int32_t found = 0;
    for (int32_t s0 = 0; s0 < n_slots && found < N; s0 += PLAN) {
        const int32_t s = s0 + t;
        const bool free = s < n_slots && refs[s] <= 0;
        int total;
        const int32_t i = found + rank_of(free, waves, total);
        if (free && i < N) {
            children[i] = s;
            refs[s] = 1;
        }
        found += total;
    }
    for (int32_t i = found + t; i < N; i += PLAN) children[i] = -1;
}

// With U used slots: the used slots from U on go to the free ones before U, both in order.  to[s]: where slot s is
// afterwards (-1: free).
__global__ void __launch_bounds__(PLAN) compact_plan_kernel(int32_t* refs, int32_t* __restrict__ src,
                                                            int32_t* __restrict__ dst, int32_t* to,
                                                            int32_t* __restrict__ count, int32_t* __restrict__ used,
                                                            int32_t n_slots) {
    __shared__ int32_t waves[PLAN / 64];
    const int t = threadIdx.x;
    int32_t mine = 0;
    for (int32_t s = t; s < n_slots; s += PLAN) mine += refs[s] > 0;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) mine += __shfl_xor(mine, off, 64);
    if ((t & 63) == 0) waves[t >> 6] = mine;
    __syncthreads();
    int32_t U = 0;
    for (int w = 0; w < PLAN / 64; ++w) U += waves[w];
    __syncthreads();
    int32_t holes = 0, movers = 0;
    for (int32_t s0 = 0; s0 < n_slots; s0 += PLAN) {
        const int32_t s = s0 + t;
        const bool taken = s < n_slots && refs[s] > 0;
        const bool hole = s < U && !taken, mover = s >= U && taken;
        if (s < n_slots) to[s] = taken ? s : -1;
        int total;
        if (s0 < U) {
            const int32_t i = holes + rank_of(hole, waves, total);
            if (hole) dst[i] = s;
            holes += total;
        }
        if (s0 + PLAN > U) {
            const int32_t i = movers + rank_of(mover, waves, total);
            if (mover) src[i] = s;
            movers += total;
        }
    }
    __syncthreads();
    for (int32_t i = t; i < movers; i += PLAN) {     // as many holes as movers
        const int32_t a = src[i], b = dst[i];
        refs[b] = refs[a];
        refs[a] = 0;
        to[a] = b;
    }
    if (t == 0) {
        *count = movers;
        *used = U;
    }
}

__global__ void __launch_bounds__(THREADS) table_kernel(int32_t* table, int64_t n_table, const int32_t* __restrict__ to,
                                                        int32_t n_slots) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * THREADS + threadIdx.x;
    if (i >= n_table) return;
    const int32_t s = table[i];
    table[i] = s >= 0 && s < n_slots ? to[s] : -1;
}

int64_t total_parts(const Planes& p) {
    int64_t parts = 0;
    for (int i = 0; i < p.n; ++i) parts += (p.bytes[i] + PART - 1) / PART;
    return parts;
}
// Workgroups of a copy: eight a CU, each with 32 KB of loads under way, or one a part where there are fewer.
unsigned copy_grid(int64_t pairs, int64_t parts) {
    return static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(pairs * parts, 2048)));
}

}  // namespace

size_t slots_workspace_bytes(int32_t n_slots, int32_t N) {
    // fork: from [N]; compact: count, src and dst [n_slots / 2], to [n_slots]
    const int64_t half = n_slots / 2;
    return static_cast<size_t>(std::max<int64_t>(N, 4 + 2 * half + n_slots)) * 4;
}

hipError_t launch_slots_copy(const Planes& p, const int32_t* src_slots, const int32_t* dst_slots, int32_t N,
                             int32_t n_src, int32_t n_dst, hipStream_t stream) {
    const int64_t parts = total_parts(p);
    hipLaunchKernelGGL(pair_kernel, dim3(static_cast<unsigned>(N * parts)), dim3(THREADS), 0, stream, p, src_slots,
                       dst_slots, N, n_src, n_dst, static_cast<int32_t>(parts));
    return hipGetLastError();
}

hipError_t launch_slots_count(int32_t* refs, const int32_t* slots, int32_t N, int32_t n_slots, bool up,
                              hipStream_t stream) {
    hipLaunchKernelGGL(count_kernel, dim3((N - 1) / THREADS + 1), dim3(THREADS), 0, stream, refs, slots, N, n_slots,
                       up ? 1 : 0);
    return hipGetLastError();
}

hipError_t launch_slots_fork(const Planes& p, int32_t* refs, const int32_t* parents, int32_t* children, int32_t N,
                             int32_t n_slots, void* workspace, hipStream_t stream) {
    int32_t* from = static_cast<int32_t*>(workspace);
    hipLaunchKernelGGL(fork_plan_kernel, dim3(1), dim3(PLAN), 0, stream, refs, parents, children, from, N, n_slots);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t parts = total_parts(p);
    hipLaunchKernelGGL(plan_copy_kernel, dim3(copy_grid(N, parts)), dim3(THREADS), 0, stream, p, from, children,
                       nullptr, N, static_cast<int32_t>(parts));
    return hipGetLastError();
}

hipError_t launch_slots_compact(const Planes& p, int32_t* refs, int32_t* table, int64_t n_table, int32_t* used,
                                int32_t n_slots, void* workspace, hipStream_t stream) {
    const int64_t half = n_slots / 2;
    int32_t* count = static_cast<int32_t*>(workspace);
    int32_t *src = count + 4, *dst = src + half, *to = dst + half;
    hipLaunchKernelGGL(compact_plan_kernel, dim3(1), dim3(PLAN), 0, stream, refs, src, dst, to, count, used, n_slots);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && n_table > 0) {
        hipLaunchKernelGGL(table_kernel, dim3(static_cast<unsigned>((n_table - 1) / THREADS + 1)), dim3(THREADS), 0,
                           stream, table, n_table, to, n_slots);
        e = hipGetLastError();
    }
    if (e != hipSuccess || half == 0) return e;
    const int64_t parts = total_parts(p);
    hipLaunchKernelGGL(plan_copy_kernel, dim3(copy_grid(half, parts)), dim3(THREADS), 0, stream, p, src, dst, count,
                       0, static_cast<int32_t>(parts));
    return hipGetLastError();
}

}  // namespace kda
