// kda_state_cache.hip -- recurrent states in a pool of 8-bit codes: kda_state_store, kda_state_load.
//
// A state row (one key channel) is cut into groups of GROUP value channels; a group has one fp32
// scale, max|x| times 1 / M with M the largest code (127, or 448 for e4m3), and its codes are x / scale
// rounded to nearest even.  The quotient must not be rounded twice (an fp32 quotient next to the
// border of two codes could fall on it), which costs a few VALU operations only:
//   integers: c = rint(x * (1/scale)) is off by at most one; e = x - c scale is exact in fp32 (both
//     are multiples of the smaller ulp, and |e| <= scale), so comparing 2 |e| with scale decides.
//   e4m3: q within one ulp of x / scale, and the exact sign of x - q scale; where q is inexact and its
//     last bit even, one ulp towards the true quotient makes the last bit odd, and an odd q lies on the
//     right side of every border of the coarser format (borders have zeros there).
//
// Both kernels stream: 5 + 4 / GROUP bytes per state element and no reuse.  A lane owns four
// neighbouring channels (16-byte accesses to fp32, 4-byte ones to the codes), GROUP / 4
// neighbouring lanes a group; the maximum crosses them by shuffles.  One workgroup handles 4096
// elements, which divides every sequence's states, in four passes, loads first.  The fp32 states are
// streamed past the caches (each is touched once).
#include "kda_common.hpp"
#include "kda_linear.hpp"

namespace kda {
namespace {

typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr int PASSES = 4;                      // of 1024 elements: a sequence has a multiple of 4096

// The four codes of x under `scale` (finite, > 0), one byte each.
template <int CODE>
__device__ __forceinline__ uint32_t encode4(f32x4_t x, float scale) {
    constexpr float most = CODE == KDA_CODE_I8 ? 127.f : 448.f;
    // a scale whose reciprocal might overflow: scaled up with x, exactly
    const float lift = scale < 0x1p-100f ? 0x1p64f : 1.f;
    scale *= lift;
    x *= lift;
    const float inv = __builtin_amdgcn_rcpf(scale);                // within one ulp
    float q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = x[i] * inv;                 // within two ulps
    if constexpr (CODE == KDA_CODE_I8) {
        uint32_t out = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float c = __builtin_rintf(__builtin_amdgcn_fmed3f(q[i], -most, most));
            const float e = __builtin_fmaf(-c, scale, x[i]);
            const float d2 = 2.f * __builtin_fabsf(e);
            int ci = static_cast<int>(c);
            if (d2 > scale || (d2 == scale && (ci & 1))) ci += e > 0.f ? 1 : -1;
            ci = ci < -127 ? -127 : (ci > 127 ? 127 : ci);
            out |= (static_cast<uint32_t>(ci) & 0xffu) << (8 * i);
        }
        return out;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float y = __builtin_fmaf(__builtin_fmaf(-q[i], scale, x[i]), inv, q[i]);        // within one ulp
            y = __builtin_amdgcn_fmed3f(y, -most, most);
            const float r = __builtin_fmaf(-y, scale, x[i]);        // sign of the quotient's rest
            uint32_t u = __float_as_uint(y);
            if (r != 0.f && !(u & 1u) && __builtin_fabsf(y) < most) u = ((r > 0.f) == (y > 0.f)) ? u + 1u : u - 1u;
            // far below half the smallest code (2^-10): zero
            q[i] = __builtin_fabsf(y) < 0x1p-20f ? 0.f : __uint_as_float(u);
        }
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], w, true);
        return static_cast<uint32_t>(w);
    }
}

template <int CODE>
__device__ __forceinline__ float4 decode4(uint32_t w) {
    if constexpr (CODE == KDA_CODE_I8) {
        return make_float4(static_cast<float>(static_cast<int8_t>(w)), static_cast<float>(static_cast<int8_t>(w >> 8)),
                           static_cast<float>(static_cast<int8_t>(w >> 16)), static_cast<float>(static_cast<int8_t>(w >> 24)));
    } else {
        return make_float4(__builtin_amdgcn_cvt_f32_fp8(w, 0), __builtin_amdgcn_cvt_f32_fp8(w, 1),
                           __builtin_amdgcn_cvt_f32_fp8(w, 2), __builtin_amdgcn_cvt_f32_fp8(w, 3));
    }
}

// One workgroup: ROUNDS blocks of 4096 elements of one sequence's states (or what is left of them).  Every
// workgroup looks through the later sequences for its slot, so where there are many, one takes four blocks;
// where there are few, four blocks only leave the chip unevenly filled.  Four and one, in us, by sequences:
//     2 x 64 x 64     512: 8.8, 8.1    1024: 11.9, 11.4   2048: 20.4, 22.0   16384: 159, 202
//     8 x 128 x 128   512: 65, 64      1024: 123, 125     2048: 252, 269     16384: 2275, 3018
//     32 x 128 x 128  512: 254, 251    1024: 547, 525     2048: 1095, 1070   4096: 2178, 2233
template <int CODE, int GROUP, int ROUNDS>
__global__ void __launch_bounds__(256, 8) store_kernel(const float* __restrict__ states, const int32_t* __restrict__ slots,
                                                       uint8_t* __restrict__ codes, float* __restrict__ scales,
                                                       int32_t N, int32_t n_slots, int64_t per_seq, int32_t parts) {
    constexpr float inv_most = 1.f / (CODE == KDA_CODE_I8 ? 127.f : 448.f);
    const int32_t n = blockIdx.x / parts, part = blockIdx.x % parts;
    const int32_t slot = slots ? slots[n] : n;
    if (slot < 0 || slot >= n_slots) return;
    if (slots) {                     // a later sequence with the same slot takes it
        bool later = false;
        for (int32_t m = n + 1 + static_cast<int32_t>(threadIdx.x); m < N; m += 256) later |= slots[m] == slot;
        if (__syncthreads_or(later)) return;
    }
    const float* src = states + n * per_seq + 4 * threadIdx.x;
    uint8_t* dst = codes + slot * per_seq + 4 * threadIdx.x;
    float* sc = scales + slot * (per_seq / GROUP) + threadIdx.x / (GROUP / 4);
    for (int32_t r = 0; r < ROUNDS; ++r) {
        const int64_t e = (static_cast<int64_t>(part) * ROUNDS + r) * (PASSES * 1024);
        if (ROUNDS > 1 && e >= per_seq) break;
        f32x4_t x[PASSES];
#pragma unroll
        for (int p = 0; p < PASSES; ++p) x[p] = __builtin_nontemporal_load(reinterpret_cast<const f32x4_t*>(src + e + p * 1024));
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
            float a = __builtin_fmaxf(__builtin_fmaxf(__builtin_fabsf(x[p][0]), __builtin_fabsf(x[p][1])),
                                      __builtin_fmaxf(__builtin_fabsf(x[p][2]), __builtin_fabsf(x[p][3])));
            // 0 while all values are finite, NaN from the first infinity or NaN on
            float bad = (x[p][0] - x[p][0]) + (x[p][1] - x[p][1]) + (x[p][2] - x[p][2]) + (x[p][3] - x[p][3]);
#pragma unroll
            for (int off = 1; off < GROUP / 4; off <<= 1) {
                a = __builtin_fmaxf(a, __shfl_xor(a, off, 64));
                bad += __shfl_xor(bad, off, 64);
            }
            const float scale = bad == 0.f ? a * inv_most : __uint_as_float(0x7fc00000u);
            uint32_t w = 0;
            if (scale > 0.f) w = encode4<CODE>(x[p], scale);
            *reinterpret_cast<uint32_t*>(dst + e + p * 1024) = w;
            if (threadIdx.x % (GROUP / 4) == 0) sc[(e + p * 1024) / GROUP] = scale;
        }
    }
}

template <int CODE, int GROUP>
__global__ void __launch_bounds__(256) load_kernel(const uint8_t* __restrict__ codes, const float* __restrict__ scales,
                                                   const int32_t* __restrict__ slots, float* __restrict__ states,
                                                   int32_t n_slots, int64_t per_seq, int32_t blocks_per_seq) {
    const int32_t n = blockIdx.x / blocks_per_seq, part = blockIdx.x % blocks_per_seq;
    const int32_t slot = slots ? slots[n] : n;
    const bool have = slot >= 0 && slot < n_slots;
    const int64_t e0 = static_cast<int64_t>(part) * (PASSES * 1024) + 4 * threadIdx.x;
    const uint8_t* src = codes + (have ? slot : 0) * per_seq;
    const float* sc = scales + (have ? slot : 0) * (per_seq / GROUP);
    float* dst = states + n * per_seq;
    uint32_t w[PASSES];
    float s[PASSES];
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
        const int64_t e = e0 + p * 1024;
        w[p] = 0;
        s[p] = 0.f;
        if (have) {
            w[p] = *reinterpret_cast<const uint32_t*>(src + e);
            s[p] = sc[e / GROUP];
        }
    }
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
        const int64_t e = e0 + p * 1024;
        const float4 c = decode4<CODE>(w[p]);
        const f32x4_t y = {c.x * s[p], c.y * s[p], c.z * s[p], c.w * s[p]};
        __builtin_nontemporal_store(y, reinterpret_cast<f32x4_t*>(dst + e));
    }
}

}  // namespace

hipError_t launch_state_store(const StateCacheArgs& a, const float* states, hipStream_t stream) {
    const int64_t per_seq = int64_t(a.H) * a.dk * a.dv;
    const int64_t blocks = per_seq / (PASSES * 1024);
    const int32_t rounds = a.slots && a.N >= 2048 ? 4 : 1, parts = static_cast<int32_t>((blocks + rounds - 1) / rounds);
    const dim3 grid(static_cast<unsigned>(int64_t(a.N) * parts));
    auto go = [&](auto one, auto four) {
        hipLaunchKernelGGL(rounds == 1 ? one : four, grid, dim3(256), 0, stream, states, a.slots,
                           static_cast<uint8_t*>(a.codes), a.scales, a.N, a.n_slots, per_seq, parts);
        return hipGetLastError();
    };
    if (a.code == KDA_CODE_I8) {
        if (a.group == 32) return go(store_kernel<KDA_CODE_I8, 32, 1>, store_kernel<KDA_CODE_I8, 32, 4>);
        if (a.group == 64) return go(store_kernel<KDA_CODE_I8, 64, 1>, store_kernel<KDA_CODE_I8, 64, 4>);
        return go(store_kernel<KDA_CODE_I8, 128, 1>, store_kernel<KDA_CODE_I8, 128, 4>);
    }
    if (a.group == 32) return go(store_kernel<KDA_CODE_E4M3, 32, 1>, store_kernel<KDA_CODE_E4M3, 32, 4>);
    if (a.group == 64) return go(store_kernel<KDA_CODE_E4M3, 64, 1>, store_kernel<KDA_CODE_E4M3, 64, 4>);
    return go(store_kernel<KDA_CODE_E4M3, 128, 1>, store_kernel<KDA_CODE_E4M3, 128, 4>);
}

hipError_t launch_state_load(const StateCacheArgs& a, float* states, hipStream_t stream) {
    const int64_t per_seq = int64_t(a.H) * a.dk * a.dv;
    const int32_t bps = static_cast<int32_t>(per_seq / (PASSES * 1024));
    const dim3 grid(static_cast<unsigned>(int64_t(a.N) * bps));
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, static_cast<const uint8_t*>(a.codes), a.scales, a.slots,
                           states, a.n_slots, per_seq, bps);
        return hipGetLastError();
    };
    if (a.code == KDA_CODE_I8) {
        if (a.group == 32) return go(load_kernel<KDA_CODE_I8, 32>);
        if (a.group == 64) return go(load_kernel<KDA_CODE_I8, 64>);
        return go(load_kernel<KDA_CODE_I8, 128>);
    }
    if (a.group == 32) return go(load_kernel<KDA_CODE_E4M3, 32>);
    if (a.group == 64) return go(load_kernel<KDA_CODE_E4M3, 64>);
    return go(load_kernel<KDA_CODE_E4M3, 128>);
}

}  // namespace kda
