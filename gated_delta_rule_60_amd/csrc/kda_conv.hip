// kda_conv.hip -- short causal convolution: every channel's weighted sum of its last W inputs, with or without a
// SiLU, over packed or fixed-length sequences; its gradients; and the single-token step on windows in slots.
//     u_t = bias + sum_i w_i x_{t-W+1+i},   y_t = u_t sigmoid(u_t) or u_t,
//     du_t = dy_t y'(u_t),   dx_t = sum_k w_{W-1-k} du_{t+k},   dw_i = sum_t du_t x_{t-W+1+i},   dbias = sum_t du_t
// with the inputs before a sequence's first token from its initial window.
//
// A lane owns V neighbouring channels (prompts four: 8 bytes of 16-bit elements, 16 of fp32; the step up to 16 bytes) and
// walks SUB tokens with the last W - 1 inputs in registers; a workgroup is 32 lanes of channels by 8 walks one behind the
// other, so that the W - 1 rows a walk reads of its neighbour's come from the caches.
// 4 x 4096 tokens of 4352 channels, 4 taps, SiLU: bf16 58 us (4.9 TB/s), fp32 114 us (5.0 TB/s), bound by HBM (2 rows of
// channels a token, about 16 VALU instructions an element).  Gradients (3 rows): fp32 180 us (4.8 TB/s), bf16 115 us
// (3.7 TB/s), bound by VALU issue: 47 instructions an element of a walk, of which it takes 16 + 3 for 16 tokens (one
// exponential and one reciprocal each); the SIMDs issue all of the kernel's time.  1780 packed tokens of 2304 channels:
// gradients 19 us, of which a walk, load after load, is most.
// Sums are fp32, over a workgroup's RUN tokens, then fp64 over the workgroups in order.
#include "kda_ssm.hpp"
#include "kda_tile.hpp"

#include <algorithm>
#include <type_traits>

namespace kda {
namespace {

constexpr int SUBS = 8, LANES = 32, SUB = 16, RUN = SUBS * SUB;

struct Conv {
    const uint8_t *x, *dy;
    uint8_t* out;
    int64_t ldx, lddy, ldo;          // bytes from token to token
    const float *w, *bias;
    const uint8_t *h0, *dhT;
    uint8_t *hT, *dh0;
    const int32_t* cu;
    int64_t T;
    int32_t n_seqs, C, nvec, seg, n_seg, slots, vblocks, silu;
    float* part;                     // [slots, W + 1, C]
};

// V neighbouring elements.
template <int DT, int V>
struct Vec {
    static constexpr int ES = DT == KDA_BF16 ? 2 : 4, BYTES = V * ES;
    using raw = std::conditional_t<BYTES == 16, u32x4, std::conditional_t<BYTES == 8, u32x2, uint32_t>>;
    static __device__ __forceinline__ raw load(__amdgpu_buffer_rsrc_t r, uint32_t at) {
        if constexpr (BYTES == 16) return __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0);
        else if constexpr (BYTES == 8) return __builtin_amdgcn_raw_buffer_load_b64(r, at, 0, 0);
        else if constexpr (BYTES == 4) return __builtin_amdgcn_raw_buffer_load_b32(r, at, 0, 0);
        else return __builtin_amdgcn_raw_buffer_load_b16(r, at, 0, 0);
    }
    static __device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t r, uint32_t at, raw x) {
        if constexpr (BYTES == 16) __builtin_amdgcn_raw_buffer_store_b128(x, r, at, 0, CP_NT);
        else if constexpr (BYTES == 8) __builtin_amdgcn_raw_buffer_store_b64(x, r, at, 0, CP_NT);
        else if constexpr (BYTES == 4) __builtin_amdgcn_raw_buffer_store_b32(x, r, at, 0, 0);
        else __builtin_amdgcn_raw_buffer_store_b16(static_cast<uint16_t>(x), r, at, 0, 0);
    }
    static __device__ __forceinline__ raw get(const uint8_t* p) {
        if constexpr (BYTES == 2) return *reinterpret_cast<const uint16_t*>(p);
        else return *reinterpret_cast<const raw*>(p);
    }
    static __device__ __forceinline__ void put(uint8_t* p, raw x) {
        if constexpr (BYTES == 2) *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(x);
        else *reinterpret_cast<raw*>(p) = x;
    }
    static __device__ __forceinline__ raw zero() {
        if constexpr (BYTES >= 8) return raw{};
        else return 0u;
    }
    static __device__ __forceinline__ void open(raw x, float (&f)[V]) {
        if constexpr (ES == 4) {
            if constexpr (V == 1) f[0] = __uint_as_float(x);
            else
#pragma unroll
                for (int i = 0; i < V; ++i) f[i] = __uint_as_float(x[i]);
        } else if constexpr (V == 1) {
            f[0] = __uint_as_float(x << 16);
        } else {
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                f[2 * i] = __uint_as_float(x[i] << 16);
                f[2 * i + 1] = __uint_as_float(x[i] & 0xffff0000u);
            }
        }
    }
    static __device__ __forceinline__ raw close(const float (&f)[V]) {
        if constexpr (ES == 4) {
            if constexpr (V == 1) return __float_as_uint(f[0]);
            else {
                raw x;
#pragma unroll
                for (int i = 0; i < V; ++i) x[i] = __float_as_uint(f[i]);
                return x;
            }
        } else if constexpr (V == 1) {
            return bf16_bits(f[0]);
        } else {
            raw x;
#pragma unroll
            for (int i = 0; i < V / 2; ++i) x[i] = pack_bf16(f[2 * i], f[2 * i + 1]);
            return x;
        }
    }
};

// 1 / (1 + e^-u): e^-u from 2^p with p's rounding error carried along, the quotient within 1.5 ulp.
__device__ __forceinline__ float sigmoid(float u) {
    constexpr float LOG2E = 1.44269504088896340736f, LOG2E_LO = 1.925963033500e-8f;
    const float c = __builtin_amdgcn_fmed3f(u, -87.f, 87.f);       // beyond: 1 to fp32's accuracy, or below 2^-125: 0
    const float p = -c * LOG2E;
    const float rest = __builtin_fmaf(-c, LOG2E_LO, __builtin_fmaf(-c, LOG2E, -p));
    float e = __builtin_amdgcn_exp2f(p);
    e = __builtin_fmaf(e, rest * 0.69314718055994531f, e);
    const float d = 1.f + e, r = __builtin_amdgcn_rcpf(d);
    return u < -87.f ? 0.f : __builtin_fmaf(__builtin_fmaf(-d, r, 1.f), r, r);
}

// What a lane of the two prompt kernels works on.
struct Walk {
    Where w;
    int64_t first;                   // the sequence's first token
    int vec, sub;
    int32_t n;                       // tokens of the walk
    int64_t t0;                      // its first one
};
__device__ __forceinline__ bool start_walk(const Conv& c, Walk& k) {
    const int32_t slot = blockIdx.x / c.vblocks;
    k.vec = static_cast<int>(blockIdx.x % c.vblocks) * LANES + (threadIdx.x & (LANES - 1));
    k.sub = threadIdx.x / LANES;
    if (!locate(c, slot, k.w)) return false;
    k.first = k.w.lo - static_cast<int64_t>(k.w.s) * RUN;
    k.t0 = k.w.lo + k.sub * SUB;
    const int64_t left = k.w.hi - k.t0;
    k.n = left <= 0 ? 0 : (left < SUB ? static_cast<int32_t>(left) : SUB);
    return true;
}

// Weights of a lane's channels, by taps.
template <int V, int W>
__device__ __forceinline__ void load_weights(const Conv& c, int vec, float (&w)[W][V], float (&b)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int i = 0; i < W; ++i) w[i][v] = c.w[(static_cast<int64_t>(vec) * V + v) * W + i];
        b[v] = c.bias ? c.bias[vec * V + v] : 0.f;
    }
}

// Rows of the run from `back` tokens before it (0 in a sequence's first run: nothing there) to `ahead` behind it.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t run_rows(const uint8_t* p, int64_t ld, const Where& w, int back,
                                                           int64_t end, uint32_t row_bytes) {
    const int64_t n = end - w.lo + back;
    return make_rsrc_u(p + (w.lo - back) * ld, n > 0 ? static_cast<uint32_t>((n - 1) * ld) + row_bytes : 0);
}

template <int DT, int V, int W>
__global__ void __launch_bounds__(256) conv_fwd_kernel(Conv c, uint32_t main_blocks) {
    using X = Vec<DT, V>;
    if (blockIdx.x >= main_blocks) {                 // the windows behind the last tokens
        const int64_t i = static_cast<int64_t>(blockIdx.x - main_blocks) * 256 + threadIdx.x;
        if (i >= static_cast<int64_t>(c.n_seqs) * (W - 1) * c.nvec) return;
        const int32_t vec = i % c.nvec, k = i / c.nvec % (W - 1), n = i / c.nvec / (W - 1);
        int64_t lo, hi;
        seq_range(c, n, lo, hi);
        const int64_t at = hi - (W - 1) + k;
        typename X::raw x = X::zero();
        if (at >= lo) x = X::get(c.x + at * c.ldx + vec * X::BYTES);
        else if (c.h0) x = X::get(c.h0 + ((static_cast<int64_t>(n) * (W - 1) + (at - lo + W - 1)) * c.nvec + vec) * X::BYTES);
        X::put(c.hT + i * X::BYTES, x);
        return;
    }
    Walk k;
    if (!start_walk(c, k) || k.n == 0 || k.vec >= c.nvec) return;
    const uint32_t row = c.C * X::ES, ldx = static_cast<uint32_t>(c.ldx), ldo = static_cast<uint32_t>(c.ldo);
    const int back = k.w.s > 0 ? W - 1 : 0;
    const __amdgpu_buffer_rsrc_t rx = run_rows(c.x, c.ldx, k.w, back, k.w.hi, row);
    const __amdgpu_buffer_rsrc_t ro = run_rows(c.out, c.ldo, k.w, 0, k.w.hi, row);
    const uint32_t at_x = (k.sub * SUB + back) * ldx + k.vec * X::BYTES, at_o = k.sub * SUB * ldo + k.vec * X::BYTES;
    constexpr int STEP = 8;
    typename X::raw next[STEP];
#pragma unroll
    for (int j = 0; j < STEP; ++j) next[j] = X::load(rx, at_x + j * ldx);
    float w[W][V], b[V], win[W][V];                  // win[i]: the input of tap i
    load_weights<V, W>(c, k.vec, w, b);
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
        typename X::raw x = X::zero();
        if (k.sub > 0 || back) x = X::load(rx, at_x - (W - 1 - i) * ldx);
        else if (c.h0) x = X::get(c.h0 + ((static_cast<int64_t>(k.w.n) * (W - 1) + i) * c.nvec + k.vec) * X::BYTES);
        X::open(x, win[i + 1]);
    }
    for (int t0 = 0; t0 < SUB && t0 < k.n; t0 += STEP) {
        typename X::raw cur[STEP];
#pragma unroll
        for (int j = 0; j < STEP; ++j) cur[j] = next[j];
        if (t0 + STEP < SUB)
#pragma unroll
            for (int j = 0; j < STEP; ++j) next[j] = X::load(rx, at_x + (t0 + STEP + j) * ldx);
#pragma unroll
        for (int j = 0; j < STEP; ++j) {
            if (t0 + j >= k.n) break;
#pragma unroll
            for (int i = 0; i < W - 1; ++i)
#pragma unroll
                for (int v = 0; v < V; ++v) win[i][v] = win[i + 1][v];
            X::open(cur[j], win[W - 1]);
            float u[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                u[v] = b[v];
#pragma unroll
                for (int i = 0; i < W; ++i) u[v] = __builtin_fmaf(w[i][v], win[i][v], u[v]);
            }
            if (c.silu)
#pragma unroll
                for (int v = 0; v < V; ++v) u[v] *= sigmoid(u[v]);
            X::store(ro, at_o + (t0 + j) * ldo, X::close(u));
        }
    }
}

template <int DT, int V, int W>
__global__ void __launch_bounds__(256) conv_bwd_kernel(Conv c) {
    using X = Vec<DT, V>;
    __shared__ float red[4][W + 1][LANES * V];
    Walk k;
    const bool used = start_walk(c, k);
    const int32_t slot = blockIdx.x / c.vblocks, vec0 = static_cast<int32_t>(blockIdx.x % c.vblocks) * LANES;
    float dw[W][V] = {}, db[V] = {};
    // an empty walk has nothing to do, but a sequence's first one hands out the initial window's gradient
    if (used && k.vec < c.nvec && (k.n > 0 || (k.sub == 0 && k.w.s == 0))) {
        const uint32_t row = c.C * X::ES, ldx = static_cast<uint32_t>(c.ldx), lddy = static_cast<uint32_t>(c.lddy),
                       ldo = static_cast<uint32_t>(c.ldo);
        const int back = k.w.s > 0 ? W - 1 : 0;
        // the sequence's last token, or the last one a walk of this run looks at
        int64_t lo, end;
        seq_range(c, k.w.n, lo, end);
        const int64_t hi = end;
        end = end < k.w.hi + (W - 1) ? end : k.w.hi + (W - 1);
        const __amdgpu_buffer_rsrc_t rx = run_rows(c.x, c.ldx, k.w, back, end, row);
        const __amdgpu_buffer_rsrc_t ry = run_rows(c.dy, c.lddy, k.w, 0, end, row);
        const __amdgpu_buffer_rsrc_t ro = run_rows(c.out, c.ldo, k.w, 0, k.w.hi, row);
        const uint32_t at_x = (k.sub * SUB + back) * ldx + k.vec * X::BYTES;
        const uint32_t at_y = k.sub * SUB * lddy + k.vec * X::BYTES, at_o = k.sub * SUB * ldo + k.vec * X::BYTES;
        constexpr int STEP = 4;
        typename X::raw nx[STEP], ny[STEP];
#pragma unroll
        for (int j = 0; j < STEP; ++j) {
            nx[j] = X::load(rx, at_x + j * ldx);
            ny[j] = X::load(ry, at_y + j * lddy);
        }
        float w[W][V], b[V], win[W][V], du[W][V];    // du[i]: of W - 1 - i tokens ago
        load_weights<V, W>(c, k.vec, w, b);
#pragma unroll
        for (int i = 0; i < W; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v) du[i][v] = 0.f;
#pragma unroll
        for (int i = 0; i < W - 1; ++i) {
            typename X::raw x = X::zero();
            if (k.sub > 0 || back) x = X::load(rx, at_x - (W - 1 - i) * ldx);
            else if (c.h0) x = X::get(c.h0 + ((static_cast<int64_t>(k.w.n) * (W - 1) + i) * c.nvec + k.vec) * X::BYTES);
            X::open(x, win[i + 1]);
        }
        const int32_t steps = k.n + W - 1;
        const int64_t rest = hi - k.t0;              // tokens of the sequence from the walk on
        for (int t0 = 0; t0 < steps; t0 += STEP) {
            typename X::raw cx[STEP], cy[STEP];
#pragma unroll
            for (int j = 0; j < STEP; ++j) {
                cx[j] = nx[j];
                cy[j] = ny[j];
            }
            if (t0 + STEP < steps)
#pragma unroll
                for (int j = 0; j < STEP; ++j) {
                    nx[j] = X::load(rx, at_x + (t0 + STEP + j) * ldx);
                    ny[j] = X::load(ry, at_y + (t0 + STEP + j) * lddy);
                }
#pragma unroll
            for (int j = 0; j < STEP; ++j) {
                const int t = t0 + j;
                if (t >= steps) break;
#pragma unroll
                for (int i = 0; i < W - 1; ++i)
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        win[i][v] = win[i + 1][v];
                        du[i][v] = du[i + 1][v];
                    }
                X::open(cx[j], win[W - 1]);
                float g[V];
                X::open(cy[j], g);
                if (c.silu) {
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        float u = b[v];
#pragma unroll
                        for (int i = 0; i < W; ++i) u = __builtin_fmaf(w[i][v], win[i][v], u);
                        const float s = sigmoid(u);
                        g[v] *= __builtin_fmaf(s * u, 1.f - s, s);
                    }
                }
                const bool inside = t < rest;
#pragma unroll
                for (int v = 0; v < V; ++v) du[W - 1][v] = inside ? g[v] : 0.f;
                if (t < k.n) {
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        db[v] += du[W - 1][v];
#pragma unroll
                        for (int i = 0; i < W; ++i) dw[i][v] = __builtin_fmaf(du[W - 1][v], win[i][v], dw[i][v]);
                    }
                }
                const int s = t - (W - 1);           // the token whose gradient is complete now
                if (s < 0 && !(k.sub == 0 && k.w.s == 0 && c.dh0)) continue;
                float d[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    d[v] = 0.f;
#pragma unroll
                    for (int i = 0; i < W; ++i) d[v] = __builtin_fmaf(w[W - 1 - i][v], du[i][v], d[v]);
                }
                if (c.dhT && s >= rest - (W - 1)) {  // it is in the final window
                    float f[V];
                    X::open(X::get(c.dhT + ((static_cast<int64_t>(k.w.n) * (W - 1) + (s - rest + W - 1)) * c.nvec + k.vec) * X::BYTES), f);
#pragma unroll
                    for (int v = 0; v < V; ++v) d[v] += f[v];
                }
                if (s >= 0) X::store(ro, at_o + s * ldo, X::close(d));
                else X::put(c.dh0 + ((static_cast<int64_t>(k.w.n) * (W - 1) + (s + W - 1)) * c.nvec + k.vec) * X::BYTES, X::close(d));
            }
        }
    }
    // sums over the run: the two walks of a wave, the four waves
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int i = 0; i <= W; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float s = i < W ? dw[i < W ? i : 0][v] : db[v];
            s += __shfl_xor(s, 32, 64);
            if (lane < 32) red[wave][i][lane * V + v] = s;
        }
    __syncthreads();
    float* part = c.part + static_cast<int64_t>(slot) * (W + 1) * c.C;
    for (int e = threadIdx.x; e < (W + 1) * LANES * V; e += 256) {
        const int i = e / (LANES * V), ch = e % (LANES * V);
        if (vec0 * V + ch < c.C)
            part[static_cast<int64_t>(i) * c.C + vec0 * V + ch] = (red[0][i][ch] + red[1][i][ch]) + (red[2][i][ch] + red[3][i][ch]);
    }
}

// Sums over the runs, in order within a lane: 64 channels by four lanes of runs, row blockIdx.y of W + 1.
__global__ void __launch_bounds__(256) conv_sum_kernel(const float* __restrict__ part, int32_t slots, int32_t C, int32_t W,
                                                       float* __restrict__ dw, float* __restrict__ db) {
    __shared__ double red[4][64];
    const int32_t i = blockIdx.y, ch = blockIdx.x * 64 + (threadIdx.x & 63), q = threadIdx.x >> 6;
    double s = 0.0;
    if (ch < C) {
#pragma unroll 8
        for (int32_t r = q; r < slots; r += 4) s += static_cast<double>(part[(static_cast<int64_t>(r) * (W + 1) + i) * C + ch]);
    }
    red[q][threadIdx.x & 63] = s;
    __syncthreads();
    if (q == 0 && ch < C) {
        const int x = threadIdx.x & 63;
        const float sum = static_cast<float>((red[0][x] + red[1][x]) + (red[2][x] + red[3][x]));
        if (i < W) dw[static_cast<int64_t>(ch) * W + i] = sum;
        else if (db) db[ch] = sum;
    }
}

// One token of every sequence: blockIdx.x / blocks is the sequence, a lane V channels.
template <int DT, int V, int W>
__global__ void __launch_bounds__(256) conv_step_kernel(Conv c, uint8_t* windows, const int32_t* __restrict__ slots,
                                                        int32_t N, int32_t n_slots, int32_t blocks) {
    using X = Vec<DT, V>;
    const int32_t n = blockIdx.x / blocks, vec = static_cast<int32_t>(blockIdx.x % blocks) * 256 + threadIdx.x;
    const bool mine = vec < c.nvec;
    const int32_t slot = slots ? slots[n] : n;
    bool live = slot >= 0 && slot < n_slots;
    typename X::raw x[W];
    float w[W][V], b[V];
    uint8_t* win = windows + ((live ? slot : 0) * static_cast<int64_t>(W - 1) * c.nvec + vec) * X::BYTES;
    if (mine) {
        x[W - 1] = X::get(c.x + n * c.ldx + static_cast<int64_t>(vec) * X::BYTES);
#pragma unroll
        for (int i = 0; i < W - 1; ++i) x[i] = X::get(win + static_cast<int64_t>(i) * c.nvec * X::BYTES);
        load_weights<V, W>(c, vec, w, b);
    }
    if (slots && live) {                             // a later sequence with the same slot takes it
        bool later = false;
        for (int32_t m = n + 1 + static_cast<int32_t>(threadIdx.x); m < N; m += 256) later |= slots[m] == slot;
        if (__syncthreads_or(later)) live = false;
    }
    if (!mine) return;
    float u[V] = {};
    if (live) {
#pragma unroll
        for (int v = 0; v < V; ++v) u[v] = b[v];
#pragma unroll
        for (int i = 0; i < W; ++i) {
            float f[V];
            X::open(x[i], f);
#pragma unroll
            for (int v = 0; v < V; ++v) u[v] = __builtin_fmaf(w[i][v], f[v], u[v]);
        }
        if (c.silu)
#pragma unroll
            for (int v = 0; v < V; ++v) u[v] *= sigmoid(u[v]);
#pragma unroll
        for (int i = 0; i < W - 1; ++i) X::put(win + static_cast<int64_t>(i) * c.nvec * X::BYTES, x[i + 1]);
    }
    X::put(c.out + n * c.ldo + static_cast<int64_t>(vec) * X::BYTES, X::close(u));
}

// ---------------------------------------------------------------- host side

bool fits(const void* p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

// The widest accesses that the channels, the strides and the addresses allow, up to `most` channels: 16 bytes, 8 (16-bit
// elements), one element.  Prompts take four channels at most: with eight 16-bit ones a lane's registers (162, gradients
// 251) leave too few waves to keep loads under way (4 x 4096 x 4352: 67 us against 58, gradients 152 against 115).
constexpr int PROMPT = 4, STEP_ONE = 8;
int vector_width(const ConvArgs& a, const void* windows, int most) {
    const int64_t es = a.dtype == KDA_BF16 ? 2 : 4;
    for (int64_t bytes : {16, 8}) {
        const int64_t v = bytes / es;
        if (v < 4 || v > most || a.C % v || a.x.ld % v || a.dy.ld % v || a.out.ld % v) continue;
        bool ok = true;
        for (const void* p : {a.x.p, a.dy.p, static_cast<const void*>(a.out.p), a.h0, static_cast<const void*>(a.hT), a.dhT,
                              static_cast<const void*>(a.dh0), windows})
            ok = ok && fits(p, bytes);
        if (ok) return static_cast<int>(v);
    }
    return 1;
}

int64_t run_slots(int32_t n_seqs, int64_t total, bool packed) {
    if (packed) return total / RUN + n_seqs;
    return n_seqs * std::max<int64_t>(1, (total / n_seqs + RUN - 1) / RUN);
}

Conv base(const ConvArgs& a, int V) {
    const int64_t es = a.dtype == KDA_BF16 ? 2 : 4;
    Conv c{};
    c.x = static_cast<const uint8_t*>(a.x.p); c.dy = static_cast<const uint8_t*>(a.dy.p); c.out = static_cast<uint8_t*>(a.out.p);
    c.ldx = a.x.ld * es; c.lddy = a.dy.ld * es; c.ldo = a.out.ld * es;
    c.w = a.weight; c.bias = a.bias;
    c.h0 = static_cast<const uint8_t*>(a.h0); c.dhT = static_cast<const uint8_t*>(a.dhT);
    c.hT = static_cast<uint8_t*>(a.hT); c.dh0 = static_cast<uint8_t*>(a.dh0);
    c.cu = a.cu; c.T = a.T; c.n_seqs = a.n_seqs; c.C = a.C; c.nvec = a.C / V; c.silu = a.silu;
    c.vblocks = (c.nvec + LANES - 1) / LANES;
    c.seg = RUN;
    if (a.n_seqs > 0) {
        c.slots = static_cast<int32_t>(run_slots(a.n_seqs, int64_t(a.B) * a.T, a.cu != nullptr));
        c.n_seg = c.slots / a.n_seqs;
    }
    c.part = static_cast<float*>(a.workspace);
    return c;
}

// go(DT, V, W) as compile-time constants.
template <int MOST, typename F>
hipError_t by_kind(int dtype, int V, int W, F go) {
    auto taps = [&](auto dt, auto v) {
        if (W == 2) return go(dt, v, std::integral_constant<int, 2>{});
        if (W == 3) return go(dt, v, std::integral_constant<int, 3>{});
        return go(dt, v, std::integral_constant<int, 4>{});
    };
    using One = std::integral_constant<int, 1>;
    using Four = std::integral_constant<int, 4>;
    if (dtype == KDA_BF16) {
        using Bf = std::integral_constant<int, KDA_BF16>;
        if constexpr (MOST == 8)
            if (V == 8) return taps(Bf{}, std::integral_constant<int, 8>{});
        return V == 4 ? taps(Bf{}, Four{}) : taps(Bf{}, One{});
    }
    using F32 = std::integral_constant<int, KDA_F32>;
    return V == 4 ? taps(F32{}, Four{}) : taps(F32{}, One{});
}

}  // namespace

size_t conv_workspace_bytes(int32_t n_seqs, int64_t total, int32_t C, int32_t W) {
    const int64_t slots = std::max(run_slots(n_seqs, total, false), run_slots(n_seqs, total, true));
    return static_cast<size_t>(slots) * (W + 1) * C * 4;
}

hipError_t launch_conv_fwd(const ConvArgs& a, hipStream_t stream) {
    const int V = vector_width(a, nullptr, PROMPT);
    const Conv c = base(a, V);
    return by_kind<PROMPT>(a.dtype, V, a.W, [&](auto dt, auto v, auto w) {
        constexpr int W = decltype(w)::value;
        const int64_t blocks = int64_t(c.slots) * c.vblocks;
        const int64_t windows = c.hT ? (int64_t(c.n_seqs) * (W - 1) * c.nvec + 255) / 256 : 0;
        hipLaunchKernelGGL((conv_fwd_kernel<decltype(dt)::value, decltype(v)::value, W>),
                           dim3(static_cast<unsigned>(blocks + windows)), dim3(256), 0, stream, c,
                           static_cast<uint32_t>(blocks));
        return hipGetLastError();
    });
}

hipError_t launch_conv_bwd(const ConvArgs& a, hipStream_t stream) {
    const int V = vector_width(a, nullptr, PROMPT);
    const Conv c = base(a, V);
    const hipError_t e = by_kind<PROMPT>(a.dtype, V, a.W, [&](auto dt, auto v, auto w) {
        hipLaunchKernelGGL((conv_bwd_kernel<decltype(dt)::value, decltype(v)::value, decltype(w)::value>),
                           dim3(static_cast<unsigned>(int64_t(c.slots) * c.vblocks)), dim3(256), 0, stream, c);
        return hipGetLastError();
    });
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(conv_sum_kernel, dim3((a.C + 63) / 64, a.W + 1), dim3(256), 0, stream, c.part, c.slots, a.C, a.W,
                       a.dw, a.db);
    return hipGetLastError();
}

hipError_t launch_conv_step(const ConvArgs& a, void* windows, const int32_t* slots, int32_t N, int32_t n_slots,
                            hipStream_t stream) {
    const int V = vector_width(a, windows, STEP_ONE);
    const Conv c = base(a, V);
    const int32_t blocks = (c.nvec + 255) / 256;
    return by_kind<STEP_ONE>(a.dtype, V, a.W, [&](auto dt, auto v, auto w) {
        hipLaunchKernelGGL((conv_step_kernel<decltype(dt)::value, decltype(v)::value, decltype(w)::value>),
                           dim3(static_cast<unsigned>(int64_t(N) * blocks)), dim3(256), 0, stream, c,
                           static_cast<uint8_t*>(windows), slots, N, n_slots, blocks);
        return hipGetLastError();
    });
}

}  // namespace kda
