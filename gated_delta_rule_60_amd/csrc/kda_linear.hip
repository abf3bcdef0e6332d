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
    int32_t m_transposed;
};

// Token by token: one workgroup per (sequence, head), 256 lanes, lane t owns column t % DC of
// DA * DC / 256 state rows.  lam is carried as hi + lo: a rounded lam alone would shift the state by
// half an ulp per token the same way each time.
template <int DT, int ODT, int DA, int DC, bool BACK>
__global__ void __launch_bounds__(256) linear_token_kernel(Pass p) {
    constexpr int RG = 256 / DC, RPT = DA / RG;
    __shared__ float sa[DA], sb[DA], red[RG][DC];
    const int t = threadIdx.x, c = t % DC, rg = t / DC;
    const int32_t n = blockIdx.x / p.H, h = blockIdx.x % p.H;
    int64_t lo = n * p.T, hi = lo + p.T;
    if (p.cu) {
        const int64_t x = p.cu[n], y = p.cu[n + 1];
        lo = x < 0 ? 0 : (x > p.T ? p.T : x);
        hi = y < lo ? lo : (y > p.T ? p.T : y);
    }
    float m[RPT];
    const int64_t base = static_cast<int64_t>(blockIdx.x) * (DA * DC);
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int r = rg * RPT + i;
        m[i] = p.m_in ? p.m_in[base + (p.m_transposed ? c * DA + r : r * DC + c)] : 0.f;
    }
    float lam = 1.f, lam_lo = 0.f;
    if (lo < hi) {
        const double l = exp(static_cast<double>(p.g[h]));
        lam = static_cast<float>(l);
        lam_lo = static_cast<float>(l - static_cast<double>(lam));
    }
    for (int64_t i = lo; i < hi; ++i) {
        const int64_t row = (BACK ? hi - 1 - (i - lo) : i) * p.H + h;
        if (t < DA) {
            sa[t] = load_as_f32<DT>(p.a, row * DA + t);
            sb[t] = p.ub * load_as_f32<DT>(p.b, row * DA + t);
        }
        const float cc = load_as_f32<DT>(p.c, row * DC + c);
        __syncthreads();
        float acc = 0.f;
#pragma unroll
        for (int j = 0; j < RPT; ++j) {
            const int r = rg * RPT + j;
            if constexpr (!BACK) m[j] = __builtin_fmaf(m[j], lam_lo, m[j] * lam);
            m[j] = __builtin_fmaf(sb[r], cc, m[j]);
            acc = __builtin_fmaf(sa[r], m[j], acc);
            if constexpr (BACK) m[j] = __builtin_fmaf(m[j], lam_lo, m[j] * lam);
        }
        red[rg][c] = acc;
        __syncthreads();
        if (rg == 0) {
            float s = 0.f;
#pragma unroll
            for (int r = 0; r < RG; ++r) s += red[r][c];
            store_from_f32<ODT>(p.out, row * DC + c, p.so * s);
        }
    }
    if (p.m_out)
#pragma unroll
        for (int i = 0; i < RPT; ++i) p.m_out[base + (rg * RPT + i) * DC + c] = m[i];
}

template <int DT, int ODT, bool BACK>
hipError_t launch_pass(const Pass& p, int32_t da, int32_t dc, hipStream_t stream) {
    const dim3 grid(static_cast<unsigned>(p.n_seqs * p.H));
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, p);
        return hipGetLastError();
    };
    if (da == 128 && dc == 128) return go(linear_token_kernel<DT, ODT, 128, 128, BACK>);
    if (da == 128) return go(linear_token_kernel<DT, ODT, 128, 64, BACK>);
    if (dc == 128) return go(linear_token_kernel<DT, ODT, 64, 128, BACK>);
    return go(linear_token_kernel<DT, ODT, 64, 64, BACK>);
}

Pass base_pass(const LinearArgs& a) {
    Pass p{};
    p.g = a.g; p.cu = a.cu; p.T = a.T; p.n_seqs = a.n_seqs; p.H = a.H; p.so = 1.f; p.ub = 1.f;
    return p;
}

}  // namespace

size_t linear_workspace_bytes(int32_t, int64_t, int32_t, int32_t, int32_t, int32_t, bool) { return 0; }

hipError_t launch_linear_fwd(const LinearArgs& a, hipStream_t stream) {
    Pass p = base_pass(a);
    p.a = a.q; p.b = a.k; p.c = a.v; p.out = a.o; p.so = a.scale; p.m_in = a.h0; p.m_out = a.hT;
    if (a.in_dtype == KDA_BF16)
        return a.o_dtype == KDA_BF16 ? launch_pass<KDA_BF16, KDA_BF16, false>(p, a.dk, a.dv, stream)
                                     : launch_pass<KDA_BF16, KDA_F32, false>(p, a.dk, a.dv, stream);
    return a.o_dtype == KDA_BF16 ? launch_pass<KDA_F32, KDA_BF16, false>(p, a.dk, a.dv, stream)
                                 : launch_pass<KDA_F32, KDA_F32, false>(p, a.dk, a.dv, stream);
}

hipError_t launch_linear_bwd(const LinearArgs& a, hipStream_t stream) {
    Pass q = base_pass(a), k = q, v = q;
    q.a = a.d_o; q.b = a.v; q.c = a.k; q.out = a.dq; q.so = a.scale; q.m_in = a.h0; q.m_transposed = 1;
    k.a = a.v; k.b = a.d_o; k.c = a.q; k.out = a.dkk; k.ub = a.scale; k.m_in = a.dhT; k.m_transposed = 1;
    v.a = a.k; v.b = a.q; v.c = a.d_o; v.out = a.dvv; v.ub = a.scale; v.m_in = a.dhT; v.m_out = a.dh0;
    auto go = [&](auto fwd, auto back) {
        hipError_t e = fwd(q, a.dv, a.dk, stream);
        if (e == hipSuccess) e = back(k, a.dv, a.dk, stream);
        if (e == hipSuccess) e = back(v, a.dk, a.dv, stream);
        return e;
    };
    if (a.in_dtype == KDA_BF16) return go(launch_pass<KDA_BF16, KDA_BF16, false>, launch_pass<KDA_BF16, KDA_BF16, true>);
    return go(launch_pass<KDA_F32, KDA_F32, false>, launch_pass<KDA_F32, KDA_F32, true>);
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
