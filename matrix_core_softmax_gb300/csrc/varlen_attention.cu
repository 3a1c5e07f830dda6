// varlen_attention.cu -- softmax attention over packed sequences of different
// lengths with grouped heads, optionally causal.
//
// Sequence b has the query rows cu_q[b] .. cu_q[b + 1] - 1 and the keys cu_k[b]
// .. cu_k[b + 1] - 1; with `causal` its query i sees keys j <= nk - nq + i (the
// queries are the last ones).  A row that sees no key gets o = 0 and -inf;
// rows outside every sequence are left as they were.
//
// One warp per query row and head, one key at a time, everything in FP32.
#include <cuda_bf16.h>

#include <cmath>

#include "fsa_internal.h"

namespace fsa {
namespace {

struct Params {
    const uint16_t *q, *k, *v;
    uint16_t* o;
    float* lse;
    const int *cu_q, *cu_k;
    int64_t q_stride, k_stride, v_stride;
    int B, Tq, Tk, Hq, Hkv, causal;
    float sm;
    unsigned int* err_word;
};

__device__ __forceinline__ float bf(uint16_t x) { return __uint_as_float(static_cast<uint32_t>(x) << 16); }

template <int D>
__global__ void __launch_bounds__(128) varlen_attn_kernel(const Params p) {
    constexpr int kN = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t row = blockIdx.x * 4ll + (threadIdx.x >> 5);
    if (blockIdx.x == 0)  // the first block looks at the bounds
        for (int b = threadIdx.x; b < p.B; b += blockDim.x)
            if (p.cu_q[b] < 0 || p.cu_q[b] > p.cu_q[b + 1] || p.cu_q[b + 1] > p.Tq || p.cu_k[b] < 0 ||
                p.cu_k[b] > p.cu_k[b + 1] || p.cu_k[b + 1] > p.Tk)
                atomicOr(p.err_word, kErrBadIndex);
    if (row >= static_cast<int64_t>(p.Tq) * p.Hq) return;
    const int h = static_cast<int>(row % p.Hq), tok = static_cast<int>(row / p.Hq);
    const int hk = h / (p.Hq / p.Hkv);
    int b = 0;
    while (b < p.B && !(tok >= p.cu_q[b] && tok < p.cu_q[b + 1])) ++b;
    if (b == p.B) return;
    const int q0 = p.cu_q[b], nq = p.cu_q[b + 1] - q0, k0 = p.cu_k[b], nk = p.cu_k[b + 1] - k0;
    if (k0 < 0 || k0 > p.cu_k[b + 1] || p.cu_k[b + 1] > p.Tk) return;
    const int n = p.causal ? nk - nq + 1 + (tok - q0) : nk;
    float q[kN], o[kN] = {}, m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int c = 0; c < kN; ++c)
        q[c] = bf(p.q[tok * p.q_stride + h * D + 32 * c + lane]) * p.sm * 1.4426950408889634f;
    for (int j = 0; j < n; ++j) {
        const uint16_t* kr = p.k + (k0 + j) * p.k_stride + hk * D + lane;
        const uint16_t* vr = p.v + (k0 + j) * p.v_stride + hk * D + lane;
        float s = 0.0f;
#pragma unroll
        for (int c = 0; c < kN; ++c) s += q[c] * bf(kr[32 * c]);
        for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, x);
        const float mn = fmaxf(m, s), f = exp2f(m - mn), w = exp2f(s - mn);
        l = l * f + w;
        m = mn;
#pragma unroll
        for (int c = 0; c < kN; ++c) o[c] = o[c] * f + w * bf(vr[32 * c]);
    }
    for (int c = 0; c < kN; ++c) {
        const __nv_bfloat16 x = __float2bfloat16_rn(l > 0.0f ? o[c] / l : 0.0f);
        p.o[row * D + 32 * c + lane] = *reinterpret_cast<const uint16_t*>(&x);
    }
    if (p.lse && lane == 0) p.lse[row] = l > 0.0f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

}  // namespace

cudaError_t launch_varlen_attention(const VarlenLaunch& a, cudaStream_t st) {
    const Params p{static_cast<const uint16_t*>(a.q), static_cast<const uint16_t*>(a.k), static_cast<const uint16_t*>(a.v),
                   static_cast<uint16_t*>(a.o), a.lse, a.cu_q, a.cu_k, a.q_stride, a.k_stride, a.v_stride, a.B, a.Tq, a.Tk,
                   a.Hq, a.Hkv, a.causal, a.sm_scale, a.err_word};
    const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(a.Tq) * a.Hq + 3) / 4);
    if (a.D == 128)
        varlen_attn_kernel<128><<<grid, 128, 0, st>>>(p);
    else
        varlen_attn_kernel<64><<<grid, 128, 0, st>>>(p);
    return cudaGetLastError();
}

}  // namespace fsa
