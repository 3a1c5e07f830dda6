// kv4_attention.cu -- attention of a few query tokens per sequence over the
// four-bit key/value cache.
//
// Query i of sequence b (Sq queries, the last ones of its len keys) sees keys
// j <= len - Sq + i: s_j = sm q.k^_j, o = sum_j softmax(s)_j v^_j, and the
// log-sum-exp of s.  A row that sees no key gets o = 0 and -inf.
//
// One warp per query row and head, one key at a time, everything in FP32.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>

#include "fsa_internal.h"
#include "kv4.cuh"
#include "mx_scale.cuh"

namespace fsa {
namespace {

struct Params {
    const uint16_t* q;
    const uint8_t* cache;
    const int* page_table;
    const int* seq_lens;
    uint16_t* o;
    float* lse;
    int64_t q_stride, num_pages;
    int B, Sq, Hq, Hkv, page_size, max_pages;
    float sm;
    unsigned int* err_word;
};

__device__ __forceinline__ float e2m1(uint32_t c) {
    const uint32_t e = (c >> 1) & 3u, m = c & 1u;
    const float a = e ? static_cast<float>(2u + m) * static_cast<float>(1u << (e - 1)) * 0.5f : 0.5f * m;
    return (c & 8u) ? -a : a;
}

template <int D>
__global__ void __launch_bounds__(128) kv4_attn_kernel(const Params p) {
    constexpr int kN = D / 32;  // d per lane: lane + 32 b
    constexpr Kv4Layout L = kv4_layout(D);
    const int lane = threadIdx.x & 31;
    const int64_t row = blockIdx.x * 4ll + (threadIdx.x >> 5);
    if (row >= static_cast<int64_t>(p.B) * p.Sq * p.Hq) return;
    const int h = static_cast<int>(row % p.Hq);
    const int64_t tok = row / p.Hq;
    const int i = static_cast<int>(tok % p.Sq), b = static_cast<int>(tok / p.Sq);
    const int hk = h / (p.Hq / p.Hkv);
    const int64_t cap = static_cast<int64_t>(p.max_pages) * p.page_size;
    int64_t len = p.seq_lens[b];
    if (len < 0 || len > cap) {
        if (lane == 0) atomicOr(p.err_word, kErrBadIndex);
        len = len < 0 ? 0 : cap;
    }
    const int64_t n = len - p.Sq + 1 + i;
    float q[kN], o[kN] = {}, m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int c = 0; c < kN; ++c)
        q[c] = __uint_as_float(static_cast<uint32_t>(p.q[tok * p.q_stride + h * D + 32 * c + lane]) << 16) * p.sm *
               1.4426950408889634f;
    const int kb = (lane >> 3) * (D / 8) + ((lane & 7) >> 1);
    const int vb = (lane >> 2) * (D / 16) + ((lane & 3) >> 1);
    for (int64_t j = 0; j < n; ++j) {
        const int page = p.page_table[static_cast<int64_t>(b) * p.max_pages + j / p.page_size];
        if (page < 0 || page >= p.num_pages) {
            if (lane == 0) atomicOr(p.err_word, kErrBadIndex);
            continue;
        }
        const int r = static_cast<int>(j % p.page_size);
        const uint8_t* g = p.cache + ((static_cast<int64_t>(page) * p.Hkv + hk) * (p.page_size / kKv4Group) + r / kKv4Group) *
                                         kv4_group_bytes(D);
        const int rr = r % kKv4Group;
        float s = 0.0f;
#pragma unroll
        for (int c = 0; c < kN; ++c)
            s += q[c] * e2m1(g[rr * L.row + kb + 4 * c] >> (4 * (lane & 1))) * pow2f(g[L.kscales + rr * L.srow + c] - 127);
        for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, x);
        const float mn = fmaxf(m, s), f = exp2f(m - mn), w = exp2f(s - mn);
        l = l * f + w;
        m = mn;
#pragma unroll
        for (int c = 0; c < kN; ++c)
            o[c] = o[c] * f + w * e2m1(g[L.vcodes + rr * L.row + vb + 2 * c] >> (4 * (lane & 1))) *
                                  pow2f(g[L.vscales + rr * L.srow + c] - 127);
    }
    for (int c = 0; c < kN; ++c) {
        const __nv_bfloat16 x = __float2bfloat16_rn(l > 0.0f ? o[c] / l : 0.0f);
        p.o[row * D + 32 * c + lane] = *reinterpret_cast<const uint16_t*>(&x);
    }
    if (p.lse && lane == 0) p.lse[row] = l > 0.0f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

}  // namespace

size_t kv4_attention_workspace_bytes(int, int, int, int, int, int, int) { return 0; }

cudaError_t launch_kv4_attention(const Kv4AttnLaunch& a, cudaStream_t st) {
    const Params p{static_cast<const uint16_t*>(a.q), a.cache, a.page_table, a.seq_lens, static_cast<uint16_t*>(a.o),
                   a.lse, a.q_stride, a.num_pages, a.B, a.Sq, a.Hq, a.Hkv, a.page_size, a.max_pages, a.sm_scale,
                   a.err_word};
    const int64_t rows = static_cast<int64_t>(a.B) * a.Sq * a.Hq;
    const unsigned grid = static_cast<unsigned>((rows + 3) / 4);
    if (a.D == 128)
        kv4_attn_kernel<128><<<grid, 128, 0, st>>>(p);
    else
        kv4_attn_kernel<64><<<grid, 128, 0, st>>>(p);
    return cudaGetLastError();
}

}  // namespace fsa
