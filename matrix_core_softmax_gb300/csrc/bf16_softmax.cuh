// bf16_softmax.cuh -- row arithmetic of the softmax warps of the BF16
// attention kernels: maxima, masks and exponentials of 32 scores of a row held
// in registers.
#pragma once
#include <cstdint>

#include "sm100_ptx.cuh"

namespace fsa {

__device__ __forceinline__ float fmax3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Maximum of 32 raw scores (three-input max in a depth-4 tree).
__device__ __forceinline__ float max32(const uint32_t (&v)[32]) {
    float a[11];
#pragma unroll
    for (int i = 0; i < 10; ++i)
        a[i] = fmax3(__uint_as_float(v[3 * i]), __uint_as_float(v[3 * i + 1]), __uint_as_float(v[3 * i + 2]));
    a[10] = fmaxf(__uint_as_float(v[30]), __uint_as_float(v[31]));
    return fmax3(fmax3(fmax3(a[0], a[1], a[2]), fmax3(a[3], a[4], a[5]), fmax3(a[6], a[7], a[8])), a[9],
                 a[10]);
}

__device__ __forceinline__ void mask32(uint32_t (&v)[32], int n_valid) {
#pragma unroll
    for (int j = 0; j < 32; ++j)
        if (j >= n_valid) v[j] = 0xFF800000u;
}

// p = 2^(s c - m) for 32 scores, packed to 16 bf16 pairs in w; returns their FP32 sum.
__device__ __forceinline__ float exp32(const uint32_t (&v)[32], float c, float m, uint32_t (&w)[16]) {
    const float2 c2 = make_float2(c, c), nm2 = make_float2(-m, -m);
    float2 acc = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float2 x = __ffma2_rn(make_float2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), c2, nm2);
        const float2 pp = make_float2(ex2(x.x), ex2(x.y));
        acc = __fadd2_rn(acc, pp);
        w[i] = bf16x2(pp.x, pp.y);
    }
    return acc.x + acc.y;
}

__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

}  // namespace fsa
