// mx_scale.cuh -- the block scale rule of the MX element types (E8M0 scales:
// the smallest power of two 2^X with amax <= max_elem * 2^X), for the quantizer,
// and powers of two, for it and the four-bit key/value cache (whose kernels have
// the rule in a closed form for E2M1).
#pragma once
#include <cstdint>

#include "fsa_internal.h"

namespace fsa {

struct FmtConsts {
    int emax;       // exponent of the largest finite element
    uint32_t mthr;  // largest element = (1 + mthr / 128) * 2^emax in bf16 mantissa units
};

__device__ __forceinline__ FmtConsts fmt_consts(int elem) {
    if (elem == ELEM_E4M3) return {8, 0x60};  // 448 = 1.75 * 2^8
    if (elem == ELEM_E2M3) return {2, 0x70};  // 7.5 = 1.875 * 2^2
    return {2, 0x40};                         // 6   = 1.5 * 2^2
}

// Smallest integer X with amax <= max_elem * 2^X, clamped to [-127, 127];
// -127 for an all-zero block.  amax is given as the bit pattern of a
// non-negative bf16 (its magnitude bits, 15 bits).
__device__ __forceinline__ int mx_scale_exp(uint32_t amax_bf16, FmtConsts f) {
    if (amax_bf16 == 0) return -127;
    int E = static_cast<int>(amax_bf16 >> 7);
    uint32_t m = amax_bf16 & 0x7Fu;
    int e;
    if (E == 0) {  // bf16 subnormal: m * 2^-133, renormalise
        int nb = 32 - __clz(m);
        e = nb - 134;
        m = (m << (8 - nb)) & 0x7Fu;
    } else {
        e = E - 127;
    }
    int X = e - f.emax + (m > f.mthr ? 1 : 0);
    return min(127, max(-127, X));
}

// 2^-X as an FP32 (X in [-127, 126] for any bf16 block maximum).
__device__ __forceinline__ float pow2_neg(int X) {
    return __int_as_float((127 - X) << 23);
}

// 2^X as an FP32 for X in [-127, 127] (2^-127 is subnormal).
__device__ __forceinline__ float pow2f(int X) {
    return X >= -126 ? __int_as_float((127 + X) << 23) : __int_as_float(0x00400000);
}

}  // namespace fsa
