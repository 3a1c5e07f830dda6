// mx_operand.cuh -- layout of a matrix in an MX format as an operand of
// fsa_mx_linear, and the arithmetic that writes one.
//
// Rows of K elements, E2M1 (two to a byte, low nibble first) or E4M3, in lines of
// `pitch` bytes that hold whole 128-element pieces (codes behind K are zero).  One
// E8M0 byte per 32 elements, in atoms of 128 rows x 4 blocks: 512 bytes that the
// tensor core's scale copy takes as they are.  Row r, block b: atom [r / 128][b / 4],
// byte (r % 32) 16 + (r % 128 / 32) 4 + b % 4.  Blocks behind K have scale 1; the
// bytes of rows behind the last one are nobody's (those rows are zeros by the copy's
// own bounds, and no output comes of them).
#pragma once
#include <cstdint>

#include "fsa_internal.h"
#include "sm100_ptx.cuh"

namespace fsa {

template <int kElem>
struct MxElem;
// X = e - emax, one more where the largest magnitude passes the largest element's
// mantissa: adding `carry` to the bits of an FP32 carries into the exponent there.
template <>
struct MxElem<ELEM_E2M1> {
    static constexpr int emax = 2;             // 6 = 1.5 * 2^2
    static constexpr uint32_t carry = 0x3FFFFF;
    static constexpr int piece_bytes = 4;      // codes of 8 elements
};
template <>
struct MxElem<ELEM_E4M3> {
    static constexpr int emax = 8;             // 448 = 1.75 * 2^8
    static constexpr uint32_t carry = 0x1FFFFF;
    static constexpr int piece_bytes = 8;
};

__host__ __device__ constexpr int64_t mx_atoms(int64_t n) { return (n + 127) / 128; }
__host__ __device__ constexpr int64_t mx_pitch(int64_t cols, int elem) {
    return mx_atoms(cols) * (elem == ELEM_E2M1 ? 64 : 128);
}

// Address of the four scale bytes of row r and 128-element piece a.
__device__ __forceinline__ int64_t mx_scale_word(int64_t r, int a, int n_atoms) {
    return ((r >> 7) * n_atoms + a) * kAtomBytes + (r & 31) * 16 + ((r & 127) >> 5) * 4;
}

// Quantizes the 8 values of this lane, which with the other three of its quad are a
// block (all four call it): the block's E8M0 byte, and the codes, element i in bits
// 4 i (E2M1) or 8 i (E4M3, two words).
// A block's scale is the least power of two 2^X with max |v| <= m 2^X, X in -127 ..
// 127; codes are v / 2^X (exact: a power of two, no product leaves FP32's range)
// rounded to the nearest element, ties to even.
template <int kElem>
__device__ __forceinline__ uint32_t mx_quantize8(const float2 (&v)[4], uint2& codes) {
    float m = fmaxf(fmaxf(fmaxf(fabsf(v[0].x), fabsf(v[0].y)), fmaxf(fabsf(v[1].x), fabsf(v[1].y))),
                    fmaxf(fmaxf(fabsf(v[2].x), fabsf(v[2].y)), fmaxf(fabsf(v[3].x), fabsf(v[3].y))));
    m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    const int e = static_cast<int>((__float_as_uint(m) + MxElem<kElem>::carry) >> 23) - MxElem<kElem>::emax;
    const uint32_t byte = static_cast<uint32_t>(max(e, 0));
    const float f = __uint_as_float((254u - byte) << 23);
    float2 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __fmul2_rn(v[i], make_float2(f, f));
    if constexpr (kElem == ELEM_E2M1) {
        asm("{\n.reg .b8 a, b, c, d;\n"
            "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n"
            "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
            "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n"
            "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
            "mov.b32 %0, {a, b, c, d};\n}"
            : "=r"(codes.x)
            : "f"(w[0].x), "f"(w[0].y), "f"(w[1].x), "f"(w[1].y), "f"(w[2].x), "f"(w[2].y), "f"(w[3].x), "f"(w[3].y));
        codes.y = 0;
    } else {
        codes.x = cvt_e4m3x4(w[0].x, w[0].y, w[1].x, w[1].y);
        codes.y = cvt_e4m3x4(w[2].x, w[2].y, w[3].x, w[3].y);
    }
    return byte;
}

// Where a row of an operand is: its codes, and the four scale bytes of its first piece.
struct MxRow {
    uint8_t *codes, *scales;
};
template <int kElem>
__device__ __forceinline__ MxRow mx_row(uint8_t* codes, uint8_t* scales, int64_t r, int n_atoms) {
    return {codes + r * (n_atoms * 16 * MxElem<kElem>::piece_bytes), scales + mx_scale_word(r, 0, n_atoms)};
}

// Quantizes and stores piece p (8 elements; 16 lanes in a row hold a 128-element
// piece, all of the warp calls it) of a row.
template <int kElem>
__device__ __forceinline__ void mx_store8(const float2 (&v)[4], MxRow row, int p, int cols, int n_atoms) {
    uint2 c;
    uint32_t byte = mx_quantize8<kElem>(v, c);
    if (8 * (p & ~3) >= cols) byte = 127u;  // a block behind the row's end
    uint32_t word = byte << (8 * ((p >> 2) & 3));
    word |= __shfl_xor_sync(0xFFFFFFFFu, word, 4);
    word |= __shfl_xor_sync(0xFFFFFFFFu, word, 8);
    if (p >= 16 * n_atoms) return;
    if constexpr (kElem == ELEM_E2M1)
        *reinterpret_cast<uint32_t*>(row.codes + 4 * p) = c.x;
    else
        *reinterpret_cast<uint2*>(row.codes + 8 * p) = c;
    if ((p & 15) == 0) *reinterpret_cast<uint32_t*>(row.scales + (p >> 4) * kAtomBytes) = word;
}

}  // namespace fsa
