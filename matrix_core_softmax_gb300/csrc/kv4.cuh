// kv4.cuh -- layout of the four-bit key/value cache.
//
// A cache is [page][kv head][page_size / 32] groups of 32 keys of one head.
// A group is 34 D contiguous bytes:
//   key codes    32 rows of D / 2 bytes
//   value codes  32 rows of D / 2 bytes
//   key scales   32 rows of D / 32 E8M0 bytes (one per 32-element block)
//   value scales 32 rows of D / 32 E8M0 bytes
// so that one bulk copy brings everything a warp needs for 32 keys.  Codes are
// E2M1, two to a byte, low nibble first.  Inside a row the bytes follow the
// A fragments of a 16 x 8 x 16 tensor-core product, so that a lane finds its
// part of a row in one contiguous piece:
//   key row:   byte t (D / 8) + 4 b + j holds d = 32 b + 8 t + 2 j and d + 1
//              (t < 4: the lane of its quad; b: the block; j < 4);
//   value row: byte g (D / 16) + 2 b + j holds d = 32 b + 4 g + 2 j and d + 1
//              (g < 8: the quad; j < 2).
#pragma once
#include <cstdint>

namespace fsa {

constexpr int kKv4Group = 32;  // keys of a group

__host__ __device__ constexpr int kv4_group_bytes(int D) { return kKv4Group * (D + D / 16); }

struct Kv4Layout {  // byte offsets inside a group
    int vcodes, kscales, vscales, row, srow;
};
__host__ __device__ constexpr Kv4Layout kv4_layout(int D) {
    return {kKv4Group * D / 2, kKv4Group * D, kKv4Group * (D + D / 32), D / 2, D / 32};
}

// Packed unsigned 16-bit maximum.
__device__ __forceinline__ uint32_t max16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Eight E2M1 codes of a word to four f16 pairs (exact); pair i from byte i.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&r)[4]) {
    asm("{\n.reg .b8 a, b, c, d;\n"
        "mov.b32 {a, b, c, d}, %4;\n"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n}"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(w));
}

}  // namespace fsa
