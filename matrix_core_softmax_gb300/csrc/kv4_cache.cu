// kv4_cache.cu -- writes bf16 keys and values into the four-bit cache and
// reads them back.
//
// Per token, head and 32-element block along D (the quantizer's rule): X the
// smallest integer with max |x| <= 6 * 2^X, clamped to [-127, 127] (-127 for
// a zero block), codes E2M1(x / 2^X) rounded to nearest even.
//
// Both kernels move each byte once: per token and head 4 D bytes of bf16 and
// 2 (D / 2 + D / 32) bytes of cache.  HBM-bound at length, launch-bound for a
// decoding step.  Four lanes take one row of K or of V; lane t holds
// d = 32 b + 8 t .. + 7 of every block b, which is both a contiguous 16-byte
// load per block (the quad covers the block's 64 bytes) and one contiguous
// 16-byte (D = 128) piece of the row's codes in the cache's order.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fsa_internal.h"
#include "kv4.cuh"
#include "mx_scale.cuh"
#include "sm100_ptx.cuh"

namespace fsa {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = kThreads / 4;  // tokens of a block, all of one head

// Byte address of the group and the row in it that slot s of head h lives in.
__device__ __forceinline__ int64_t group_of(int64_t s, int h, int H, int page_size, int gbytes, int* row) {
    const int64_t page = s / page_size;
    const int r = static_cast<int>(s - page * page_size);
    *row = r & (kKv4Group - 1);
    return ((page * H + h) * (page_size / kKv4Group) + (r / kKv4Group)) * gbytes;
}

// X + 127 of the scale rule for a block whose largest magnitude has the bf16
// pattern `amax`: e - 2, one more beyond 1.5 * 2^e (the 0x3F carries into the
// exponent from mantissa 0x41 on), at least 0 -- where every subnormal lands.
__device__ __forceinline__ uint32_t e2m1_scale_byte(uint32_t amax) {
    return static_cast<uint32_t>(max(static_cast<int>((amax + 0x3Fu) >> 7) - 2, 0));
}

// Eight bf16 values (four pairs) times f, rounded to E2M1 codes, value i in
// nibble i.  (f is a power of two and no product leaves FP32's normal range.)
__device__ __forceinline__ uint32_t e2m1x8(const uint32_t (&u)[4], float f) {
    float2 v[4];
    const float2 f2 = make_float2(f, f);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = __fmul2_rn(make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xFFFF0000u)), f2);
    uint32_t r;
    asm("{\n.reg .b8 a, b, c, d;\n"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
        "mov.b32 %0, {a, b, c, d};\n}"
        : "=r"(r)
        : "f"(v[0].x), "f"(v[0].y), "f"(v[1].x), "f"(v[1].y), "f"(v[2].x), "f"(v[2].y), "f"(v[3].x), "f"(v[3].y));
    return r;
}

template <int D>
__global__ void __launch_bounds__(kThreads) kv4_append_kernel(
    const uint16_t* __restrict__ k, const uint16_t* __restrict__ v, int64_t k_stride, int64_t v_stride,
    const int64_t* __restrict__ slots, int64_t T, int H, uint8_t* __restrict__ cache, int64_t capacity,
    int page_size, unsigned int* err_word) {
    constexpr int kB = D / 32;
    constexpr Kv4Layout L = kv4_layout(D);
    const bool is_v = blockIdx.y != 0;
    const int t = threadIdx.x & 3;
    const unsigned chunk = blockIdx.x / H;
    const int h = blockIdx.x - chunk * H;
    const int64_t tok = chunk * static_cast<int64_t>(kTokens) + (threadIdx.x >> 2);
    // a quad's four lanes take the same way through every branch, so the
    // shuffles below name the quad
    if (tok >= T) return;
    const int64_t s = __ldg(slots + tok);
    if (s < 0) return;
    if (s >= capacity) {
        if (t == 0) atomicOr(err_word, kErrBadIndex);
        return;
    }
    const uint16_t* src = (is_v ? v + tok * v_stride : k + tok * k_stride) + static_cast<int64_t>(h) * D + 8 * t;
    uint4 x[kB];
#pragma unroll
    for (int b = 0; b < kB; ++b) x[b] = __ldg(reinterpret_cast<const uint4*>(src + 32 * b));
    const unsigned quad = 0xFu << (threadIdx.x & 28);
    uint32_t w[kB], sc = 0;
#pragma unroll
    for (int b = 0; b < kB; ++b) {
        const uint32_t u[4] = {x[b].x, x[b].y, x[b].z, x[b].w};
        // magnitudes of bf16 values order like their bit patterns
        uint32_t m = max16x2(max16x2(u[0] & 0x7FFF7FFFu, u[1] & 0x7FFF7FFFu), max16x2(u[2] & 0x7FFF7FFFu, u[3] & 0x7FFF7FFFu));
        m = max16x2(m, __shfl_xor_sync(quad, m, 1));
        m = max16x2(m, __shfl_xor_sync(quad, m, 2));
        const uint32_t byte = e2m1_scale_byte(max(m & 0xFFFFu, m >> 16));
        w[b] = e2m1x8(u, __uint_as_float((254u - byte) << 23));
        sc |= byte << (8 * b);
    }
    int row;
    uint8_t* g = cache + group_of(s, h, H, page_size, kv4_group_bytes(D), &row);
    uint8_t* dst = g + (is_v ? L.vcodes : 0) + row * L.row + t * (D / 8);
    // a key row keeps the words in block order; in a value row the halves of a
    // word (four d each) belong to two quads, block after block
    if (D == 128) {
        uint4 o = make_uint4(w[0], w[1], w[kB - 2], w[kB - 1]);
        if (is_v)
            o = make_uint4(__byte_perm(w[0], w[1], 0x5410), __byte_perm(w[kB - 2], w[kB - 1], 0x5410),
                           __byte_perm(w[0], w[1], 0x7632), __byte_perm(w[kB - 2], w[kB - 1], 0x7632));
        *reinterpret_cast<uint4*>(dst) = o;
        if (t == 0) *reinterpret_cast<uint32_t*>(g + (is_v ? L.vscales : L.kscales) + row * L.srow) = sc;
    } else {
        uint2 o = make_uint2(w[0], w[1]);
        if (is_v) o = make_uint2(__byte_perm(w[0], w[1], 0x5410), __byte_perm(w[0], w[1], 0x7632));
        *reinterpret_cast<uint2*>(dst) = o;
        if (t == 0)
            *reinterpret_cast<uint16_t*>(g + (is_v ? L.vscales : L.kscales) + row * L.srow) = static_cast<uint16_t>(sc);
    }
}

// A pair of f16 values times sc, as packed bf16 (exact: two significant bits).
__device__ __forceinline__ uint32_t f16x2_scaled_bf16(uint32_t h2, float sc) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
    const __nv_bfloat162 r = __floats2bfloat162_rn(f.x * sc, f.y * sc);
    return *reinterpret_cast<const uint32_t*>(&r);
}

template <int D>
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(
    const uint8_t* __restrict__ cache, const int64_t* __restrict__ slots, int64_t T, int H,
    int64_t capacity, int page_size, uint16_t* __restrict__ k, uint16_t* __restrict__ v,
    int64_t k_stride, int64_t v_stride, unsigned int* err_word) {
    constexpr int kB = D / 32;
    constexpr Kv4Layout L = kv4_layout(D);
    const bool is_v = blockIdx.y != 0;
    const int t = threadIdx.x & 3;
    const unsigned chunk = blockIdx.x / H;
    const int h = blockIdx.x - chunk * H;
    const int64_t tok = chunk * static_cast<int64_t>(kTokens) + (threadIdx.x >> 2);
    if (tok >= T) return;
    const int64_t s = __ldg(slots + tok);
    uint32_t w[kB] = {}, sc = 0;
    if (s >= capacity && t == 0) atomicOr(err_word, kErrBadIndex);
    if (s >= 0 && s < capacity) {
        int row;
        const uint8_t* g = cache + group_of(s, h, H, page_size, kv4_group_bytes(D), &row);
        const uint8_t* src = g + (is_v ? L.vcodes : 0) + row * L.row + t * (D / 8);
        const uint8_t* ss = g + (is_v ? L.vscales : L.kscales) + row * L.srow;
        if (D == 128) {
            const uint4 o = __ldg(reinterpret_cast<const uint4*>(src));
            sc = __ldg(reinterpret_cast<const uint32_t*>(ss));
            w[0] = o.x; w[1] = o.y; w[kB - 2] = o.z; w[kB - 1] = o.w;
            if (is_v) {
                w[0] = __byte_perm(o.x, o.z, 0x5410); w[1] = __byte_perm(o.x, o.z, 0x7632);
                w[kB - 2] = __byte_perm(o.y, o.w, 0x5410); w[kB - 1] = __byte_perm(o.y, o.w, 0x7632);
            }
        } else {
            const uint2 o = __ldg(reinterpret_cast<const uint2*>(src));
            sc = __ldg(reinterpret_cast<const uint16_t*>(ss));
            w[0] = o.x; w[1] = o.y;
            if (is_v) { w[0] = __byte_perm(o.x, o.y, 0x5410); w[1] = __byte_perm(o.x, o.y, 0x7632); }
        }
    }
    uint16_t* dst = (is_v ? v + tok * v_stride : k + tok * k_stride) + static_cast<int64_t>(h) * D + 8 * t;
#pragma unroll
    for (int b = 0; b < kB; ++b) {
        uint32_t p[4];
        e2m1x8_to_f16(w[b], p);
        const float f = pow2f(static_cast<int>((sc >> (8 * b)) & 0xFFu) - 127);
        *reinterpret_cast<uint4*>(dst + 32 * b) =
            make_uint4(f16x2_scaled_bf16(p[0], f), f16x2_scaled_bf16(p[1], f), f16x2_scaled_bf16(p[2], f),
                       f16x2_scaled_bf16(p[3], f));
    }
}

// Blocks of the heads of one token chunk are neighbours, so a token's rows are
// read or written together.
dim3 grid_of(const Kv4Rows& a) { return dim3(static_cast<unsigned>((a.T + kTokens - 1) / kTokens * a.H), 2); }

}  // namespace

cudaError_t launch_kv4_append(const Kv4Rows& a, uint8_t* cache, cudaStream_t st) {
    const uint16_t* k = static_cast<const uint16_t*>(a.k);
    const uint16_t* v = static_cast<const uint16_t*>(a.v);
    const dim3 grid = grid_of(a);
    if (a.D == 128)
        kv4_append_kernel<128><<<grid, kThreads, 0, st>>>(k, v, a.k_stride, a.v_stride, a.slots, a.T, a.H, cache,
                                                          a.capacity, a.page_size, a.err_word);
    else
        kv4_append_kernel<64><<<grid, kThreads, 0, st>>>(k, v, a.k_stride, a.v_stride, a.slots, a.T, a.H, cache,
                                                         a.capacity, a.page_size, a.err_word);
    return cudaGetLastError();
}

cudaError_t launch_kv4_read(const Kv4Rows& a, const uint8_t* cache, cudaStream_t st) {
    uint16_t* k = static_cast<uint16_t*>(const_cast<void*>(a.k));
    uint16_t* v = static_cast<uint16_t*>(const_cast<void*>(a.v));
    const dim3 grid = grid_of(a);
    if (a.D == 128)
        kv4_read_kernel<128><<<grid, kThreads, 0, st>>>(cache, a.slots, a.T, a.H, a.capacity, a.page_size, k, v,
                                                        a.k_stride, a.v_stride, a.err_word);
    else
        kv4_read_kernel<64><<<grid, kThreads, 0, st>>>(cache, a.slots, a.T, a.H, a.capacity, a.page_size, k, v,
                                                       a.k_stride, a.v_stride, a.err_word);
    return cudaGetLastError();
}

}  // namespace fsa
