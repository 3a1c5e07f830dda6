// mx_operand.cu -- operands of the MX product: bf16 rows quantized into one, one
// read back as bf16, and the root-mean-square norm (with the residual's addition)
// that writes its output as one.
//
// All three move each byte once and are HBM-bound at length, launch-bound for a
// token.  A lane holds pieces of 8 elements (16 bytes of bf16), a quad a 32-element
// block, 16 lanes the four blocks whose scales are one word of an atom; a row
// belongs to 1 to 32 warps, by how many rows there are.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fsa.h"
#include "fsa_internal.h"
#include "mx_operand.cuh"
#include "sm100_ptx.cuh"

namespace fsa {
namespace {

constexpr int kSms = 152;
constexpr int kWarps = 8;   // warps of a block, unless a row has more
constexpr int kUnroll = 4;  // pieces that a lane has under way

// Elements 8 p .. 8 p + 7 of a row that starts on `align` (16, 8, 4 or 2) bytes, zeros
// from column `cols` on.  (Ordinary loads: the norm's sum may replace what it reads.)
__device__ __forceinline__ uint4 load8(const uint16_t* row, int p, int cols, int align) {
    if (8 * p + 8 <= cols) {
        const uint16_t* src = row + 8 * p;
        if (align == 16) return *reinterpret_cast<const uint4*>(src);
        if (align == 8) {
            const uint2 a = *reinterpret_cast<const uint2*>(src), b = *reinterpret_cast<const uint2*>(src + 4);
            return make_uint4(a.x, a.y, b.x, b.y);
        }
        if (align == 4) {
            const uint32_t* w = reinterpret_cast<const uint32_t*>(src);
            return make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    uint32_t h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = 8 * p + i < cols ? row[8 * p + i] : 0u;
    return make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
}

__device__ __forceinline__ void store8(uint16_t* row, int p, int cols, int align, uint4 u) {
    if (8 * p + 8 <= cols) {
        uint16_t* dst = row + 8 * p;
        if (align == 16) {
            *reinterpret_cast<uint4*>(dst) = u;
            return;
        }
        if (align == 8) {
            reinterpret_cast<uint2*>(dst)[0] = make_uint2(u.x, u.y);
            reinterpret_cast<uint2*>(dst)[1] = make_uint2(u.z, u.w);
            return;
        }
        if (align == 4) {
            uint32_t* w = reinterpret_cast<uint32_t*>(dst);
            w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
            return;
        }
    }
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (8 * p + i < cols) row[8 * p + i] = static_cast<uint16_t>(w[i / 2] >> (16 * (i & 1)));
}

__device__ __forceinline__ void widen(uint4 u, float (&v)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ void widen2(uint4 u, float2 (&v)[4]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}

__device__ __forceinline__ uint32_t pair_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// 2^lg warps a row.  Two at least for long rows, four in the way back (with one, blocks
// of 8 x 8192 elements leave SMs idle at the end: 8192 x 8192 in four bits 31.9 -> 28.6
// us, back 34.4 -> 27.2).
template <int kElem>
__global__ void __launch_bounds__(32 * kWarps) mx_pack_kernel(const uint16_t* x, int64_t stride, int64_t rows, int cols, int lg,
                                                              int align, uint8_t* codes, uint8_t* scales) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t r = blockIdx.x * static_cast<int64_t>(kWarps >> lg) + (warp >> lg);
    grid_launch_next();
    grid_wait();
    if (r >= rows) return;
    const int n_atoms = static_cast<int>(mx_atoms(cols)), step = 32 << lg;
    const uint16_t* row = x + r * stride;
    const MxRow out = mx_row<kElem>(codes, scales, r, n_atoms);
    // whole warps: every lane takes part in the shuffles
    for (int p0 = (warp & ((1 << lg) - 1)) * 32; p0 < 16 * n_atoms; p0 += kUnroll * step) {
        uint4 u[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) u[i] = load8(row, p0 + i * step + lane, cols, align);
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            if (p0 + i * step >= 16 * n_atoms) break;
            float2 v[4];
            widen2(u[i], v);
            mx_store8<kElem>(v, out, p0 + i * step + lane, cols, n_atoms);
        }
    }
}

// Rows of one 128-element piece: half a warp a row, kUnroll rows one after another.
template <int kElem>
__global__ void __launch_bounds__(32 * kWarps) mx_pack_short_kernel(const uint16_t* x, int64_t stride, int64_t rows, int cols,
                                                                    int align, uint8_t* codes, uint8_t* scales) {
    const int64_t half = blockIdx.x * static_cast<int64_t>(2 * kWarps) + (threadIdx.x >> 4);
    const int p = threadIdx.x & 15;
    grid_launch_next();
    grid_wait();
    uint4 u[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
        const int64_t r = half * kUnroll + i;
        u[i] = r < rows ? load8(x + r * stride, p, cols, align) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
        const int64_t r = half * kUnroll + i;
        float2 v[4];
        widen2(u[i], v);
        mx_store8<kElem>(v, mx_row<kElem>(codes, scales, r, 1), p, cols, r < rows ? 1 : 0);
    }
}

// Values of a piece: E2M1 and E4M3 are exact in f16, and f16 times a power of two in
// FP32; one rounding to bf16, which only a value below bf16's normal range needs.
template <int kElem>
__device__ __forceinline__ uint4 values8(uint2 c, uint32_t byte) {
    // 2^X, and 2^-127 (byte 0) as a subnormal; byte 255 is NaN
    const float f = byte == 0 ? __uint_as_float(0x00400000u) : byte == 255 ? __uint_as_float(0x7FC00000u) : __uint_as_float(byte << 23);
    uint32_t h[4];
    if constexpr (kElem == ELEM_E2M1) {
        asm("{\n.reg .b8 a, b, c, d;\n"
            "mov.b32 {a, b, c, d}, %4;\n"
            "cvt.rn.f16x2.e2m1x2 %0, a;\n"
            "cvt.rn.f16x2.e2m1x2 %1, b;\n"
            "cvt.rn.f16x2.e2m1x2 %2, c;\n"
            "cvt.rn.f16x2.e2m1x2 %3, d;\n}"
            : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(c.x));
    } else {
        asm("{\n.reg .b16 a, b, c, d;\n"
            "mov.b32 {a, b}, %4;\n"
            "mov.b32 {c, d}, %5;\n"
            "cvt.rn.f16x2.e4m3x2 %0, a;\n"
            "cvt.rn.f16x2.e4m3x2 %1, b;\n"
            "cvt.rn.f16x2.e4m3x2 %2, c;\n"
            "cvt.rn.f16x2.e4m3x2 %3, d;\n}"
            : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(c.x), "r"(c.y));
    }
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
        o[i] = pair_bf16(v.x * f, v.y * f);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// The codes and the scale byte of piece p of a row.  (Ordinary loads: the kernel before
// may still write them when this one begins.)
template <int kElem>
__device__ __forceinline__ uint32_t read8(const uint8_t* codes, const uint8_t* scales, int64_t r, int p, int n_atoms, uint2& c) {
    const uint8_t* src = codes + (r * n_atoms * 16 + p) * MxElem<kElem>::piece_bytes;
    if constexpr (kElem == ELEM_E2M1)
        c = make_uint2(*reinterpret_cast<const uint32_t*>(src), 0u);
    else
        c = *reinterpret_cast<const uint2*>(src);
    return scales[mx_scale_word(r, p >> 4, n_atoms) + ((p >> 2) & 3)];
}

template <int kElem>
__global__ void __launch_bounds__(32 * kWarps) mx_unpack_kernel(const uint8_t* codes, const uint8_t* scales, int64_t rows,
                                                                int cols, int lg, int align, uint16_t* out, int64_t stride) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t r = blockIdx.x * static_cast<int64_t>(kWarps >> lg) + (warp >> lg);
    grid_launch_next();
    grid_wait();
    if (r >= rows) return;
    const int n_atoms = static_cast<int>(mx_atoms(cols)), step = 32 << lg;
    uint16_t* row = out + r * stride;
    for (int p0 = (warp & ((1 << lg) - 1)) * 32 + lane; 8 * p0 < cols; p0 += kUnroll * step) {
        uint2 c[kUnroll];
        uint32_t s[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i)
            if (8 * (p0 + i * step) < cols) s[i] = read8<kElem>(codes, scales, r, p0 + i * step, n_atoms, c[i]);
#pragma unroll
        for (int i = 0; i < kUnroll; ++i)
            if (8 * (p0 + i * step) < cols) store8(row, p0 + i * step, cols, align, values8<kElem>(c[i], s[i]));
    }
}

// As mx_pack_short_kernel.
template <int kElem>
__global__ void __launch_bounds__(32 * kWarps) mx_unpack_short_kernel(const uint8_t* codes, const uint8_t* scales, int64_t rows,
                                                                      int cols, int align, uint16_t* out, int64_t stride) {
    const int64_t r0 = (blockIdx.x * static_cast<int64_t>(2 * kWarps) + (threadIdx.x >> 4)) * kUnroll;
    const int p = threadIdx.x & 15;
    grid_launch_next();
    grid_wait();
    if (8 * p >= cols) return;
    uint2 c[kUnroll];
    uint32_t s[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i)
        if (r0 + i < rows) s[i] = read8<kElem>(codes, scales, r0 + i, p, 1, c[i]);
#pragma unroll
    for (int i = 0; i < kUnroll; ++i)
        if (r0 + i < rows) store8(out + (r0 + i) * stride, p, cols, align, values8<kElem>(c[i], s[i]));
}

// h = x + residual, rounded to bf16.
__device__ __forceinline__ uint4 add8(uint4 x, uint4 d) {
    float2 u[4], v[4];
    widen2(x, u);
    widen2(d, v);
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 t = __fadd2_rn(u[i], v[i]);
        o[i] = pair_bf16(t.x, t.y);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// The 2^lg warps of a row wait for one another; rows of a block do not.
__device__ __forceinline__ void row_sync(int lg) {
    if (lg == 0)
        __syncwarp();
    else
        asm volatile("bar.sync %0, %1;" ::"r"(1 + (static_cast<int>(threadIdx.x) >> (5 + lg))), "r"(32 << lg) : "memory");
}

// Sum (or maximum) of s over the row's warps, the same in each of them.  `part`: a word
// a warp; it may be written again behind the row's next wait.
__device__ __forceinline__ float over_row(float s, bool most, int lg, float* part) {
    const int warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const float other = __shfl_xor_sync(0xFFFFFFFFu, s, o);
        s = most ? fmaxf(s, other) : s + other;
    }
    if (lg > 0) {
        if ((threadIdx.x & 31) == 0) part[warp] = s;
        row_sync(lg);
        const int w0 = warp & ~((1 << lg) - 1);
        s = 0.0f;  // (of squares or magnitudes: none is below)
        for (int w = 0; w < 1 << lg; ++w) s = most ? fmaxf(s, part[w0 + w]) : s + part[w0 + w];
    }
    return s;
}

// 1 / sqrt(m) within 2^-24 (1 + 2^-18) of itself, m far from either end of FP32: rsqrtf's r
// (within 2 units) and a step of Newton, r + r / 2 (1 - m r^2), m r in two parts.  The
// error of a root is a whole row's: rsqrtf alone put values on the wrong side of a border
// between two codes that a rounded root gets right (777 x 4096 in eight bits: 5.1e-5 off 64
// bits in the 2-norm, with this 4.8e-5).  16384 x 8192 takes 154 us with either, 156 with
// __frsqrt_rn.
__device__ __forceinline__ float root_inverse(float m) {
    const float r = rsqrtf(m), q = m * r, low = __fmaf_rn(m, r, -q);
    return __fmaf_rn(0.5f * r, __fmaf_rn(-low, r, __fmaf_rn(-q, r, 1.0f)), r);
}

// The norm of row r, whose h and gains this lane holds kV pieces of, into the operand;
// 2^lg warps a row.  `turn` alternates from row to row; `read` is called once all of
// the row's warps have h.
template <int kElem, int kV, class Read>
__device__ __forceinline__ void norm_row(const RmsNormMx& a, int64_t r, const uint4 (&h)[kV], const uint4 (&g)[kV], int lg,
                                         float (&part)[4][32], int turn, Read read) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int first = (warp & ((1 << lg) - 1)) * 32 + lane, step = 32 << lg;
    const int n_atoms = static_cast<int>(mx_atoms(a.cols));
    float2 acc = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < kV; ++i) {
        float2 v[4];
        widen2(h[i], v);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc = __ffma2_rn(v[j], v[j], acc);
    }
    float f = 1.0f, s = over_row(acc.x + acc.y, false, lg, part[turn]);
    read();
    // y = h (f inv) g with f = 1, except where squares leave FP32 (or get lost below it and
    // no larger eps covers them): there f is a power of two that brings the larger of the
    // row's maximum and sqrt(eps) near 1
    if (!(s <= 1e36f) || (s < 1e-25f && a.eps < 1e-12f)) {
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            float v[8];
            widen(h[i], v);
#pragma unroll
            for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(v[j]));
        }
        m = fmaxf(over_row(m, true, lg, part[2]), sqrtf(a.eps));
        // (2^-100 at least, so that f inv keeps its bits)
        f = __uint_as_float((254u - min(__float_as_uint(m) >> 23, 227u)) << 23);
        float t = 0.0f;
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            float v[8];
            widen(h[i], v);
#pragma unroll
            for (int j = 0; j < 8; ++j) t = __fmaf_rn(v[j] * f, v[j] * f, t);
        }
        s = over_row(t, false, lg, part[3]);
    }
    const float inv = f * root_inverse(s * a.inv_cols + a.eps * f * f);
    const float2 inv2 = make_float2(inv, inv);
    const MxRow out = mx_row<kElem>(a.codes, a.scales, r, n_atoms);
#pragma unroll
    for (int i = 0; i < kV; ++i) {
        const int p = first + i * step;
        if (p - lane >= 16 * n_atoms) break;  // (the whole warp is behind the row's end)
        float2 v[4], w[4];
        widen2(h[i], v);
        widen2(g[i], w);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = __fmul2_rn(__fmul2_rn(v[j], inv2), w[j]);
        mx_store8<kElem>(v, out, p, a.cols, n_atoms);
    }
}

// y = h / sqrt(mean(h^2) + eps) g of the sum h = bf16(x + residual), or of h = x,
// quantized.  A row's h stays in registers (bf16, as it is stored) between the sum
// of its squares and its output, so x and the residual are read once.  kV pieces a
// lane, 2^lg warps a row; kWide: a block of 32 warps for one row.
template <int kElem, int kV, bool kWide>
__global__ void __launch_bounds__(kWide ? 1024 : 512) rms_norm_mx_kernel(const RmsNormMx a, int lg) {
    __shared__ float part[4][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n_warps = blockDim.x >> 5;
    const int64_t r = blockIdx.x * static_cast<int64_t>(n_warps >> lg) + (warp >> lg);
    const int first = (warp & ((1 << lg) - 1)) * 32 + lane, step = 32 << lg;
    grid_launch_next();
    grid_wait();
    if (r >= a.rows) return;
    uint4 h[kV], g[kV];
    const uint16_t* x = static_cast<const uint16_t*>(a.x) + r * a.x_stride;
#pragma unroll
    for (int i = 0; i < kV; ++i) h[i] = load8(x, first + i * step, a.cols, a.x_align);
    if (a.residual) {
        const uint16_t* res = static_cast<const uint16_t*>(a.residual) + r * a.residual_stride;
        uint4 d[kV];
#pragma unroll
        for (int i = 0; i < kV; ++i) d[i] = load8(res, first + i * step, a.cols, a.residual_align);
        uint16_t* sum = static_cast<uint16_t*>(a.sum) + r * a.sum_stride;
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            h[i] = add8(h[i], d[i]);
            if (8 * (first + i * step) < a.cols) store8(sum, first + i * step, a.cols, a.sum_align, h[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < kV; ++i) g[i] = load8(static_cast<const uint16_t*>(a.gain), first + i * step, a.cols, a.gain_align);
    norm_row<kElem, kV>(a, r, h, g, lg, part, 0, [] {});
}

// The same for many rows that start on 16 bytes: the warps of a row stay and take every
// gridDim'th group's row, which bulk copies bring into a ring of shared memory ahead of
// them, so that the copies wait for no row's sum; the gains stay in registers.  (Its
// arguments are one word more than the other kernel's; as many, and it took 2 to 6 % longer:
// 65536 x 1024 55.5 us, with the word 51.6.)
constexpr int kMaxRing = 4;

template <int kElem, int kV, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads == 256 ? 3 : 1) rms_norm_mx_ring_kernel(const RmsNormMxLaunch a, int lg, int stages) {
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ float part[4][32];
    __shared__ uint64_t full[kMaxRing][kThreads / 32];
    __shared__ int gone;  // some row's copy did not arrive
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int per = (kThreads / 32) >> lg, mine = warp >> lg;  // rows of a group, this warp's
    const int first = (warp & ((1 << lg) - 1)) * 32 + lane, step = 32 << lg;
    const uint32_t row_bytes = 2 * a.cols;                      // (a multiple of 16)
    const uint32_t slot_bytes = row_bytes * (a.residual ? 2 : 1);
    const bool leader = lane == 0 && (warp & ((1 << lg) - 1)) == 0;  // of a row
    uint8_t* at = ring + mine * stages * slot_bytes;
    if (threadIdx.x == 0) {
        gone = 0;
        for (int i = 0; i < stages; ++i)
            for (int j = 0; j < per; ++j) mbar_init(&full[i][j], i == 1 && (a.debug_flags & FSA_DEBUG_SKIP_KV_ARRIVE) ? 2 : 1);
        fence_mbar_init();
    }
    grid_launch_next();
    __syncthreads();
    grid_wait();
    const int64_t hop = static_cast<int64_t>(per) * gridDim.x;
    int64_t r = static_cast<int64_t>(blockIdx.x) * per + mine;
    auto fetch = [&](int64_t r, int st) {
        if (r >= a.rows) return;
        uint8_t* dst = at + st * slot_bytes;
        uint64_t* bar = &full[st][mine];
        mbar_arrive_expect_tx(bar, slot_bytes);
        bulk_load(dst, static_cast<const uint16_t*>(a.x) + r * a.x_stride, row_bytes, bar);
        if (a.residual) bulk_load(dst + row_bytes, static_cast<const uint16_t*>(a.residual) + r * a.residual_stride, row_bytes, bar);
    };
    if (leader)
        for (int i = 0; i < stages; ++i) fetch(r + i * hop, i);
    uint4 g[kV];
#pragma unroll
    for (int i = 0; i < kV; ++i) g[i] = load8(static_cast<const uint16_t*>(a.gain), first + i * step, a.cols, a.gain_align);
    int st = 0, turn = 0;
    uint32_t ph = 0;
    bool lost = false;
    // test use: the place of the ring at which this lane gives up
    const int lose_at = (a.debug_flags & FSA_DEBUG_LOSE_ONE_WAIT) && lane == 31 && ((warp + 1) & ((1 << lg) - 1)) == 0 ? 1 : -1;
    for (; r < a.rows; r += hop) {
        // a copy that any lane gave up waiting for is reported, and the outputs from its row
        // on are undefined.  A leader that gives up fetches nothing more and waits for what
        // is in flight; one that does not goes on fetching, and waiting for, the rows of
        // lanes that did.  (The row's warps still meet, so that none waits for another.)
        if (!lost && (!mbar_wait(&full[st][mine], ph, a.timeout_ns, &gone) || st == lose_at)) {
            lost = true;
            gone = 1;
            atomicOr(a.err_word, kErrTimeout);
            int dummy = 0;
            for (int i = 0; leader && i < stages; ++i)
                if (r + i * hop < a.rows)
                    mbar_wait(&full[(st + i) % stages][mine], st + i < stages ? ph : ph ^ 1u, a.timeout_ns, &dummy);
        }
        __syncwarp();
        const uint8_t* src = at + st * slot_bytes;
        uint16_t* sum = static_cast<uint16_t*>(a.sum) + r * a.sum_stride;
        uint4 h[kV];
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const int p = first + i * step;
            h[i] = make_uint4(0, 0, 0, 0);
            if (8 * p < a.cols) {
                h[i] = *reinterpret_cast<const uint4*>(src + 16 * p);
                if (a.residual) {
                    h[i] = add8(h[i], *reinterpret_cast<const uint4*>(src + row_bytes + 16 * p));
                    store8(sum, p, a.cols, a.sum_align, h[i]);
                }
            }
        }
        norm_row<kElem, kV>(a, r, h, g, lg, part, turn, [&] {
            if (lg == 0) __syncwarp();
            if (leader && !lost) fetch(r + stages * hop, st);
        });
        turn ^= 1;
        if (++st == stages) {
            st = 0;
            ph ^= 1u;
        }
    }
}

// log2 of the warps for a row of `pieces` pieces, so that `rows` rows fill the GPU
// (kSms x 32 warps) as far as the row has work for them.
int warps_log2(int64_t rows, int64_t pieces, int most) {
    int lg = 0;
    while (lg < most && (rows << lg) < kSms * 32 && (int64_t{64} << lg) <= pieces) ++lg;
    return lg;
}

// The same for packing and reading back, whose rows are cut further, up to 2^least
// warps, as long as a warp keeps kUnroll pieces a lane.
int row_warps(int64_t rows, int cols, int least) {
    const int64_t pieces = 16 * mx_atoms(cols);
    int lg = warps_log2(rows, pieces, 3);
    while (lg < least && (int64_t{32} * kUnroll << (lg + 1)) <= pieces) ++lg;
    return lg;
}

// The largest of 16, 8, 4 and 2 bytes on which all rows start.
int row_align(const void* p, int64_t stride) {
    const uintptr_t bits = reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(2 * stride) | 16;
    return static_cast<int>(bits & -bits);
}

// Blocks an SM and stages of the ring for a stage of that many bytes; none: no ring.
struct NormRing {
    int blocks, stages, smem;
};
NormRing norm_ring(int64_t stage) {
    for (int blocks = 3; blocks >= 1; --blocks) {
        const int64_t room = (blocks == 3 ? 72 : blocks == 2 ? 110 : 222) * 1024;
        const int n = static_cast<int>(room / stage < kMaxRing ? room / stage : kMaxRing);
        if (n >= (blocks == 3 ? 2 : 3)) return {blocks, n, static_cast<int>(n * stage)};
    }
    return {0, 0, 0};
}

template <int kElem, int kV>
cudaError_t norm_launch(const RmsNormMxLaunch& a, int lg, cudaStream_t st) {
    const int warps = 1 << lg > kWarps ? 1 << lg : kWarps;
    const int64_t per = warps >> lg, groups = (a.rows + per - 1) / per;
    if (lg <= 4 && a.x_align == 16 && a.cols % 8 == 0 && (!a.residual || a.residual_align == 16)) {
        const NormRing ring = norm_ring(per * 2 * a.cols * (a.residual ? 2 : 1));
        const int blocks = warps == 8 ? ring.blocks : ring.blocks > 1 ? 1 : ring.blocks;
        if (blocks && groups >= 2 * kSms * blocks) {
            static KernelSetup small, large;
            const auto kernel = warps == 8 ? rms_norm_mx_ring_kernel<kElem, kV, 256> : rms_norm_mx_ring_kernel<kElem, kV, 512>;
            const cudaError_t e = (warps == 8 ? small : large)(reinterpret_cast<const void*>(kernel), 222 * 1024, 0);
            if (e != cudaSuccess) return e;
            return launch_early(kernel, kSms * blocks, 32 * warps, ring.smem, st, 1, a, lg, ring.stages);
        }
    }
    return launch_early(lg == 5 ? rms_norm_mx_kernel<kElem, kV, true> : rms_norm_mx_kernel<kElem, kV, false>,
                        static_cast<unsigned>(groups), 32 * warps, 0, st, 1, static_cast<const RmsNormMx&>(a), lg);
}

template <int kElem>
cudaError_t norm_pieces(const RmsNormMxLaunch& a, int lg, int v, cudaStream_t st) {
    switch (v) {
        case 1: return norm_launch<kElem, 1>(a, lg, st);
        case 2: return norm_launch<kElem, 2>(a, lg, st);
        case 3: return norm_launch<kElem, 3>(a, lg, st);
        default: return norm_launch<kElem, 4>(a, lg, st);
    }
}

}  // namespace

cudaError_t launch_mx_pack(const void* x, int64_t stride, int64_t rows, int cols, int elem, uint8_t* codes, uint8_t* scales,
                           cudaStream_t st) {
    const uint16_t* src = static_cast<const uint16_t*>(x);
    const int align = row_align(x, stride);
    if (cols <= 128 && rows >= kSms * 32) {
        const int64_t per = 2 * kWarps * kUnroll;
        return launch_early(elem == ELEM_E2M1 ? mx_pack_short_kernel<ELEM_E2M1> : mx_pack_short_kernel<ELEM_E4M3>,
                            static_cast<unsigned>((rows + per - 1) / per), 32 * kWarps, 0, st, 1, src, stride, rows, cols, align, codes,
                            scales);
    }
    const int lg = row_warps(rows, cols, 1);
    return launch_early(elem == ELEM_E2M1 ? mx_pack_kernel<ELEM_E2M1> : mx_pack_kernel<ELEM_E4M3>,
                        static_cast<unsigned>((rows + (kWarps >> lg) - 1) / (kWarps >> lg)), 32 * kWarps, 0, st, 1, src, stride, rows,
                        cols, lg, align, codes, scales);
}

cudaError_t launch_mx_unpack(const uint8_t* codes, const uint8_t* scales, int64_t rows, int cols, int elem, void* out,
                             int64_t stride, cudaStream_t st) {
    uint16_t* dst = static_cast<uint16_t*>(out);
    const int align = row_align(out, stride);
    if (cols <= 128 && rows >= kSms * 32) {
        const int64_t per = 2 * kWarps * kUnroll;
        return launch_early(elem == ELEM_E2M1 ? mx_unpack_short_kernel<ELEM_E2M1> : mx_unpack_short_kernel<ELEM_E4M3>,
                            static_cast<unsigned>((rows + per - 1) / per), 32 * kWarps, 0, st, 1, codes, scales, rows, cols, align, dst,
                            stride);
    }
    const int lg = row_warps(rows, cols, 2);
    return launch_early(elem == ELEM_E2M1 ? mx_unpack_kernel<ELEM_E2M1> : mx_unpack_kernel<ELEM_E4M3>,
                        static_cast<unsigned>((rows + (kWarps >> lg) - 1) / (kWarps >> lg)), 32 * kWarps, 0, st, 1, codes, scales, rows,
                        cols, lg, align, dst, stride);
}

cudaError_t launch_rms_norm_mx(const RmsNormMxLaunch& args, int elem, cudaStream_t st) {
    RmsNormMxLaunch a = args;
    a.x_align = row_align(a.x, a.x_stride);
    a.residual_align = row_align(a.residual, a.residual_stride);
    a.sum_align = row_align(a.sum, a.sum_stride);
    a.gain_align = row_align(a.gain, 0);
    a.inv_cols = 1.0f / static_cast<float>(a.cols);
    // up to four pieces a lane where the rows alone fill the GPU, fewer where they do
    // not; 32 warps take all of the 32768 columns a row may have
    const int64_t pieces = 16 * mx_atoms(a.cols);
    int lg = warps_log2(a.rows, pieces, 5);
    while (lg < 5 && (int64_t{4} * 32 << lg) < pieces) ++lg;
    const int v = static_cast<int>((pieces + (32 << lg) - 1) / (32 << lg));
    return elem == ELEM_E2M1 ? norm_pieces<ELEM_E2M1>(a, lg, v, st) : norm_pieces<ELEM_E4M3>(a, lg, v, st);
}

}  // namespace fsa
