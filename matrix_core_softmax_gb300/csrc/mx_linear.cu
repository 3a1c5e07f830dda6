// mx_linear.cu -- y[t][n] = sum over k of x^[t][k] w^[n][k]: the product of
// activations and weights that are both in an MX format, on the block-scaled tensor
// cores, with FP32 sums and one rounding to bf16.
//
//   x E2M1, w E2M1   kind::mxf4      64 elements an instruction, both packed
//   x E4M3, w E2M1   kind::mxf8f6f4  32 elements; the copy spreads 16 four-bit codes
//                                    over 16 bytes of shared memory
//   x E4M3, w E4M3   kind::mxf8f6f4
//
// A step is 128 bytes of shared memory a row in each of them: 256 elements of K (two
// scale atoms) in the first, 128 (one) in the others, and four instructions.
//
// Few tokens are bound by the weights' way out of HBM (one token, 16384 x 16384: 25.0 us
// in four bits, 5.7 TB/s; 43.4 in eight, 6.4), small products by their start and end
// (3 us), many tokens by the tensor core and, when they keep on, by the power that it may
// draw (8192 x 16384 x 8192: 290 to 330 us in four bits, 6.7 to 7.6 PFLOP/s, 585 to 620 in
// eight, 3.5 to 3.8, by what a box allows; in one product of 4096 x 8192 x 8192 the tensor pipe
// is active for 85 and 92 % of the SMs' time).
#include <cuda_bf16.h>

#include "fsa_internal.h"
#include "mx_operand.cuh"
#include "sm100_ptx.cuh"

namespace fsa {
namespace {

enum Mode : int { X4W4 = 0, X8W4 = 1, X8W8 = 2 };

// ---- few tokens --------------------------------------------------------------
// The weights' rows are the accumulator's lanes and the tokens its columns, so that
// one token costs 16 columns and not 128 rows.  A CTA: 128 outputs of n_tok tokens,
// over its part of K; the `split` CTAs of a cluster add their sums up through
// distributed shared memory, each for its share of the outputs, in the order of
// their ranks.
constexpr int kSms = 152;
constexpr int kFixed = 8;           // (see mx_linear_plan)
// warps 0-3 output; 4, 5 copies of w and of x (one warp for both: 560 clocks a step); 6
// products; 7 copies of scales
constexpr int kThreads = 256;
constexpr int kWarpLoad = 4, kWarpLoadX = 5, kWarpMma = 6, kWarpScales = 7;
constexpr int kMaxStages = 12;
// Scales come for 512 elements of K at once, in a ring of their own, so that a step costs
// a warp one copy (some 150 clocks to issue, and 120 for a wait that is over).  Two slots
// held one token over weights in four bits up by 700 clocks a step.
constexpr int kSfAtoms = 4, kSfSlots = 4, kSfBytes = 2 * kSfAtoms * kAtomBytes;
constexpr int kSmemTwo = 112 * 1024, kSmemOne = 224 * 1024;  // of a CTA, two or one an SM
constexpr uint32_t kTmemCols = 256; // of two CTAs: all 512
constexpr uint32_t kColSf = 128;    // accumulator at 0, scales of slot s at 128 + 32 s
constexpr int kMaxSplit = 8;       // portable cluster
constexpr int kPartRow = 132;       // FP32 of a token's 128 outputs in shared memory, padded

struct Params {
    const uint8_t *xs, *ws;
    __nv_bfloat16* y;
    int64_t y_stride;
    int T, N, n_atoms, n_tok, split, stages, slots, t_tiles, vec;
    uint64_t timeout_ns;
    unsigned int* err_word;
    int skip;  // test use: stage 1 never arrives
};

struct Bars {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t sf_full[kSfSlots], sf_empty[kSfSlots];
    uint64_t done;
    uint32_t tmem_base;
    int abort;
};

constexpr int stage_atoms(int mode) { return mode == X4W4 ? 2 : 1; }
constexpr int stage_bytes(int n_tok) { return 128 * 128 + n_tok * 128; }

__device__ __forceinline__ void raise_abort(Bars& sm, const Params& p) {
    sm.abort = 1;
    atomicOr(p.err_word, kErrTimeout);
}

template <int kMode>
__global__ void __launch_bounds__(kThreads, 2)
    mx_linear_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w, const Params p) {
    extern __shared__ __align__(1024) uint8_t ring[];
    __shared__ Bars sm;
    constexpr int kAtoms = stage_atoms(kMode), kSfSteps = kSfAtoms / kAtoms;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // (dynamic shared memory begins behind `sm`; swizzled tiles want 1024 bytes)
    const uint32_t pad = (1024u - (smem_u32(ring) & 1023u)) & 1023u;
    uint8_t* w_tiles = ring + pad;
    uint8_t* x_tiles = w_tiles + p.stages * 16384;
    uint8_t* sf_tiles = x_tiles + p.stages * p.n_tok * 128;

    const int tile = blockIdx.x / p.split, rank = blockIdx.x - tile * p.split;
    const int n_tile = tile / p.t_tiles, t_tile = tile - n_tile * p.t_tiles;
    const int n0 = n_tile * 128, t0 = t_tile * p.n_tok;
    const int steps = (p.n_atoms + kAtoms - 1) / kAtoms;
    const int first = static_cast<int>(static_cast<int64_t>(steps) * rank / p.split);
    const int mine = static_cast<int>(static_cast<int64_t>(steps) * (rank + 1) / p.split) - first;

    // w's, or x's, part of step i of this CTA's into stage st (one lane)
    const bool is_x = warp == kWarpLoadX;
    auto load = [&](int i, int st) {
        // (a spread copy counts the bytes that it reads, 64 a row)
        mbar_arrive_expect_tx(&sm.full[st], is_x ? p.n_tok * 128 : 128 * (kMode == X8W4 ? 64 : 128));
        if (is_x)
            tma_load_2d(x_tiles + st * p.n_tok * 128, &tm_x, &sm.full[st], (first + i) * 128, t0);
        else
            tma_load_2d(w_tiles + st * 16384, &tm_w, &sm.full[st], (first + i) * 128, n0);
    };
    const int ahead = min(mine, p.stages);
    if (warp == kWarpLoad && lane == 0) {
        sm.abort = 0;
        for (int i = 0; i < p.stages; ++i) {
            mbar_init(&sm.full[i], i == 1 && p.skip ? 3 : 2);
            mbar_init(&sm.empty[i], 1);
        }
        for (int i = 0; i < p.slots; ++i) {
            mbar_init(&sm.sf_full[i], 1);
            mbar_init(&sm.sf_empty[i], 1);
        }
        mbar_init(&sm.done, 1);
        fence_mbar_init();
        grid_wait();
        for (int i = 0; i < ahead; ++i) load(i, i);  // (the other warps need not be there yet)
    }
    if (warp == kWarpMma) {
        tmem_alloc(&sm.tmem_base, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    grid_launch_next();  // (the next kernel's CTAs find this one's tensor memory taken)
    const uint32_t tmem = sm.tmem_base;
    bool ok = true;
    // give-up and exit of a loader: every copy lands before the CTA goes on, whoever gives
    // up and when (in a call that ends well they have landed)
    auto settle = [&](uint64_t* full, int stages, int issued) {
        if (!ok) raise_abort(sm, p);
        int dummy = 0;
        for (int i = max(0, issued - stages); i < issued; ++i) mbar_wait(full + i % stages, (i / stages) & 1, p.timeout_ns, &dummy);
    };

    if (warp == kWarpLoad || is_x) {
        if (lane == 0) {
            int st = 0, issued = 0;
            if (is_x) grid_wait();
            for (; issued < ahead; ++issued)
                if (is_x) load(issued, issued);  // (w's are under way)
            if (ahead < p.stages) st = ahead;
            uint32_t ph = 1;
            for (; issued < mine; ++issued) {
                ok = mbar_wait(&sm.empty[st], ph ^ 1u, p.timeout_ns, &sm.abort);
                if (!ok) break;
                load(issued, st);
                if (++st == p.stages) {
                    st = 0;
                    ph ^= 1u;
                }
            }
            settle(sm.full, p.stages, issued);
        }
    } else if (warp == kWarpScales) {
        if (lane == 0) {
            grid_wait();
            const int64_t at = static_cast<int64_t>(first) * kAtoms * kAtomBytes;
            const uint8_t* ws = p.ws + static_cast<int64_t>(n_tile) * p.n_atoms * kAtomBytes + at;
            const uint8_t* xs = p.xs + static_cast<int64_t>(t0 / 128) * p.n_atoms * kAtomBytes + at;
            const int atoms = min(mine * kAtoms, p.n_atoms - first * kAtoms);  // (the last step may hold one atom)
            int issued = 0, slot = 0;
            uint32_t ph = 1;
            for (int a = 0; a < atoms; a += kSfAtoms, ++issued) {
                if (issued >= p.slots) ok = mbar_wait(&sm.sf_empty[slot], ph, p.timeout_ns, &sm.abort);
                if (!ok) break;
                const uint32_t bytes = min(kSfAtoms, atoms - a) * kAtomBytes;
                uint8_t* dst = sf_tiles + slot * kSfBytes;
                mbar_arrive_expect_tx(&sm.sf_full[slot], 2 * bytes);
                bulk_load(dst, ws + static_cast<int64_t>(a) * kAtomBytes, bytes, &sm.sf_full[slot]);
                bulk_load(dst + kSfBytes / 2, xs + static_cast<int64_t>(a) * kAtomBytes, bytes, &sm.sf_full[slot]);
                if (++slot == p.slots) {
                    slot = 0;
                    ph ^= 1u;
                }
            }
            settle(sm.sf_full, p.slots, issued);
        }
    } else if (warp == kWarpMma) {
        const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
        const uint64_t dw = smem_desc(smem_u32(w_tiles), 16, 1024, SWZ_128B), dx = smem_desc(smem_u32(x_tiles), 16, 1024, SWZ_128B);
        const uint64_t dsf = smem_desc(smem_u32(sf_tiles), 0, 128, SWZ_NONE);
        const uint32_t id = kMode == X4W4 ? idesc_mxf8f6f4(128, p.n_tok, 1, 1, 0, 0)
                                          : idesc_mxf8f6f4(128, p.n_tok, kMode == X8W4 ? 5 : 0, 0, 0, 0);
        auto wait = [&](uint64_t* bar, uint32_t phase) {
            return __all_sync(0xFFFFFFFFu, mbar_wait(bar, phase & 1u, p.timeout_ns, &sm.abort)) != 0;
        };
        int st = 0, slot = 0;
        uint32_t ph = 0, sf_ph = 0;
        for (int i = 0; i < mine; ++i) {
            const int in = i % kSfSteps;
            if (in == 0) ok = wait(&sm.sf_full[slot], sf_ph);
            ok = ok && wait(&sm.full[st], ph);
            if (!ok) break;
            tc_fence_after();
            const uint32_t sfw = tm + kColSf + 8 * kSfAtoms * slot + 4 * kAtoms * in, sfx = sfw + 4 * kSfAtoms;
            const uint64_t sf = dsf + slot * (kSfBytes >> 4) + in * (kAtoms * kAtomBytes >> 4);
            const bool half = kAtoms == 2 && p.n_atoms - (first + i) * kAtoms == 1;
#pragma unroll
            for (int a = 0; a < kAtoms; ++a) {
                if (a && half) break;
                tc_cp_32x128b_x4_one(sfw + 4 * a, sf + a * (kAtomBytes >> 4));
                tc_cp_32x128b_x4_one(sfx + 4 * a, sf + (kSfAtoms + a) * (kAtomBytes >> 4));
            }
            const uint64_t aw = dw + st * (16384 >> 4), ax = dx + st * (p.n_tok * 128 >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                const uint32_t acc = (i > 0 || kk > 0) ? 1u : 0u;
                if constexpr (kMode == X4W4) {
                    if (kk >= 2 && half) break;
                    const uint32_t s = (kk & 1) * 2;  // scale bytes 0-1 or 2-3 of the atom
                    mma_mxf4_one(tm, aw + 2 * kk, ax + 2 * kk, id | s << 4 | s << 29, sfw + 4 * (kk >> 1), sfx + 4 * (kk >> 1), acc);
                } else {
                    mma_mxf8f6f4_one(tm, aw + 2 * kk, ax + 2 * kk, id | kk << 4 | static_cast<uint32_t>(kk) << 29, sfw, sfx, acc);
                }
            }
            tc_commit_one(&sm.empty[st]);
            if (in == kSfSteps - 1) {
                tc_commit_one(&sm.sf_empty[slot]);
                if (++slot == p.slots) {
                    slot = 0;
                    sf_ph ^= 1u;
                }
            }
            if (++st == p.stages) {
                st = 0;
                ph ^= 1u;
            }
        }
        if (!ok && lane == 0) raise_abort(sm, p);
        tc_commit_one(&sm.done);  // every product issued retires before its sums are read or TMEM is freed
        int dummy = 0;
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(&sm.done, 0, p.timeout_ns, &dummy)) && lane == 0) raise_abort(sm, p);
    }
    // (all copies have landed: the products that read them are done, or the loader waited)
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    float* part = reinterpret_cast<float*>(w_tiles);
    const int rows = min(p.n_tok, p.T - t0);
    if (warp < 4) {
        const uint32_t col = tmem + (static_cast<uint32_t>(32 * warp) << 16);
        const bool put = p.split == 1 && n0 + tid < p.N && !sm.abort;
        __nv_bfloat16* dst = p.y + t0 * p.y_stride + n0 + tid;
        for (int c = 0; c < rows; c += 16) {
            uint32_t v[16];
            tmem_ld16(col + c, v);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j) asm volatile("" : "+r"(v[j]));  // (not before the wait)
            if (p.split > 1) {
#pragma unroll
                for (int j = 0; j < 16; ++j) part[(c + j) * kPartRow + tid] = __uint_as_float(v[j]);
            } else if (put) {
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (c + j < rows) dst[(c + j) * p.y_stride] = __float2bfloat16_rn(__uint_as_float(v[j]));
            }
        }
    }
    tc_fence_before();
    __syncwarp();
    if (p.split > 1)
        cluster_sync();
    else
        __syncthreads();
    if (warp == kWarpMma) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
    if (p.split > 1 && !sm.abort) {
        // this CTA's share: 128 / split outputs of each token, four a thread
        const int lg = __ffs(32 / p.split) - 1;
        const uint32_t base = smem_u32(part);
        for (int e = tid; e < rows << lg; e += kThreads) {
            const int t = e >> lg, n = 4 * ((e & ((1 << lg) - 1)) + (rank << lg));
            if (n0 + n >= p.N) continue;
            // all parts asked for before the first is added (a load from another SM takes
            // some 600 clocks)
            float4 v[kMaxSplit];
#pragma unroll
            for (int r = 0; r < kMaxSplit; ++r)
                if (r < p.split) v[r] = ld_cluster_f4(mapa(base + 4 * (t * kPartRow + n), r));
            float4 s = v[0];
#pragma unroll
            for (int r = 1; r < kMaxSplit; ++r)
                if (r < p.split) s = make_float4(s.x + v[r].x, s.y + v[r].y, s.z + v[r].z, s.w + v[r].w);
            __nv_bfloat16* dst = p.y + (t0 + t) * p.y_stride + n0 + n;
            const __nv_bfloat162 lo = __floats2bfloat162_rn(s.x, s.y), hi = __floats2bfloat162_rn(s.z, s.w);
            if (p.vec && n0 + n + 4 <= p.N) {
                *reinterpret_cast<uint2*>(dst) =
                    make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
            } else {
                const __nv_bfloat16 v[4] = {lo.x, lo.y, hi.x, hi.y};
                for (int j = 0; j < 4 && n0 + n + j < p.N; ++j) dst[j] = v[j];
            }
        }
    }
    __syncwarp();
    if (p.split > 1) cluster_sync();  // no CTA leaves while another reads its sums
}

// ---- many tokens: pairs of CTAs --------------------------------------------
// Tokens are the accumulator's lanes here, so that a thread of the output holds
// neighbouring outputs of one token.  A pair of CTAs works on 256 tokens x 256
// outputs: each has 128 tokens' rows and half of the weights' in its shared memory
// and its tokens' sums in its tensor memory, so a step brings an SM 32 KB of codes for
// twice the operations that a 128 x 128 tile's 32 KB serve (8192 x 16384 x 8192 in 128 x
// 128 tiles, two CTAs an SM: 550 us in four bits, 941 in eight, 17 to 19 TB/s out of L2).
// An output tile leaves through registers, so that the next tile's products begin 450
// clocks after the last one's end.
//
// warps 0-7 output; 8, 9, 10 copies; 11 the products (rank 0).  The copies into either CTA's
// memory count on rank 0's barriers, so that the products' wait is for the copies themselves:
// a warp of rank 1 that waited and then told rank 0 would have to release to the cluster's
// scope, 1450 clocks a step.  (The barriers expect fixed bytes: scales come by tensor copies,
// too, which fill what is behind the matrix.  4096 x 5120 x 5120 in four bits 38.9 us, with
// word from rank 1 39.2.)
// An SM begins a copy every 110 clocks, whatever its size, where a step's products take 540,
// and a warp takes 150 to issue one and 120 for a wait that is over, so three warps share a
// step's copies (one for all 815 clocks a step of 256 outputs, three warps 545), each in a
// loop of its own (one loop that asks what to copy: 2048 x 5120 x 5120 in eight by four bits
// 32.2 -> 35.9 us).  Narrower tiles' products take less, so their scales come for 512
// elements of K at once, in a ring of their own (kRing; 512 x 5120 x 5120 in eight by four
// bits 16.5 -> 13.7 us); tiles of 256 outputs keep them in the stages, because the second wait
// holds the products up (in four bits 24.0 us for 1024 x 8192 x 8192, with the ring 25.5;
// 8192 x 16384 x 4096 in eight by four 282, 288).
constexpr int kPairThreads = 384;
constexpr int kPairLoadX = 8, kPairLoadW = 9, kPairLoadSf = 10, kPairMma = 11;
constexpr int kPairStages = 6, kPairSlots = 3;
constexpr int kPairSf = 3 * kPairSlots * kSfAtoms * kAtomBytes;  // scales: x, w's rows in two groups of 128
constexpr uint32_t kPairCols = 512;
constexpr uint32_t kPairColSf = 256;  // accumulator at 0, scales of slot s at 256 + 12 s times a slot's atoms
constexpr int kPairGroup = 8;         // token tiles that are walked side by side
static_assert(kPairSlots * kSfAtoms >= kPairStages * 2, "scales in the stages take the ring's room");

struct PairBars {
    uint64_t full[kPairStages];       // rank 0's: both CTAs' copies
    uint64_t empty[kPairStages];      // a commit of rank 0's products arrives in both
    uint64_t sf_full[kPairSlots], sf_empty[kPairSlots];  // the same of scales (kRing)
    uint64_t acc_full, acc_empty;     // (acc_empty: rank 0's, an arrival a warp of both CTAs' output)
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
};

constexpr int kOutBytes = 8 * 32 * 64;  // per output warp: 32 rows x 32 outputs on their way
constexpr int kPairSmem = kPairStages * 2 * 16384 + kPairSf + kOutBytes + static_cast<int>(sizeof(PairBars));
static_assert(kPairSmem <= 232448, "shared memory beyond the 227 KB a CTA may use");

// A place in a ring of n.
template <int n>
struct Turn {
    int at = 0;
    uint32_t ph = 0;
    __device__ __forceinline__ void next() {
        if (++at == n) {
            at = 0;
            ph ^= 1u;
        }
    }
};

struct PairParams {
    __nv_bfloat16* y;
    int64_t y_stride;
    int T, N, n_atoms, t_tiles, n_tiles, bn, vec;  // bn: outputs of a tile, 256, 192 or 128
    uint64_t timeout_ns;
    unsigned int* err_word;
    int skip;
};

// Token and output tile of number i: groups of kPairGroup token tiles, in a group
// token tiles first, so that the pairs at work share a square of the product.
__device__ __forceinline__ void pair_tile(const PairParams& p, int i, int& t_tile, int& n_tile) {
    const int per = kPairGroup * p.n_tiles, group = i / per, in = i - group * per;
    const int width = min(kPairGroup, p.t_tiles - group * kPairGroup);
    n_tile = in / width;
    t_tile = group * kPairGroup + in - n_tile * width;
}

template <int kMode, bool kRing>
__global__ void __launch_bounds__(kPairThreads, 1)
    mx_linear_pair_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                          const __grid_constant__ CUtensorMap tm_xs, const __grid_constant__ CUtensorMap tm_ws, const PairParams p) {
    extern __shared__ __align__(1024) uint8_t ring[];
    // the 128-byte-swizzled tiles need a 1024-byte aligned base (the same in both CTAs)
    if (smem_u32(ring) & 1023u) {
        if (threadIdx.x == 0) atomicOr(p.err_word, kErrMisaligned);
        return;
    }
    constexpr int kAtoms = stage_atoms(kMode);                           // of a step
    constexpr int kSlot = kRing ? kSfAtoms : kAtoms;                     // of a slot of scales
    constexpr int kSfSteps = kSlot / kAtoms, kSfGroup = kSlot * kAtomBytes;
    const int bn = kRing ? p.bn : 256;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_ctarank();
    const int first_tile = blockIdx.x >> 1, tile_step = gridDim.x >> 1, tiles = p.t_tiles * p.n_tiles;
    const int steps = (p.n_atoms + kAtoms - 1) / kAtoms;
    uint8_t* x_tiles = ring;
    uint8_t* w_tiles = x_tiles + kPairStages * 16384;
    uint8_t* sf_tiles = w_tiles + kPairStages * 16384;
    uint4* out = reinterpret_cast<uint4*>(sf_tiles + kPairSf);
    PairBars& sm = *reinterpret_cast<PairBars*>(out + kOutBytes / 16);

    if (tid == 0) {
        sm.abort = 0;
        for (int i = 0; i < kPairStages; ++i) {
            mbar_init(&sm.full[i], (kRing ? 2 : 3) + (i == 1 && p.skip));
            mbar_init(&sm.empty[i], 1);
        }
        for (int i = 0; i < kPairSlots; ++i) {
            mbar_init(&sm.sf_full[i], 1);
            mbar_init(&sm.sf_empty[i], 1);
        }
        mbar_init(&sm.acc_full, 1);
        mbar_init(&sm.acc_empty, 16);
        mbar_init(&sm.drain, 1);
        fence_mbar_init();
    }
    if (warp == kPairMma) pair_tmem_alloc(&sm.tmem_base, kPairCols);
    tc_fence_before();
    __syncthreads();
    // both CTAs' barriers are there behind the wait; rank 0's loaders only use their own CTA's
    cluster_arrive();
    const bool loader = warp >= kPairLoadX && warp <= kPairLoadSf, early = loader && rank == 0;
    if (!early) cluster_wait();
    tc_fence_after();
    grid_launch_next();  // (the next kernel's CTAs find this one's tensor memory taken)
    grid_wait();         // in all warps: the time of the kernel before is not their waits'
    const uint32_t tmem = sm.tmem_base;
    auto give_up = [&] {
        sm.abort = 1;
        atomicOr(p.err_word, kErrTimeout);
    };
    auto wait = [&](uint64_t* bar, uint32_t phase) {
        return __all_sync(0xFFFFFFFFu, mbar_wait_cluster(bar, phase & 1u, p.timeout_ns, &sm.abort)) != 0;
    };
    bool ok = true;
    Turn<kPairStages> st;
    Turn<kPairSlots> slot;

    if (loader) {
        if (lane == 0) {
            // copies of `per` scale atoms' part of K at once into n places, tile by tile; `bytes`:
            // those that they bring one CTA (a spread copy counts the 64 a row that it reads;
            // rows and scales behind the matrix come as zeros and count)
            auto fill = [&](uint64_t* full, uint64_t* empty, int n, int per, uint32_t bytes, auto copy) {
                const uint32_t full0 = mapa(smem_u32(full), 0);
                int issued = 0, at = 0;
                uint32_t ph = 1;
                for (int i = first_tile; ok && i < tiles; i += tile_step) {
                    int t_tile, n_tile;
                    pair_tile(p, i, t_tile, n_tile);
                    const int xg = 2 * t_tile + static_cast<int>(rank), n0 = bn * n_tile;
                    for (int a = 0; a < p.n_atoms; a += per, ++issued) {
                        if (issued >= n) ok = mbar_wait_cluster(&empty[at], ph, p.timeout_ns, &sm.abort);
                        if (!ok) break;
                        if (rank == 0) mbar_arrive_expect_tx(&full[at], 2 * bytes);
                        copy(at, full0 + 8 * at, a, xg, n0);
                        if (++at == n) {
                            at = 0;
                            ph ^= 1u;
                        }
                    }
                }
                if (!ok) give_up();
                // the products that read them are done before the CTA goes on; where they are
                // not because someone gave up, the copies have the waits' limit to land
                int dummy = 0;
                for (int i = max(0, issued - n); i < issued; ++i)
                    if (!mbar_wait_cluster(&empty[i % n], (i / n) & 1, p.timeout_ns, &dummy)) break;
            };
            constexpr int kSfWords = kAtomBytes / 8;
            auto x_scales = [&](int at, uint32_t bar, int a, int xg) {
                pair_tma_load_2d(sf_tiles + at * 3 * kSfGroup, &tm_xs, bar, a * kSfWords, xg);
            };
            auto w_scales = [&](int at, uint32_t bar, int a, int n0) {
                pair_tma_load_2d(sf_tiles + (at * 3 + 1) * kSfGroup, &tm_ws, bar, a * kSfWords, n0 / 128);
            };
            const int w_groups = bn > 128 ? 2 : 1;
            if (warp == kPairLoadX)
                fill(sm.full, sm.empty, kPairStages, kAtoms, 128 * 128 + (kRing ? 0 : kSfGroup), [&](int at, uint32_t bar, int a, int xg, int) {
                    pair_tma_load_2d(x_tiles + at * 16384, &tm_x, bar, a / kAtoms * 128, 128 * xg);
                    if (!kRing) x_scales(at, bar, a, xg);
                });
            else if (warp == kPairLoadW)
                fill(sm.full, sm.empty, kPairStages, kAtoms, bn / 2 * (kMode == X8W4 ? 64 : 128), [&](int at, uint32_t bar, int a, int, int n0) {
                    pair_tma_load_2d(w_tiles + at * 16384, &tm_w, bar, a / kAtoms * 128, n0 + bn / 2 * static_cast<int>(rank));
                });
            else if (kRing)
                fill(sm.sf_full, sm.sf_empty, kPairSlots, kSlot, (1 + w_groups) * kSfGroup, [&](int at, uint32_t bar, int a, int xg, int n0) {
                    x_scales(at, bar, a, xg);
                    w_scales(at, bar, a, n0);
                });
            else
                fill(sm.full, sm.empty, kPairStages, kAtoms, 2 * kSfGroup, [&](int at, uint32_t bar, int a, int, int n0) { w_scales(at, bar, a, n0); });
        }
    } else if (warp == kPairMma && rank == 0) {
        const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
        const uint64_t dx = smem_desc(smem_u32(x_tiles), 16, 1024, SWZ_128B), dw = smem_desc(smem_u32(w_tiles), 16, 1024, SWZ_128B);
        const uint64_t dsf = smem_desc(smem_u32(sf_tiles), 0, 128, SWZ_NONE);
        const uint32_t id = kMode == X4W4 ? idesc_mxf8f6f4(256, bn, 1, 1, 0, 0)
                                          : idesc_mxf8f6f4(256, bn, 0, kMode == X8W4 ? 5 : 0, 0, 0);
        uint32_t acc_ph = 1;  // (the first tile finds the accumulator empty)
        for (int i = first_tile; ok && i < tiles; i += tile_step, acc_ph ^= 1u) {
            if (i != first_tile) ok = wait(&sm.acc_empty, acc_ph);
            int t_tile, n_tile;
            pair_tile(p, i, t_tile, n_tile);
            // scales of a tile that begins inside a group, 32 rows a column (an odd column would
            // be a misaligned address: tiles begin at multiples of 64)
            const uint32_t skew = bn * n_tile % 128 / 32;
            for (int k = 0; ok && k < steps; ++k) {
                const int in = k % kSfSteps;
                if (kRing && in == 0) ok = wait(&sm.sf_full[slot.at], slot.ph);
                ok = ok && wait(&sm.full[st.at], st.ph);
                if (!ok) break;
                tc_fence_after();
                // scale columns of a slot: x's atoms, then for each atom both groups of w
                const int at = kRing ? slot.at : st.at;
                const uint32_t sfx = tm + kPairColSf + 12 * kSlot * at + 4 * kAtoms * in;
                const uint32_t sfw = tm + kPairColSf + 12 * kSlot * at + 4 * kSlot + 8 * kAtoms * in;
                const uint64_t sf = dsf + at * (3 * kSfGroup >> 4) + in * (kAtoms * kAtomBytes >> 4);
                const bool half = kAtoms == 2 && p.n_atoms - k * kAtoms == 1;
#pragma unroll
                for (int a = 0; a < kAtoms; ++a) {
                    if (a && half) break;
                    pair_cp_32x128b_x4_one(sfx + 4 * a, sf + a * (kAtomBytes >> 4));
                    pair_cp_32x128b_x4_one(sfw + 8 * a, sf + (kSlot + a) * (kAtomBytes >> 4));
                    if (bn > 128) pair_cp_32x128b_x4_one(sfw + 8 * a + 4, sf + (2 * kSlot + a) * (kAtomBytes >> 4));
                }
                const uint64_t ax = dx + st.at * (16384 >> 4), aw = dw + st.at * (16384 >> 4);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    const uint32_t acc = (k > 0 || kk > 0) ? 1u : 0u;
                    if constexpr (kMode == X4W4) {
                        if (kk >= 2 && half) break;
                        const uint32_t s = (kk & 1) * 2;
                        pair_mma_mxf4_one(tm, ax + 2 * kk, aw + 2 * kk, id | s << 4 | s << 29, sfx + 4 * (kk >> 1),
                                          sfw + 8 * (kk >> 1) + skew, acc);
                    } else {
                        pair_mma_mxf8f6f4_one(tm, ax + 2 * kk, aw + 2 * kk, id | kk << 4 | static_cast<uint32_t>(kk) << 29, sfx, sfw + skew,
                                              acc);
                    }
                }
                pair_commit_one(&sm.empty[st.at], 3);
                st.next();
                if (kRing && (in == kSfSteps - 1 || k + 1 == steps)) {
                    pair_commit_one(&sm.sf_empty[slot.at], 3);
                    slot.next();
                }
            }
            if (ok) pair_commit_one(&sm.acc_full, 3);
        }
        if (!ok && lane == 0) give_up();
        pair_commit_one(&sm.drain, 1);  // every product issued retires before anything is freed
        int dummy = 0;
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(&sm.drain, 0, p.timeout_ns, &dummy)) && lane == 0) give_up();
    } else if (warp < kPairLoadX) {
        // four warps for each half of the tile's outputs, 32 at a time
        const int half = bn / 2 * (warp >> 2), pieces = bn / 64;
        const uint32_t col = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + half;
        const uint32_t acc_empty = mapa(smem_u32(&sm.acc_empty), 0);
        uint4* mine = out + warp * 128;  // 32 rows x 4 pieces of 8 outputs
        uint32_t acc_ph = 0;
        for (int i = first_tile; i < tiles; i += tile_step, acc_ph ^= 1u) {
            ok = wait(&sm.acc_full, acc_ph);
            if (!ok) break;
            tc_fence_after();
            // sums into registers first: the next tile's products wait for no store
            uint32_t v[64];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                if (c >= pieces) break;
                uint32_t r[32];
                tmem_ld32(col + 32 * c, r);
                tmem_ld_wait();
                tmem_reg_dep(r);
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
                    v[16 * c + j] = *reinterpret_cast<const uint32_t*>(&b);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(acc_empty);
            int t_tile, n_tile;
            pair_tile(p, i, t_tile, n_tile);
            const int t0 = 256 * t_tile + 128 * static_cast<int>(rank) + 32 * (warp & 3), n0 = bn * n_tile + half;
            // through shared memory, so that a store covers eight rows' 64 bytes
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                if (c >= pieces) break;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    mine[4 * lane + (j ^ ((lane >> 1) & 3))] = make_uint4(v[16 * c + 4 * j], v[16 * c + 4 * j + 1], v[16 * c + 4 * j + 2],
                                                                         v[16 * c + 4 * j + 3]);
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int wr = 8 * j + (lane >> 2), t = t0 + wr, n = n0 + 32 * c + 8 * (lane & 3);
                    const uint4 u = mine[4 * wr + ((lane & 3) ^ ((wr >> 1) & 3))];
                    if (t < p.T && n < p.N) {
                        __nv_bfloat16* dst = p.y + t * p.y_stride + n;
                        if (p.vec && n + 8 <= p.N) {
                            *reinterpret_cast<uint4*>(dst) = u;
                        } else {
                            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                if (n + e < p.N)
                                    reinterpret_cast<uint16_t*>(dst)[e] = static_cast<uint16_t>(w[e / 2] >> (16 * (e & 1)));
                        }
                    }
                }
                __syncwarp();
            }
        }
        if (!ok && lane == 0) give_up();
    }
    tc_fence_before();
    __syncwarp();
    if (early) cluster_wait();
    cluster_sync();  // no CTA leaves while the other reads its memory or arrives at its barriers
    if (warp == kPairMma) {
        tc_fence_after();
        pair_tmem_dealloc(tmem, kPairCols);
    }
}

template <int kMode, bool kRing>
cudaError_t launch_pair(const MxLinearLaunch& a, int bn, cudaStream_t st) {
    static KernelSetup setup;
    cudaError_t e = setup(reinterpret_cast<const void*>(mx_linear_pair_kernel<kMode, kRing>), kPairSmem, 0);
    if (e != cudaSuccess) return e;
    PairParams p{};
    p.y = static_cast<__nv_bfloat16*>(a.y);
    p.y_stride = a.y_stride;
    p.T = a.T;
    p.N = a.N;
    p.n_atoms = static_cast<int>(mx_atoms(a.K));
    p.t_tiles = (a.T + 255) / 256;
    p.bn = bn;
    p.n_tiles = (a.N + bn - 1) / bn;
    p.vec = (reinterpret_cast<uintptr_t>(a.y) & 15) == 0 && a.y_stride % 8 == 0;
    p.timeout_ns = a.timeout_ns;
    p.err_word = a.err_word;
    p.skip = a.debug_flags & 1;
    const int tiles = p.t_tiles * p.n_tiles;
    return launch_early(mx_linear_pair_kernel<kMode, kRing>, 2 * (tiles < kSms / 2 ? tiles : kSms / 2), kPairThreads, kPairSmem, st, 2,
                        *a.tm_x, *a.tm_w, *a.tm_xs, *a.tm_ws, p);
}

// Tiles that run at once, each split between `split` CTAs of a cluster, one CTA or two an SM.
// A cluster stays within a group of SMs that are not all as many, so clusters of eight leave
// some SMs out (a token by 4096 columns in eight by four bits with one CTA an SM: 15 tiles
// split by 8 4.9 us, 16 tiles 8.1; 36 tiles split by 4 5.6, 37 tiles 8.4; 74 tiles split by 2
// 7.9, 75 tiles 12.0. With two an SM: 36 and 37 tiles 5.5 and 8.1; 74 and 75 7.6 and 12.2;
// 152 and 153 10.6 and 11.8).  GB300's numbers as constants: the split decides the order of a
// sum, which is not to depend on the chip at hand.  (cudaOccupancyMaxActiveClusters says the
// same there, but for 76 with two CTAs on SMs of their own, where 75 and 76 tiles take 8.4 us
// against 8.1 with two CTAs an SM.)
int64_t tiles_at_once(int split, int per_sm) {
    const int64_t one = split == 1 ? kSms : split == 2 ? 74 : split == 4 ? 36 : 15;
    const int64_t two = split == 1 ? 2 * kSms : split == 2 ? 152 : split == 4 ? 74 : 36;
    return per_sm == 1 ? one : two;
}

int mode_of(int x_elem, int w_elem) { return w_elem == ELEM_E4M3 ? X8W8 : x_elem == ELEM_E4M3 ? X8W4 : X4W4; }

template <int kMode>
cudaError_t launch(const MxLinearLaunch& a, Params p, int tiles, cudaStream_t st) {
    static KernelSetup setup;
    cudaError_t e = setup(reinterpret_cast<const void*>(mx_linear_kernel<kMode>), kSmemOne, 0);
    if (e != cudaSuccess) return e;
    const int smem = tiles <= tiles_at_once(p.split, 1) ? kSmemOne : kSmemTwo;
    // scales as far ahead as codes: a slot is two steps in four bits and four in eight
    for (p.slots = kMode == X4W4 || smem == kSmemOne ? kSfSlots : 2; p.slots >= 2; p.slots /= 2) {
        p.stages = (smem - 1024 - p.slots * kSfBytes) / stage_bytes(p.n_tok);
        if (p.stages >= 3) break;
    }
    if (p.stages > kMaxStages) p.stages = kMaxStages;
    return launch_early(mx_linear_kernel<kMode>, static_cast<unsigned>(tiles) * p.split, kThreads, smem, st, p.split, *a.tm_x,
                        *a.tm_w, p);
}

}  // namespace

MxLinearPlan mx_linear_plan(int T, int N, int K, int x_elem, int w_elem) {
    MxLinearPlan plan{};
    plan.w_rows = plan.x_rows = 128;
    // More than 128 tokens: 128 x 128 tiles where four CTAs to a tile run at once, one an SM,
    // pairs of CTAs otherwise (256 tokens by 4096 columns, 16 / 32 / 36 / 38 / 64 tiles: 7.7 /
    // 8.6 / 8.9 / 9.7 / 10.4 us against 9.7 / 9.8 / 9.8 / 9.8 / 10.0 in pairs in eight by four
    // bits, 6.8 / 7.6 / 7.9 / 8.2 / 8.9 against 7.5 / 7.6 / 7.5 / 7.5 / 7.8 in four bits).
    const int64_t tiles = mx_atoms(N) * mx_atoms(T);
    const int kAtoms = stage_atoms(mode_of(x_elem, w_elem));
    const int64_t steps = (mx_atoms(K) + kAtoms - 1) / kAtoms;
    if (T > 128 && tiles > tiles_at_once(4, 1)) {
        // Tiles of 256, 192 or 128 outputs, whichever take the fewest rounds of pairs' time
        // together (a step of fewer than 144 outputs is held up by its copies, a tile costs
        // two steps more).
        int64_t best = 0;
        for (int bn = 256; bn >= 128; bn -= 64) {
            const int64_t n = static_cast<int64_t>((T + 255) / 256) * ((N + bn - 1) / bn);
            const int64_t cost = (n + kSms / 2 - 1) / (kSms / 2) * (steps * (bn > 144 ? bn : 144) + 2 * 256);
            if (bn == 256 || cost < best) {
                best = cost;
                plan.w_rows = bn / 2;
            }
        }
        plan.sf_atoms = plan.w_rows == 128 ? kAtoms : kSfAtoms;
        plan.sf_rows = plan.w_rows == 64 ? 1 : 2;
        return plan;
    }
    if (T <= 128) plan.x_rows = (T + 15) / 16 * 16;
    // The time goes with the rounds of tiles (two CTAs an SM), times the steps of each and kFixed
    // more for its start and end; where two CTAs of an SM add up parts of K, the parts' way
    // through the SMs counts as a step for eight tokens (4096 outputs of 6144 columns in
    // eight by four bits, 1 / 64 / 128 tokens: split by 8, 256 CTAs, 6.4 / 10.2 / 13.9 us;
    // by 4 7.4 / 8.2 / 9.5; by 1 12.8 / 14.0 / 15.9).
    plan.split = 1;
    int64_t best = 0;
    for (int s = 1; s <= kMaxSplit && s <= steps; s *= 2) {
        int64_t cost = ((tiles - 1) / tiles_at_once(s, 2) + 1) * ((steps + s - 1) / s + kFixed);
        if (s > 1 && tiles > tiles_at_once(s, 1)) cost += plan.x_rows / 8;
        if (s == 1 || cost < best) {
            best = cost;
            plan.split = s;
        }
    }
    return plan;
}

cudaError_t launch_mx_linear(const MxLinearLaunch& a, const MxLinearPlan& plan, cudaStream_t st) {
    const int mode = mode_of(a.x_elem, a.w_elem);
    if (plan.split == 0) {
        const int bn = 2 * plan.w_rows;
        switch (mode) {
            case X4W4: return bn == 256 ? launch_pair<X4W4, false>(a, bn, st) : launch_pair<X4W4, true>(a, bn, st);
            case X8W4: return bn == 256 ? launch_pair<X8W4, false>(a, bn, st) : launch_pair<X8W4, true>(a, bn, st);
            default: return bn == 256 ? launch_pair<X8W8, false>(a, bn, st) : launch_pair<X8W8, true>(a, bn, st);
        }
    }
    Params p{};
    p.xs = a.xs;
    p.ws = a.ws;
    p.y = static_cast<__nv_bfloat16*>(a.y);
    p.y_stride = a.y_stride;
    p.T = a.T;
    p.N = a.N;
    p.n_atoms = static_cast<int>(mx_atoms(a.K));
    p.n_tok = plan.x_rows;
    p.split = plan.split;
    p.t_tiles = (a.T + p.n_tok - 1) / p.n_tok;
    p.vec = (reinterpret_cast<uintptr_t>(a.y) & 7) == 0 && a.y_stride % 4 == 0;
    p.timeout_ns = a.timeout_ns;
    p.err_word = a.err_word;
    p.skip = a.debug_flags & 1;
    const int tiles = static_cast<int>(mx_atoms(a.N)) * p.t_tiles;
    switch (mode) {
        case X4W4: return launch<X4W4>(a, p, tiles, st);
        case X8W4: return launch<X8W4>(a, p, tiles, st);
        default: return launch<X8W8>(a, p, tiles, st);
    }
}

}  // namespace fsa
