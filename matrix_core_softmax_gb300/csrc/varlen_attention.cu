// varlen_attention.cu -- softmax attention over packed sequences of different
// lengths with grouped heads, optionally causal, on tcgen05.
//
// Sequence b has the query rows cu_q[b] .. cu_q[b + 1] - 1 and the keys cu_k[b]
// .. cu_k[b + 1] - 1; with `causal` its query i sees keys j <= nk - nq + i (the
// queries are the last ones).  A row that sees no key gets o = 0 and -inf;
// rows outside every sequence are left as they were.
//
// A CTA owns two query tiles of one key head.  A tile is 128 rows: 128 / G
// whole tokens times the G query heads that share the key head, so a key tile
// brought in once serves every head of the group and short prompts still fill
// rows.  Both tiles work on the same 128-key tiles, which halves the K and V
// traffic out of L2 against one tile a CTA (64 KB per 128 x 128 tile pair of
// products, at the full tensor rate more than L2 delivers).
//
//   warps 0-3 / 4-7  softmax of tile 0 / tile 1 (thread = row = TMEM lane);
//   warp 8           TMA of Q and the K ring; warp 10 of the V ring;
//   warp 9           TMEM allocator and the issuer of every product.
// TMEM: S0, S1 (128 columns each, P overlays the first 64 of its S in bf16),
// O0, O1 (D columns each).
//
// The products of one thread run in the order of issue:
//   Q0 K(0), Q1 K(0), then per key tile t
//   P0 V(t), Q0 K(t+1), P1 V(t), Q1 K(t+1)
// so while one tile's softmax works on its scores the other tile's two products
// run.  A score product's commit also says that the tile's P V before it has
// finished, so between s_full and p_full a softmax thread owns its row of O and
// may rescale it: that happens only when the running maximum is passed by more
// than 2^8 (weights up to 2^8 are exact enough in bf16, sums are FP32).
//
// Exponentials: 128 x 128 per tile and product pair are 512 clocks of the
// SFU (32 a clock and SM, measured) against 1024 clocks of the tensor core at
// D = 128, 512 at D = 64.
#include <cuda_bf16.h>

#include <cmath>

#include "bf16_softmax.cuh"
#include "fsa_internal.h"
#include "sm100_ptx.cuh"

namespace fsa {
namespace {

constexpr int kKStages = 2, kVStages = 2;
constexpr int kThreads = 384;
constexpr int kWarpLoad = 8, kWarpMma = 9, kWarpLoadV = 10;
// launched at 168 registers per thread; helpers drop to 32, softmax takes 232
constexpr int kLaunchRegs = 168, kSoftmaxRegs = 232, kHelperRegs = 40;
static_assert(2 * 128 * kSoftmaxRegs + 128 * kHelperRegs <= kThreads * kLaunchRegs,
              "register split exceeds the launch allocation");
constexpr int kAtom = 128 * 128;       // 128 rows x 128 bytes (64 bf16)
constexpr int kTileBytes = 2 * kAtom;  // 128 rows x 128 bf16
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 256;        // S0 at 0, S1 at 128, O0 at 256, O1 at 384
constexpr float kNoMax = -1e30f;
constexpr float kLag = 8.0f;           // how far the reference may lag behind the maximum (log2)

struct __align__(1024) Smem {
    uint8_t q[2][kTileBytes];
    uint8_t k[kKStages][kTileBytes];
    uint8_t v[kVStages][kTileBytes];
    uint64_t bar_q;
    uint64_t k_full[kKStages], k_empty[kKStages];
    uint64_t v_full[kVStages], v_empty[kVStages], v_clean[kVStages];
    uint64_t s_full[2], p_full[2], o_full[2];
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
    int scan[kThreads / 32];
    int first_bad;
    int seq, tile;  // this CTA's sequence (-1: none) and pair of tiles in it
};

static_assert(sizeof(Smem) <= 232448, "shared memory beyond the 227 KB a CTA may use");

struct Params {
    __nv_bfloat16* o;
    float* lse;
    const int *cu_q, *cu_k;
    unsigned int* err_word;
    int B, Tq, Tk, Hq, Hkv, G, n_tok, causal;  // n_tok: tokens of a query tile
    float c;  // sm_scale * log2(e)
    uint64_t timeout_ns;
};

__device__ __forceinline__ void raise_abort(Smem& sm, const Params& p) {
    sm.abort = 1;
    atomicOr(p.err_word, kErrTimeout);
}

// Finds the sequence and the pair of query tiles of CTA number `idx`: sequence
// after sequence, the last pair (the longest one when causal) first.  Sequences
// from the first wrong bound on have none.
__device__ __forceinline__ void find_work(Smem& sm, const Params& p, int idx, bool report) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (p.B + kThreads - 1) / kThreads;
    const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
    const int rows = 2 * p.n_tok;
    int bad = p.B, sum = 0;
    int q0 = b0 < p.B ? __ldg(p.cu_q + b0) : 0, k0 = b0 < p.B ? __ldg(p.cu_k + b0) : 0;
    for (int b = b0; b < b1; ++b) {
        const int q1 = __ldg(p.cu_q + b + 1), k1 = __ldg(p.cu_k + b + 1);
        if (q0 < 0 || q1 < q0 || q1 > p.Tq || k0 < 0 || k1 < k0 || k1 > p.Tk) bad = min(bad, b);
        if (b < bad) sum += (q1 - q0 + rows - 1) / rows;
        q0 = q1;
        k0 = k1;
    }
    if (bad < p.B) atomicMin(&sm.first_bad, bad);
    int inc = sum;
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += x;
    }
    if (lane == 31) sm.scan[warp] = inc;
    __syncthreads();
    int before = inc - sum;
    for (int w = 0; w < warp; ++w) before += sm.scan[w];
    // counts of threads behind the first wrong bound are off, but their
    // sequences are behind it, too
    if (idx >= before && idx < before + sum) {
        int b = b0, at = before;
        int q = __ldg(p.cu_q + b);
        while (true) {
            const int q1 = __ldg(p.cu_q + b + 1);
            const int n = (q1 - q + rows - 1) / rows;
            if (idx < at + n) {
                if (b < sm.first_bad) {
                    sm.seq = b;
                    sm.tile = n - 1 - (idx - at);
                }
                break;
            }
            at += n;
            q = q1;
            ++b;
        }
    }
    if (tid == 0 && report && sm.first_bad < p.B) atomicOr(p.err_word, kErrBadIndex);
}

// One key tile t for this thread's row: scores out of TMEM, the maximum, the
// rare rescale of O, P back into TMEM.  `lim`: keys the row sees in all;
// `masked`: some row of the tile sees less than this whole key tile.
template <int D>
__device__ __forceinline__ bool softmax_tile(Smem& sm, const Params& p, int t, int i, uint32_t s_col, uint32_t o_col, int lim,
                                             bool masked, float& m, float& l) {
    const bool ok = mbar_wait(&sm.s_full[i], t & 1, p.timeout_ns, &sm.abort);
    tc_fence_after();
    uint32_t s0[32], s1[32], s2[32], s3[32];
    float top;
#ifdef FSA_HAVE_TMEM_REDUCE
    if (!masked) {
        float r0, r1, r2, r3;
        tmem_ld32_red<true>(s_col, s0, r0);
        tmem_ld32_red<true>(s_col + 32, s1, r1);
        tmem_ld32_red<true>(s_col + 64, s2, r2);
        tmem_ld32_red<true>(s_col + 96, s3, r3);
        tmem_ld_wait();
        tmem_reg_dep(s0);
        tmem_reg_dep(s1);
        tmem_reg_dep(s2);
        tmem_reg_dep(s3);
        tmem_reg_dep1(r0);
        tmem_reg_dep1(r1);
        tmem_reg_dep1(r2);
        tmem_reg_dep1(r3);
        top = fmaxf(fmax3(r0, r1, r2), r3);
    } else
#endif
    {
        tmem_ld32(s_col, s0);
        tmem_ld32(s_col + 32, s1);
        tmem_ld32(s_col + 64, s2);
        tmem_ld32(s_col + 96, s3);
        tmem_ld_wait();
        tmem_reg_dep(s0);
        tmem_reg_dep(s1);
        tmem_reg_dep(s2);
        tmem_reg_dep(s3);
        if (masked) {
            const int n_valid = lim - t * kTile;
            mask32(s0, n_valid);
            mask32(s1, n_valid - 32);
            mask32(s2, n_valid - 64);
            mask32(s3, n_valid - 96);
        }
        top = fmaxf(fmaxf(max32(s0), max32(s1)), fmaxf(max32(s2), max32(s3)));
    }
    top *= p.c;
    const bool grew = top > m + kLag;
    if (__any_sync(0xFFFFFFFFu, grew)) {
        const float mn = grew ? top : m;
        const float f = ex2(m - mn);
        l *= f;
        m = mn;
        if (t > 0) {  // O holds the tiles before t
            uint32_t rr[32];
            for (int c = 0; c < D / 32; ++c) {
                tmem_ld32(o_col + 32 * c, rr);
                tmem_ld_wait();
                tmem_reg_dep(rr);
#pragma unroll
                for (int j = 0; j < 32; ++j) rr[j] = __float_as_uint(__uint_as_float(rr[j]) * f);
                tmem_st32(o_col + 32 * c, rr);
            }
        }
    }
    uint32_t lo[32], hi[32];
    {
        uint32_t w0[16], w1[16];
        l += exp32(s0, p.c, m, w0);
        l += exp32(s1, p.c, m, w1);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            lo[j] = w0[j];
            lo[16 + j] = w1[j];
        }
        tmem_st32(s_col, lo);
        l += exp32(s2, p.c, m, w0);
        l += exp32(s3, p.c, m, w1);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            hi[j] = w0[j];
            hi[16 + j] = w1[j];
        }
        tmem_st32(s_col + 32, hi);
    }
    tmem_st_wait();
    tc_fence_before();
    warp_arrive(&sm.p_full[i]);
    return __all_sync(0xFFFFFFFFu, ok);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    varlen_attn_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const Params p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    // the 128-byte-swizzled TMA/MMA tiles need a 1024-byte aligned base
    if (smem_u32(smem_raw) & 1023u) {
        if (threadIdx.x == 0) atomicOr(p.err_word, kErrMisaligned);
        return;
    }
    Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    constexpr int n_atoms = D / 64;
    const int idx = blockIdx.x / p.Hkv, hk = blockIdx.x - idx * p.Hkv;

    if (tid == 0) {
        sm.abort = 0;
        sm.first_bad = p.B;
        sm.seq = -1;
        mbar_init(&sm.bar_q, 1);
        for (int i = 0; i < kKStages; ++i) {
            mbar_init(&sm.k_full[i], 1);
            mbar_init(&sm.k_empty[i], 1);
        }
        for (int i = 0; i < kVStages; ++i) {
            mbar_init(&sm.v_full[i], 1);
            mbar_init(&sm.v_empty[i], 1);
            mbar_init(&sm.v_clean[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.s_full[i], 1);
            mbar_init(&sm.p_full[i], 4);  // one arrival per softmax warp
            mbar_init(&sm.o_full[i], 1);
        }
        mbar_init(&sm.drain, 1);
        fence_mbar_init();
    }
    __syncthreads();
    find_work(sm, p, idx, blockIdx.x == 0);
    if (warp == kWarpMma) {
        tmem_alloc(&sm.tmem_base, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;
    const int b = sm.seq;

    if (b >= 0) {
        const int q0 = __ldg(p.cu_q + b), nq = __ldg(p.cu_q + b + 1) - q0;
        const int k0 = __ldg(p.cu_k + b), nk = __ldg(p.cu_k + b + 1) - k0;
        const int tok0 = sm.tile * 2 * p.n_tok;  // first token of the pair in its sequence
        // key tiles of query tile i: those that its last token sees
        int n_t[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int first = tok0 + i * p.n_tok, last = min(first + p.n_tok, nq) - 1;
            const int see = first >= nq ? 0 : p.causal ? min(nk, max(0, nk - nq + 1 + last)) : nk;
            n_t[i] = (see + kTile - 1) / kTile;
        }
        const int n_max = max(n_t[0], n_t[1]);  // (a missing second tile has none)
        const int t_ragged = (nk % kTile) ? nk / kTile : -1;  // key tile that ends inside, if any

        if (warp == kWarpLoad || warp == kWarpLoadV) {
            warpgroup_reg_dec<kHelperRegs>();
            const bool is_k = warp == kWarpLoad;
            const int stages = is_k ? kKStages : kVStages;
            uint64_t* full = is_k ? sm.k_full : sm.v_full;
            uint64_t* empty = is_k ? sm.k_empty : sm.v_empty;
            const CUtensorMap* map = is_k ? &tm_k : &tm_v;
            bool ok = true;
            bool q_issued = false;
            int issued = 0, st = 0;
            uint32_t ph = 0;
            if (lane == 0 && is_k && n_max > 0) {
                const int n_q = n_t[1] > 0 ? 2 : 1;
                mbar_arrive_expect_tx(&sm.bar_q, n_q * n_atoms * p.G * p.n_tok * 128);
                for (int i = 0; i < n_q; ++i)
                    for (int a = 0; a < n_atoms; ++a)
                        tma_load_3d(sm.q[i] + a * kAtom, &tm_q, &sm.bar_q, 64 * a, hk * p.G, q0 + tok0 + i * p.n_tok);
                q_issued = true;
            }
            for (int t = 0; t < n_max; ++t) {
                if (t >= stages) ok = mbar_wait(&empty[st], ph ^ 1u, p.timeout_ns, &sm.abort);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                uint8_t* dst = is_k ? sm.k[st] : sm.v[st];
                if (lane == 0) {
                    mbar_arrive_expect_tx(&full[st], kAtom * n_atoms);
                    for (int a = 0; a < n_atoms; ++a) tma_load_3d(dst + a * kAtom, map, &full[st], 64 * a, hk, k0 + t * kTile);
                }
                issued = t + 1;
                if (!is_k && t == t_ragged) {
                    // the rows behind the sequence's last key belong to others: a
                    // weight of zero does not hide a NaN, so they become zeros
                    ok = __all_sync(0xFFFFFFFFu, mbar_wait(&full[st], ph, p.timeout_ns, &sm.abort));
                    if (!ok) break;
                    const int r0 = nk - t * kTile;
                    for (int a = 0; a < n_atoms; ++a)
                        for (int e = r0 * 8 + lane; e < kTile * 8; e += 32)
                            reinterpret_cast<uint4*>(dst + a * kAtom)[e] = make_uint4(0, 0, 0, 0);
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.v_clean[st]);
                }
                if (++st == stages) {
                    st = 0;
                    ph ^= 1u;
                }
            }
            if (lane == 0) {
                if (!ok) raise_abort(sm, p);
                if (sm.abort) {
                    // let the copies still in flight land before the CTA exits
                    int dummy = 0;
                    if (q_issued) mbar_wait(&sm.bar_q, 0, p.timeout_ns, &dummy);
                    for (int t = max(0, issued - stages); t < issued; ++t)
                        mbar_wait(&full[t % stages], (t / stages) & 1, p.timeout_ns, &dummy);
                }
            }
        } else if (warp == kWarpMma) {
            warpgroup_reg_dec<kHelperRegs>();
            if (n_max > 0) {
                // the whole warp walks this, one elected lane issues.  Descriptors:
                // + 2 advances a K-major operand by one 16-element K step, + kAtom /
                // 16 by one swizzle atom; V is MN-major, 64-wide d atoms kAtom apart
                // (LBO), 8-key groups 1024 apart (SBO), one 16-key step 2048 bytes
                constexpr uint32_t id_qk = idesc_bf16(128, 128, 0, 0), id_pv = idesc_bf16(128, D, 0, 1);
                const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
                const uint64_t dq = smem_desc(smem_u32(sm.q[0]), 16, 1024, SWZ_128B);
                const uint64_t dk = smem_desc(smem_u32(sm.k[0]), 16, 1024, SWZ_128B);
                const uint64_t dv = smem_desc(smem_u32(sm.v[0]), kAtom, 1024, SWZ_128B);
                auto scores = [&](int i, int t) {
                    const uint64_t a = dq + (kTileBytes >> 4) * i, bk = dk + (kTileBytes >> 4) * (t % kKStages);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t off = (kk >> 2) * (kAtom >> 4) + 2 * (kk & 3);
                        mma_bf16_one(tm + 128 * i, a + off, bk + off, id_qk, kk > 0 ? 1u : 0u);
                    }
                    tc_commit_one(&sm.s_full[i]);
                };
                auto values = [&](int i, int t) {
                    const uint64_t bv = dv + (kTileBytes >> 4) * (t % kVStages);
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        mma_bf16_tmem_a_one(tm + kColO + 128 * i, tm + 128 * i + 8 * kk, bv + 128 * kk, id_pv,
                                            (t > 0 || kk > 0) ? 1u : 0u);
                };
                auto wait = [&](uint64_t* bar, int phase) {
                    return __all_sync(0xFFFFFFFFu, mbar_wait(bar, phase & 1, p.timeout_ns, &sm.abort)) != 0;
                };
                bool ok = wait(&sm.bar_q, 0) && wait(&sm.k_full[0], 0);
                if (ok) {
                    tc_fence_after();
                    if (n_t[0] > 0) scores(0, 0);
                    if (n_t[1] > 0) scores(1, 0);
                    tc_commit_one(&sm.k_empty[0]);
                }
                for (int t = 0; ok && t < n_max; ++t) {
                    bool have_v = false, have_k = false;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        if (!ok || t >= n_t[i]) continue;
                        ok = wait(&sm.p_full[i], t);
                        if (ok && !have_v) {
                            ok = wait(&sm.v_full[t % kVStages], t / kVStages) &&
                                 (t != t_ragged || wait(&sm.v_clean[t % kVStages], 0));
                            have_v = true;
                        }
                        if (!ok) continue;
                        tc_fence_after();
                        values(i, t);
                        if (t + 1 == n_t[i]) {
                            tc_commit_one(&sm.o_full[i]);
                            continue;
                        }
                        if (!have_k) {
                            ok = wait(&sm.k_full[(t + 1) % kKStages], (t + 1) / kKStages);
                            have_k = true;
                            if (!ok) continue;
                            tc_fence_after();
                        }
                        scores(i, t + 1);
                    }
                    if (!ok) break;
                    tc_commit_one(&sm.v_empty[t % kVStages]);
                    if (t + 1 < n_max) tc_commit_one(&sm.k_empty[(t + 1) % kKStages]);
                }
                if (!ok) {
                    if (lane == 0) raise_abort(sm, p);
                    int dummy = 0;
                    tc_commit_one(&sm.drain);  // wait until every product issued has retired
                    mbar_wait(&sm.drain, 0, p.timeout_ns, &dummy);
                }
            }
        } else if (warp < 8) {
            warpgroup_reg_inc<kSoftmaxRegs>();
            const int i = warp >> 2, r = tid & 127;
            const uint32_t lane_addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
            const uint32_t s_col = lane_addr + 128 * i, o_col = lane_addr + kColO + 128 * i;
            const int first = tok0 + i * p.n_tok;
            const int tl = r / p.G, h = r - tl * p.G, tok = first + tl;
            const bool row_valid = tl < p.n_tok && tok < nq;
            // keys that this row and the tile's first row see
            const int lim = p.causal ? min(nk, nk - nq + 1 + tok) : nk;
            const int lim0 = p.causal ? min(nk, nk - nq + 1 + first) : nk;
            float m = kNoMax, l = 0.0f;
            bool ok = true;
            for (int t = 0; ok && t < n_t[i]; ++t)
                ok = softmax_tile<D>(sm, p, t, i, s_col, o_col, lim, (t + 1) * kTile > lim0, m, l);
            if (ok && n_t[i] > 0) ok = __all_sync(0xFFFFFFFFu, mbar_wait(&sm.o_full[i], 0, p.timeout_ns, &sm.abort));
            if (!ok) raise_abort(sm, p);
            if (ok && first < nq) {
                const int64_t row = static_cast<int64_t>(q0 + tok) * p.Hq + hk * p.G + h;
                const float inv = l == 0.0f ? 0.0f : 1.0f / l;
                tc_fence_after();
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t rr[32];
                    if (n_t[i] > 0) {
                        tmem_ld32(o_col + 32 * c, rr);
                        tmem_ld_wait();
                        tmem_reg_dep(rr);
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j) rr[j] = 0u;
                    }
                    if (row_valid) {
                        uint32_t packed[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            packed[j] = bf16x2(__uint_as_float(rr[2 * j]) * inv, __uint_as_float(rr[2 * j + 1]) * inv);
                        uint4* dst = reinterpret_cast<uint4*>(p.o + row * D + 32 * c);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            dst[j] = make_uint4(packed[4 * j], packed[4 * j + 1], packed[4 * j + 2], packed[4 * j + 3]);
                    }
                }
                if (row_valid && p.lse) p.lse[row] = l == 0.0f ? -INFINITY : (m + __log2f(l)) * 0.6931471805599453f;
            }
        } else {
            warpgroup_reg_dec<kHelperRegs>();
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == kWarpMma) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

template <int D>
cudaError_t launch(const VarlenLaunch& a, const Params& p, cudaStream_t st) {
    const size_t smem = sizeof(Smem);
    // the in-kernel register split assumes exactly kLaunchRegs per thread at
    // launch; anything else could make the increase wait forever
    static KernelSetup setup;
    const cudaError_t e = setup(reinterpret_cast<const void*>(varlen_attn_kernel<D>), static_cast<int>(smem), kLaunchRegs);
    if (e != cudaSuccess) return e;
    // a sequence of n tokens has at most n / (2 n_tok) + 1 pairs
    const int64_t pairs = a.Tq / (2 * p.n_tok) + static_cast<int64_t>(a.B);
    if (pairs * a.Hkv > 0x7FFFFFFF) return cudaErrorInvalidValue;
    varlen_attn_kernel<D><<<static_cast<unsigned>(pairs * a.Hkv), kThreads, smem, st>>>(*a.tm_q, *a.tm_k, *a.tm_v, p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_varlen_attention(const VarlenLaunch& a, cudaStream_t st) {
    Params p{};
    p.o = reinterpret_cast<__nv_bfloat16*>(a.o);
    p.lse = a.lse;
    p.cu_q = a.cu_q;
    p.cu_k = a.cu_k;
    p.err_word = a.err_word;
    p.B = a.B;
    p.Tq = a.Tq;
    p.Tk = a.Tk;
    p.Hq = a.Hq;
    p.Hkv = a.Hkv;
    p.G = a.Hq / a.Hkv;
    p.n_tok = kTile / p.G;
    p.causal = a.causal;
    p.c = static_cast<float>(static_cast<double>(a.sm_scale) * 1.4426950408889634);
    p.timeout_ns = a.timeout_ns;
    return a.D == 128 ? launch<128>(a, p, st) : launch<64>(a, p, st);
}

}  // namespace fsa
