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
//   warp 9           TMEM allocator and the issuer of every product;
//   warp 11          finds the CTA's next pair of tiles.
// A CTA stays on its SM: when it has taken a pair, warp 11 cancels the launch of
// a CTA that has not started yet and takes over its number, so pairs (those of
// most keys first) go to whichever SM is free, and the next pair's Q,
// K and first scores are under way while the softmax warps still write the last
// one's output.
// TMEM: S0, S1 (128 columns each, P overlays the first 64 of its S in bf16),
// O0, O1 (D columns each).
//
// The products of one thread run in the order of issue:
//   Q0 K(0), Q1 K(0), then per key tile t
//   P0 V(t), Q0 K(t+1), P1 V(t), Q1 K(t+1)
// so while one tile's softmax works on its scores the other tile's two products
// run.  P is handed over in halves of 64 keys, so that P V begins under the second
// half's exponentials: a step is bound by this chain, from scores to weights to
// the next scores, as much as by the products (16 prompts of up to 1000 tokens
// 73.5 -> 71 us with the halves and V waited for ahead of P, 24 of up to 2000 at
// D = 64 208 -> 199, 32 / 8 heads; quarters no better).  A score product's commit also says that
// the tile's P V before it has finished, so between s_full and p_half a softmax
// thread owns its row of O and may rescale it: that happens only when the running
// maximum is passed by more than 2^8 (weights up to 2^8 are exact enough in bf16,
// sums are FP32).
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
constexpr unsigned kSms = 152;
constexpr int kWarpLoad = 8, kWarpMma = 9, kWarpLoadV = 10, kWarpPlan = 11;
// launched at 168 registers per thread; helpers drop to 40, softmax takes 232
constexpr int kLaunchRegs = 168, kSoftmaxRegs = 232, kHelperRegs = 40;
static_assert(2 * 128 * kSoftmaxRegs + 128 * kHelperRegs <= kThreads * kLaunchRegs,
              "register split exceeds the launch allocation");
constexpr int kAtom = 128 * 128;       // 128 rows x 128 bytes (64 bf16)
constexpr int kTileBytes = 2 * kAtom;  // 128 rows x 128 bf16
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 256;        // S0 at 0, S1 at 128, O0 at 256, O1 at 384
constexpr float kNoMax = -3.402823466e38f;  // before a row's first key: the least finite value
constexpr float kLag = 8.0f;           // how far the reference may lag behind the maximum (log2)
// A weight is 2^(s c - m) in one rounding, m the rounded reference: all weights of
// the row are off by the same 2^d, |d| <= 2^-25 |m|, which cancels in the output
// while it stays in range.  From scores of this size on (d = 8) both are rounded
// before they are subtracted.
constexpr float kFar = 268435456.0f;

// A pair of query tiles of one key head: sequence bounds, first token of the pair
// in its sequence, key head (-1: no more work).
struct Item {
    int q0, nq, k0, nk, tok0, hk;
};

struct __align__(1024) Smem {
    uint8_t q[2][kTileBytes];
    uint8_t k[kKStages][kTileBytes];
    uint8_t v[kVStages][kTileBytes];
    uint4 out[8][32][4];  // per softmax warp: 32 rows x 32 channels of output on their way
    uint4 next;           // the launch control's answer
    uint64_t next_full;
    uint64_t item_full[2], item_empty[2];
    uint64_t q_full, q_empty;
    uint64_t k_full[kKStages], k_empty[kKStages];
    uint64_t v_full[kVStages], v_empty[kVStages], v_clean[kVStages];
    uint64_t s_full[2], p_half[2], p_full[2], o_full[2];
    uint64_t drain;
    Item item[2];
    uint32_t tmem_base;
    int abort;
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
    int skip;  // test use: K tile 1 never arrives
};

__device__ __forceinline__ void raise_abort(Smem& sm, const Params& p) {
    sm.abort = 1;
    atomicOr(p.err_word, kErrTimeout);
}

// Where the plan warp's search for pair numbers stands: 32 sequences from b on,
// whose pairs' numbers begin with `first`.
struct Cursor {
    int b, first;
};

// Finds pair number idx, by the whole warp: 32 sequences after 32 from the cursor
// on (numbers grow from call to call as a rule), among the pairs of these the
// one with the most key tiles first, so that no long one is left for the end
// (eight ragged sequences in the order of the pack: SMs idle a tenth of the
// time).  Sequences from the first wrong bound on have none.  False: no such pair.
__device__ __forceinline__ bool find_pair(const Params& p, int idx, Cursor& at, Item& it) {
    const int lane = threadIdx.x & 31, rows = 2 * p.n_tok;
    if (idx < at.first) at = {0, 0};
    while (at.b < p.B) {
        const int b = min(at.b + lane, p.B - 1);
        const int q0 = __ldg(p.cu_q + b), q1 = __ldg(p.cu_q + b + 1), k0 = __ldg(p.cu_k + b), k1 = __ldg(p.cu_k + b + 1);
        const bool bad = q0 < 0 || q1 < q0 || q1 > p.Tq || k0 < 0 || k1 < k0 || k1 > p.Tk;
        const unsigned wrong = __ballot_sync(0xFFFFFFFFu, bad);
        const int good = min(p.B - at.b, wrong ? __ffs(wrong) - 1 : 32);  // sequences of this window
        const int nq = q1 - q0, nk = k1 - k0;
        const int n = lane < good ? (nq + rows - 1) / rows : 0;
        const int local = idx - at.first, total = __reduce_add_sync(0xFFFFFFFFu, n);
        if (local < total) {
            // pairs of this lane's sequence that see at least `tiles` key tiles: the
            // later ones, from the one whose last token sees key 128 (tiles - 1) on
            auto longer = [&](int tiles) {
                const int key = kTile * (tiles - 1);
                if (tiles <= 0 || n == 0) return n;
                if (nk <= key) return 0;
                const int token = key - (nk - nq);
                return !p.causal || token < 0 ? n : n - token / rows;
            };
            // the length of pair idx: the largest with more than `local` pairs that
            // long (where every CTA starts at once the order is of no use, and the
            // 0.7 us of the search would stand before the first load)
            int more = 0, same = n;
            if (gridDim.x > kSms) {
                int lo = 0, hi = __reduce_max_sync(0xFFFFFFFFu, n ? nk / kTile + 2 : 1);
                while (hi - lo > 1) {
                    const int mid = (lo + hi) / 2;
                    if (__reduce_add_sync(0xFFFFFFFFu, longer(mid)) > local)
                        lo = mid;
                    else
                        hi = mid;
                }
                more = longer(lo + 1);
                same = longer(lo) - more;
            }
            int inc = same;
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xFFFFFFFFu, inc, o);
                if (lane >= o) inc += x;
            }
            const int rest = local - __reduce_add_sync(0xFFFFFFFFu, more);
            const int src = __ffs(__ballot_sync(0xFFFFFFFFu, rest < inc)) - 1;
            const int pair = n - 1 - more - (rest - (inc - same));
            it.q0 = __shfl_sync(0xFFFFFFFFu, q0, src);
            it.nq = __shfl_sync(0xFFFFFFFFu, nq, src);
            it.k0 = __shfl_sync(0xFFFFFFFFu, k0, src);
            it.nk = __shfl_sync(0xFFFFFFFFu, nk, src);
            it.tok0 = __shfl_sync(0xFFFFFFFFu, pair, src) * rows;
            return true;
        }
        if (good < min(32, p.B - at.b)) {
            if (lane == 0) atomicOr(p.err_word, kErrBadIndex);
            return false;
        }
        at.first += total;
        at.b += 32;
    }
    return false;
}

// Asks the hardware for a CTA of this grid that has not started: its number, or
// that there is none, arrives in `answer` and on `bar`.
__device__ __forceinline__ void ask_next_cta(uint4* answer, uint64_t* bar) {
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                     smem_u32(answer)),
                 "r"(smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ int next_cta(const uint4* answer) {  // -1: none
    uint32_t ok, x;
    asm volatile(
        "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\t"
        "ld.shared.b128 h, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t"
        "mov.u32 %1, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n\t}"
        : "=r"(ok), "=r"(x)
        : "r"(smem_u32(answer))
        : "memory");
    return ok ? static_cast<int>(x) : -1;
}

// Key tiles that query tile i of an item works on: those that its last token sees.
__device__ __forceinline__ int key_tiles(const Params& p, const Item& it, int i) {
    const int first = it.tok0 + i * p.n_tok, last = min(first + p.n_tok, it.nq) - 1;
    const int see = first >= it.nq ? 0 : p.causal ? min(it.nk, max(0, it.nk - it.nq + 1 + last)) : it.nk;
    return (see + kTile - 1) / kTile;
}

// O of this thread's row times f.
template <int D>
__device__ __forceinline__ void rescale_output(uint32_t o_col, float f) {
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

// The rest of softmax_tile, reading the scores once more, where some row's are
// beyond kFar (`far`: this row's); the other rows' arithmetic is the same as there.
template <int D>
__device__ __forceinline__ void far_tile(Smem& sm, const Params& p, int t, int i, uint32_t s_col, uint32_t o_col, int n_valid,
                                         float top, bool far, float& m, float& l) {
    const float mn = top > m + kLag ? top : m, f = ex2(m - mn);
    l *= f;
    m = mn;
    if (t > 0) rescale_output<D>(o_col, f);
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
        uint32_t s[32], w[16];
        tmem_ld32(s_col + 32 * c, s);
        tmem_ld_wait();
        tmem_reg_dep(s);
        mask32(s, n_valid - 32 * c);
        if (far) {
#pragma unroll
            for (int j = 0; j < 32; ++j) s[j] = __float_as_uint(__fsub_rn(__fmul_rn(__uint_as_float(s[j]), p.c), m));
        }
        l += exp32(s, far ? 1.0f : p.c, far ? 0.0f : m, w);
        tmem_st16(s_col + 16 * c, w);  // (ends below the next 32 scores)
        if (c & 1) {
            tmem_st_wait();
            tc_fence_before();
            warp_arrive(c == 1 ? &sm.p_half[i] : &sm.p_full[i]);
        }
    }
}

// One key tile t for this thread's row: scores out of TMEM, the maximum, the
// rare rescale of O, P back into TMEM.  `lim`: keys the row sees in all; `ph`:
// phase of s_full;
// `masked`: some row of the tile sees less than this whole key tile.
template <int D>
__device__ __forceinline__ bool softmax_tile(Smem& sm, const Params& p, int t, int i, uint32_t ph, uint32_t s_col, uint32_t o_col,
                                             int lim, bool masked, float& m, float& l) {
    const bool ok = mbar_wait(&sm.s_full[i], ph, p.timeout_ns, &sm.abort);
    tc_fence_after();
    uint32_t s0[32], s1[32], s2[32], s3[32];
    float top;
    bool half = false;  // no row of the warp sees the tile's second 64 keys
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
        const int n_valid = masked ? lim - t * kTile : kTile;
        half = __reduce_max_sync(0xFFFFFFFFu, n_valid) <= 64;
        tmem_ld32(s_col, s0);
        tmem_ld32(s_col + 32, s1);
        if (!half) {
            tmem_ld32(s_col + 64, s2);
            tmem_ld32(s_col + 96, s3);
        }
        tmem_ld_wait();
        tmem_reg_dep(s0);
        tmem_reg_dep(s1);
        tmem_reg_dep(s2);
        tmem_reg_dep(s3);
        const int least = __reduce_min_sync(0xFFFFFFFFu, n_valid);  // of the warp's rows
        if (least < 32) mask32(s0, n_valid);
        if (least < 64) mask32(s1, n_valid - 32);
        top = fmaxf(max32(s0), max32(s1));
        if (!half) {
            if (least < 96) mask32(s2, n_valid - 64);
            if (least < 128) mask32(s3, n_valid - 96);
            top = fmaxf(top, fmaxf(max32(s2), max32(s3)));
        }
    }
    top *= p.c;
    const bool grew = top > m + kLag, far = fabsf(top) >= kFar && top >= kNoMax;
    if (__any_sync(0xFFFFFFFFu, grew || far)) {
        if (__builtin_expect(__any_sync(0xFFFFFFFFu, far), 0)) {
            far_tile<D>(sm, p, t, i, s_col, o_col, masked ? lim - t * kTile : kTile, top, far, m, l);
            return __all_sync(0xFFFFFFFFu, ok);
        }
        const float mn = grew ? top : m;
        const float f = ex2(m - mn);
        l *= f;
        m = mn;
        if (t > 0) rescale_output<D>(o_col, f);  // O holds the tiles before t
    }
    // the weights of 64 keys
    auto weights = [&](const uint32_t (&a)[32], const uint32_t (&b)[32], uint32_t col) {
        uint32_t w0[16], w1[16], w[32];
        l += exp32(a, p.c, m, w0);
        l += exp32(b, p.c, m, w1);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            w[j] = w0[j];
            w[16 + j] = w1[j];
        }
        tmem_st32(col, w);
    };
    auto hand_over = [&](uint64_t* bar) {
        tmem_st_wait();
        tc_fence_before();
        warp_arrive(bar);
    };
    if (half) {
        // (a branch around the second half alone cost all tiles 3 % at D = 64)
        uint32_t none[32] = {};
        tmem_st32(s_col + 32, none);
        weights(s0, s1, s_col);
        hand_over(&sm.p_half[i]);
        hand_over(&sm.p_full[i]);
    } else {
        weights(s0, s1, s_col);
        hand_over(&sm.p_half[i]);
        weights(s2, s3, s_col + 32);
        hand_over(&sm.p_full[i]);
    }
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

    if (tid == 0) {
        sm.abort = 0;
        mbar_init(&sm.next_full, 1);
        mbar_init(&sm.q_full, 1);
        mbar_init(&sm.q_empty, 1);
        for (int i = 0; i < kKStages; ++i) {
            mbar_init(&sm.k_full[i], i == 1 && p.skip ? 2 : 1);
            mbar_init(&sm.k_empty[i], 1);
        }
        for (int i = 0; i < kVStages; ++i) {
            mbar_init(&sm.v_full[i], 1);
            mbar_init(&sm.v_empty[i], 1);
            mbar_init(&sm.v_clean[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.item_full[i], 1);
            mbar_init(&sm.item_empty[i], 11);  // every warp but the plan warp
            mbar_init(&sm.s_full[i], 1);
            mbar_init(&sm.p_half[i], 4);  // one arrival per softmax warp
            mbar_init(&sm.p_full[i], 4);
            mbar_init(&sm.o_full[i], 1);
        }
        mbar_init(&sm.drain, 1);
        fence_mbar_init();
    }
    // rows behind a query tile's last whole token are loaded by no copy: zeros, so
    // that their scores are none that would have to be followed
#pragma unroll 1
    for (int e = tid + p.G * p.n_tok * 8; e < kTile * 8; e += kThreads)
#pragma unroll 1
        for (int a = 0; a < 2 * n_atoms; ++a)
            reinterpret_cast<uint4*>(sm.q[a / n_atoms] + a % n_atoms * kAtom)[e] = make_uint4(0, 0, 0, 0);
    if (p.G * p.n_tok < kTile) fence_async_smem();
    if (warp == kWarpMma) {
        tmem_alloc(&sm.tmem_base, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;

    auto wait = [&](uint64_t* bar, uint32_t phase) {
        return __all_sync(0xFFFFFFFFu, mbar_wait(bar, phase & 1u, p.timeout_ns, &sm.abort)) != 0;
    };
    // the n-th item of this CTA; false: no more, or a wait ran out
    auto take = [&](int n, Item& it, bool& ok) {
        ok = wait(&sm.item_full[n & 1], n >> 1);
        if (!ok) return false;
        it = sm.item[n & 1];
        return it.hk >= 0;
    };
    auto give_back = [&](int n) { warp_arrive(&sm.item_empty[n & 1]); };

    if (warp == kWarpPlan) {
        warpgroup_reg_dec<kHelperRegs>();
        Cursor at{0, 0};
        int cta = blockIdx.x, n = 0;
        uint32_t asked = 0;  // phase of next_full
        bool ok = true;
        while (true) {
            // the next number is asked for while this one is looked up
            if (cta >= 0 && lane == 0) {
                mbar_arrive_expect_tx(&sm.next_full, 16);
                ask_next_cta(&sm.next, &sm.next_full);
            }
            Item it{};
            it.hk = -1;
            bool have = false;
            if (cta >= 0) {
                const int idx = cta / p.Hkv;
                have = find_pair(p, idx, at, it);
                it.hk = have ? cta - idx * p.Hkv : -1;
            }
            if (have || cta < 0) {
                if (n >= 2) ok = wait(&sm.item_empty[n & 1], (n >> 1) + 1);
                if (ok && lane == 0) {
                    sm.item[n & 1] = it;
                    mbar_arrive(&sm.item_full[n & 1]);
                }
                ++n;
            }
            if (cta < 0) break;
            int dummy = 0;  // (an answer under way is waited for in any case)
            const bool got = __all_sync(0xFFFFFFFFu, mbar_wait(&sm.next_full, asked, p.timeout_ns, &dummy)) != 0;
            asked ^= 1u;
            ok = ok && got;
            if (!ok) break;
            cta = next_cta(&sm.next);
            fence_async_smem();
            __syncwarp();
        }
        if (!ok && lane == 0) raise_abort(sm, p);
    } else if (warp == kWarpLoad || warp == kWarpLoadV) {
        warpgroup_reg_dec<kHelperRegs>();
        const bool is_k = warp == kWarpLoad;
        const int stages = is_k ? kKStages : kVStages;
        uint64_t* full = is_k ? sm.k_full : sm.v_full;
        uint64_t* empty = is_k ? sm.k_empty : sm.v_empty;
        const CUtensorMap* map = is_k ? &tm_k : &tm_v;
        int issued = 0, st = 0, n_q = 0;  // key tiles and query pairs loaded so far, stage of the next
        uint32_t ph = 0;
        bool ok = true;
        Item it;
        for (int n = 0; take(n, it, ok); ++n) {
            const int n0 = key_tiles(p, it, 0), n1 = key_tiles(p, it, 1), n_max = max(n0, n1);
            if (is_k && n_max > 0) {
                if (n_q > 0) ok = wait(&sm.q_empty, n_q - 1);
                if (!ok) break;
                if (lane == 0) {
                    const int tiles = n1 > 0 ? 2 : 1;
                    mbar_arrive_expect_tx(&sm.q_full, tiles * n_atoms * p.G * p.n_tok * 128);
                    for (int i = 0; i < tiles; ++i)
                        for (int a = 0; a < n_atoms; ++a)
                            tma_load_3d(sm.q[i] + a * kAtom, &tm_q, &sm.q_full, 64 * a, it.hk * p.G,
                                        it.q0 + it.tok0 + i * p.n_tok);
                }
                ++n_q;
            }
            const int t_ragged = (it.nk % kTile) ? it.nk / kTile : -1;  // key tile that ends inside, if any
            for (int t = 0; t < n_max; ++t) {
                if (issued >= stages) ok = wait(&empty[st], ph ^ 1u);
                if (!ok) break;
                uint8_t* dst = is_k ? sm.k[st] : sm.v[st];
                if (lane == 0) {
                    mbar_arrive_expect_tx(&full[st], kAtom * n_atoms);
                    for (int a = 0; a < n_atoms; ++a)
                        tma_load_3d(dst + a * kAtom, map, &full[st], 64 * a, it.hk, it.k0 + t * kTile);
                }
                ++issued;
                if (!is_k && t == t_ragged) {
                    // the rows behind the sequence's last key belong to others: a
                    // weight of zero does not hide a NaN, so they become zeros
                    ok = wait(&full[st], ph);
                    if (!ok) break;
                    const int r0 = it.nk - t * kTile;
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
            if (!ok) break;
            give_back(n);
        }
        if (lane == 0) {
            if (!ok) raise_abort(sm, p);
            // the copies still in flight land before the CTA exits, whoever gives up
            // and when (in a call that ends well they have landed)
            int dummy = 0;
            if (n_q > 0) mbar_wait(&sm.q_full, (n_q - 1) & 1, p.timeout_ns, &dummy);
            for (int t = max(0, issued - stages); t < issued; ++t)
                mbar_wait(&full[t % stages], (t / stages) & 1, p.timeout_ns, &dummy);
        }
    } else if (warp == kWarpMma) {
        warpgroup_reg_dec<kHelperRegs>();
        // the whole warp walks this, one elected lane issues.  Descriptors: + 2
        // advances a K-major operand by one 16-element K step, + kAtom / 16 by one
        // swizzle atom; V is MN-major, 64-wide d atoms kAtom apart (LBO), 8-key
        // groups 1024 apart (SBO), one 16-key step 2048 bytes
        constexpr uint32_t id_qk = idesc_bf16(128, 128, 0, 0), id_pv = idesc_bf16(128, D, 0, 1);
        const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
        const uint64_t dq = smem_desc(smem_u32(sm.q[0]), 16, 1024, SWZ_128B);
        const uint64_t dk = smem_desc(smem_u32(sm.k[0]), 16, 1024, SWZ_128B);
        const uint64_t dv = smem_desc(smem_u32(sm.v[0]), kAtom, 1024, SWZ_128B);
        auto scores = [&](int i, int st) {
            const uint64_t a = dq + (kTileBytes >> 4) * i, bk = dk + (kTileBytes >> 4) * st;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t off = (kk >> 2) * (kAtom >> 4) + 2 * (kk & 3);
                mma_bf16_one(tm + 128 * i, a + off, bk + off, id_qk, kk > 0 ? 1u : 0u);
            }
            tc_commit_one(&sm.s_full[i]);
        };
        auto values = [&](int i, int st, int half, bool add) {
            const uint64_t bv = dv + (kTileBytes >> 4) * st;
#pragma unroll
            for (int kk = 4 * half; kk < 4 * half + 4; ++kk)
                mma_bf16_tmem_a_one(tm + kColO + 128 * i, tm + 128 * i + 8 * kk, bv + 128 * kk, id_pv,
                                    (add || kk > 0) ? 1u : 0u);
        };
        int tiles = 0, n_q = 0;      // key tiles and query pairs used so far
        uint32_t p_ph[2] = {0, 0};   // phases of p_full
        uint32_t clean_ph = 0;       // phases of v_clean, a bit per stage
        bool ok = true;
        Item it;
        for (int n = 0; take(n, it, ok); ++n) {
            const int n_t[2] = {key_tiles(p, it, 0), key_tiles(p, it, 1)};
            const int n_max = max(n_t[0], n_t[1]);
            const int t_ragged = (it.nk % kTile) ? it.nk / kTile : -1;
            if (n_max > 0) {
                ok = wait(&sm.q_full, n_q) && wait(&sm.k_full[tiles % kKStages], tiles / kKStages);
                if (!ok) break;
                tc_fence_after();
                if (n_t[0] > 0) scores(0, tiles % kKStages);
                if (n_t[1] > 0) scores(1, tiles % kKStages);
                tc_commit_one(&sm.k_empty[tiles % kKStages]);
                if (n_max == 1) tc_commit_one(&sm.q_empty);
                ++n_q;
            }
            for (int t = 0; ok && t < n_max; ++t, ++tiles) {
                const int sv = tiles % kVStages, sk = (tiles + 1) % kKStages;
                // (before the weights, so that these are waited for alone: a wait takes
                // some 100 clocks even when there is nothing to wait for)
                ok = wait(&sm.v_full[sv], tiles / kVStages);
                if (ok && t == t_ragged) {
                    ok = wait(&sm.v_clean[sv], clean_ph >> sv);
                    clean_ph ^= 1u << sv;
                }
                bool have_k = false;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (!ok || t >= n_t[i]) continue;
                    ok = wait(&sm.p_half[i], p_ph[i]);
                    if (!ok) continue;
                    tc_fence_after();
                    values(i, sv, 0, t > 0);
                    ok = wait(&sm.p_full[i], p_ph[i]);
                    p_ph[i] ^= 1u;
                    if (!ok) continue;
                    tc_fence_after();
                    values(i, sv, 1, true);
                    if (t + 1 == n_t[i]) {
                        tc_commit_one(&sm.o_full[i]);
                        continue;
                    }
                    if (!have_k) {
                        ok = wait(&sm.k_full[sk], (tiles + 1) / kKStages);
                        have_k = true;
                        if (!ok) continue;
                        tc_fence_after();
                    }
                    scores(i, sk);
                }
                if (!ok) break;
                tc_commit_one(&sm.v_empty[sv]);
                if (t + 1 < n_max) tc_commit_one(&sm.k_empty[sk]);
                if (t + 2 == n_max) tc_commit_one(&sm.q_empty);
            }
            if (!ok) break;
            give_back(n);
        }
        if (!ok && lane == 0) raise_abort(sm, p);
        int dummy = 0;
        tc_commit_one(&sm.drain);  // every product issued retires before TMEM is freed
        mbar_wait(&sm.drain, 0, p.timeout_ns, &dummy);
    } else {
        warpgroup_reg_inc<kSoftmaxRegs>();
        const int i = warp >> 2, r = tid & 127;
        const uint32_t lane_addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const uint32_t s_col = lane_addr + 128 * i, o_col = lane_addr + kColO + 128 * i;
        const int tl = r / p.G, h = r - tl * p.G;
        // the four rows that this lane stores a piece of: token in the tile and
        // row in the packed output from the tile's first on
        int out_tok[4], out_row[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int wr = 32 * (warp & 3) + 8 * j + (lane >> 2);
            out_tok[j] = wr / p.G;
            out_row[j] = out_tok[j] * p.Hq + wr - out_tok[j] * p.G;
        }
        uint32_t s_ph = 0, o_ph = 0;
        bool ok = true;
        Item it;
        for (int n = 0; take(n, it, ok); ++n) {
            const int n_t = key_tiles(p, it, i);
            const int first = it.tok0 + i * p.n_tok, tok = first + tl;
            const bool row_valid = tl < p.n_tok && tok < it.nq;
            // keys that this row and the tile's first row see
            const int lim = p.causal ? min(it.nk, it.nk - it.nq + 1 + tok) : it.nk;
            const int lim0 = p.causal ? min(it.nk, it.nk - it.nq + 1 + first) : it.nk;
            float m = kNoMax, l = 0.0f;
            for (int t = 0; ok && t < n_t; ++t, s_ph ^= 1u)
                ok = softmax_tile<D>(sm, p, t, i, s_ph, s_col, o_col, lim, (t + 1) * kTile > lim0, m, l);
            if (ok && n_t > 0) {
                ok = wait(&sm.o_full[i], o_ph);
                o_ph ^= 1u;
            }
            if (!ok) break;
            if (first < it.nq) {
                // through shared memory, so that a store covers eight rows' 64 bytes
                // and not 32 rows' 16 (which held the next pair up by 0.8 us)
                const float inv = l == 0.0f ? 0.0f : 1.0f / l;
                const int64_t row0 = static_cast<int64_t>(it.q0 + first) * p.Hq + it.hk * p.G;
                tc_fence_after();
#pragma unroll
                for (int c2 = 0; c2 < D / 64; ++c2) {
                    uint32_t rr[2][32];
                    if (n_t > 0) {
                        tmem_ld32(o_col + 64 * c2, rr[0]);
                        tmem_ld32(o_col + 64 * c2 + 32, rr[1]);
                        tmem_ld_wait();
                        tmem_reg_dep(rr[0]);
                        tmem_reg_dep(rr[1]);
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j) rr[0][j] = rr[1][j] = 0u;
                    }
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        uint32_t packed[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            packed[j] = bf16x2(__uint_as_float(rr[half][2 * j]) * inv, __uint_as_float(rr[half][2 * j + 1]) * inv);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            sm.out[warp][lane][j ^ ((lane >> 1) & 3)] =
                                make_uint4(packed[4 * j], packed[4 * j + 1], packed[4 * j + 2], packed[4 * j + 3]);
                        __syncwarp();
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int wr = 8 * j + (lane >> 2);
                            const uint4 v = sm.out[warp][wr][(lane & 3) ^ ((wr >> 1) & 3)];
                            if (out_tok[j] < p.n_tok && first + out_tok[j] < it.nq)
                                *reinterpret_cast<uint4*>(p.o + (row0 + out_row[j]) * D + 64 * c2 + 32 * half + 8 * (lane & 3)) = v;
                        }
                        __syncwarp();
                    }
                }
                if (row_valid && p.lse)
                    p.lse[row0 + static_cast<int64_t>(tl) * p.Hq + h] = l == 0.0f ? -INFINITY : (m + __log2f(l)) * 0.6931471805599453f;
            }
            give_back(n);
        }
        if (!ok) raise_abort(sm, p);
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
    p.skip = a.debug_flags & 1;
    return a.D == 128 ? launch<128>(a, p, st) : launch<64>(a, p, st);
}

}  // namespace fsa
