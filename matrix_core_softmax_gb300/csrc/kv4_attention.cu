// kv4_attention.cu -- attention of a few query tokens per sequence over the
// four-bit key/value cache.
//
// Query i of sequence b (Sq queries, the last ones of its len keys) sees keys
// j <= len - Sq + i: s_j = sm q.k^_j, o = sum_j softmax(s)_j v^_j, and the
// log-sum-exp of s.  A row that sees no key gets o = 0 and -inf.
//
// What bounds it: 34 D / 32 bytes of cache per key and key head (136 at
// D = 128) are read once, so at 6.8 TB/s an SM has to finish a key of one head
// every 5.8 clocks, with all query heads of the group at once.  A CUDA-core
// product is far too slow for that; a product needs the codes as 16-bit values
// in registers, and that unpacking (256 values a key) is what has to be cheap:
//  - both products run on m16n8k16 f16 MMAs with the keys (S^T = K Q^T) or the
//    value channels (O^T = V^T P^T) as the 16 rows and the query rows as the 8
//    columns, so that up to 8 query rows cost the same as one;
//  - the cache's byte order is the A fragments' order: a lane finds its codes
//    of a row in one 16-byte (keys) or 8-byte (values) piece, and cvt
//    (E2M1 pair -> f16 pair, 64 lanes a clock and SM, three times the rate of
//    placing the bits by shifts and masks) turns a byte into a register of the
//    fragment.  For the values, whose pairs run along the keys, the nibbles of
//    two keys are first interleaved (4 integer instructions for 16 values);
//  - the scales are never multiplied into the codes.  The key scale of a block
//    multiplies the 8-column product of that block (FP32); the value scale,
//    which differs along the product's contraction, goes into the weights: one
//    weight fragment per 32-channel block.
//
// Weights.  With X the scale exponent of a key's value block b, R_b the largest
// one so far and y = min_b (R_b - X_b) (at most 90) the kernel takes
//   p = 2^(s - y - M)  rounded to f16, M the running maximum of s - y,
//   w_b = p 2^(y - (R_b - X_b) + 11),
//   O_b += sum w_b code,  l += p 2^y (before the rounding),
// so the weights are relative to the largest product of weight and value scale
// and neither a large nor a small value row leaves f16's range; a weight's
// error is 2^-11 of itself or 2^-25 of that largest product.  M and R_b follow
// lazily (M may lag by 2^4, which the 2^11 leaves room for), so O is rescaled
// only when one of them really grows.  Where the R_b grow, s - y of every key
// before falls by the least of the steps and M with it (else the keys after a
// large value of little weight would have p far below 1), but only as far as
// keeps l below 2^100: a key without value that leads the others by 2^g has
// added 2^min(g, 90) to it.  A later key adds less than 2^(4 + 90), so a lane's
// share of 2^30 keys stays below 2^122 and a row's sum below 2^125.  O, l and
// the scores are FP32.  q is scaled by a power of two to [1, 2) per row, in
// which f16 holds a bf16 value exactly down to 2^-14 of the row's largest and to
// 2^-25 of it below.
// Pieces of a row are kept as their own output and its log-sum-exp, not as
// unnormalised sums, whose scale 2^(M + R_b) may lie outside of FP32.
//
// Work split.  The cache's groups of all (sequence, key head, 8- or 16-row tile)
// segments form one line (kSegmentCost places before each segment's groups),
// cut into equal shares, one per team of eight warps (two on an SM), and a share
// into equal parts, one per warp: long contexts spread over the GPU and
// ragged batches balance.  A warp runs along its part on its own: a ring of
// bulk copies (one 32-key group, 4352 bytes at D = 128, a copy) that reaches
// over the segments' ends, its own softmax state, and the output of every
// segment that lies in its part as a whole.  Of the others it leaves at most
// two pieces, the segment it starts in and the one it ends in; the team joins
// its warps' pieces, leaves at most two of its own, and a second kernel joins
// those.  (With teams that walked over segments together and met at each end,
// 64 ragged sequences of up to 2000 keys took 40.7 us.)  Where no sequence can
// be longer than kWholeGroups groups, or twice as many with many segments, a block
// takes one segment and there is no second kernel.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>

#include "fsa_internal.h"
#include "kv4.cuh"
#include "mx_scale.cuh"
#include "sm100_ptx.cuh"

namespace fsa {
namespace {

// Warps that share a part of the line of the split form, a team: one a block and
// two blocks on an SM, or, where a warp's part may be kLongPart groups or more,
// two a block.  (Of two blocks on an SM the first is served first, 8 of the 152
// SMs get two of the first ones or two of the later ones, and the later ones are
// the call's end; the warps of one block are served evenly.  But the second kernel
// cannot start before a block ends.)  One team a block / two, 32 / 8 heads of 128:
// 64 sequences of up to 32768 keys 208.6 / 198.3 us, of up to 8000 64.7 / 62.3, of
// up to 4000 42.2 / 41.4; 16 of up to 8000 24.1 / 25.6, of up to 4000 19.2 / 21.6.
constexpr int kTeamWarps = 8, kLongPart = 16;
constexpr int kJoinThreads = 256;
constexpr int kStages = 2;        // (three: 1 % slower, they leave less L1)
constexpr int kTeams = 304;       // of the split form: two on each of 152 SMs
constexpr int kMinShare = kTeamWarps; // places of a team, at least one a warp
// A block takes a whole segment up to this many groups, twice as many where
// there are many segments.  32 / 8 heads of 128, whole / split: one sequence of
// 1000 keys 9.3 / 9.6 us, of 2000 13.9 / 9.9; 16 of up to 1000 9.6 / 13.2, 64 of
// them 16.6 / 20.4, 256 48.0 / 49.8; up to 2000 keys: 8 sequences 14.0 / 13.5, 16
// 14.0 / 15.2, 32 17.5 / 19.4, 64 30.1 / 27.6, 128 45.6 / 46.4, 256 79.8 / 78.7 (no
// clear side: the longest segment sets the whole form's time); 16 of up to 4000
// 22.8 / 19.3, 64 of them 44.6 / 41.3.
constexpr int kWholeGroups = 32;
constexpr int kManySegments = 64; // from here on the join takes four rows a block, too
// More whole segments than fit the GPU in blocks of eight warps run in blocks of
// four: twice as many segments at a time wait for their first keys.  32 / 8 heads
// of 128, four warps / eight: 64 sequences of up to 500 keys 11.2 / 15.6 us, of up
// to 1000 16.6 / 21.6, of up to 2000 30.1 / 31.5; 32 of up to 1000 12.3 / 12.2; 8 of
// up to 1000 10.8 / 9.6, of up to 2000 17.2 / 14.0.
constexpr int kFewWarps = 8, kManyWarps = 4;
// A segment takes this many places of the line before its groups, for what a
// warp spends on taking it up and writing it and for the joins of its pieces
// (without them the warps that meet many short sequences finished last).  One,
// two and three places, 32 / 8 heads: 64 sequences of up to 8000 keys 70.0 / 62.7 /
// 62.3 us, at D = 64 51.7 / 46.9 / 44.0, of up to 4000 44.1 / 41.3 / 41.4, of up to
// 32768 200.5 / 199.4 / 198.3; 16 of up to 4000 with four queries 30.9 / 29.6 / 28.9.
constexpr int kSegmentCost = 3;
constexpr uint32_t kNoGroup = 0xFFFFFFFFu, kNoPlace = 0xFFFFFFFEu;
constexpr float kNoMax = -3.402823466e38f;  // of a row without keys: the least finite value, below every score
constexpr float kLag = 4.0f;      // how far M may lag behind (log2)
constexpr unsigned kMostY = 90;   // largest y
constexpr int kMostL = 100;       // l is not rescaled to 2^100 or more
constexpr int kHeadroom = 11;     // weights carry 2^11: 2^11 * 2^4 = 2^15 < 65504
constexpr float kUnit = 1.0f / (1 << kHeadroom);
// A key's products of codes and the scaled q, below 2^11 in sum, take the key
// scales over 2^kKeyShift and the scores the rest: scales go up to 2^127, and
// nothing on the way to a score of normal size leaves FP32's range.
constexpr int kKeyShift = 10;
constexpr float kKeyUnit = 1.0f / (1 << kKeyShift);
constexpr int kMostE = 240;       // largest exponent that q is scaled by: below 2^15 in f16

struct Params {
    const uint16_t* q;
    const uint8_t* cache;
    const int* page_table;
    const int* seq_lens;
    uint16_t* o;
    float* lse;
    float* partial;  // [team][2]: 8 NT rows of D, then their log2-sum-exp2; null: whole segments
    int64_t q_stride, num_pages;
    int B, Sq, Hq, Hkv, G, n_rt, page_size, max_pages;
    float c;  // sm_scale * log2(e)
    uint64_t timeout_ns;
    unsigned int* err_word;
    int skip;  // test use: a warp's second group never arrives
};

// A piece of a segment: what one warp made of the groups of it in its part.
struct Piece {
    int64_t seg_x;  // the place of the segment's first group
    int b, seg, ng; // sequence (-1: no piece), segment of it, its groups
};

template <int D, int NT, int kWarps>
struct __align__(128) Smem {
    static constexpr int kPitch = D + 4;  // floats of a row of a piece
    uint8_t ring[kWarps][kStages][kv4_group_bytes(D)];  // in the end: the warp's last piece
    float first[kWarps][8 * NT][kPitch];                // the segment a warp starts in
    float4 kscale[kWarps][kKv4Group];      // 2^X of the key blocks, by row position
    float2 ykey[kWarps][kKv4Group];        // -y and 2^y of each key, by row position
    uint32_t vscale[kWarps][4][2][2][4];   // f16 pairs: [t][16-key step][half][block]
    uint64_t full[kWarps][kStages];
    float lse2[kWarps][2][8 * NT];  // log2-sum-exp2 of the pieces' rows
    Piece piece[kWarps][2];  // [0] in first, [1] in ring
    int64_t scan[kWarps];
    int64_t first_x;
    int first_b;
    int abort;
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_f16_zero(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                             uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// Packed unsigned 16-bit minimum.
__device__ __forceinline__ uint32_t min16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Keys of a sequence, clamped to its page table.
__device__ __forceinline__ int seq_len(const Params& p, int b, bool* bad) {
    const int cap = p.max_pages * p.page_size, n = __ldg(p.seq_lens + b);
    *bad = n < 0 || n > cap;
    return min(max(n, 0), cap);
}
__device__ __forceinline__ int seq_groups(const Params& p, int b) {
    bool bad;
    return (seq_len(p, b, &bad) + kKv4Group - 1) / kKv4Group;
}
// Places on the line of a segment of ng groups (of the split form).
__device__ __forceinline__ int places_of(int ng) { return ng ? ng + kSegmentCost : 0; }

// Row position of a key in its group and back (an involution within each 8):
// position r of a 16-row tile is key r with its low bit flipped by bit 1, so
// that the 128-byte key loads and the 8-byte value loads of a warp spread over
// the banks.
__device__ __forceinline__ int swap_pos(int r) { return r ^ ((r >> 1) & 1); }

// A query row of a segment: token i of the sequence, query head h of the group.
struct Row {
    int i, h;
};
__device__ __forceinline__ Row row_of(const Params& p, int r) { return {r / p.G, r % p.G}; }

// Segment of a sequence with segments of `places` places that its place `rel`
// lies in (a 64-bit division takes 1 us, and every warp waits for two of these).
__device__ __forceinline__ int segment_at(int64_t rel, int places) {
    if (rel <= 0x7FFFFFFF) return static_cast<int>(static_cast<uint32_t>(rel) / static_cast<uint32_t>(places));
    return static_cast<int>(rel / places);
}

// Places of a team's share of a line of `all` places.
__device__ __forceinline__ int64_t share_of(int64_t all, int n_teams) {
    return max(static_cast<int64_t>(kMinShare), (all + n_teams - 1) / n_teams);
}

// Four channels of row r of a segment, and the row's log-sum-exp from its log2.
template <int D>
__device__ __forceinline__ void write_row(const Params& p, int b, int hk, int r, int d4, float4 a, float lse2) {
    const Row w = row_of(p, r);
    const int64_t row = (static_cast<int64_t>(b) * p.Sq + w.i) * p.Hq + hk * p.G + w.h;
    const __nv_bfloat162 lo = __floats2bfloat162_rn(a.x, a.y), hi = __floats2bfloat162_rn(a.z, a.w);
    *reinterpret_cast<uint2*>(p.o + row * D + 4 * d4) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    if (p.lse && d4 == 0) p.lse[row] = lse2 == kNoMax ? -INFINITY : lse2 * 0.6931471805599453f;
}

// kWhole: a block takes one segment, without a walk over sequences, segments
// that end inside a warp's part or pieces left to the second kernel; the short
// calls that it serves wait for the kernel's instructions, too (300 keys: 7.5 us
// with the general form).
template <int D, int NT, bool kWhole, int kWarps, int kBlockTeams>
__global__ void __launch_bounds__(32 * kWarps * kBlockTeams, (NT == 1 ? 16 : 8) / (kWarps * kBlockTeams))
    kv4_attn_kernel(const Params p) {
    constexpr int kThreads = 32 * kWarps;  // of a team
    constexpr int kB = D / 32;
    constexpr int kGroupBytes = kv4_group_bytes(D);
    constexpr Kv4Layout L = kv4_layout(D);
    constexpr int kRows = 8 * NT;
    constexpr int kPitch = Smem<D, NT, kWarps>::kPitch;
    static_assert(kRows * kPitch * 4 <= kStages * kGroupBytes, "a piece exceeds a warp's ring");
    extern __shared__ __align__(128) uint8_t smem_raw[];
    const int block_team = kBlockTeams == 1 ? 0 : static_cast<int>(threadIdx.x) / kThreads;
    const int tid = threadIdx.x - block_team * kThreads, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t = lane & 3;
    const int team = blockIdx.x + gridDim.x * block_team;  // few teams' work goes to as many SMs
    Smem<D, NT, kWarps>& sm = reinterpret_cast<Smem<D, NT, kWarps>*>(smem_raw)[block_team];
    auto sync = [&]() {
        if constexpr (kBlockTeams == 1)
            __syncthreads();
        else
            asm volatile("bar.sync %0, %1;" ::"r"(1 + block_team), "n"(kThreads) : "memory");
    };

    if (tid == 0) sm.abort = 0;
    if (lane < 2) sm.piece[warp][lane].b = -1;
    if (lane < kStages) mbar_init(&sm.full[warp][lane], lane == 1 && p.skip ? 2 : 1);
    fence_mbar_init();

    // this team's share [x, x_end) of the line, and where it starts: sequence b,
    // whose places begin at x_seq
    int64_t x, x_end, x_seq;
    int b, len;
    const int n_seg = p.Hkv * p.n_rt;  // segments of a sequence
    if constexpr (kWhole) {
        sync();
        b = blockIdx.x / n_seg;
        bool bad;
        len = seq_len(p, b, &bad);
        const int ng = (len + kKv4Group - 1) / kKv4Group;
        if (bad && tid == 0) atomicOr(p.err_word, kErrBadIndex);
        const int seg = blockIdx.x - b * n_seg;
        x_seq = 0;
        x = static_cast<int64_t>(seg) * ng;
        x_end = x + ng;
        if (ng == 0) {  // an empty sequence: zeros
            const int hk = seg / p.n_rt, r0 = (seg % p.n_rt) * kRows;
            for (int e = tid; e < kRows * D; e += kThreads) {
                const int r = r0 + e / D;
                if (r < p.Sq * p.G) {
                    const Row w = row_of(p, r);
                    const int64_t row = (static_cast<int64_t>(b) * p.Sq + w.i) * p.Hq + hk * p.G + w.h;
                    p.o[row * D + e % D] = 0;
                    if (p.lse && e % D == 0) p.lse[row] = -INFINITY;
                }
            }
            return;
        }
    } else {
        const int per = (p.B + kThreads - 1) / kThreads;
        const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
        int64_t sum = 0;
        for (int i = b0; i < b1; ++i) {
            bool bad;
            sum += places_of((seq_len(p, i, &bad) + kKv4Group - 1) / kKv4Group);
            if (bad && team == 0) atomicOr(p.err_word, kErrBadIndex);
        }
        // inclusive scan over the warp, then over the warps
        int64_t inc = sum;
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
            if (lane >= o) inc += v;
        }
        if (lane == 31) sm.scan[warp] = inc;
        sync();
        int64_t before = inc - sum, total = 0;
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) before += sm.scan[w];
            total += sm.scan[w];
        }
        const int64_t all = total * n_seg;
        const int64_t share = share_of(all, gridDim.x * kBlockTeams);
        x = share * team;
        x_end = min(x + share, all);
        if (x >= x_end) return;
        if (before * n_seg <= x && x < (before + sum) * n_seg) {
            int i = b0;
            int64_t at = before * n_seg;
            while (true) {
                const int64_t next = at + static_cast<int64_t>(places_of(seq_groups(p, i))) * n_seg;
                if (x < next) break;
                at = next;
                ++i;
            }
            sm.first_b = i;
            sm.first_x = at;
        }
        sync();
        b = sm.first_b;
        x_seq = sm.first_x;
        bool bad;
        len = seq_len(p, b, &bad);
    }
    const int gpp = p.page_size / kKv4Group;
    // this warp's part of the share
    const int64_t pos_begin = x + (x_end - x) * warp / kWarps, pos_end = x + (x_end - x) * (warp + 1) / kWarps;
    const int count = static_cast<int>(pos_end - pos_begin);

    // copies: the next place to look at, and the copies issued so far (copy k in
    // stage k mod kStages)
    int next = 0, n_in = 0;
    uint32_t ids = 0;        // lane i: the cache's group number at place 32 n + i of the part
    uint32_t bad_stage = 0;  // stages whose group has no page
    int ib = b;              // sequence that the next ids are looked for from,
    int64_t ix = x_seq;      // where its places begin, and the groups of its segments
    int ing = (len + kKv4Group - 1) / kKv4Group;
    auto issue = [&]() {
        while (next < count) {
            if ((next & 31) == 0) {
                const int64_t pos = pos_begin + next + lane;
                ids = kNoPlace;
                if (pos < pos_end) {
                    int seg, gi;
                    if constexpr (kWhole) {
                        seg = blockIdx.x - b * n_seg;
                        gi = static_cast<int>(pos - x);
                    } else {
                        while (pos >= ix + static_cast<int64_t>(places_of(ing)) * n_seg) {
                            ix += static_cast<int64_t>(places_of(ing)) * n_seg;
                            ing = seq_groups(p, ++ib);
                        }
                        seg = segment_at(pos - ix, places_of(ing));
                        gi = static_cast<int>(pos - ix - static_cast<int64_t>(seg) * places_of(ing)) - kSegmentCost;
                    }
                    if (gi >= 0) {
                        const int pi = gi / gpp;
                        const int page = __ldg(p.page_table + static_cast<int64_t>(ib) * p.max_pages + pi);
                        ids = kNoGroup;
                        if (page >= 0 && page < p.num_pages)  // (a 9 TB cache would have 2^32 - 2 groups)
                            ids = (static_cast<uint32_t>(page) * p.Hkv + seg / p.n_rt) * gpp + (gi - pi * gpp);
                        else
                            atomicOr(p.err_word, kErrBadIndex);
                    }
                }
                if constexpr (!kWhole) {
                    const int last = min(31, count - 1 - next);
                    ib = __shfl_sync(0xFFFFFFFFu, ib, last);
                    ix = __shfl_sync(0xFFFFFFFFu, ix, last);
                    ing = __shfl_sync(0xFFFFFFFFu, ing, last);
                }
            }
            const uint32_t id = __shfl_sync(0xFFFFFFFFu, ids, next & 31);
            ++next;
            if (!kWhole && id == kNoPlace) continue;
            const int st = n_in % kStages;
            ++n_in;
            bad_stage &= ~(1u << st);
            if (id == kNoGroup) bad_stage |= 1u << st;
            if (lane == 0) {
                if (id == kNoGroup) {
                    mbar_arrive(&sm.full[warp][st]);
                } else {
                    mbar_arrive_expect_tx(&sm.full[warp][st], kGroupBytes);
                    bulk_load(sm.ring[warp][st], p.cache + static_cast<uint64_t>(id) * kGroupBytes, kGroupBytes, &sm.full[warp][st]);
                }
            }
            return;
        }
    };
#pragma unroll 1
    for (int k = 0; k < kStages; ++k) issue();

    int i = 0, n_out = 0;  // places passed, groups done
    bool ok = true;
    while (ok && i < count) {
        const int64_t pos = pos_begin + i;
        int ng = (len + kKv4Group - 1) / kKv4Group;
        while (!kWhole && pos >= x_seq + static_cast<int64_t>(places_of(ng)) * n_seg) {
            x_seq += static_cast<int64_t>(places_of(ng)) * n_seg;
            bool bad;
            len = seq_len(p, ++b, &bad);
            ng = (len + kKv4Group - 1) / kKv4Group;
        }
        const int seg = kWhole ? blockIdx.x - b * n_seg : segment_at(pos - x_seq, places_of(ng));
        const int64_t seg_x = kWhole ? x : x_seq + static_cast<int64_t>(seg) * places_of(ng) + kSegmentCost;
        if (!kWhole && pos < seg_x) {
            i = static_cast<int>(min(seg_x, pos_end) - pos_begin);
            continue;
        }
        const int i_end = kWhole ? count : static_cast<int>(min(seg_x + ng, pos_end) - pos_begin);  // end of the segment's groups
        const int hk = seg / p.n_rt, r0 = (seg % p.n_rt) * kRows;

        // the query rows as B fragments, in f16 relative to each row's largest
        uint32_t qf[NT][kB][4];
        float cs[NT][2];      // sm log2(e) 2^(e + kKeyShift) of the rows of this lane's columns
        int seen[NT][2];      // keys that they see
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = r0 + 8 * n + g;
            uint4 raw[kB] = {};
            if (r < p.Sq * p.G) {
                const Row w = row_of(p, r);
                const uint16_t* src = p.q + (static_cast<int64_t>(b) * p.Sq + w.i) * p.q_stride + (hk * p.G + w.h) * D + 8 * t;
#pragma unroll
                for (int c = 0; c < kB; ++c) raw[c] = __ldg(reinterpret_cast<const uint4*>(src + 32 * c));
            }
            uint32_t mx = 0;
#pragma unroll
            for (int c = 0; c < kB; ++c) {
                const uint32_t u[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) mx = max(mx, max(u[i] & 0x7FFFu, (u[i] >> 16) & 0x7FFFu));
            }
            mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
            mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
            const int E = min(max(static_cast<int>(mx >> 7), 1), kMostE);
            const float f = __int_as_float((254 - E) << 23);
#pragma unroll
            for (int c = 0; c < kB; ++c) {
                const uint32_t u[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    qf[n][c][i] = f16x2(__uint_as_float(u[i] << 16) * f, __uint_as_float(u[i] & 0xFFFF0000u) * f);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                cs[n][j] = p.c * __int_as_float((__shfl_sync(0xFFFFFFFFu, E, 8 * t + 4 * j) + kKeyShift) << 23);
                const int rr = r0 + 8 * n + 2 * t + j;
                seen[n][j] = rr < p.Sq * p.G ? len - p.Sq + 1 + rr / p.G : 0;
            }
        }
        const int all_see = len - p.Sq + 1;  // keys that every row sees

        float O[NT][kB][2][4] = {};
        float M[NT][2], l[NT][2] = {};
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j) M[n][j] = kNoMax;
        uint32_t R02 = 0, R13 = 0;  // largest value scale bytes so far

        for (; i < i_end; ++i) {
            const int st = n_out % kStages;
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(&sm.full[warp][st], (n_out / kStages) & 1, p.timeout_ns, &sm.abort));
            if (!ok) break;
            if (!((bad_stage >> st) & 1u)) {
                const uint8_t* buf = sm.ring[warp][st];
                const int key0 = static_cast<int>(pos_begin + i - seg_x) * kKv4Group;

                // scales: lane = key.  2^(X - kKeyShift) of the key blocks (byte 0, 2^-127, is
                // the one without an exponent field).  Value scale bytes as 16-bit pairs,
                // blocks 0 and 2, 1 and 3.
                {
                    const int pos = swap_pos(lane);
                    uint32_t ks, vs;
                    if (D == 128) {
                        ks = *reinterpret_cast<const uint32_t*>(buf + L.kscales + lane * L.srow);
                        vs = *reinterpret_cast<const uint32_t*>(buf + L.vscales + lane * L.srow);
                    } else {
                        ks = *reinterpret_cast<const uint16_t*>(buf + L.kscales + lane * L.srow);
                        vs = *reinterpret_cast<const uint16_t*>(buf + L.vscales + lane * L.srow);
                    }
                    if (key0 + lane >= len) vs = 0;
                    float kf[4];
                    kf[0] = __uint_as_float(max((ks & 0xFFu) << 23, 0x00400000u)) * kKeyUnit;
                    kf[1] = __uint_as_float(max((ks << 15) & 0x7F800000u, 0x00400000u)) * kKeyUnit;
                    kf[2] = __uint_as_float(max((ks << 7) & 0x7F800000u, 0x00400000u)) * kKeyUnit;
                    kf[3] = __uint_as_float(max((ks >> 1) & 0x7F800000u, 0x00400000u)) * kKeyUnit;
                    if (D == 128)
                        sm.kscale[warp][pos] = make_float4(kf[0], kf[1], kf[2], kf[3]);
                    else
                        *reinterpret_cast<float2*>(&sm.kscale[warp][pos]) = make_float2(kf[0], kf[1]);
                    const uint32_t v02 = vs & 0x00FF00FFu, v13 = (vs >> 8) & 0x00FF00FFu;
                    const uint32_t t02 = max16x2(v02, R02), t13 = max16x2(v13, R13);
                    if (__any_sync(0xFFFFFFFFu, t02 != R02 || t13 != R13)) {
                        uint32_t n02 = t02, n13 = t13;
                        for (int o = 16; o; o >>= 1) {
                            n02 = max16x2(n02, __shfl_xor_sync(0xFFFFFFFFu, n02, o));
                            n13 = max16x2(n13, __shfl_xor_sync(0xFFFFFFFFu, n13, o));
                        }
                        int d[kB], least = 255;
#pragma unroll
                        for (int c = 0; c < kB; ++c) {
                            const int sh = 16 * (c >> 1);
                            d[c] = static_cast<int>(((c & 1 ? n13 : n02) >> sh) & 0xFFu) -
                                   static_cast<int>(((c & 1 ? R13 : R02) >> sh) & 0xFFu);
                            least = min(least, d[c]);
                        }
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                // l < 2^(exp - 126) in every lane of the column.  (Rolled and unrolled: 64 x
                                // 32768 keys 197.6 / 199.0 us, but one of 300 6.7 / 6.5)
                                int exp = __float_as_int(l[n][j]) >> 23;
#pragma unroll (kWhole ? 3 : 1)
                                for (int o = 4; o < 32; o <<= 1) exp = max(exp, __shfl_xor_sync(0xFFFFFFFFu, exp, o));
                                const int room = min(least, max(kMostL + 126 - exp, 0));
                                float to = M[n][j] - static_cast<float>(room), drop = M[n][j] - to;
                                if (drop > static_cast<float>(room + 1)) {  // an M of 2^25 or more takes no small steps
                                    to = M[n][j];
                                    drop = 0.0f;
                                }
                                M[n][j] = to;
                                l[n][j] *= ex2(drop);
#pragma unroll
                                for (int c = 0; c < kB; ++c) {
                                    const float f = ex2(drop - static_cast<float>(d[c]));
#pragma unroll
                                    for (int h = 0; h < 2; ++h) {
                                        O[n][c][h][j] *= f;
                                        O[n][c][h][2 + j] *= f;
                                    }
                                }
                            }
                        R02 = n02;
                        R13 = n13;
                    }
                    const uint32_t z02 = R02 - v02, z13 = R13 - v13;  // no borrow: R is the larger in every half
                    const uint32_t zm = D == 128 ? min16x2(z02, z13) : min(z02, z13);
                    const uint32_t y = D == 128 ? min(min(zm & 0xFFFFu, zm >> 16), kMostY) : min(zm, kMostY);
                    sm.ykey[warp][pos] = make_float2(-static_cast<float>(y), __uint_as_float((127u + y) << 23));
                    // f16 2^(kHeadroom - (z - y)), zero where that has no exponent left
                    const uint32_t top = (15 + kHeadroom + y) * 0x00010001u;
                    const uint32_t f02 = (top - min16x2(z02, top)) << 10, f13 = (top - min16x2(z13, top)) << 10;
                    // position pos = 16 step + 8 half + 2 t + e
                    uint16_t* dst = reinterpret_cast<uint16_t*>(&sm.vscale[warp][(pos >> 1) & 3][pos >> 4][(pos >> 3) & 1][0]) + (pos & 1);
                    dst[0] = static_cast<uint16_t>(f02);
                    dst[2] = static_cast<uint16_t>(f13);
                    if (D == 128) {
                        dst[4] = static_cast<uint16_t>(f02 >> 16);
                        dst[6] = static_cast<uint16_t>(f13 >> 16);
                    }
                }
                __syncwarp();

                // scores: position r of tile mt is key 16 mt + swap_pos(r); a pair of
                // columns (query rows) at a time
                float2 s[NT][2][2];
#pragma unroll
                for (int mt = 0; mt < 2; ++mt) {
                    uint32_t ka[kB], kb[kB];
                    const uint8_t* ra = buf + (16 * mt + swap_pos(g)) * L.row + t * (D / 8);
                    if (D == 128) {
                        const uint4 u = *reinterpret_cast<const uint4*>(ra), v = *reinterpret_cast<const uint4*>(ra + 8 * L.row);
                        ka[0] = u.x; ka[1] = u.y; ka[kB - 2] = u.z; ka[kB - 1] = u.w;
                        kb[0] = v.x; kb[1] = v.y; kb[kB - 2] = v.z; kb[kB - 1] = v.w;
                    } else {
                        const uint2 u = *reinterpret_cast<const uint2*>(ra), v = *reinterpret_cast<const uint2*>(ra + 8 * L.row);
                        ka[0] = u.x; ka[1] = u.y;
                        kb[0] = v.x; kb[1] = v.y;
                    }
                    const float4 fa4 = sm.kscale[warp][16 * mt + g], fb4 = sm.kscale[warp][16 * mt + 8 + g];
                    const float fa[4] = {fa4.x, fa4.y, fa4.z, fa4.w}, fb[4] = {fb4.x, fb4.y, fb4.z, fb4.w};
#pragma unroll
                    for (int c = 0; c < kB; ++c) {
                        uint32_t xa[4], xb[4];
                        e2m1x8_to_f16(ka[c], xa);
                        e2m1x8_to_f16(kb[c], xb);
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            float acc[4];
                            mma_f16_zero(acc, xa[0], xb[0], xa[1], xb[1], qf[n][c][0], qf[n][c][1]);
                            mma_f16(acc, xa[2], xb[2], xa[3], xb[3], qf[n][c][2], qf[n][c][3]);
                            const float2 a0 = make_float2(acc[0], acc[1]), a1 = make_float2(acc[2], acc[3]);
                            const float2 f0 = make_float2(fa[c], fa[c]), f1 = make_float2(fb[c], fb[c]);
                            s[n][mt][0] = c == 0 ? __fmul2_rn(a0, f0) : __ffma2_rn(a0, f0, s[n][mt][0]);
                            s[n][mt][1] = c == 0 ? __fmul2_rn(a1, f1) : __ffma2_rn(a1, f1, s[n][mt][1]);
                        }
                    }
                }

                // s - y in log2, masked; the running maximum
                float y2[2][2];
#pragma unroll
                for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float2 yy = sm.ykey[warp][16 * mt + 8 * h + g];
                        y2[mt][h] = yy.y;
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            s[n][mt][h] = __ffma2_rn(s[n][mt][h], make_float2(cs[n][0], cs[n][1]), make_float2(yy.x, yy.x));
                    }
                if (key0 + kKv4Group > all_see) {
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int key = key0 + 16 * mt + 8 * h + swap_pos(g);
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                if (key >= seen[n][0]) s[n][mt][h].x = -INFINITY;
                                if (key >= seen[n][1]) s[n][mt][h].y = -INFINITY;
                            }
                        }
                }
                float top[NT][2];
                bool grew = false;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    top[n][0] = fmaxf(fmaxf(s[n][0][0].x, s[n][0][1].x), fmaxf(s[n][1][0].x, s[n][1][1].x));
                    top[n][1] = fmaxf(fmaxf(s[n][0][0].y, s[n][0][1].y), fmaxf(s[n][1][0].y, s[n][1][1].y));
                    grew |= top[n][0] > M[n][0] + kLag || top[n][1] > M[n][1] + kLag;
                }
                if (__any_sync(0xFFFFFFFFu, grew)) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            float m = top[n][j];
                            for (int o = 4; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
                            m = fmaxf(m, M[n][j]);
                            const float f = ex2(M[n][j] - m);
                            M[n][j] = m;
                            l[n][j] *= f;
#pragma unroll
                            for (int c = 0; c < kB; ++c)
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    O[n][c][h][j] *= f;
                                    O[n][c][h][2 + j] *= f;
                                }
                        }
                }
                // weights, transposed into B fragments (keys along k)
                uint32_t pf[NT][2][2];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float2 lv = make_float2(l[n][0], l[n][1]);
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const float2 d = __fadd2_rn(s[n][mt][h], make_float2(-M[n][0], -M[n][1]));
                            const float2 w = make_float2(ex2(d.x), ex2(d.y));
                            lv = __ffma2_rn(w, make_float2(y2[mt][h], y2[mt][h]), lv);
                            pf[n][mt][h] = transpose8x8(f16x2(w.x, w.y));
                        }
                    l[n][0] = lv.x;
                    l[n][1] = lv.y;
                }
                // O^T += V^T P^T: k of a step = positions 2t, 2t + 1, 8 + 2t, 9 + 2t
#pragma unroll
                for (int ks = 0; ks < 2; ++ks) {
                    uint32_t u[4][kB / 2];
                    const uint8_t* rv = buf + L.vcodes + 16 * ks * L.row + g * (D / 16);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint8_t* src = rv + (8 * (j >> 1) + swap_pos(2 * t + (j & 1))) * L.row;
                        if (D == 128) {
                            const uint2 v = *reinterpret_cast<const uint2*>(src);
                            u[j][0] = v.x;
                            u[j][kB / 2 - 1] = v.y;
                        } else {
                            u[j][0] = *reinterpret_cast<const uint32_t*>(src);
                        }
                    }
                    const uint4 sa4 = *reinterpret_cast<const uint4*>(sm.vscale[warp][t][ks][0]);
                    const uint4 sb4 = *reinterpret_cast<const uint4*>(sm.vscale[warp][t][ks][1]);
                    const uint32_t sa[4] = {sa4.x, sa4.y, sa4.z, sa4.w}, sb[4] = {sb4.x, sb4.y, sb4.z, sb4.w};
#pragma unroll
                    for (int c2 = 0; c2 < kB / 2; ++c2) {
                        uint32_t e01[4], o01[4], e23[4], o23[4];
                        const uint32_t lo = 0x0F0F0F0Fu, hi = 0xF0F0F0F0u;
                        e2m1x8_to_f16((u[0][c2] & lo) | ((u[1][c2] << 4) & hi), e01);
                        e2m1x8_to_f16(((u[0][c2] >> 4) & lo) | (u[1][c2] & hi), o01);
                        e2m1x8_to_f16((u[2][c2] & lo) | ((u[3][c2] << 4) & hi), e23);
                        e2m1x8_to_f16(((u[2][c2] >> 4) & lo) | (u[3][c2] & hi), o23);
#pragma unroll
                        for (int cc = 0; cc < 2; ++cc) {
                            const int c = 2 * c2 + cc;
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                const uint32_t w0 = hmul2(pf[n][ks][0], sa[c]), w1 = hmul2(pf[n][ks][1], sb[c]);
                                mma_f16(O[n][c][0], e01[2 * cc], o01[2 * cc], e23[2 * cc], o23[2 * cc], w0, w1);
                                mma_f16(O[n][c][1], e01[2 * cc + 1], o01[2 * cc + 1], e23[2 * cc + 1], o23[2 * cc + 1], w0, w1);
                            }
                        }
                    }
                }
            }
            __syncwarp();
            ++n_out;
            issue();
        }
        if (!ok) break;

        // the outputs of this part, and their log-sum-exp
        float L2[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float lt = l[n][j];
                for (int o = 4; o < 32; o <<= 1) lt += __shfl_xor_sync(0xFFFFFFFFu, lt, o);
                L2[n][j] = lt == 0.0f ? kNoMax : M[n][j] + __log2f(lt);
                const float inv = lt == 0.0f ? 0.0f : 1.0f / lt;
#pragma unroll
                for (int c = 0; c < kB; ++c) {
                    const float f = kUnit * pow2f(static_cast<int>(((c & 1 ? R13 : R02) >> (16 * (c >> 1))) & 0xFFu) - 127);  // exact
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        O[n][c][h][j] = O[n][c][h][j] * inv * f;
                        O[n][c][h][2 + j] = O[n][c][h][2 + j] * inv * f;
                    }
                }
            }
        // written where the segment is complete, kept as a piece where it is not
        const bool complete = !kWhole && seg_x >= pos_begin && seg_x + ng <= pos_end;
        const int slot = kWhole || i == count ? 1 : 0;  // (the ring is free at the end only)
        float* piece = slot ? reinterpret_cast<float*>(sm.ring[warp][0]) : &sm.first[warp][0][0];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int r = 8 * n + 2 * t + j;
                if (!complete) {
                    if (g == 0) sm.lse2[warp][slot][r] = L2[n][j];
#pragma unroll
                    for (int c = 0; c < kB; ++c)
                        *reinterpret_cast<float4*>(piece + r * kPitch + 32 * c + 4 * g) =
                            make_float4(O[n][c][0][j], O[n][c][0][2 + j], O[n][c][1][j], O[n][c][1][2 + j]);
                } else if (r0 + r < p.Sq * p.G) {
#pragma unroll
                    for (int c = 0; c < kB; ++c)
                        write_row<D>(p, b, hk, r0 + r, 8 * c + g,
                                     make_float4(O[n][c][0][j], O[n][c][0][2 + j], O[n][c][1][j], O[n][c][1][2 + j]), L2[n][j]);
                }
            }
        if (!complete && lane == 0) sm.piece[warp][slot] = {seg_x, b, seg, ng};
    }
    if (!ok) {
        // give up: let this warp's copies in flight land, then leave together
        if (lane == 0) {
            sm.abort = 1;
            atomicOr(p.err_word, kErrTimeout);
        }
        int dummy = 0;
        for (int k = n_out; k < n_in; ++k) mbar_wait(&sm.full[warp][k % kStages], (k / kStages) & 1, p.timeout_ns, &dummy);
    }
    // the second kernel's blocks may start as these finish
    if constexpr (!kWhole) asm volatile("griddepcontrol.launch_dependents;");
    sync();
    if (sm.abort) return;

    // join the warps' pieces: bit k of a mask is piece k & 1 of warp k / 2
    const Piece& own = sm.piece[(lane >> 1) % kWarps][lane & 1];
    const int own_b = lane < 2 * kWarps ? own.b : -1;
    const int64_t own_x = own.seg_x;
    unsigned left = __ballot_sync(0xFFFFFFFFu, own_b >= 0);
    int turn = warp;  // rows until this warp's next
    while (left) {
        const int k0 = __ffs(left) - 1;
        const int64_t seg_x = __shfl_sync(0xFFFFFFFFu, own_x, k0);
        const unsigned group = __ballot_sync(0xFFFFFFFFu, own_b >= 0 && own_x == seg_x);
        left &= ~group;
        const Piece pc = sm.piece[k0 >> 1][k0 & 1];
        const int hk = pc.seg / p.n_rt, r0 = (pc.seg % p.n_rt) * kRows;
        const int n_rows = min(kRows, p.Sq * p.G - r0);
        const bool whole = kWhole || (seg_x >= x && seg_x + pc.ng <= x_end);
        float* part = whole ? nullptr : p.partial + (2 * static_cast<int64_t>(team) + (seg_x < x ? 0 : 1)) * (kRows * (D + 1));
        if constexpr (!kWhole && NT == 1) {
            // the rows of all segments go around the warps (one segment after the
            // other by the whole team held the teams with many of them up by 20
            // us); with 16 rows or one segment a block that is no gain
            int r = turn;
            for (; r < n_rows; r += kWarps) {
                const bool in = (group >> lane) & 1u;
                const float x2 = in ? sm.lse2[(lane >> 1) % kWarps][lane & 1][r] : kNoMax;
                float m = x2;
                for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
                const float f = in ? ex2(x2 - m) : 0.0f;
                float sum = f;
                for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
                float4 v = make_float4(0, 0, 0, 0);
                for (unsigned rest = group; rest; rest &= rest - 1) {
                    const int k = __ffs(rest) - 1;
                    const float fk = __shfl_sync(0xFFFFFFFFu, f, k);
                    const float* src = (k & 1) ? reinterpret_cast<const float*>(sm.ring[k >> 1][0]) : &sm.first[k >> 1][0][0];
                    if (lane < D / 4) {
                        const float4 y = *reinterpret_cast<const float4*>(src + r * kPitch + 4 * lane);
                        v.x = fmaf(fk, y.x, v.x);
                        v.y = fmaf(fk, y.y, v.y);
                        v.z = fmaf(fk, y.z, v.z);
                        v.w = fmaf(fk, y.w, v.w);
                    }
                }
                const float inv = 1.0f / sum;
                v = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
                m += __log2f(sum);
                if (lane < D / 4) {
                    if (whole) {
                        write_row<D>(p, pc.b, hk, r0 + r, lane, v, m);
                    } else {
                        reinterpret_cast<float4*>(part)[r * (D / 4) + lane] = v;
                        if (lane == 0) part[kRows * D + r] = m;
                    }
                }
            }
            turn = r - n_rows;
        } else {
            for (int e = tid; e < n_rows * (D / 4); e += kThreads) {
                const int r = e / (D / 4), d4 = e % (D / 4);
                // (selected rather than branched on, so that the loads overlap; unrolled
                // no further, since a short call waits for the instructions themselves)
                float m = kNoMax, sum = 0.0f;
                float4 v = make_float4(0, 0, 0, 0);
#pragma unroll 4
                for (int k = kWhole ? 1 : 0; k < 2 * kWarps; k += kWhole ? 2 : 1)
                    m = fmaxf(m, (group >> k) & 1u ? sm.lse2[k >> 1][k & 1][r] : kNoMax);
#pragma unroll 4
                for (int k = kWhole ? 1 : 0; k < 2 * kWarps; k += kWhole ? 2 : 1) {
                    const bool in = (group >> k) & 1u;
                    const float* src = (k & 1) ? reinterpret_cast<const float*>(sm.ring[k >> 1][0]) : &sm.first[k >> 1][0][0];
                    const float4 y = in ? *reinterpret_cast<const float4*>(src + r * kPitch + 4 * d4) : make_float4(0, 0, 0, 0);
                    const float f = in ? ex2(sm.lse2[k >> 1][k & 1][r] - m) : 0.0f;
                    sum += f;
                    v.x = fmaf(f, y.x, v.x);
                    v.y = fmaf(f, y.y, v.y);
                    v.z = fmaf(f, y.z, v.z);
                    v.w = fmaf(f, y.w, v.w);
                }
                const float inv = 1.0f / sum;
                v = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
                m += __log2f(sum);
                if (whole) {
                    write_row<D>(p, pc.b, hk, r0 + r, d4, v, m);
                } else {
                    reinterpret_cast<float4*>(part)[r * (D / 4) + d4] = v;
                    if (d4 == 0) part[kRows * D + r] = m;
                }
            }
        }
    }
}

// Joins the parts of the segments that several teams worked on, and writes the
// rows of empty sequences.  A block takes kPer rows of a segment: a warp a row
// weighs the parts, then kSlices groups of kPer * D / 4 threads each add every
// kSlices-th part, so that a row split over all teams still waits for
// few loads in turn (8 segments of 38 parts: 12 us less than with one thread
// adding all of an element's parts).  One row a block where segments are few,
// four where they are many and their parts few (16 sequences, 64 segments: 20.7
// us for the whole call with one row a block, 18.7 with four).  Launched to
// overlap the end of the first kernel: what precedes the wait depends on the
// lengths alone, and every block waits before it ends, so that this kernel's end
// is the first one's, too.
template <int D, int NT, int kPer>
__global__ void __launch_bounds__(kJoinThreads) kv4_join_kernel(const Params p, int n_teams) {
    constexpr int kRows = 8 * NT, kLanes = D / 4, kSlices = kJoinThreads / (kLanes * kPer);
    __shared__ int64_t warp_sum[2][kJoinThreads / 32];
    __shared__ float row_lse2[kPer], row_inv[kPer];
    __shared__ float fac[kPer][kTeams];
    __shared__ float4 red[kSlices][kPer * kLanes];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n_seg = p.Hkv * p.n_rt;
    const int b = blockIdx.x / n_seg, seg = blockIdx.x - b * n_seg;
    const int r_first = blockIdx.y * kPer;
    const int hk = seg / p.n_rt, r0 = (seg % p.n_rt) * kRows;
    if (r0 + r_first >= p.Sq * p.G) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        return;
    }
    int64_t before = 0, total = 0;
    for (int i = tid; i < p.B; i += kJoinThreads) {
        const int n = places_of(seq_groups(p, i));
        total += n;
        if (i < b) before += n;
    }
    for (int o = 16; o; o >>= 1) {
        before += __shfl_xor_sync(0xFFFFFFFFu, before, o);
        total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
    }
    if (lane == 0) {
        warp_sum[0][warp] = before;
        warp_sum[1][warp] = total;
    }
    __syncthreads();
    before = total = 0;
    for (int w = 0; w < kJoinThreads / 32; ++w) {
        before += warp_sum[0][w];
        total += warp_sum[1][w];
    }
    const int ng = seq_groups(p, b);
    const int64_t share = share_of(total * n_seg, n_teams);
    const int64_t s0 = before * n_seg + static_cast<int64_t>(seg) * places_of(ng) + kSegmentCost;
    const int c0 = static_cast<int>(s0 / share), c1 = ng ? static_cast<int>((s0 + ng - 1) / share) : c0 - 1;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (c0 == c1) return;  // one team wrote the result

    // the segment starts in team c0's share, as its second part, and is the first
    // part of every later team
    const int n_parts = c1 - c0 + 1;
    auto part_of = [&](int j) {
        return p.partial + (2 * static_cast<int64_t>(c0 + j) + (j == 0 ? 1 : 0)) * (kRows * (D + 1));
    };
    if (warp < kPer) {
        const int r = r_first + warp;
        float m = kNoMax, sum = 0.0f;
        for (int j = lane; j < n_parts; j += 32) {
            const float x = part_of(j)[kRows * D + r];
            fac[warp][j] = x;
            m = fmaxf(m, x);
        }
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        for (int j = lane; j < n_parts; j += 32) {
            const float f = ex2(fac[warp][j] - m);
            fac[warp][j] = f;
            sum += f;
        }
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        if (lane == 0) {
            row_lse2[warp] = n_parts ? m + __log2f(sum) : kNoMax;
            row_inv[warp] = n_parts ? 1.0f / sum : 0.0f;
        }
    }
    __syncthreads();

    const int e = tid % (kPer * kLanes), slice = tid / (kPer * kLanes);
    const int k = e / kLanes, d4 = e % kLanes, r = r_first + k;
    float4 a = make_float4(0, 0, 0, 0);
#pragma unroll 4
    for (int j = slice; j < n_parts; j += kSlices) {
        const float f = fac[k][j];
        const float4 v = reinterpret_cast<const float4*>(part_of(j))[r * kLanes + d4];
        a.x = fmaf(f, v.x, a.x);
        a.y = fmaf(f, v.y, a.y);
        a.z = fmaf(f, v.z, a.z);
        a.w = fmaf(f, v.w, a.w);
    }
    red[slice][e] = a;
    __syncthreads();
    if (slice == 0 && r0 + r < p.Sq * p.G) {
#pragma unroll
        for (int i = 1; i < kSlices; ++i) {
            const float4 v = red[i][e];
            a.x += v.x;
            a.y += v.y;
            a.z += v.z;
            a.w += v.w;
        }
        const float inv = row_inv[k];
        write_row<D>(p, b, hk, r0 + r, d4, make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv), row_lse2[k]);
    }
}

// Query rows of a block: 8 or, beyond 8 rows to a key head, 16.
int row_tiles(int rows) { return rows <= 8 ? 1 : 2; }

bool takes_whole(int64_t segments, int page_size, int max_pages) {
    return static_cast<int64_t>(max_pages) * (page_size / kKv4Group) <= (segments >= kManySegments ? 2 : 1) * kWholeGroups;
}

int64_t segments_of(int B, int Sq, int Hq, int Hkv) {
    const int rows = Sq * (Hq / Hkv), per = 8 * row_tiles(rows);
    return static_cast<int64_t>(B) * Hkv * ((rows + per - 1) / per);
}

// The whole form in blocks of W warps.
template <int D, int NT, int W>
cudaError_t launch_whole(const Params& p, int segments, cudaStream_t st) {
    static KernelSetup setup;
    constexpr int smem = sizeof(Smem<D, NT, W>);
    const cudaError_t e = setup(reinterpret_cast<const void*>(kv4_attn_kernel<D, NT, true, W, 1>), smem, 0);
    if (e != cudaSuccess) return e;
    kv4_attn_kernel<D, NT, true, W, 1><<<segments, 32 * W, smem, st>>>(p);
    return cudaGetLastError();
}

// The split form in blocks of T teams, and the join.
template <int D, int NT, int T>
cudaError_t launch_split(const Params& p, int segments, cudaStream_t st) {
    static KernelSetup setup;
    constexpr int n_teams = kTeams / NT, smem = T * sizeof(Smem<D, NT, kTeamWarps>);
    static_assert(smem <= 232448, "shared memory beyond the 227 KB a block may use");
    cudaError_t e = setup(reinterpret_cast<const void*>(kv4_attn_kernel<D, NT, false, kTeamWarps, T>), smem, 0);
    if (e != cudaSuccess) return e;
    kv4_attn_kernel<D, NT, false, kTeamWarps, T><<<n_teams / T, 32 * kTeamWarps * T, smem, st>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const bool many = segments >= kManySegments;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(segments), static_cast<unsigned>(8 * NT / (many ? 4 : 1)));
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    e = many ? cudaLaunchKernelEx(&cfg, kv4_join_kernel<D, NT, 4>, p, n_teams)
             : cudaLaunchKernelEx(&cfg, kv4_join_kernel<D, NT, 1>, p, n_teams);
    if (e != cudaSuccess) cudaGetLastError();
    return e;
}

template <int D, int NT>
cudaError_t launch(const Params& p, int segments, cudaStream_t st) {
    if (!p.partial)
        return segments > kTeams / NT ? launch_whole<D, NT, kManyWarps>(p, segments, st)
                                       : launch_whole<D, NT, kFewWarps>(p, segments, st);
    if constexpr (NT == 1) {
        const int64_t most = static_cast<int64_t>(segments) * p.max_pages * (p.page_size / kKv4Group);
        if (most >= static_cast<int64_t>(kLongPart) * kTeams * kTeamWarps) return launch_split<D, NT, 2>(p, segments, st);
    }
    return launch_split<D, NT, 1>(p, segments, st);
}

}  // namespace

size_t kv4_attention_workspace_bytes(int B, int Sq, int Hq, int Hkv, int D, int page_size, int max_pages) {
    if (takes_whole(segments_of(B, Sq, Hq, Hkv), page_size, max_pages)) return 0;
    const int nt = row_tiles(Sq * (Hq / Hkv));
    return static_cast<size_t>(kTeams / nt) * 2 * (8 * nt) * (D + 1) * sizeof(float);
}

cudaError_t launch_kv4_attention(const Kv4AttnLaunch& a, cudaStream_t st) {
    Params p{};
    p.q = static_cast<const uint16_t*>(a.q);
    p.cache = a.cache;
    p.page_table = a.page_table;
    p.seq_lens = a.seq_lens;
    p.o = static_cast<uint16_t*>(a.o);
    p.lse = a.lse;
    const int64_t segments = segments_of(a.B, a.Sq, a.Hq, a.Hkv);
    p.partial = takes_whole(segments, a.page_size, a.max_pages) ? nullptr : static_cast<float*>(a.workspace);
    p.q_stride = a.q_stride;
    p.num_pages = a.num_pages;
    p.B = a.B;
    p.Sq = a.Sq;
    p.Hq = a.Hq;
    p.Hkv = a.Hkv;
    p.G = a.Hq / a.Hkv;
    const int rows = a.Sq * p.G, nt = row_tiles(rows);
    p.n_rt = (rows + 8 * nt - 1) / (8 * nt);
    p.page_size = a.page_size;
    p.max_pages = a.max_pages;
    p.c = static_cast<float>(static_cast<double>(a.sm_scale) * 1.4426950408889634);
    p.timeout_ns = a.timeout_ns;
    p.skip = a.debug_flags & 1;
    p.err_word = a.err_word;
    const int n = static_cast<int>(segments);
    if (a.D == 128) return nt == 1 ? launch<128, 1>(p, n, st) : launch<128, 2>(p, n, st);
    return nt == 1 ? launch<64, 1>(p, n, st) : launch<64, 2>(p, n, st);
}

}  // namespace fsa
