// capi.cu -- the C ABI of libfsa.so (declared in include/fsa.h): argument
// validation, the cached per-device workspace, TMA tensor maps and launches.
#include <cmath>
#include <cstring>
#include <mutex>

#include "fsa.h"
#include "fsa_internal.h"
#include "mx_operand.cuh"

namespace fsa {

namespace {

constexpr int kMaxDevices = 64;

// Library-owned resources of the host-buffer entry points: two chunk buffer
// sets (bf16 Q, K, V and O of a chunk of heads plus the chunk's MX
// workspace), a copy-in and a copy-out stream, a second compute stream, and
// the events that order them.
struct HostPipe {
    void* buf = nullptr;
    size_t bytes = 0;
    cudaStream_t h2d = nullptr, d2h = nullptr, comp1 = nullptr;
    cudaEvent_t in_ready[2] = {}, in_free[2] = {}, out_ready[2] = {}, out_free[2] = {};
    cudaEvent_t start = nullptr, copies_done = nullptr, comp1_done = nullptr;
    bool init = false;
    // buffer-set layout of the last call (heads per chunk and the shape it
    // was carved for); a call with another layout starts its copies only
    // after all of the last call's work
    int64_t last_G = 0, last_Sq = 0, last_Sk = 0, last_D = 0;
};

struct DeviceState {
    std::mutex mu;
    void* ws = nullptr;
    size_t ws_bytes = 0;
    unsigned int* err = nullptr;
    int arch_ok = -1;  // -1 unknown, 0 no, 1 yes
    HostPipe hp;
};
DeviceState g_dev[kMaxDevices];

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_tiled() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                             cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

// 3-D byte tensor map: dims (inner first), row strides in bytes, box.
bool make_map_u8(CUtensorMap* m, void* base, uint64_t d0, uint64_t d1, uint64_t d2,
                 uint64_t stride1, uint64_t stride2, uint32_t b0, uint32_t b1,
                 CUtensorMapSwizzle swz) {
    EncodeTiledFn fn = encode_tiled();
    if (!fn) return false;
    cuuint64_t dims[3] = {d0, d1, d2};
    cuuint64_t strides[2] = {stride1, stride2};
    cuuint32_t box[3] = {b0, b1, 1};
    cuuint32_t es[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, base, dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, swz, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 3-D bf16 tensor map.
bool make_map_bf16(CUtensorMap* m, void* base, uint64_t d0, uint64_t d1, uint64_t d2,
                   uint64_t stride1, uint64_t stride2, uint32_t b0, uint32_t b1,
                   CUtensorMapSwizzle swz) {
    EncodeTiledFn fn = encode_tiled();
    if (!fn) return false;
    cuuint64_t dims[3] = {d0, d1, d2};
    cuuint64_t strides[2] = {stride1, stride2};
    cuuint32_t box[3] = {b0, b1, 1};
    cuuint32_t es[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, swz, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// bf16 rows [T][H][D] (heads contiguous, tokens `stride` elements apart) in boxes
// of 64 channels x bh heads x bt tokens.
bool make_map_heads(CUtensorMap* m, const void* base, int D, int H, int T, int64_t stride, int bh, int bt) {
    EncodeTiledFn fn = encode_tiled();
    if (!fn) return false;
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(T)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(stride) * 2};
    cuuint32_t box[3] = {64, static_cast<cuuint32_t>(bh), static_cast<cuuint32_t>(bt)};
    cuuint32_t es[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Codes of an operand of the MX product in boxes of 128 bytes of shared memory x
// `box` rows; E2M1 codes stay packed, or are spread 16 to 16 bytes.
bool make_map_mx(CUtensorMap* m, const uint8_t* codes, int64_t rows, int64_t cols, int elem, bool spread, int box) {
    EncodeTiledFn fn = encode_tiled();
    if (!fn) return false;
    const int64_t pitch = mx_pitch(cols, elem);
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(spread ? 2 * pitch : pitch), static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(pitch)};
    cuuint32_t boxes[2] = {128, static_cast<cuuint32_t>(box)};
    cuuint32_t es[2] = {1, 1};
    return fn(m, spread ? CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2,
              const_cast<uint8_t*>(codes), dims, strides, boxes, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Its scales in boxes of `atoms` atoms (8-byte elements) of `groups` groups of 128 rows.
bool make_map_mx_scales(CUtensorMap* m, const uint8_t* scales, int64_t rows, int64_t cols, int atoms, int groups) {
    EncodeTiledFn fn = encode_tiled();
    if (!fn) return false;
    constexpr int kWords = kAtomBytes / 8;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(mx_atoms(cols) * kWords), static_cast<cuuint64_t>(mx_atoms(rows))};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(mx_atoms(cols) * kAtomBytes)};
    cuuint32_t boxes[2] = {static_cast<cuuint32_t>(atoms * kWords), static_cast<cuuint32_t>(groups)};
    cuuint32_t es[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT64, 2, const_cast<uint8_t*>(scales), dims, strides, boxes, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Current device, its state, and the architecture check (sm_100 / sm_103).
fsa_status current_device(int* dev_out, DeviceState** st_out) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return FSA_ERR_CUDA;
    if (dev < 0 || dev >= kMaxDevices) return FSA_ERR_UNSUPPORTED;
    DeviceState& st = g_dev[dev];
    std::lock_guard<std::mutex> lk(st.mu);
    if (st.arch_ok < 0) {
        int major = 0, minor = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
            return FSA_ERR_CUDA;
        st.arch_ok = (major == 10 && (minor == 0 || minor == 3)) ? 1 : 0;
    }
    if (!st.arch_ok) return FSA_ERR_UNSUPPORTED;
    if (!st.err) {
        if (cudaMalloc(&st.err, sizeof(unsigned int)) != cudaSuccess) return FSA_ERR_OUT_OF_MEMORY;
        if (cudaMemset(st.err, 0, sizeof(unsigned int)) != cudaSuccess) return FSA_ERR_CUDA;
    }
    *dev_out = dev;
    *st_out = &st;
    return FSA_OK;
}

fsa_status validate_attention(const void* q, const void* k, const void* v, const void* o, int B,
                              int H, int Sq, int Sk, int D) {
    if (!q || !k || !v || !o) return FSA_ERR_INVALID_ARGUMENT;
    if (B < 1 || H < 1 || Sq < 1 || Sk < 1) return FSA_ERR_INVALID_ARGUMENT;
    if (D != 64 && D != 128) return FSA_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(B) * H > 65535) return FSA_ERR_INVALID_ARGUMENT;
    if (Sq > (1 << 30) || Sk > (1 << 30)) return FSA_ERR_INVALID_ARGUMENT;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o))
        return FSA_ERR_INVALID_ARGUMENT;
    return FSA_OK;
}

}  // namespace

size_t attn_workspace_bytes(int64_t BH, int64_t Sq, int64_t Sk, int D) {
    const int64_t Sk16 = (Sk + 15) / 16 * 16;
    const int64_t ntq = (Sq + kTile - 1) / kTile, ntk = (Sk + kTile - 1) / kTile;
    return align256(BH * Sq * D) + align256(BH * Sk * D) + align256(BH * D * Sk16) +
           align256((ntq + 2 * ntk) * BH * static_cast<int64_t>(kAtomBytes)) +
           align256(BH * Sq * 4) + align256(BH * ntk * 4);
}

AttnWorkspace attn_workspace_carve(void* base, int64_t BH, int64_t Sq, int64_t Sk, int D) {
    const int64_t Sk16 = (Sk + 15) / 16 * 16;
    const int64_t ntq = (Sq + kTile - 1) / kTile, ntk = (Sk + kTile - 1) / kTile;
    uint8_t* p = static_cast<uint8_t*>(base);
    AttnWorkspace w{};
    w.qc = p; p += align256(BH * Sq * D);
    w.kc = p; p += align256(BH * Sk * D);
    w.vt = p; p += align256(BH * D * Sk16);
    const size_t atoms_q = static_cast<size_t>(BH * ntq) * kAtomBytes;
    const size_t atoms_k = static_cast<size_t>(BH * ntk) * kAtomBytes;
    w.qsf = p;
    w.ksf = p + atoms_q;
    w.vsf = p + atoms_q + atoms_k;
    w.sf_bytes_total = atoms_q + 2 * atoms_k;
    p += align256(static_cast<int64_t>(w.sf_bytes_total));
    w.qnorm = reinterpret_cast<float*>(p); p += align256(BH * Sq * 4);
    w.knorm = reinterpret_cast<float*>(p);
    return w;
}

}  // namespace fsa

namespace fsa {
namespace {

fsa_status check_run_args(int fmt, float threshold, const fsa_options& op) {
    if (fmt < 0 || fmt > 3) return FSA_ERR_INVALID_ARGUMENT;
    if (!std::isfinite(threshold) || threshold < 0.0f || threshold > 80.0f)
        return FSA_ERR_INVALID_ARGUMENT;
    if (!std::isfinite(op.sm_scale)) return FSA_ERR_INVALID_ARGUMENT;
    if (fmt == FSA_MXFP4_EFQ && (!std::isfinite(op.efq_tau) || !std::isfinite(op.efq_h)))
        return FSA_ERR_INVALID_ARGUMENT;
    if (op.gate_mode != 0 && op.gate_mode != 1) return FSA_ERR_INVALID_ARGUMENT;
    return FSA_OK;
}

fsa_status check_workspace(const void* ws, uint64_t bytes, int64_t BH, int Sq, int Sk, int D) {
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255)) return FSA_ERR_INVALID_ARGUMENT;
    if (bytes < attn_workspace_bytes(BH, Sq, Sk, D)) return FSA_ERR_INVALID_ARGUMENT;
    return FSA_OK;
}

// Quantizes Q, K (blocks along D) and V (blocks along keys, transposed).
fsa_status prepare_impl(const void* q, const void* k, const void* v, int64_t BH, int Sq, int Sk,
                        int D, int fmt, void* ws_base, cudaStream_t st) {
    AttnWorkspace ws = attn_workspace_carve(ws_base, BH, Sq, Sk, D);
    const int elem = fmt == FSA_MXFP8 ? ELEM_E4M3 : (fmt == FSA_MXFP6 ? ELEM_E2M3 : ELEM_E2M1);
    const int64_t Sk16 = (static_cast<int64_t>(Sk) + 15) / 16 * 16;
    // six-bit P: norm bounds of the quantized rows of Q and (per KV tile) of K,
    // from which the fused kernel proves that no weight of a row can underflow
    const bool norms = fmt == FSA_MXFP6 || fmt == FSA_MXFP4;
    const int64_t ntk = (static_cast<int64_t>(Sk) + kTile - 1) / kTile;
    if (cudaMemsetAsync(ws.qsf, 0x7F, ws.sf_bytes_total, st) != cudaSuccess) return FSA_ERR_CUDA;
    if (norms && cudaMemsetAsync(ws.knorm, 0, static_cast<size_t>(BH * ntk) * 4, st) != cudaSuccess)
        return FSA_ERR_CUDA;
    if (launch_quant_rows(static_cast<const uint16_t*>(q), BH * Sq, D, elem, QL_ATTN, ws.qc, ws.qsf,
                          Sq, st, ws.qnorm, norms ? NORM_ROW : NORM_NONE) != cudaSuccess ||
        launch_quant_rows(static_cast<const uint16_t*>(k), BH * Sk, D, elem, QL_ATTN, ws.kc, ws.ksf,
                          Sk, st, ws.knorm, norms ? NORM_TILE_MAX : NORM_NONE) != cudaSuccess ||
        launch_quant_cols(static_cast<const uint16_t*>(v), BH, Sk, D, elem, QL_ATTN, ws.vt, Sk16,
                          ws.vsf, st) != cudaSuccess)
        return FSA_ERR_CUDA;
    return FSA_OK;
}

// The fused attention kernel on a prepared workspace.
fsa_status run_impl(void* ws_base, void* o, int64_t BH, int Sq, int Sk, int D, int fmt,
                    float threshold, const fsa_options& op, unsigned int* err, cudaStream_t st) {
    AttnWorkspace ws = attn_workspace_carve(ws_base, BH, Sq, Sk, D);
    const int64_t Sk16 = (static_cast<int64_t>(Sk) + 15) / 16 * 16;
    CUtensorMap tq, tk, tv;
    const CUtensorMapSwizzle qk_swz =
        D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
    if (!make_map_u8(&tq, ws.qc, D, Sq, BH, D, static_cast<uint64_t>(Sq) * D, D, kTile, qk_swz) ||
        !make_map_u8(&tk, ws.kc, D, Sk, BH, D, static_cast<uint64_t>(Sk) * D, D, kTile, qk_swz) ||
        !make_map_u8(&tv, ws.vt, Sk16, D, BH, Sk16, static_cast<uint64_t>(Sk16) * D, kTile, D,
                     CU_TENSOR_MAP_SWIZZLE_128B))
        return FSA_ERR_CUDA;
    AttnLaunch a{};
    a.tm_q = &tq;
    a.tm_k = &tk;
    a.tm_v = &tv;
    a.ws = ws;
    a.o = o;
    a.BH = BH;
    a.Sq = Sq;
    a.Sk = Sk;
    a.D = D;
    a.fmt = fmt;
    a.sm_scale = op.sm_scale > 0.0f ? op.sm_scale : 1.0f / std::sqrt(static_cast<float>(D));
    a.threshold = threshold;
    // EFQ affine rule: the library's offline calibration unless given
    a.efq_tau = op.efq_h > 0.0f ? op.efq_tau : -2.44f;
    a.efq_h = op.efq_h > 0.0f ? op.efq_h : 0.61f;
    a.rollback_bits = op.rollback_bits;
    a.rollback_count = op.rollback_count;
    a.timeout_ns = static_cast<uint64_t>(op.wait_timeout_ms > 0 ? op.wait_timeout_ms : 2000) *
                   1000000ull;
    a.debug_flags = op.debug_flags;
    a.gate_mode = op.gate_mode;
    a.err_word = err;
    // the kernel writes only the bytes of firings
    if (op.rollback_bits &&
        cudaMemsetAsync(op.rollback_bits, 0, static_cast<size_t>(BH) * Sq * ((Sk + kTile - 1) / kTile), st) !=
            cudaSuccess)
        return FSA_ERR_CUDA;
    return launch_fsa_attention(a, st) == cudaSuccess ? FSA_OK : FSA_ERR_CUDA;
}

// Lazily creates the streams and events of the host-buffer pipeline.
fsa_status host_pipe_init(HostPipe& hp) {
    if (hp.init) return FSA_OK;
    if (cudaStreamCreateWithFlags(&hp.h2d, cudaStreamNonBlocking) != cudaSuccess ||
        cudaStreamCreateWithFlags(&hp.d2h, cudaStreamNonBlocking) != cudaSuccess ||
        cudaStreamCreateWithFlags(&hp.comp1, cudaStreamNonBlocking) != cudaSuccess)
        return FSA_ERR_CUDA;
    cudaEvent_t* evs[] = {&hp.in_ready[0], &hp.in_ready[1], &hp.in_free[0], &hp.in_free[1],
                          &hp.out_ready[0], &hp.out_ready[1], &hp.out_free[0], &hp.out_free[1],
                          &hp.start, &hp.copies_done, &hp.comp1_done};
    for (cudaEvent_t* e : evs)
        if (cudaEventCreateWithFlags(e, cudaEventDisableTiming) != cudaSuccess) return FSA_ERR_CUDA;
    hp.init = true;
    return FSA_OK;
}

// Heads per chunk of the host-buffer pipeline: about eight chunks, each at
// least two waves of 152-SM query-tile CTAs, never more heads than exist.
int64_t host_chunk_heads(int64_t BH, int Sq) {
    const int64_t n_qt = (static_cast<int64_t>(Sq) + kTile - 1) / kTile;
    int64_t g = (BH + 7) / 8;
    const int64_t min_g = (304 + n_qt - 1) / n_qt;
    if (g < min_g) g = min_g;
    return g < BH ? g : BH;
}

// The attention of host-resident q, k, v into host o, streamed through the
// device in chunks of heads.  Chunk c uses buffer set c % 2 and runs its
// quantizer and fused kernel on the caller's stream (even c) or the
// library's second compute stream (odd c), so consecutive chunks' kernels
// overlap at their tails; its inputs are copied in on the copy-in stream
// while the previous chunk computes, and its output copied out on the
// copy-out stream while the next one computes.  Each buffer's reuse waits
// on the event of its last reader.  The caller's stream finally waits for
// the last copy-out and the second compute stream.
fsa_status host_fwd_impl(DeviceState& ds, const uint16_t* q, const uint16_t* k, const uint16_t* v,
                         uint16_t* o, int64_t BH, int Sq, int Sk, int D, int fmt, float threshold,
                         const fsa_options& op, cudaStream_t st) {
    HostPipe& hp = ds.hp;
    fsa_status s = host_pipe_init(hp);
    if (s != FSA_OK) return s;
    const int64_t G = host_chunk_heads(BH, Sq);
    const size_t q_bytes = static_cast<size_t>(G) * Sq * D * 2, kv_bytes = static_cast<size_t>(G) * Sk * D * 2;
    const size_t ws_bytes = attn_workspace_bytes(G, Sq, Sk, D);
    const size_t set_bytes = 2 * align256(q_bytes) + 2 * align256(kv_bytes) + align256(ws_bytes);
    if (hp.bytes < 2 * set_bytes) {
        if (hp.buf) {
            cudaDeviceSynchronize();
            cudaFree(hp.buf);
            hp.buf = nullptr;
            hp.bytes = 0;
        }
        if (cudaMalloc(&hp.buf, 2 * set_bytes) != cudaSuccess) {
            cudaGetLastError();
            return FSA_ERR_OUT_OF_MEMORY;
        }
        hp.bytes = 2 * set_bytes;
    }
    uint8_t* dq[2], *dk[2], *dv[2], *dout[2], *dws[2];
    for (int i = 0; i < 2; ++i) {
        uint8_t* p = static_cast<uint8_t*>(hp.buf) + i * set_bytes;
        dq[i] = p; p += align256(q_bytes);
        dout[i] = p; p += align256(q_bytes);
        dk[i] = p; p += align256(kv_bytes);
        dv[i] = p; p += align256(kv_bytes);
        dws[i] = p;
    }
    // a different layout carves the buffer sets at other offsets, so a
    // region this call writes may be one the last call's kernels or copies
    // still use under another name: the copy-in (and through its events
    // everything after it) waits for the whole last call, whose copy-outs
    // follow all of its kernels.  With the same layout the per-set events
    // below order every reuse.
    const bool relayout = hp.last_G != G || hp.last_Sq != Sq || hp.last_Sk != Sk || hp.last_D != D;
    if (relayout && (cudaStreamWaitEvent(hp.h2d, hp.copies_done, 0) != cudaSuccess ||
                     cudaStreamWaitEvent(hp.h2d, hp.comp1_done, 0) != cudaSuccess))
        return FSA_ERR_CUDA;
    hp.last_G = G;
    hp.last_Sq = Sq;
    hp.last_Sk = Sk;
    hp.last_D = D;
    // everything already on the caller's stream comes first (for the
    // copy-in only unless the caller declared the host inputs final)
    if (cudaEventRecord(hp.start, st) != cudaSuccess ||
        (!op.host_inputs_ready && cudaStreamWaitEvent(hp.h2d, hp.start, 0) != cudaSuccess) ||
        cudaStreamWaitEvent(hp.comp1, hp.start, 0) != cudaSuccess ||
        cudaStreamWaitEvent(hp.d2h, hp.start, 0) != cudaSuccess)
        return FSA_ERR_CUDA;
    const int64_t n_t = (static_cast<int64_t>(Sk) + kTile - 1) / kTile;
    for (int64_t h0 = 0, c = 0; h0 < BH; h0 += G, ++c) {
        const int i = static_cast<int>(c & 1);
        const int64_t g = BH - h0 < G ? BH - h0 : G;
        const size_t qb = static_cast<size_t>(g) * Sq * D * 2, kb = static_cast<size_t>(g) * Sk * D * 2;
        const size_t qo = static_cast<size_t>(h0) * Sq * D, ko = static_cast<size_t>(h0) * Sk * D;
        cudaStream_t cs = i ? hp.comp1 : st;
        // copy in once the quantizer of the chunk two back has read the buffers
        if (cudaStreamWaitEvent(hp.h2d, hp.in_free[i], 0) != cudaSuccess ||
            cudaMemcpyAsync(dq[i], q + qo, qb, cudaMemcpyHostToDevice, hp.h2d) != cudaSuccess ||
            cudaMemcpyAsync(dk[i], k + ko, kb, cudaMemcpyHostToDevice, hp.h2d) != cudaSuccess ||
            cudaMemcpyAsync(dv[i], v + ko, kb, cudaMemcpyHostToDevice, hp.h2d) != cudaSuccess ||
            cudaEventRecord(hp.in_ready[i], hp.h2d) != cudaSuccess)
            return FSA_ERR_CUDA;
        // quantize (once the inputs landed and the last fused kernel that read
        // this workspace -- possibly a previous call's on another stream --
        // finished), then attend once the copy-out of the chunk two back is done
        if (cudaStreamWaitEvent(cs, hp.in_ready[i], 0) != cudaSuccess ||
            cudaStreamWaitEvent(cs, hp.out_ready[i], 0) != cudaSuccess)
            return FSA_ERR_CUDA;
        s = prepare_impl(dq[i], dk[i], dv[i], g, Sq, Sk, D, fmt, dws[i], cs);
        if (s != FSA_OK) return s;
        if (cudaEventRecord(hp.in_free[i], cs) != cudaSuccess ||
            cudaStreamWaitEvent(cs, hp.out_free[i], 0) != cudaSuccess)
            return FSA_ERR_CUDA;
        fsa_options oc = op;
        oc.rollback_bits = op.rollback_bits ? op.rollback_bits + static_cast<size_t>(h0) * Sq * n_t : nullptr;
        s = run_impl(dws[i], dout[i], g, Sq, Sk, D, fmt, threshold, oc, ds.err, cs);
        if (s != FSA_OK) return s;
        if (cudaEventRecord(hp.out_ready[i], cs) != cudaSuccess ||
            cudaStreamWaitEvent(hp.d2h, hp.out_ready[i], 0) != cudaSuccess ||
            cudaMemcpyAsync(o + qo, dout[i], qb, cudaMemcpyDeviceToHost, hp.d2h) != cudaSuccess ||
            cudaEventRecord(hp.out_free[i], hp.d2h) != cudaSuccess)
            return FSA_ERR_CUDA;
    }
    if (cudaEventRecord(hp.copies_done, hp.d2h) != cudaSuccess ||
        cudaEventRecord(hp.comp1_done, hp.comp1) != cudaSuccess ||
        cudaStreamWaitEvent(st, hp.copies_done, 0) != cudaSuccess ||
        cudaStreamWaitEvent(st, hp.comp1_done, 0) != cudaSuccess)
        return FSA_ERR_CUDA;
    return FSA_OK;
}

// Device address of the non-allocating entry point's status word on device
// dev, or null before that entry point was set up there.
unsigned int* noalloc_status_word(int dev);

}  // namespace
}  // namespace fsa

using namespace fsa;

extern "C" {

const char* fsa_status_string(fsa_status s) {
    switch (s) {
        case FSA_OK: return "ok";
        case FSA_ERR_INVALID_ARGUMENT: return "invalid argument";
        case FSA_ERR_UNSUPPORTED: return "unsupported device or shape";
        case FSA_ERR_CUDA: return "CUDA error";
        case FSA_ERR_OUT_OF_MEMORY: return "out of device memory";
        case FSA_ERR_TIMEOUT: return "a kernel's bounded wait timed out";
    }
    return "unknown status";
}

fsa_status fsa_quantize_mx(const void* x, int64_t batch, int64_t rows, int64_t cols,
                           int block_axis, int elem_fmt, uint8_t* codes, uint8_t* scales,
                           void* stream) {
    if (!x || !codes || !scales) return FSA_ERR_INVALID_ARGUMENT;
    if (batch < 0 || rows < 0 || cols < 0) return FSA_ERR_INVALID_ARGUMENT;
    if (elem_fmt < 0 || elem_fmt > 2 || (block_axis != 0 && block_axis != 1))
        return FSA_ERR_INVALID_ARGUMENT;
    if ((reinterpret_cast<uintptr_t>(x) & 1) != 0) return FSA_ERR_INVALID_ARGUMENT;
    if (block_axis == 0 && (batch > 65535 || cols > (int64_t(65535) * 128)))
        return FSA_ERR_INVALID_ARGUMENT;
    if (batch == 0 || rows == 0 || cols == 0) return FSA_OK;
    int dev;
    DeviceState* ds;
    fsa_status s = current_device(&dev, &ds);
    if (s != FSA_OK) return s;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (block_axis == 1)
        e = launch_quant_rows(static_cast<const uint16_t*>(x), batch * rows, cols, elem_fmt,
                              QL_PLAIN, codes, scales, 0, st);
    else
        e = launch_quant_cols(static_cast<const uint16_t*>(x), batch, rows, cols, elem_fmt,
                              QL_PLAIN, codes, rows, scales, st);
    return e == cudaSuccess ? FSA_OK : FSA_ERR_CUDA;
}

uint64_t fsa_kv4_page_bytes(int H_kv, int page_size, int D) {
    if (H_kv < 1 || H_kv > 65535 || page_size < 32 || page_size > 65536 || page_size % 32 != 0 || (D != 64 && D != 128))
        return 0;
    return static_cast<uint64_t>(H_kv) * (page_size / 32) * (34 * D);
}

namespace {

// Shape of a four-bit cache and its address.
fsa_status check_kv4(const void* cache, int64_t num_pages, int page_size, int H_kv, int D) {
    if (!cache || !aligned16(cache)) return FSA_ERR_INVALID_ARGUMENT;
    if (D != 64 && D != 128) return FSA_ERR_UNSUPPORTED;
    // (groups are numbered in 32 bits, two numbers set aside: 2^32 of them would be 9 TB)
    if (num_pages < 1 || num_pages > INT32_MAX || fsa_kv4_page_bytes(H_kv, page_size, D) == 0 ||
        num_pages * H_kv * (page_size / 32) >= int64_t{UINT32_MAX})
        return FSA_ERR_INVALID_ARGUMENT;
    return FSA_OK;
}

uint64_t wait_limit_ns(const fsa_options& op) {
    return static_cast<uint64_t>(op.wait_timeout_ms > 0 ? op.wait_timeout_ms : 2000) * 1000000ull;
}

bool token_stride_ok(int64_t stride, int64_t least) { return stride >= least && stride % 8 == 0 && stride < (int64_t{1} << 36); }

fsa_status kv4_rows(const void* k, const void* v, int64_t k_stride, int64_t v_stride, const int64_t* slots, int64_t T,
                    int H_kv, int D, const void* cache, int64_t num_pages, int page_size, int64_t least, Kv4Rows* a) {
    fsa_status s = check_kv4(cache, num_pages, page_size, H_kv, D);
    if (s != FSA_OK) return s;
    if (T < 0 || T > INT32_MAX || (T + 63) / 64 * H_kv > INT32_MAX) return FSA_ERR_INVALID_ARGUMENT;
    if (T > 0 && (!k || !v || !slots || !aligned16(k) || !aligned16(v) || (reinterpret_cast<uintptr_t>(slots) & 7) ||
                  !token_stride_ok(k_stride, least) || !token_stride_ok(v_stride, least)))
        return FSA_ERR_INVALID_ARGUMENT;
    *a = Kv4Rows{k, v, k_stride, v_stride, slots, T, num_pages * page_size, H_kv, D, page_size, nullptr};
    return FSA_OK;
}

}  // namespace

fsa_status fsa_kv4_append(const void* k, const void* v, int64_t k_stride, int64_t v_stride, const int64_t* slots,
                          int64_t T, int H_kv, int D, void* cache, int64_t num_pages, int page_size, void* stream) {
    Kv4Rows a;
    fsa_status s = kv4_rows(k, v, k_stride, v_stride, slots, T, H_kv, D, cache, num_pages, page_size, 0, &a);
    if (s != FSA_OK || T == 0) return s;
    int dev;
    DeviceState* ds;
    s = current_device(&dev, &ds);
    if (s != FSA_OK) return s;
    a.err_word = ds->err;
    return launch_kv4_append(a, static_cast<uint8_t*>(cache), static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? FSA_OK : FSA_ERR_CUDA;
}

fsa_status fsa_kv4_read(const void* cache, int64_t num_pages, int page_size, const int64_t* slots, int64_t T, int H_kv,
                        int D, void* k, void* v, int64_t k_stride, int64_t v_stride, void* stream) {
    Kv4Rows a;
    fsa_status s = kv4_rows(k, v, k_stride, v_stride, slots, T, H_kv, D, cache, num_pages, page_size,
                            static_cast<int64_t>(H_kv) * D, &a);
    if (s != FSA_OK || T == 0) return s;
    int dev;
    DeviceState* ds;
    s = current_device(&dev, &ds);
    if (s != FSA_OK) return s;
    a.err_word = ds->err;
    return launch_kv4_read(a, static_cast<const uint8_t*>(cache), static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? FSA_OK : FSA_ERR_CUDA;
}

namespace {

fsa_status check_kv4_attention(int B, int Sq, int Hq, int Hkv, int D, int page_size, int max_pages) {
    if (D != 64 && D != 128) return FSA_ERR_UNSUPPORTED;
    if (B < 1 || B > 65535 || Sq < 1 || Hq < 1 || Hkv < 1 || Hkv > 65535 || Hq % Hkv != 0 ||
        static_cast<int64_t>(Sq) * (Hq / Hkv) > 65535 || max_pages < 1 ||
        fsa_kv4_page_bytes(Hkv, page_size, D) == 0 || static_cast<int64_t>(max_pages) * page_size > (1 << 30))
        return FSA_ERR_INVALID_ARGUMENT;
    // (eight-row tiles of all sequences and key heads number the blocks of a grid;
    // a warp counts the 32-key groups of its part in 32 bits)
    const int64_t tiles = static_cast<int64_t>(B) * Hkv * ((static_cast<int64_t>(Sq) * (Hq / Hkv) + 7) / 8);
    if (tiles > INT32_MAX || tiles > (int64_t{1} << 40) / (max_pages * static_cast<int64_t>(page_size / 32) + 4))
        return FSA_ERR_INVALID_ARGUMENT;
    return FSA_OK;
}

}  // namespace

uint64_t fsa_kv4_attention_workspace_size(int B, int Sq, int Hq, int Hkv, int D, int page_size, int max_pages) {
    if (check_kv4_attention(B, Sq, Hq, Hkv, D, page_size, max_pages) != FSA_OK) return 0;
    return kv4_attention_workspace_bytes(B, Sq, Hq, Hkv, D, page_size, max_pages);
}

fsa_status fsa_kv4_attention_fwd(const void* q, int64_t q_stride, const void* cache, const int32_t* page_table,
                                 const int32_t* seq_lens, void* o, float* lse, int B, int Sq, int Hq, int Hkv, int D,
                                 int64_t num_pages, int page_size, int max_pages, float sm_scale, void* workspace,
                                 uint64_t workspace_bytes, void* stream) {
    fsa_options op{};
    op.sm_scale = sm_scale;
    op.workspace = workspace;
    op.workspace_bytes = workspace_bytes;
    return fsa_kv4_attention_fwd_ex(q, q_stride, cache, page_table, seq_lens, o, lse, B, Sq, Hq, Hkv, D, num_pages,
                                    page_size, max_pages, &op, stream);
}

fsa_status fsa_kv4_attention_fwd_ex(const void* q, int64_t q_stride, const void* cache, const int32_t* page_table,
                                    const int32_t* seq_lens, void* o, float* lse, int B, int Sq, int Hq, int Hkv, int D,
                                    int64_t num_pages, int page_size, int max_pages, const fsa_options* opt,
                                    void* stream) {
    const fsa_options op = opt ? *opt : fsa_options{};
    fsa_status s = check_kv4_attention(B, Sq, Hq, Hkv, D, page_size, max_pages);
    if (s != FSA_OK) return s;
    s = check_kv4(cache, num_pages, page_size, Hkv, D);
    if (s != FSA_OK) return s;
    if (!q || !o || !page_table || !seq_lens || !aligned16(q) || !aligned16(o) ||
        (reinterpret_cast<uintptr_t>(page_table) & 3) || (reinterpret_cast<uintptr_t>(seq_lens) & 3) ||
        (reinterpret_cast<uintptr_t>(lse) & 3) || !token_stride_ok(q_stride, 0) || !std::isfinite(op.sm_scale))
        return FSA_ERR_INVALID_ARGUMENT;
    const uint64_t need = kv4_attention_workspace_bytes(B, Sq, Hq, Hkv, D, page_size, max_pages);
    if (need && (!op.workspace || (reinterpret_cast<uintptr_t>(op.workspace) & 255) || op.workspace_bytes < need))
        return FSA_ERR_INVALID_ARGUMENT;
    int dev;
    DeviceState* ds;
    s = current_device(&dev, &ds);
    if (s != FSA_OK) return s;
    Kv4AttnLaunch a{};
    a.q = q;
    a.q_stride = q_stride;
    a.cache = static_cast<const uint8_t*>(cache);
    a.page_table = page_table;
    a.seq_lens = seq_lens;
    a.o = o;
    a.lse = lse;
    a.workspace = op.workspace;
    a.num_pages = num_pages;
    a.B = B;
    a.Sq = Sq;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.D = D;
    a.page_size = page_size;
    a.max_pages = max_pages;
    a.sm_scale = op.sm_scale > 0.0f ? op.sm_scale : 1.0f / std::sqrt(static_cast<float>(D));
    a.timeout_ns = wait_limit_ns(op);
    a.debug_flags = op.debug_flags;
    a.err_word = ds->err;
    return launch_kv4_attention(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FSA_OK : FSA_ERR_CUDA;
}

fsa_status fsa_varlen_attention_fwd(const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride,
                                    int64_t v_stride, const int32_t* cu_q, const int32_t* cu_k, void* o, float* lse,
                                    int B, int Tq, int Tk, int Hq, int Hkv, int D, int causal, float sm_scale,
                                    void* stream) {
    fsa_options op{};
    op.sm_scale = sm_scale;
    return fsa_varlen_attention_fwd_ex(q, k, v, q_stride, k_stride, v_stride, cu_q, cu_k, o, lse, B, Tq, Tk, Hq, Hkv, D,
                                       causal, &op, stream);
}

fsa_status fsa_varlen_attention_fwd_ex(const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride,
                                       int64_t v_stride, const int32_t* cu_q, const int32_t* cu_k, void* o, float* lse,
                                       int B, int Tq, int Tk, int Hq, int Hkv, int D, int causal,
                                       const fsa_options* opt, void* stream) {
    const fsa_options op = opt ? *opt : fsa_options{};
    if (D != 64 && D != 128) return FSA_ERR_UNSUPPORTED;
    // (with more keys one pair of query tiles could outlast the kernel's bounded waits)
    if (B < 1 || Tq < 0 || Tk < 0 || Tq > (1 << 26) || Tk > (1 << 26) || Hq < 1 || Hkv < 1 || Hkv > 65535 ||
        Hq % Hkv != 0 || Hq / Hkv > 128 || (causal != 0 && causal != 1) || !std::isfinite(op.sm_scale))
        return FSA_ERR_INVALID_ARGUMENT;
    if ((Tq / (2 * (128 / (Hq / Hkv))) + static_cast<int64_t>(B)) * Hkv > INT32_MAX) return FSA_ERR_INVALID_ARGUMENT;
    if (!cu_q || !cu_k || (reinterpret_cast<uintptr_t>(cu_q) & 3) || (reinterpret_cast<uintptr_t>(cu_k) & 3) ||
        (reinterpret_cast<uintptr_t>(lse) & 3))
        return FSA_ERR_INVALID_ARGUMENT;
    if (Tq > 0 && (!q || !o || !aligned16(q) || !aligned16(o) || !token_stride_ok(q_stride, static_cast<int64_t>(Hq) * D)))
        return FSA_ERR_INVALID_ARGUMENT;
    if (Tk > 0 && (!k || !v || !aligned16(k) || !aligned16(v) ||
                   !token_stride_ok(k_stride, static_cast<int64_t>(Hkv) * D) ||
                   !token_stride_ok(v_stride, static_cast<int64_t>(Hkv) * D)))
        return FSA_ERR_INVALID_ARGUMENT;
    if (Tq == 0) return FSA_OK;
    int dev;
    DeviceState* ds;
    fsa_status s = current_device(&dev, &ds);
    if (s != FSA_OK) return s;
    // a query tile is 128 / G whole tokens of the G heads of a key head; without
    // any keys the maps of K and V are never used
    const int G = Hq / Hkv;
    CUtensorMap tq, tk, tv;
    if (!make_map_heads(&tq, q, D, Hq, Tq, q_stride, G, 128 / G) ||
        (Tk > 0 && (!make_map_heads(&tk, k, D, Hkv, Tk, k_stride, 1, 128) ||
                    !make_map_heads(&tv, v, D, Hkv, Tk, v_stride, 1, 128))))
        return FSA_ERR_CUDA;
    if (Tk == 0) tk = tv = tq;
    VarlenLaunch a{};
    a.tm_q = &tq;
    a.tm_k = &tk;
    a.tm_v = &tv;
    a.o = o;
    a.lse = lse;
    a.cu_q = cu_q;
    a.cu_k = cu_k;
    a.B = B;
    a.Tq = Tq;
    a.Tk = Tk;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.D = D;
    a.causal = causal;
    a.sm_scale = op.sm_scale > 0.0f ? op.sm_scale : 1.0f / std::sqrt(static_cast<float>(D));
    a.timeout_ns = wait_limit_ns(op);
    a.debug_flags = op.debug_flags;
    a.err_word = ds->err;
    return launch_varlen_attention(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FSA_OK : FSA_ERR_CUDA;
}

namespace {

// Shape and addresses of an operand of the MX product.
fsa_status check_operand(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, int elem) {
    if (elem == FSA_ELEM_E2M3) return FSA_ERR_UNSUPPORTED;
    if (elem != FSA_ELEM_E4M3 && elem != FSA_ELEM_E2M1) return FSA_ERR_INVALID_ARGUMENT;
    if (rows < 0 || rows > (1 << 30) || cols < 1 || cols > (1 << 20)) return FSA_ERR_INVALID_ARGUMENT;
    if (rows > 0 && (!codes || !scales || (reinterpret_cast<uintptr_t>(codes) & 31) || !aligned16(scales)))
        return FSA_ERR_INVALID_ARGUMENT;
    return FSA_OK;
}

// Rows of bf16, `least` elements apart or more.
bool rows_ok(const void* x, int64_t stride, int64_t least) {
    return x && (reinterpret_cast<uintptr_t>(x) & 1) == 0 && stride >= least && stride < (int64_t{1} << 36);
}

}  // namespace

fsa_status fsa_mx_pack(const void* x, int64_t x_stride, int64_t rows, int64_t cols, int elem, uint8_t* codes,
                       uint8_t* scales, void* stream) {
    fsa_status s = check_operand(codes, scales, rows, cols, elem);
    if (s != FSA_OK) return s;
    if (rows == 0) return FSA_OK;
    if (!rows_ok(x, x_stride, 0)) return FSA_ERR_INVALID_ARGUMENT;
    int dev;
    DeviceState* ds;
    s = current_device(&dev, &ds);
    if (s != FSA_OK) return s;
    return launch_mx_pack(x, x_stride, rows, static_cast<int>(cols), elem, codes, scales,
                          static_cast<cudaStream_t>(stream)) == cudaSuccess ? FSA_OK : FSA_ERR_CUDA;
}

fsa_status fsa_mx_unpack(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, int elem, void* out,
                         int64_t out_stride, void* stream) {
    fsa_status s = check_operand(codes, scales, rows, cols, elem);
    if (s != FSA_OK) return s;
    if (rows == 0) return FSA_OK;
    if (!rows_ok(out, out_stride, rows > 1 ? cols : 0)) return FSA_ERR_INVALID_ARGUMENT;
    int dev;
    DeviceState* ds;
    s = current_device(&dev, &ds);
    if (s != FSA_OK) return s;
    return launch_mx_unpack(codes, scales, rows, static_cast<int>(cols), elem, out, out_stride,
                            static_cast<cudaStream_t>(stream)) == cudaSuccess ? FSA_OK : FSA_ERR_CUDA;
}

fsa_status fsa_rms_norm_mx(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                           const void* gain, float eps, int64_t rows, int64_t cols, int elem, void* sum,
                           int64_t sum_stride, uint8_t* codes, uint8_t* scales, void* stream) {
    return fsa_rms_norm_mx_ex(x, x_stride, residual, residual_stride, gain, eps, rows, cols, elem, sum, sum_stride, codes,
                              scales, nullptr, stream);
}

fsa_status fsa_rms_norm_mx_ex(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                              const void* gain, float eps, int64_t rows, int64_t cols, int elem, void* sum,
                              int64_t sum_stride, uint8_t* codes, uint8_t* scales, const fsa_options* opt, void* stream) {
    const fsa_options op = opt ? *opt : fsa_options{};
    fsa_status s = check_operand(codes, scales, rows, cols, elem);
    if (s != FSA_OK) return s;
    if (cols > kNormMaxCols || !std::isfinite(eps) || !(eps > 0.0f)) return FSA_ERR_INVALID_ARGUMENT;
    if (rows == 0) return FSA_OK;
    if (!rows_ok(x, x_stride, 0) || !rows_ok(gain, 0, 0)) return FSA_ERR_INVALID_ARGUMENT;
    if (residual && (!rows_ok(residual, residual_stride, 0) || !rows_ok(sum, sum_stride, rows > 1 ? cols : 0)))
        return FSA_ERR_INVALID_ARGUMENT;
    int dev;
    DeviceState* ds;
    s = current_device(&dev, &ds);
    if (s != FSA_OK) return s;
    RmsNormMxLaunch a{};
    a.x = x;
    a.residual = residual;
    a.gain = gain;
    a.sum = sum;
    a.x_stride = x_stride;
    a.residual_stride = residual_stride;
    a.sum_stride = sum_stride;
    a.rows = rows;
    a.cols = static_cast<int>(cols);
    a.eps = eps;
    a.codes = codes;
    a.scales = scales;
    a.timeout_ns = wait_limit_ns(op);
    a.debug_flags = op.debug_flags;
    a.err_word = ds->err;
    return launch_rms_norm_mx(a, elem, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FSA_OK : FSA_ERR_CUDA;
}

fsa_status fsa_mx_linear(const uint8_t* x_codes, const uint8_t* x_scales, int x_elem, const uint8_t* w_codes,
                         const uint8_t* w_scales, int w_elem, int64_t T, int64_t N, int64_t K, void* y, int64_t y_stride,
                         const fsa_options* opt, void* stream) {
    const fsa_options op = opt ? *opt : fsa_options{};
    fsa_status s = check_operand(x_codes, x_scales, T, K, x_elem);
    if (s != FSA_OK) return s;
    s = check_operand(w_codes, w_scales, N, K, w_elem);
    if (s != FSA_OK) return s;
    if (x_elem == FSA_ELEM_E2M1 && w_elem == FSA_ELEM_E4M3) return FSA_ERR_UNSUPPORTED;
    // (128 x 128 tiles, up to eight CTAs each, number the blocks of a grid)
    if (mx_atoms(T) * mx_atoms(N) > (1 << 27)) return FSA_ERR_INVALID_ARGUMENT;
    if (T == 0 || N == 0) return FSA_OK;
    if (!rows_ok(y, y_stride, T > 1 ? N : 0)) return FSA_ERR_INVALID_ARGUMENT;
    int dev;
    DeviceState* ds;
    s = current_device(&dev, &ds);
    if (s != FSA_OK) return s;
    const MxLinearPlan plan = mx_linear_plan(static_cast<int>(T), static_cast<int>(N), static_cast<int>(K), x_elem, w_elem);
    CUtensorMap tx, tw, txs, tws;
    if (!make_map_mx(&tx, x_codes, T, K, x_elem, false, plan.x_rows) ||
        !make_map_mx(&tw, w_codes, N, K, w_elem, w_elem == FSA_ELEM_E2M1 && x_elem == FSA_ELEM_E4M3, plan.w_rows))
        return FSA_ERR_CUDA;
    if (plan.split == 0 && (!make_map_mx_scales(&txs, x_scales, T, K, plan.sf_atoms, 1) ||
                            !make_map_mx_scales(&tws, w_scales, N, K, plan.sf_atoms, plan.sf_rows)))
        return FSA_ERR_CUDA;
    MxLinearLaunch a{};
    a.tm_x = &tx;
    a.tm_w = &tw;
    a.tm_xs = &txs;
    a.tm_ws = &tws;
    a.xs = x_scales;
    a.ws = w_scales;
    a.y = y;
    a.y_stride = y_stride;
    a.T = static_cast<int>(T);
    a.N = static_cast<int>(N);
    a.K = static_cast<int>(K);
    a.x_elem = x_elem;
    a.w_elem = w_elem;
    a.timeout_ns = wait_limit_ns(op);
    a.debug_flags = op.debug_flags;
    a.err_word = ds->err;
    return launch_mx_linear(a, plan, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FSA_OK : FSA_ERR_CUDA;
}

uint64_t fsa_attention_workspace_size(int B, int H, int S, int D, int fmt) {
    return fsa_cross_attention_workspace_size(B, H, S, S, D, fmt);
}

uint64_t fsa_cross_attention_workspace_size(int B, int H, int Sq, int Sk, int D, int fmt) {
    if (B < 1 || H < 1 || Sq < 1 || Sk < 1 || (D != 64 && D != 128) || fmt < 0 || fmt > 3) return 0;
    return attn_workspace_bytes(static_cast<int64_t>(B) * H, Sq, Sk, D);
}

fsa_status fsa_attention_prepare(const void* q, const void* k, const void* v, int B, int H, int S,
                                 int D, int fmt, void* workspace, uint64_t workspace_bytes,
                                 void* stream) {
    return fsa_cross_attention_prepare(q, k, v, B, H, S, S, D, fmt, workspace, workspace_bytes,
                                       stream);
}

fsa_status fsa_cross_attention_prepare(const void* q, const void* k, const void* v, int B, int H,
                                       int Sq, int Sk, int D, int fmt, void* workspace,
                                       uint64_t workspace_bytes, void* stream) {
    fsa_status s = validate_attention(q, k, v, q, B, H, Sq, Sk, D);
    if (s != FSA_OK) return s;
    if (fmt < 0 || fmt > 3) return FSA_ERR_INVALID_ARGUMENT;
    const int64_t BH = static_cast<int64_t>(B) * H;
    s = check_workspace(workspace, workspace_bytes, BH, Sq, Sk, D);
    if (s != FSA_OK) return s;
    int dev;
    DeviceState* ds;
    s = current_device(&dev, &ds);
    if (s != FSA_OK) return s;
    return prepare_impl(q, k, v, BH, Sq, Sk, D, fmt, workspace, static_cast<cudaStream_t>(stream));
}

fsa_status fsa_attention_run(const void* workspace, uint64_t workspace_bytes, void* o, int B,
                             int H, int S, int D, int fmt, float threshold, const fsa_options* opt,
                             void* stream) {
    return fsa_cross_attention_run(workspace, workspace_bytes, o, B, H, S, S, D, fmt, threshold, opt,
                                   stream);
}

fsa_status fsa_cross_attention_run(const void* workspace, uint64_t workspace_bytes, void* o, int B,
                                   int H, int Sq, int Sk, int D, int fmt, float threshold,
                                   const fsa_options* opt, void* stream) {
    fsa_status s = validate_attention(o, o, o, o, B, H, Sq, Sk, D);
    if (s != FSA_OK) return s;
    fsa_options defaults{};
    const fsa_options& op = opt ? *opt : defaults;
    s = check_run_args(fmt, threshold, op);
    if (s != FSA_OK) return s;
    const int64_t BH = static_cast<int64_t>(B) * H;
    s = check_workspace(workspace, workspace_bytes, BH, Sq, Sk, D);
    if (s != FSA_OK) return s;
    int dev;
    DeviceState* ds;
    s = current_device(&dev, &ds);
    if (s != FSA_OK) return s;
    return run_impl(const_cast<void*>(workspace), o, BH, Sq, Sk, D, fmt, threshold, op, ds->err,
                    static_cast<cudaStream_t>(stream));
}

fsa_status fsa_attention_fwd_ex(const void* q, const void* k, const void* v, void* o, int B,
                                int H, int S, int D, int fmt, float threshold,
                                const fsa_options* opt, void* stream) {
    return fsa_cross_attention_fwd(q, k, v, o, B, H, S, S, D, fmt, threshold, opt, stream);
}

fsa_status fsa_cross_attention_fwd(const void* q, const void* k, const void* v, void* o, int B,
                                   int H, int Sq, int Sk, int D, int fmt, float threshold,
                                   const fsa_options* opt, void* stream) {
    fsa_status s = validate_attention(q, k, v, o, B, H, Sq, Sk, D);
    if (s != FSA_OK) return s;
    fsa_options defaults{};
    const fsa_options& op = opt ? *opt : defaults;
    s = check_run_args(fmt, threshold, op);
    if (s != FSA_OK) return s;
    int dev;
    DeviceState* ds;
    s = current_device(&dev, &ds);
    if (s != FSA_OK) return s;
    const int64_t BH = static_cast<int64_t>(B) * H;
    const size_t need = attn_workspace_bytes(BH, Sq, Sk, D);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (op.workspace) {
        s = check_workspace(op.workspace, op.workspace_bytes, BH, Sq, Sk, D);
        if (s != FSA_OK) return s;
        s = prepare_impl(q, k, v, BH, Sq, Sk, D, fmt, op.workspace, st);
        if (s != FSA_OK) return s;
        return run_impl(op.workspace, o, BH, Sq, Sk, D, fmt, threshold, op, ds->err, st);
    }
    // library-owned cached workspace, grown on demand; the lock serialises
    // host-side use of it
    std::lock_guard<std::mutex> lk(ds->mu);
    if (ds->ws_bytes < need) {
        if (ds->ws) {
            cudaDeviceSynchronize();
            cudaFree(ds->ws);
            ds->ws = nullptr;
            ds->ws_bytes = 0;
        }
        if (cudaMalloc(&ds->ws, need) != cudaSuccess) {
            cudaGetLastError();
            return FSA_ERR_OUT_OF_MEMORY;
        }
        ds->ws_bytes = need;
    }
    s = prepare_impl(q, k, v, BH, Sq, Sk, D, fmt, ds->ws, st);
    if (s != FSA_OK) return s;
    return run_impl(ds->ws, o, BH, Sq, Sk, D, fmt, threshold, op, ds->err, st);
}

fsa_status fsa_cross_attention_fwd_host(const void* q, const void* k, const void* v, void* o, int B,
                                        int H, int Sq, int Sk, int D, int fmt, float threshold,
                                        const fsa_options* opt, void* stream) {
    if (!q || !k || !v || !o) return FSA_ERR_INVALID_ARGUMENT;
    if (B < 1 || H < 1 || Sq < 1 || Sk < 1) return FSA_ERR_INVALID_ARGUMENT;
    if (D != 64 && D != 128) return FSA_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(B) * H > 65535) return FSA_ERR_INVALID_ARGUMENT;
    if (Sq > (1 << 30) || Sk > (1 << 30)) return FSA_ERR_INVALID_ARGUMENT;
    fsa_options defaults{};
    const fsa_options& op = opt ? *opt : defaults;
    fsa_status s = check_run_args(fmt, threshold, op);
    if (s != FSA_OK) return s;
    int dev;
    DeviceState* ds;
    s = current_device(&dev, &ds);
    if (s != FSA_OK) return s;
    // the lock serialises host-side use of the library's buffers, streams and events
    std::lock_guard<std::mutex> lk(ds->mu);
    return host_fwd_impl(*ds, static_cast<const uint16_t*>(q), static_cast<const uint16_t*>(k),
                         static_cast<const uint16_t*>(v), static_cast<uint16_t*>(o),
                         static_cast<int64_t>(B) * H, Sq, Sk, D, fmt, threshold, op,
                         static_cast<cudaStream_t>(stream));
}

fsa_status fsa_attention_fwd_host(const void* q, const void* k, const void* v, void* o, int B, int H,
                                  int S, int D, int fmt, float threshold, const fsa_options* opt,
                                  void* stream) {
    return fsa_cross_attention_fwd_host(q, k, v, o, B, H, S, S, D, fmt, threshold, opt, stream);
}

fsa_status fsa_attention_fwd(const void* q, const void* k, const void* v, void* o, int B, int H,
                             int S, int D, int fmt, float threshold, void* stream) {
    return fsa_attention_fwd_ex(q, k, v, o, B, H, S, D, fmt, threshold, nullptr, stream);
}

fsa_status fsa_bf16_attention_fwd(const void* q, const void* k, const void* v, void* o, int B,
                                  int H, int S, int D, void* stream) {
    fsa_status s = validate_attention(q, k, v, o, B, H, S, S, D);
    if (s != FSA_OK) return s;
    int dev;
    DeviceState* ds;
    s = current_device(&dev, &ds);
    if (s != FSA_OK) return s;
    const int64_t BH = static_cast<int64_t>(B) * H;
    CUtensorMap tq, tk, tv;
    // bf16 rows of D elements: 128 (D = 64) or 256 (D = 128) bytes, loaded
    // as boxes of 64 elements (128 bytes, one 128-byte swizzle span)
    if (!make_map_bf16(&tq, const_cast<void*>(q), D, S, BH, 2ull * D, 2ull * S * D, 64, kTile,
                       CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_map_bf16(&tk, const_cast<void*>(k), D, S, BH, 2ull * D, 2ull * S * D, 64, kTile,
                       CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_map_bf16(&tv, const_cast<void*>(v), D, S, BH, 2ull * D, 2ull * S * D, 64, kTile,
                       CU_TENSOR_MAP_SWIZZLE_128B))
        return FSA_ERR_CUDA;
    Bf16Launch a{};
    a.tm_q = &tq;
    a.tm_k = &tk;
    a.tm_v = &tv;
    a.o = o;
    a.BH = BH;
    a.S = S;
    a.D = D;
    a.sm_scale = 1.0f / std::sqrt(static_cast<float>(D));
    a.timeout_ns = 2000ull * 1000000ull;
    a.err_word = ds->err;
    return launch_bf16_attention(a, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? FSA_OK
               : FSA_ERR_CUDA;
}

fsa_status fsa_mma_rate_probe(int kind, int ctas, int iters, double* flops_per_launch,
                              void* stream) {
    if (kind < 0 || kind > 4 || ctas < 1 || ctas > 65535 || iters < 1 || iters > (1 << 24))
        return FSA_ERR_INVALID_ARGUMENT;
    int dev;
    DeviceState* ds;
    fsa_status s = current_device(&dev, &ds);
    if (s != FSA_OK) return s;
    if (flops_per_launch) *flops_per_launch = mma_probe_flops(kind, ctas, iters);
    return launch_mma_probe(kind, ctas, iters, 2000ull * 1000000ull, ds->err,
                            static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? FSA_OK
               : FSA_ERR_CUDA;
}

fsa_status fsa_get_device_error(void* stream) {
    if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return FSA_ERR_CUDA;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return FSA_ERR_CUDA;
    if (dev < 0 || dev >= kMaxDevices) return FSA_ERR_UNSUPPORTED;
    // two words may hold a status: the one of the allocating entry points
    // (allocated on their first call) and the non-allocating entry point's
    // static one (once it was set up on this device); nothing is allocated
    // here, so a caller of the non-allocating entry point may use this too
    unsigned int* words[2] = {nullptr, noalloc_status_word(dev)};
    {
        std::lock_guard<std::mutex> lk(g_dev[dev].mu);
        words[0] = g_dev[dev].err;
    }
    unsigned int w = 0;
    for (unsigned int* word : words) {
        if (!word) continue;
        unsigned int x = 0;
        if (cudaMemcpy(&x, word, sizeof(x), cudaMemcpyDeviceToHost) != cudaSuccess) return FSA_ERR_CUDA;
        if (x) {
            const unsigned int zero = 0;
            if (cudaMemcpy(word, &zero, sizeof(zero), cudaMemcpyHostToDevice) != cudaSuccess)
                return FSA_ERR_CUDA;
        }
        w |= x;
    }
    return error_word_status(w);
}

void fsa_release_workspace(void) {
    int n = 0;
    if (cudaGetDeviceCount(&n) != cudaSuccess) return;
    int cur = 0;
    cudaGetDevice(&cur);
    for (int d = 0; d < n && d < kMaxDevices; ++d) {
        std::lock_guard<std::mutex> lk(g_dev[d].mu);
        if (g_dev[d].ws || g_dev[d].hp.buf) {
            cudaSetDevice(d);
            cudaDeviceSynchronize();
            cudaFree(g_dev[d].ws);
            g_dev[d].ws = nullptr;
            g_dev[d].ws_bytes = 0;
            cudaFree(g_dev[d].hp.buf);
            g_dev[d].hp.buf = nullptr;
            g_dev[d].hp.bytes = 0;
        }
    }
    cudaSetDevice(cur);
}

}  // extern "C"

// --------------------------------------------------------------------------
// fsa_attention_fwd_noalloc: the fused attention with its scratch in a
// fixed-size device array that belongs to the library image, for callers
// that must not allocate or free device memory once running.
namespace fsa {
namespace {

constexpr size_t kNoAllocBytes = size_t(64) << 20;  // 64 MiB per device, held until exit
static __device__ __align__(256) uint8_t g_noalloc_ws[kNoAllocBytes];
static __device__ __align__(256) unsigned int g_noalloc_status;  // kernels' bounded-wait status

struct NoAllocDevice {
    void* ws = nullptr;
    unsigned int* status = nullptr;
    int arch_ok = -1;
};
std::mutex g_noalloc_mu;
NoAllocDevice g_noalloc[kMaxDevices];

// Device addresses of the two arrays on the current device (looked up once
// per device, with that device current); no allocation.
fsa_status noalloc_setup(int dev, NoAllocDevice** out) {
    std::lock_guard<std::mutex> lk(g_noalloc_mu);
    NoAllocDevice& d = g_noalloc[dev];
    if (d.arch_ok < 0) {
        int major = 0, minor = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
            return FSA_ERR_CUDA;
        d.arch_ok = (major == 10 && (minor == 0 || minor == 3)) ? 1 : 0;
    }
    if (!d.arch_ok) return FSA_ERR_UNSUPPORTED;
    if (!d.ws) {
        void* ws = nullptr;
        void* st = nullptr;
        if (cudaGetSymbolAddress(&ws, g_noalloc_ws) != cudaSuccess ||
            cudaGetSymbolAddress(&st, g_noalloc_status) != cudaSuccess) {
            cudaGetLastError();
            return FSA_ERR_CUDA;
        }
        // nothing needs clearing here: the status word is a static device
        // object, zero when the module loads, and fsa_get_device_error
        // clears it after reading; every call rewrites the codes and resets
        // the scale atoms of the array
        d.ws = ws;
        d.status = static_cast<unsigned int*>(st);
    }
    *out = &d;
    return FSA_OK;
}

unsigned int* noalloc_status_word(int dev) {
    std::lock_guard<std::mutex> lk(g_noalloc_mu);
    return g_noalloc[dev].status;
}

}  // namespace
}  // namespace fsa

extern "C" fsa_status fsa_attention_fwd_noalloc(const void* q, const void* k, const void* v,
                                                void* o, int B, int H, int S, int D, int fmt,
                                                float threshold, void* stream) {
    using namespace fsa;
    fsa_status s = validate_attention(q, k, v, o, B, H, S, S, D);
    if (s != FSA_OK) return s;
    fsa_options defaults{};
    s = check_run_args(fmt, threshold, defaults);
    if (s != FSA_OK) return s;
    const int64_t BH = static_cast<int64_t>(B) * H;
    if (attn_workspace_bytes(BH, S, S, D) > kNoAllocBytes) return FSA_ERR_INVALID_ARGUMENT;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return FSA_ERR_CUDA;
    if (dev < 0 || dev >= kMaxDevices) return FSA_ERR_UNSUPPORTED;
    NoAllocDevice* d = nullptr;
    s = noalloc_setup(dev, &d);
    if (s != FSA_OK) return s;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    s = prepare_impl(q, k, v, BH, S, S, D, fmt, d->ws, st);
    if (s != FSA_OK) return s;
    return run_impl(d->ws, o, BH, S, S, D, fmt, threshold, defaults, d->status, st);
}
