// dsa_kv_append: new keys and values into their pages, the position rotation
// applied on the way (and to the queries, in the same launch).
//
// A rotated pair (a, b) becomes (a c - b s, b c + a s) for the cosine c and
// sine s of the token's row of the angle table.  The kernel moves 2-byte
// elements once each way and computes three FP32 operations per element, so it
// is bound by memory; the angles of a token are read once per thread and kept
// in registers for every head that the thread turns.
//
// Measured on GB300 (call as a graph, about 4 us of it the replay), 16384 tokens
// of 32 + 2 x 8 heads of 128 columns, 411 MB, 60 us at the copy rate: 86 us with
// four head rows in flight per thread; 82 us with six; 70 us with six and
// streaming loads and stores (74 us with four; streaming only one side gains
// nothing); 66 us in CTAs of 128 threads instead of 256.
#include "elem16.cuh"
#include "host.h"

namespace dsa {

constexpr int kAppendThreads = 128;
constexpr int kAppendBatch = 6;   // most head rows a thread has in flight

struct AppendArgs {
    const uint16_t* k;
    const uint16_t* v;
    const uint16_t* q;
    uint16_t* q_out;
    uint16_t* kc;
    uint16_t* vc;
    int64_t kt, kh, vt, vh, qt, qh, ot, oh;         // element strides: token, head
    int64_t kcp, kct, kch, vcp, vct, vch;           // cache strides: page, token, head
    const int64_t* slots;
    const int64_t* positions;
    const float* cos_sin;
    int64_t cs_stride, max_pos, num_slots, n;
    int q_heads, kv_heads, units, rot_units, half, head_lanes, tokens_per_cta, batch;
    int32_t* status;
};

// Streaming: read or written once, first to leave L2.
template <bool kStreams>
__device__ __forceinline__ uint4 ld16(const uint16_t* p) {
    const uint4* v = reinterpret_cast<const uint4*>(p);
    return kStreams ? __ldcs(v) : *v;
}
template <bool kStreams>
__device__ __forceinline__ void st16(uint16_t* p, uint4 v) {
    if (kStreams)
        __stcs(reinterpret_cast<uint4*>(p), v);
    else
        *reinterpret_cast<uint4*>(p) = v;
}

// Two words of two elements each: (a, b) pairs across the words' vectors, or
// adjacent elements.  No fused multiply-add: the two products are rounded to
// FP32 and subtracted, the plainest reading of the formula.
template <typename T>
__device__ __forceinline__ void turn_halves(uint4& x, uint4& y, const float (&c)[8], const float (&s)[8]) {
    uint32_t* xw = &x.x;
    uint32_t* yw = &y.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 a = T::unpack(xw[i]), b = T::unpack(yw[i]);
        const float c0 = c[2 * i], c1 = c[2 * i + 1], s0 = s[2 * i], s1 = s[2 * i + 1];
        xw[i] = T::pack(__fsub_rn(__fmul_rn(a.x, c0), __fmul_rn(b.x, s0)),
                        __fsub_rn(__fmul_rn(a.y, c1), __fmul_rn(b.y, s1)));
        yw[i] = T::pack(__fadd_rn(__fmul_rn(b.x, c0), __fmul_rn(a.x, s0)),
                        __fadd_rn(__fmul_rn(b.y, c1), __fmul_rn(a.y, s1)));
    }
}
template <typename T>
__device__ __forceinline__ void turn_pairs(uint4& x, const float* c, const float* s) {
    uint32_t* xw = &x.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 a = T::unpack(xw[i]);
        xw[i] = T::pack(__fsub_rn(__fmul_rn(a.x, c[i]), __fmul_rn(a.y, s[i])),
                        __fadd_rn(__fmul_rn(a.y, c[i]), __fmul_rn(a.x, s[i])));
    }
}

// A head row is cut into units of 16 elements (two 16-byte vectors): unit u <
// rot_units turns vectors u and u + rot_units of the rotated columns (halves),
// or vectors 2u and 2u + 1 (adjacent pairs); the other units copy.  A token
// has units x head_lanes threads; a thread keeps its unit's eight angles and
// walks the token's query, key and value heads in steps of head_lanes.
template <typename T, bool kInterleaved, bool kStreams>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const AppendArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    const int per_token = a.units * a.head_lanes;
    const int sub = threadIdx.x / per_token;
    const int64_t tok = static_cast<int64_t>(blockIdx.x) * a.tokens_per_cta + sub;
    if (sub >= a.tokens_per_cta || tok >= a.n) return;
    const int in = threadIdx.x - sub * per_token;
    const int unit = in % a.units, lane = in / a.units;
    const int64_t slot = a.slots[tok];
    const bool cached = slot >= 0 && slot < a.num_slots;
    if (slot >= a.num_slots && in == 0 && a.status) atomicOr(a.status, DSA_STATUS_BAD_SLOT);
    const bool turns = unit < a.rot_units;
    int e0, e1;   // the unit's two vectors
    if (turns && !kInterleaved) {
        e0 = unit * 8;
        e1 = e0 + a.half;
    } else {
        e0 = unit * 16;
        e1 = e0 + 8;
    }
    float c[8], s[8];
    if (turns) {
        int64_t p = a.positions[tok];
        if (p < 0 || p >= a.max_pos) {
            if (slot >= 0 && in == 0 && a.status) atomicOr(a.status, DSA_STATUS_BAD_GEOMETRY);
            p = p < 0 ? 0 : a.max_pos - 1;
        }
        const float* row = a.cos_sin + p * a.cs_stride + unit * 8;
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
            *reinterpret_cast<float4*>(c + i) = __ldg(reinterpret_cast<const float4*>(row + i));
            *reinterpret_cast<float4*>(s + i) = __ldg(reinterpret_cast<const float4*>(row + a.half + i));
        }
    }
    const int64_t page = cached ? slot >> 6 : 0;
    const int off = static_cast<int>(slot & 63);
    uint16_t* const kdst = a.kc + page * a.kcp + off * a.kct;
    uint16_t* const vdst = a.vc + page * a.vcp + off * a.vct;
    const int heads = a.q_heads + 2 * a.kv_heads;
    const int kv0 = a.q_heads, v0 = a.q_heads + a.kv_heads;
    for (int base = lane; base < heads; base += a.batch * a.head_lanes) {
        const int end = min(heads, base - lane + a.batch * a.head_lanes);
        uint4 x[kAppendBatch], y[kAppendBatch];
#pragma unroll
        for (int i = 0; i < kAppendBatch; ++i) {
            const int h = base + i * a.head_lanes;
            if (h >= end) continue;
            const uint16_t* src;
            if (h < kv0)
                src = a.q + tok * a.qt + h * a.qh;
            else if (cached)
                src = h < v0 ? a.k + tok * a.kt + (h - kv0) * a.kh : a.v + tok * a.vt + (h - v0) * a.vh;
            else
                continue;
            // (values are copied: which 16 elements a thread takes is free)
            x[i] = ld16<kStreams>(src + e0);
            y[i] = ld16<kStreams>(src + e1);
        }
#pragma unroll
        for (int i = 0; i < kAppendBatch; ++i) {
            const int h = base + i * a.head_lanes;
            if (h >= end || (h >= kv0 && !cached)) continue;
            if (turns && h < v0) {
                if (kInterleaved) {
                    turn_pairs<T>(x[i], c, s);
                    turn_pairs<T>(y[i], c + 4, s + 4);
                } else {
                    turn_halves<T>(x[i], y[i], c, s);
                }
            }
            uint16_t* dst = h < kv0  ? a.q_out + tok * a.ot + h * a.oh
                            : h < v0 ? kdst + (h - kv0) * a.kch
                                     : vdst + (h - v0) * a.vch;
            st16<kStreams>(dst + e0, x[i]);
            st16<kStreams>(dst + e1, y[i]);
        }
    }
}

template <typename T>
static cudaError_t launch_append(const AppendArgs& a, dim3 grid, bool interleaved, bool streams, cudaStream_t stream) {
    auto* kernel = interleaved ? (streams ? kv_append_kernel<T, true, true> : kv_append_kernel<T, true, false>)
                               : (streams ? kv_append_kernel<T, false, true> : kv_append_kernel<T, false, false>);
    return launch_pdl(kernel, grid, dim3(kAppendThreads), 0, stream, a);
}

int check_kv_cache(const dsa_kv_cache* c) {
    if (!c) return DSA_ERR_INVALID;
    if (c->num_pages < 0 || c->heads < 1 || c->dim < 16) return DSA_ERR_INVALID;
    if (c->dtype != DSA_BF16 && c->dtype != DSA_FP16) return DSA_ERR_UNSUPPORTED;
    if (c->dim % 16 || c->dim > 512 || c->heads > 65535 || c->num_pages > 0x7FFFFFFF) return DSA_ERR_UNSUPPORTED;
    if (c->num_pages > 0 && (!c->k || !c->v)) return DSA_ERR_INVALID;
    const int64_t strides[6] = {c->k_page_stride, c->k_token_stride, c->k_head_stride,
                                c->v_page_stride, c->v_token_stride, c->v_head_stride};
    for (int64_t s : strides)
        if (s < 0 || s % 8) return DSA_ERR_INVALID;
    if ((reinterpret_cast<uintptr_t>(c->k) | reinterpret_cast<uintptr_t>(c->v)) & 15) return DSA_ERR_INVALID;
    return DSA_OK;
}

}  // namespace dsa

using namespace dsa;

extern "C" int dsa_kv_append(const dsa_kv_cache* cache, const void* k, int64_t k_token_stride, int64_t k_head_stride,
                             const void* v, int64_t v_token_stride, int64_t v_head_stride, const void* q,
                             int64_t q_token_stride, int64_t q_head_stride, int64_t q_heads, void* q_out,
                             int64_t qo_token_stride, int64_t qo_head_stride, int64_t n, const int64_t* slots,
                             const int64_t* positions, const float* cos_sin, int64_t cs_stride, int64_t max_pos,
                             int64_t rot_dim, int interleaved, int32_t* status, void* stream_) {
    const int rc = check_kv_cache(cache);
    if (rc != DSA_OK) return rc;
    if (n < 0 || rot_dim < 0 || rot_dim > cache->dim || (interleaved != 0 && interleaved != 1)) return DSA_ERR_INVALID;
    if (rot_dim % 16) return DSA_ERR_UNSUPPORTED;
    if ((q == nullptr) != (q_out == nullptr) || (q && q_heads < 1)) return DSA_ERR_INVALID;
    if (n == 0) return DSA_OK;
    if (!k || !v || !slots) return DSA_ERR_INVALID;
    if (rot_dim > 0 && (!positions || !cos_sin || max_pos < 1 || cs_stride < rot_dim || cs_stride % 4))
        return DSA_ERR_INVALID;
    if (q && q_heads > 65535) return DSA_ERR_UNSUPPORTED;
    const uintptr_t ptrs = reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v) |
                           reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(q_out) |
                           reinterpret_cast<uintptr_t>(cos_sin);
    const int64_t strides = k_token_stride | k_head_stride | v_token_stride | v_head_stride |
                            (q ? q_token_stride | q_head_stride | qo_token_stride | qo_head_stride : 0);
    if ((ptrs & 15) || (strides & 7)) return DSA_ERR_INVALID;
    // tokens, heads or pages written to one place
    auto one = [](int64_t extent, int64_t stride) { return extent > 1 && stride == 0; };
    if ((q && (one(n, qo_token_stride) || one(q_heads, qo_head_stride))) || one(cache->num_pages, cache->k_page_stride) ||
        one(cache->num_pages, cache->v_page_stride) || one(kPage, cache->k_token_stride) ||
        one(kPage, cache->v_token_stride) || one(cache->heads, cache->k_head_stride) ||
        one(cache->heads, cache->v_head_stride))
        return DSA_ERR_INVALID;

    AppendArgs a;
    a.k = static_cast<const uint16_t*>(k);
    a.v = static_cast<const uint16_t*>(v);
    a.q = static_cast<const uint16_t*>(q);
    a.q_out = static_cast<uint16_t*>(q_out);
    a.kc = static_cast<uint16_t*>(cache->k);
    a.vc = static_cast<uint16_t*>(cache->v);
    a.kt = k_token_stride, a.kh = k_head_stride, a.vt = v_token_stride, a.vh = v_head_stride;
    a.qt = q_token_stride, a.qh = q_head_stride, a.ot = qo_token_stride, a.oh = qo_head_stride;
    a.kcp = cache->k_page_stride, a.kct = cache->k_token_stride, a.kch = cache->k_head_stride;
    a.vcp = cache->v_page_stride, a.vct = cache->v_token_stride, a.vch = cache->v_head_stride;
    a.slots = slots;
    a.positions = positions;
    a.cos_sin = cos_sin;
    a.cs_stride = cs_stride, a.max_pos = max_pos, a.num_slots = cache->num_pages * kPage, a.n = n;
    a.q_heads = q ? static_cast<int>(q_heads) : 0;
    a.kv_heads = static_cast<int>(cache->heads);
    a.units = static_cast<int>(cache->dim / 16);
    a.rot_units = static_cast<int>(rot_dim / 16);
    a.half = static_cast<int>(rot_dim / 2);
    a.status = status;
    // Long appends: 64 threads a token, so that a thread turns several heads
    // with the angles it holds.  Short ones: a CTA a token, so that a token's
    // heads are in flight at once.  A long append's output does not stay in L2.
    // Long form against short: 608 tokens (32 + 2 x 8 heads) equal, 1216: 8.6 and
    // 10.5 us, 4864: 24 and 35; below that both are the launch.
    const bool streams = n >= 4 * device_sm_count();
    const int want = streams ? 64 : kAppendThreads;
    a.head_lanes = want / a.units > 0 ? want / a.units : 1;
    // the heads of a thread in equal rounds
    const int each = (a.q_heads + 2 * a.kv_heads + a.head_lanes - 1) / a.head_lanes;
    const int rounds = (each + kAppendBatch - 1) / kAppendBatch;
    a.batch = (each + rounds - 1) / rounds;
    a.tokens_per_cta = kAppendThreads / (a.units * a.head_lanes);
    const int64_t blocks = (n + a.tokens_per_cta - 1) / a.tokens_per_cta;
    if (blocks > 0x7FFFFFFF) return DSA_ERR_UNSUPPORTED;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    const dim3 grid(static_cast<unsigned>(blocks));
    const cudaError_t err = cache->dtype == DSA_BF16 ? launch_append<Bf16>(a, grid, interleaved, streams, stream)
                                                     : launch_append<Fp16>(a, grid, interleaved, streams, stream);
    return err == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}
