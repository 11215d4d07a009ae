// dsa_attend_paged and dsa_attend_selected: decode attention over the paged
// key/value cache.
//
// First form: one CTA per (row, query head), one pass over the row's keys with
// the running maximum and sum of the softmax.  Each warp takes every fourth
// key (four columns a lane), and the four partial results are joined at the end.
#include <math.h>

#include "elem16.cuh"
#include "host.h"

namespace dsa {

int check_kv_cache(const dsa_kv_cache* c);

struct AttendArgs {
    dsa_kv_cache c;
    const uint16_t* q;
    int64_t qr, qh;
    const int32_t* bt;
    int64_t bt_stride, max_pages;
    const int32_t* starts;
    const int32_t* row_ends;
    int R, rows, heads, group;
    const int32_t* prefix_pages;
    int64_t prefix_len;
    const int32_t* topk;
    int64_t topk_stride, k;
    float scale;
    uint16_t* out;
    int64_t orow, oh;
    float* lse;
    int32_t* status;
};

template <typename T, bool kSelected>
__global__ void __launch_bounds__(128) attend_simple_kernel(const AttendArgs a) {
    const int row = blockIdx.x, head = blockIdx.y, kvh = head / a.group;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __shared__ int s_req;
    __shared__ float sm[4], sl[4], so[4][128];
    if (threadIdx.x == 0) s_req = -1;
    __syncthreads();
    for (int j = threadIdx.x; j < a.R; j += 128) {
        const int s0 = a.starts[j], s1 = a.starts[j + 1];
        if ((s0 < 0 || s1 < s0 || s1 > a.rows) && a.status) atomicOr(a.status, DSA_STATUS_BAD_GEOMETRY);
        if (s0 <= row && row < s1) atomicMax(&s_req, j);
    }
    __syncthreads();
    const int req = s_req;
    int64_t own = 0;
    if (req >= 0) {
        own = a.row_ends[row];
        if (own < 0 || own > a.max_pages * kPage) {
            if (threadIdx.x == 0 && a.status) atomicOr(a.status, DSA_STATUS_BAD_GEOMETRY);
            own = own < 0 ? 0 : a.max_pages * kPage;
        }
    }
    const int dim = static_cast<int>(a.c.dim);
    const bool on = lane * 4 < dim;
    float q[4] = {0, 0, 0, 0};
    if (on) {
        const uint2 w = *reinterpret_cast<const uint2*>(a.q + row * a.qr + head * a.qh + lane * 4);
        const float2 x = T::unpack(w.x), y = T::unpack(w.y);
        q[0] = x.x, q[1] = x.y, q[2] = y.x, q[3] = y.y;
    }
    float m = -INFINITY, l = 0.0f, o[4] = {0, 0, 0, 0};
    const int64_t prefix = !kSelected && req >= 0 ? a.prefix_len : 0;
    const int64_t total = req < 0 ? 0 : kSelected ? a.k : prefix + own;
    for (int64_t i = warp; i < total; i += 4) {
        int page;
        int64_t t;
        if (kSelected) {
            t = a.topk[row * a.topk_stride + i];
            if (t < 0) continue;
            if (t >= own) {
                if (lane == 0 && a.status) atomicOr(a.status, DSA_STATUS_BAD_GEOMETRY);
                continue;
            }
            page = a.bt[req * a.bt_stride + t / kPage];
        } else if (i < prefix) {
            t = i;
            page = a.prefix_pages[t / kPage];
        } else {
            t = i - prefix;
            page = a.bt[req * a.bt_stride + t / kPage];
        }
        if (page < 0 || page >= a.c.num_pages) {
            if (lane == 0 && a.status) atomicOr(a.status, DSA_STATUS_BAD_PAGE);
            continue;
        }
        const uint16_t* kp = static_cast<const uint16_t*>(a.c.k) + page * a.c.k_page_stride +
                             (t % kPage) * a.c.k_token_stride + kvh * a.c.k_head_stride;
        const uint16_t* vp = static_cast<const uint16_t*>(a.c.v) + page * a.c.v_page_stride +
                             (t % kPage) * a.c.v_token_stride + kvh * a.c.v_head_stride;
        float s = 0.0f, v[4] = {0, 0, 0, 0};
        if (on) {
            const uint2 kw = *reinterpret_cast<const uint2*>(kp + lane * 4);
            const uint2 vw = *reinterpret_cast<const uint2*>(vp + lane * 4);
            const float2 x = T::unpack(kw.x), y = T::unpack(kw.y), z = T::unpack(vw.x), w = T::unpack(vw.y);
            s = q[0] * x.x + q[1] * x.y + q[2] * y.x + q[3] * y.y;
            v[0] = z.x, v[1] = z.y, v[2] = w.x, v[3] = w.y;
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
        s *= a.scale;
        const float mn = fmaxf(m, s);
        const float keep = m == -INFINITY ? 0.0f : expf(m - mn), p = expf(s - mn);
        l = l * keep + p;
#pragma unroll
        for (int d = 0; d < 4; ++d) o[d] = o[d] * keep + p * v[d];
        m = mn;
    }
    if (lane == 0) sm[warp] = m, sl[warp] = l;
#pragma unroll
    for (int d = 0; d < 4; ++d) so[warp][lane * 4 + d] = o[d];
    __syncthreads();
    const float top = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
    float sum = 0.0f, acc = 0.0f;
    for (int w = 0; w < 4; ++w) {
        const float f = sm[w] == -INFINITY ? 0.0f : expf(sm[w] - top);
        sum += sl[w] * f;
        acc += so[w][threadIdx.x] * f;
    }
    if (threadIdx.x < dim)
        a.out[row * a.orow + head * a.oh + threadIdx.x] =
            static_cast<uint16_t>(T::pack(sum == 0.0f ? 0.0f : acc / sum, 0.0f));
    if (threadIdx.x == 0 && a.lse)
        a.lse[static_cast<int64_t>(row) * a.heads + head] = sum == 0.0f ? -INFINITY : top + logf(sum);
}

static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// The checks both calls share.
static int check_attend(const dsa_kv_cache* cache, const void* q, int64_t q_row_stride, int64_t q_head_stride,
                        int64_t heads, const int32_t* block_table, int64_t bt_stride, int64_t max_pages,
                        const int32_t* starts, const int32_t* row_ends, int64_t num_requests, int64_t rows,
                        float scale, const void* out, int64_t out_row_stride, int64_t out_head_stride,
                        const void* workspace) {
    const int rc = check_kv_cache(cache);
    if (rc != DSA_OK) return rc;
    if (heads < 1 || rows < 0 || num_requests < 0 || max_pages < 0) return DSA_ERR_INVALID;
    if (heads % cache->heads) return DSA_ERR_INVALID;
    if (cache->dim > 128 || heads / cache->heads > 128 || heads > 65535) return DSA_ERR_UNSUPPORTED;
    if (!(scale > 0.0f) || !isfinite(scale)) return DSA_ERR_INVALID;
    if (rows == 0) return DSA_OK;
    if (rows > (1 << 24) || num_requests > (1 << 30) || max_pages > (int64_t(1) << 24)) return DSA_ERR_UNSUPPORTED;
    if (!q || !out || !row_ends || !starts || !workspace) return DSA_ERR_INVALID;
    if (max_pages > 0 && num_requests > 0 && (!block_table || bt_stride < max_pages)) return DSA_ERR_INVALID;
    if (!aligned16(q) || !aligned16(out) || (reinterpret_cast<uintptr_t>(workspace) & 255)) return DSA_ERR_INVALID;
    if (((q_row_stride | q_head_stride | out_row_stride | out_head_stride) & 7) || q_row_stride < 0 ||
        q_head_stride < 0 || out_row_stride < 0 || out_head_stride < 0)
        return DSA_ERR_INVALID;
    return DSA_OK;
}

}  // namespace dsa

using namespace dsa;

extern "C" size_t dsa_attend_workspace_size(int64_t rows, int64_t num_requests, int64_t heads, int64_t kv_heads,
                                            int64_t dim, int64_t max_query_len, int64_t k) {
    if (rows < 0 || num_requests < 0 || heads < 1 || kv_heads < 1 || heads % kv_heads || dim < 16 || dim % 16 ||
        dim > 128 || heads / kv_heads > 128 || max_query_len < 0 || k < 0)
        return 0;
    return 256;
}

template <bool kSelected>
static int launch_simple(const AttendArgs& a, cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>(a.rows), static_cast<unsigned>(a.heads));
    if (a.c.dtype == DSA_BF16)
        attend_simple_kernel<Bf16, kSelected><<<grid, 128, 0, stream>>>(a);
    else
        attend_simple_kernel<Fp16, kSelected><<<grid, 128, 0, stream>>>(a);
    return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

extern "C" int dsa_attend_paged(const dsa_kv_cache* cache, const void* q, int64_t q_row_stride, int64_t q_head_stride,
                                int64_t heads, const int32_t* block_table, int64_t bt_stride, int64_t max_pages,
                                const int32_t* starts, const int32_t* row_ends, int64_t num_requests, int64_t rows,
                                int64_t max_query_len, const int32_t* prefix_pages, int64_t prefix_len, float scale,
                                void* out, int64_t out_row_stride, int64_t out_head_stride, float* lse,
                                void* workspace, size_t workspace_bytes, int32_t* status, void* stream) {
    const int rc = check_attend(cache, q, q_row_stride, q_head_stride, heads, block_table, bt_stride, max_pages, starts,
                                row_ends, num_requests, rows, scale, out, out_row_stride, out_head_stride, workspace);
    if (rc != DSA_OK) return rc;
    if (max_query_len < 0 || prefix_len < 0 || (prefix_len > 0 && !prefix_pages)) return DSA_ERR_INVALID;
    if (prefix_len > (int64_t(1) << 30)) return DSA_ERR_UNSUPPORTED;
    if (rows == 0) return DSA_OK;
    if (workspace_bytes <
        dsa_attend_workspace_size(rows, num_requests, heads, cache->heads, cache->dim, max_query_len, 0))
        return DSA_ERR_INVALID;
    const AttendArgs a{*cache, static_cast<const uint16_t*>(q), q_row_stride, q_head_stride, block_table, bt_stride,
                       max_pages, starts, row_ends, static_cast<int>(num_requests), static_cast<int>(rows),
                       static_cast<int>(heads), static_cast<int>(heads / cache->heads), prefix_pages, prefix_len,
                       nullptr, 0, 0, scale, static_cast<uint16_t*>(out), out_row_stride, out_head_stride, lse, status};
    return launch_simple<false>(a, static_cast<cudaStream_t>(stream));
}

extern "C" int dsa_attend_selected(const dsa_kv_cache* cache, const void* q, int64_t q_row_stride,
                                   int64_t q_head_stride, int64_t heads, const int32_t* block_table, int64_t bt_stride,
                                   int64_t max_pages, const int32_t* starts, const int32_t* row_ends,
                                   int64_t num_requests, int64_t rows, const int32_t* topk, int64_t topk_stride,
                                   int64_t k, float scale, void* out, int64_t out_row_stride, int64_t out_head_stride,
                                   float* lse, void* workspace, size_t workspace_bytes, int32_t* status,
                                   void* stream) {
    const int rc = check_attend(cache, q, q_row_stride, q_head_stride, heads, block_table, bt_stride, max_pages, starts,
                                row_ends, num_requests, rows, scale, out, out_row_stride, out_head_stride, workspace);
    if (rc != DSA_OK) return rc;
    if (k < 0 || (k > 0 && rows > 0 && (!topk || topk_stride < k))) return DSA_ERR_INVALID;
    if (k > (int64_t(1) << 24)) return DSA_ERR_UNSUPPORTED;
    if (rows == 0) return DSA_OK;
    if (workspace_bytes < dsa_attend_workspace_size(rows, num_requests, heads, cache->heads, cache->dim, 1, k))
        return DSA_ERR_INVALID;
    const AttendArgs a{*cache, static_cast<const uint16_t*>(q), q_row_stride, q_head_stride, block_table, bt_stride,
                       max_pages, starts, row_ends, static_cast<int>(num_requests), static_cast<int>(rows),
                       static_cast<int>(heads), static_cast<int>(heads / cache->heads), nullptr, 0, topk, topk_stride,
                       k, scale, static_cast<uint16_t*>(out), out_row_stride, out_head_stride, lse, status};
    return launch_simple<true>(a, static_cast<cudaStream_t>(stream));
}
