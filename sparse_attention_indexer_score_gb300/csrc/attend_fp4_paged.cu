// dsa_attend_paged_fp4: attention of grouped decode rows over all keys of their requests.
#include "attend_fp4.cuh"

using namespace dsa;

extern "C" size_t dsa_attend_workspace_size_fp4(int64_t rows, int64_t num_requests, int64_t heads, int64_t kv_heads,
                                                int64_t dim, int64_t max_query_len, int64_t k) {
    if (rows < 0 || num_requests < 0 || heads < 1 || kv_heads < 1 || heads % kv_heads || max_query_len < 0 || k < 0 ||
        k > (1 << 24) || !sizes4_ok(rows, num_requests, heads, kv_heads, dim))
        return 0;
    return attend4_layout(rows, num_requests, heads, kv_heads, dim, max_query_len, k).total;
}

extern "C" int dsa_attend_paged_fp4(const dsa_kv_cache_fp4* cache, int32_t dtype, const void* q, int64_t q_row_stride,
                                    int64_t q_head_stride, int64_t heads, const int32_t* block_table,
                                    int64_t bt_stride, int64_t max_pages, const int32_t* starts,
                                    const int32_t* row_ends, int64_t num_requests, int64_t rows, int64_t max_query_len,
                                    float scale, void* out, int64_t out_row_stride, int64_t out_head_stride,
                                    float* lse, void* workspace, size_t workspace_bytes, int32_t* status,
                                    void* stream_) {
    const int rc = check_attend4(cache, dtype, q, q_row_stride, q_head_stride, heads, block_table, bt_stride,
                                 max_pages, starts, row_ends, num_requests, rows, scale, out, out_row_stride,
                                 out_head_stride, workspace);
    if (rc != DSA_OK) return rc;
    if (max_query_len < 0) return DSA_ERR_INVALID;
    if (rows == 0) return DSA_OK;
    const Att4Layout L = attend4_layout(rows, num_requests, heads, cache->heads, cache->dim, max_query_len, 0);
    if (workspace_bytes < L.total) return DSA_ERR_INVALID;
    Att4Params p = params4(cache, L, static_cast<uint8_t*>(workspace), scale);
    p.bf16 = dtype == DSA_BF16;
    p.q = static_cast<const uint16_t*>(q), p.qrow = q_row_stride, p.qhead = q_head_stride;
    p.out = static_cast<uint16_t*>(out), p.orow = out_row_stride, p.ohead = out_head_stride;
    p.lse = lse, p.status = status;
    p.bt = block_table, p.bt_stride = bt_stride, p.starts = starts, p.row_ends = row_ends;
    p.R = static_cast<int>(num_requests), p.rows = static_cast<int>(rows), p.heads = static_cast<int>(heads);
    p.group = p.heads / p.kv_heads;
    p.max_keys = cache->num_pages > 0 ? static_cast<int>(max_pages * kPage) : 0;
    p.plan_in_cta = p.R <= kCtaRequests && p.rows <= 4096;
    // What a unit, and an item's beginning and end, take: measured as times of warps with many and with few items.
    // Starts of 4 and 7 left those with many short items behind the others: 128 requests of 64 to 8192 keys under 32
    // rows 260 us against 247, 150 of 64 to 4096 under 16 rows 121 against 108, 200 under 8 rows 108 against 100.
    p.axis.light = 5, p.axis.heavy = p.cap > 16 ? 7 : 5, p.axis.start = p.cap > 16 ? 13 : 10;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    return launch_all4<false>(p, L.tiles, stream);
}
