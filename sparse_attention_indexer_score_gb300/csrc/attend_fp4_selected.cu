// dsa_attend_selected_fp4: attention of decode rows over the keys listed for each.
#include "attend_fp4.cuh"

using namespace dsa;

extern "C" int dsa_attend_selected_fp4(const dsa_kv_cache_fp4* cache, int32_t dtype, const void* q,
                                       int64_t q_row_stride, int64_t q_head_stride, int64_t heads,
                                       const int32_t* block_table, int64_t bt_stride, int64_t max_pages,
                                       const int32_t* starts, const int32_t* row_ends, int64_t num_requests,
                                       int64_t rows, const int32_t* topk, int64_t topk_stride, int64_t k, float scale,
                                       void* out, int64_t out_row_stride, int64_t out_head_stride, float* lse,
                                       void* workspace, size_t workspace_bytes, int32_t* status, void* stream_) {
    const int rc = check_attend4(cache, dtype, q, q_row_stride, q_head_stride, heads, block_table, bt_stride,
                                 max_pages, starts, row_ends, num_requests, rows, scale, out, out_row_stride,
                                 out_head_stride, workspace);
    if (rc != DSA_OK) return rc;
    if (k < 0 || (k > 0 && rows > 0 && (!topk || topk_stride < k))) return DSA_ERR_INVALID;
    if (k > (int64_t(1) << 24)) return DSA_ERR_UNSUPPORTED;
    if (rows == 0) return DSA_OK;
    // (an empty list is one key long in the workspace: the rows still need their zeros)
    const Att4Layout L = attend4_layout(rows, num_requests, heads, cache->heads, cache->dim, 1, k > 0 ? k : 1);
    if (workspace_bytes < L.total) return DSA_ERR_INVALID;
    Att4Params p = params4(cache, L, static_cast<uint8_t*>(workspace), scale);
    p.bf16 = dtype == DSA_BF16;
    p.q = static_cast<const uint16_t*>(q), p.qrow = q_row_stride, p.qhead = q_head_stride;
    p.out = static_cast<uint16_t*>(out), p.orow = out_row_stride, p.ohead = out_head_stride;
    p.lse = lse, p.status = status;
    p.bt = block_table, p.bt_stride = bt_stride, p.starts = starts, p.row_ends = row_ends;
    p.topk = topk, p.topk_stride = topk_stride, p.k = static_cast<int>(k);
    p.R = static_cast<int>(num_requests), p.rows = static_cast<int>(rows), p.heads = static_cast<int>(heads);
    p.group = p.heads / p.kv_heads;
    p.max_keys = cache->num_pages > 0 ? static_cast<int>(max_pages * kPage) : 0;
    p.list_units = static_cast<int>((k + kUnit - 1) / kUnit);
    p.list_tiles = (p.group + p.cap - 1) / p.cap;
    const int64_t per_row = static_cast<int64_t>(p.kv_heads) * p.list_tiles * p.list_units;
    if (per_row > 0x7FFFFFFF) return DSA_ERR_UNSUPPORTED;
    p.packed = cache->num_pages <= (1 << 25) && per_row * rows * p.section >= kPackBytes;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    return launch_all4<true>(p, L.tiles, stream);
}
