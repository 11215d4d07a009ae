// dsa_attend_paged and dsa_attend_selected: decode attention over the paged
// key/value cache, on the tensor cores.
//
//   o = sum_t softmax_t(c q . k_t) v_t over the keys a row sees, in one pass:
//   per tile of 128 keys S = Q K^T, p = 2^(s c' - m), l += sum p, O += P V with a
//   running reference m of the row; pieces of a row's keys taken by different
//   CTAs are joined by their (m, l, O).
//
// The keys of all (segment, key head) items lie on one axis of 128-key tiles: a
// segment is a run of rows that share keys (rows of one request, or rows behind
// the prefix, or one row's listed keys).  Every worker (a pipeline slot of a CTA)
// takes an equal share of the axis, so one long context and many short ones fill
// the GPU alike; an item that several workers share is joined by a last, small
// kernel.  Up to 128 segments every CTA lays out the axis itself; for more, a plan
// kernel does.  Listed keys are first packed into slots, a CTA a row; a large
// batch's prefix has a launch of its own, in pairs of 128-row tiles.
//
// What bounds it: a key and its value are 4 d bytes and cost each row that shares
// them 4 d flops, one flop a byte, so memory bounds it until some 270 rows share a
// key; a prefix under hundreds of rows and heads is bound by the tensor cores.
// Measured on GB300 (BF16, whole calls, 6.8 TB/s and 1.95 PFLOP/s by copy and matrix
// product): 64 requests of 4096 to 8192 keys, 32 heads over 8: 237 to 241 us,
// 6.7 TB/s.  64 rows of 2048 listed keys: 97 us, 5.5 TB/s (the kernel alone 87 us).
// 320 rows of 64 heads over 8 behind 32768 keys: 276 us for the prefix,
// 1.25 PFLOP/s.  One row of 1000 keys: 10 us, a chain of latencies (4600 cycles to
// the first scores, 2750 for the join of the strips, then the pieces' join as a
// launch).
#include <math.h>

#include "elem16.cuh"
#include "host.h"

namespace dsa {

int check_kv_cache(const dsa_kv_cache* c);

constexpr int kTile = 128;          // keys per tile: two pages, or 128 listed keys
constexpr int kMaxCtas = 192;       // workspace and tables are sized for at most this many CTAs
constexpr int kMaxWorkers = 2 * kMaxCtas;
constexpr int kMaxStages = 10;
constexpr int kPieces = 4;          // piece records in flight per slot: ahead, in use, being read out
constexpr int kPlanThreads = 512;
constexpr int kListThreads = 256;
constexpr int kPrefixSmem = 2048;
constexpr int kPairTiles = 12;       // tiles a CTA from which a prefix is taken by pairs of row tiles
constexpr int kPlanSegs = 128;      // up to this many segments every CTA lays out the axis itself
constexpr int kPlanRows = 4096;     // ... and up to this many rows
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// The reference m of a row is raised when a tile's maximum passes it by more
// than this many powers of two; until then weights up to 2^8 are kept as they
// are, and O and l need no rescaling.
constexpr float kSlack = 8.0f;

// A run of a segment's tiles of one key/value head, taken by one worker.
struct Piece {
    int row0, nrows;      // query rows
    int kvh, req;         // key/value head; request, -1 for the shared prefix
    int keys, minb;       // largest and smallest key bound of the rows
    int tile0, ntiles;
    int slot;             // where its partial result goes
    int direct;           // no other piece sees these rows: write the output itself
    int poison;           // a value that some of the rows must not see is not finite
    int pad;
};

// Where the join finds a row's own pieces.
struct RowInfo {
    int64_t first;        // first tile of the segment on the axis
    int seg, row0, tph;   // segment (own ones count from 0; -1 outside every request), its first row, tiles per head
    int pad;
};

// The axis: tile prefix (all key heads), {first row, rows, request or -1, largest
// bound} and smallest bound of every segment, in shared or global memory.
struct Axis {
    int64_t* prefix;
    int4* seg;
    int* minb;
};

// Workspace regions, 256-byte aligned.
struct AttLayout {
    size_t info;      // int64[2]: tiles on the axis, segments
    size_t seg, minb, prefix;   // the axis in global memory (S = max_segs)
    size_t worker;    // int[kMaxWorkers]: segment of the worker's first tile
    size_t row_info;  // RowInfo[rows]
    size_t count;     // int[rows]: listed keys of each row
    size_t list;      // int[rows][kpad]: slots of the selected keys, packed
    size_t po, pml;   // float[pieces][own_cap][dim], float2[pieces][own_cap]: partial results
    size_t xo, xml;   // the same of the prefix's pieces
    size_t total;
    int64_t max_segs, kpad, own_rps;
};

struct AttParams {
    int64_t* info;
    Axis axis;
    int* worker;
    RowInfo* row_info;
    int* count;
    int* list;
    float* po;
    float2* pml;
    float* xo;
    float2* xml;
    const int32_t* bt;
    int64_t bt_stride;
    const int32_t* starts;
    const int32_t* row_ends;
    const int32_t* prefix_pages;
    const int32_t* topk;
    int64_t topk_stride;
    const uint16_t* vbase;                 // the value pool (element strides), read where a value is not finite
    int64_t vp, vt, vh;
    int kpu, ktu, khu, vpu, vtu, vhu;      // listed keys: row numbers per page, token, head in the pools' row maps
    int k_none, v_none;                    // ... and a row outside the map
    uint16_t* out;
    int64_t orow, ohead;
    float* lse;
    int32_t* status;
    int R, rows, heads, group, kv_heads, dim, max_keys, num_pages;
    int k, kpad;
    int prefix_len;                        // shared keys; prefix_mode says who computes them
    int prefix_mode;                       // 0 none, 1 segments of the axis, 2 the paired kernel
    int px_segs;                           // mode 1: the prefix's segments, first on the axis
    int rps, rows_cap;                     // query rows and tile rows (group * rps) of a tile
    int own_rps, own_cap;                  // the same of a request's segments
    int q_half, nst;                       // Q bytes per 64 columns and ring stages per slot
    int max_segs, workers;                 // workers: 2 per CTA of the axis' kernel
    int plan_in_cta;                       // every CTA lays out the axis, no plan kernel
    int x_rps, x_pairs, x_workers, x_cap;  // prefix: query rows per row tile, pairs of them, paired workers, tile rows
    float scale_log2;
};

// ----------------------------------------------------------------- the axis
// Worker w of W takes tiles [w T / W, (w + 1) T / W).
__device__ __forceinline__ int64_t share_start(int64_t w, int64_t T, int64_t W) {
    if ((w + 1) * T < (int64_t(1) << 32)) return static_cast<uint32_t>(w * T) / static_cast<uint32_t>(W);
    return w * T / W;
}
__device__ __forceinline__ int worker_of(int64_t t, int64_t T, int64_t W) {
    if (T * W < (int64_t(1) << 32))   // (a 64-bit division takes about five times the instructions)
        return static_cast<int>((static_cast<uint32_t>(t + 1) * static_cast<uint32_t>(W) - 1) /
                                static_cast<uint32_t>(T));
    return static_cast<int>(((t + 1) * W - 1) / T);
}
__device__ __forceinline__ int tiles_of(int keys) { return (keys + kTile - 1) / kTile; }

// Inclusive scan of one int64 per thread; total in *total (shared).
__device__ __forceinline__ int64_t block_scan64(int64_t v, int64_t* warp_tmp, int64_t* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t o = __shfl_up_sync(0xFFFFFFFFu, v, d);
        if (lane >= d) v += o;
    }
    if (lane == 31) warp_tmp[warp] = v;
    __syncthreads();
    if (warp == 0) {
        int64_t s = lane < nwarps ? warp_tmp[lane] : 0;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t o = __shfl_up_sync(0xFFFFFFFFu, s, d);
            if (lane >= d) s += o;
        }
        warp_tmp[lane] = s;
        if (lane == 31) *total = s;
    }
    __syncthreads();
    if (warp > 0) v += warp_tmp[warp - 1];
    __syncthreads();
    return v;
}

// Lays out the axis in global memory (whole block).  `tmp`: 33 int64 of shared scratch; `bounds`:
// shared scratch of one int per row, or null.  One block also writes what the
// join reads (`write`).  Returns the tiles; *segs: the segments.
template <bool kSelected>
__device__ int64_t lay_out(const AttParams& p, const Axis& ax, int64_t* tmp, int* bounds, bool write, int* segs) {
    int64_t* total = tmp + 32;
    const int nt = blockDim.x;
    bool bad = false;
    int S;
    if (kSelected) {
        S = p.rows;
        for (int r = threadIdx.x; r < S; r += nt) {
            const int n = p.count[r];
            ax.seg[r] = make_int4(r, 1, 0, n);
            ax.minb[r] = n;
        }
    } else {
        if (bounds)
            for (int r = threadIdx.x; r < p.rows; r += nt) bounds[r] = p.row_ends[r];
        if (write)
            for (int r = threadIdx.x; r < p.rows; r += nt) p.row_info[r] = RowInfo{0, -1, 0, 0, 0};
        for (int i = threadIdx.x; i < p.px_segs; i += nt) {
            ax.seg[i] = make_int4(i * p.x_rps, min(p.x_rps, p.rows - i * p.x_rps), -1, p.prefix_len);
            ax.minb[i] = p.prefix_len;
        }
        int carry = p.px_segs;
        __syncthreads();
        for (int base = 0; base < p.R; base += nt) {
            const int q = base + threadIdx.x;
            int s0 = 0, s1 = 0;
            if (q < p.R) {
                const int a = p.starts[q], b = p.starts[q + 1];
                if (a < 0 || b < a || b > p.rows) bad = true;
                s0 = min(max(a, 0), p.rows);
                s1 = min(max(b, s0), p.rows);
            }
            const int nseg = (s1 - s0 + p.own_rps - 1) / p.own_rps;
            // (requests that overlap may claim more segments than 32 bits count)
            const int64_t at = carry + block_scan64(nseg, tmp, total) - nseg;
            for (int i = 0; i < nseg; ++i) {
                if (at + i >= p.max_segs) {   // overlapping requests
                    bad = true;
                    break;
                }
                const int row0 = s0 + i * p.own_rps, nr = min(p.own_rps, s1 - row0);
                int most = 0, least = 0x7FFFFFFF;
                for (int r = row0; r < row0 + nr; ++r) {
                    const int given = bounds ? bounds[r] : p.row_ends[r];
                    const int e = min(max(given, 0), p.max_keys);
                    if (e != given) bad = true;
                    most = max(most, e);
                    least = min(least, e);
                }
                ax.seg[at + i] = make_int4(row0, nr, q, most);
                ax.minb[at + i] = least;
            }
            carry = static_cast<int>(min(carry + *total, static_cast<int64_t>(p.max_segs)));
            __syncthreads();
        }
        S = carry;
    }
    __syncthreads();
    int64_t carry = 0;
    for (int base = 0; base < S; base += nt) {
        const int i = base + threadIdx.x;
        const int4 rec = i < S ? ax.seg[i] : make_int4(0, 0, 0, 0);
        const int tph = tiles_of(rec.w);
        const int64_t n = static_cast<int64_t>(tph) * p.kv_heads;
        const int64_t before = carry + block_scan64(n, tmp, total) - n;
        if (i < S) {
            ax.prefix[i] = before;
            if (write && i >= p.px_segs)
                for (int r = rec.x; r < rec.x + rec.y; ++r)
                    p.row_info[r] = RowInfo{before, i - p.px_segs, rec.x, tph, 0};
        }
        carry += *total;
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        ax.prefix[S] = carry;
        if (write) {
            p.info[0] = carry;
            p.info[1] = S;
        }
    }
    if (write && bad && p.status) atomicOr(p.status, DSA_STATUS_BAD_GEOMETRY);
    __syncthreads();
    *segs = S;
    return carry;
}

// The same for up to kPlanSegs segments of at most as many requests, in shared
// memory: one warp does it with warp scans (the block's scans and their barriers
// cost 2 us where this takes half of one), after all threads have fetched the
// bounds.
template <bool kSelected>
__device__ int64_t lay_out_few(const AttParams& p, const Axis& ax, int* bounds, int64_t* result, bool write,
                               int* segs) {
    const int lane = threadIdx.x & 31;
    const bool first = threadIdx.x < 32;
    int a_next = 0, b_next = 0;
    if (!kSelected && first && lane < p.R) {
        a_next = p.starts[lane];
        b_next = p.starts[lane + 1];
    }
    for (int r = threadIdx.x; r < p.rows; r += blockDim.x) bounds[r] = kSelected ? p.count[r] : p.row_ends[r];
    if (!kSelected && write)
        for (int r = threadIdx.x; r < p.rows; r += blockDim.x) p.row_info[r] = RowInfo{0, -1, 0, 0, 0};
    __syncthreads();
    if (first) {
        bool bad = false;
        int S = p.rows;
        if (kSelected) {
            for (int r = lane; r < S; r += 32) {
                ax.seg[r] = make_int4(r, 1, 0, bounds[r]);
                ax.minb[r] = bounds[r];
            }
        } else {
            for (int i = lane; i < p.px_segs; i += 32) {
                ax.seg[i] = make_int4(i * p.x_rps, min(p.x_rps, p.rows - i * p.x_rps), -1, p.prefix_len);
                ax.minb[i] = p.prefix_len;
            }
            S = p.px_segs;
#pragma unroll 1
            for (int base = 0; base < p.R; base += 32) {
                const int a = a_next, b = b_next, q = base + 32 + lane;
                a_next = b_next = 0;
                if (q < p.R) {
                    a_next = p.starts[q];
                    b_next = p.starts[q + 1];
                }
                if (a < 0 || b < a || b > p.rows) bad = true;
                const int s0 = min(max(a, 0), p.rows), s1 = min(max(b, s0), p.rows);
                const int nseg = (s1 - s0 + p.own_rps - 1) / p.own_rps;
                int inc = nseg;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int o = __shfl_up_sync(0xFFFFFFFFu, inc, d);
                    if (lane >= d) inc += o;
                }
                const int at = S + inc - nseg;
                for (int j = 0; j < nseg; ++j) {
                    if (at + j >= p.max_segs) {   // overlapping requests
                        bad = true;
                        break;
                    }
                    const int row0 = s0 + j * p.own_rps, nr = min(p.own_rps, s1 - row0);
                    int most = 0, least = 0x7FFFFFFF;
                    for (int r = row0; r < row0 + nr; ++r) {
                        const int e = min(max(bounds[r], 0), p.max_keys);
                        if (e != bounds[r]) bad = true;
                        most = max(most, e);
                        least = min(least, e);
                    }
                    ax.seg[at + j] = make_int4(row0, nr, base + lane, most);
                    ax.minb[at + j] = least;
                }
                S = min(S + __shfl_sync(0xFFFFFFFFu, inc, 31), p.max_segs);
            }
        }
        __syncwarp();
        int64_t carry = 0;
#pragma unroll 1
        for (int base = 0; base < S; base += 32) {
            const int i = base + lane;
            const int4 rec = i < S ? ax.seg[i] : make_int4(0, 0, 0, 0);
            const int tph = tiles_of(rec.w);
            int64_t inc = static_cast<int64_t>(tph) * p.kv_heads;
            const int64_t n = inc;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int64_t o = __shfl_up_sync(0xFFFFFFFFu, inc, d);
                if (lane >= d) inc += o;
            }
            const int64_t before = carry + inc - n;
            if (i < S) {
                ax.prefix[i] = before;
                if (write && i >= p.px_segs)
                    for (int r = rec.x; r < rec.x + rec.y; ++r)
                        p.row_info[r] = RowInfo{before, i - p.px_segs, rec.x, tph, 0};
            }
            carry += __shfl_sync(0xFFFFFFFFu, inc, 31);
        }
        if (lane == 0) {
            ax.prefix[S] = carry;
            result[0] = carry;
            result[1] = S;
            if (write) {
                p.info[0] = carry;
                p.info[1] = S;
            }
        }
        if (write && bad && p.status) atomicOr(p.status, DSA_STATUS_BAD_GEOMETRY);
    }
    __syncthreads();
    *segs = static_cast<int>(result[1]);
    return result[0];
}

// The segment with tile t: the last that starts at or before it (segments
// without tiles come before the next one's start, so the last is not empty).
__device__ __forceinline__ int segment_of(const int64_t* prefix, int S, int64_t t) {
    int lo = 0, hi = S - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (prefix[mid] <= t) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// The axis in global memory, for calls of many segments.  One CTA.
template <bool kSelected>
__global__ void __launch_bounds__(kPlanThreads) attend_plan_kernel(const AttParams p) {
    pdl_wait();
    pdl_launch_dependents();
    __shared__ int64_t tmp[33];
    __shared__ int64_t sp[kPrefixSmem];
    __shared__ int bounds[kPlanRows];
    int S;
    const int64_t T =
        lay_out<kSelected>(p, p.axis, tmp, p.rows <= kPlanRows ? bounds : nullptr, true, &S);
    const bool fits = S <= kPrefixSmem;
    if (fits)
        for (int i = threadIdx.x; i < S; i += blockDim.x) sp[i] = p.axis.prefix[i];
    __syncthreads();
    const int64_t W = p.workers < T ? p.workers : T;
    for (int w = threadIdx.x; w < W; w += blockDim.x)
        p.worker[w] = segment_of(fits ? sp : p.axis.prefix, S, share_start(w, T, W));
}

// Packs each row's listed keys into slots (page * 64 + token; -1 for a page
// outside the pool) and counts them.  One CTA a row.
__global__ void __launch_bounds__(kListThreads) attend_list_kernel(const AttParams p) {
    pdl_wait();
    pdl_launch_dependents();
    __shared__ int64_t tmp[33];
    __shared__ int s_req;
    const int row = blockIdx.x;
    // (the first entries and the bound are on their way while the row's request is looked up)
    const int32_t* src = p.topk + row * p.topk_stride;
    int* dst = p.list + static_cast<int64_t>(row) * p.kpad;
    int next[4];
    auto load = [&](int base) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int at = base + threadIdx.x * 4 + i;
            next[i] = at < p.k ? src[at] : -1;
        }
    };
    load(0);
    const int e = p.row_ends[row];
    if (threadIdx.x == 0) s_req = -1;
    __syncthreads();
    bool bad = false, bad_page = false;
    for (int j = threadIdx.x; j < p.R; j += blockDim.x) {
        const int a = p.starts[j], b = p.starts[j + 1];
        if (a < 0 || b < a || b > p.rows) bad = true;
        if (a <= row && row < b) atomicMax(&s_req, j);
    }
    __syncthreads();
    const int req = s_req;
    int count = 0;
    if (req >= 0) {
        if (e < 0 || e > p.max_keys) bad = true;
        const int bound = min(max(e, 0), p.max_keys);
        const int32_t* pages = p.bt + req * p.bt_stride;
        for (int base = 0; base < p.k; base += 4 * kListThreads) {
            int slot[4], n = 0;
            int page[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) page[i] = next[i] >= 0 && next[i] < bound ? pages[next[i] / kPage] : -1;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = next[i];
                if (t >= bound) bad = true;
                if (t >= 0 && t < bound) {
                    const bool ok = page[i] >= 0 && page[i] < p.num_pages;
                    bad_page |= !ok;
                    slot[n++] = ok ? page[i] * kPage + t % kPage : -1;
                }
            }
            if (base + 4 * kListThreads < p.k) load(base + 4 * kListThreads);
            const int o = count + static_cast<int>(block_scan64(n, tmp, tmp + 32)) - n;
            for (int i = 0; i < n; ++i) dst[o + i] = slot[i];
            count += static_cast<int>(tmp[32]);
        }
    }
    if (threadIdx.x == 0) p.count[row] = count;
    if (bad && p.status) atomicOr(p.status, DSA_STATUS_BAD_GEOMETRY);
    if (bad_page && p.status) atomicOr(p.status, DSA_STATUS_BAD_PAGE);
}

// ----------------------------------------------------------------- attention
struct AttShared {
    uint64_t full[2][kMaxStages], empty[2][kMaxStages];
    uint64_t qfull[2], qempty[2];
    uint64_t sfull[2][2], pfull[2][2];   // per half tile (wide); [0] per tile (narrow)
    uint64_t ofull[2], ofree[2], drain[2];
    uint64_t pvdone[2], xch[2][4];       // wide: products of a half tile; the two warps of 32 rows meet
    uint8_t vote[2][4][2][2];            // ... and what each of them says there, by slot, rows, parity and half
    float half[2][2][128];            // maxima (then sums) of the two halves of each row; narrow: {m, l} of the strips
    uint64_t merge[2];                // narrow: the strips of a piece meet
    Piece piece[2][kPieces];
    int abort;
    uint32_t tmem;
};
constexpr int kAttMeta = (sizeof(AttShared) + 127) / 128 * 128;
static_assert(kAttMeta <= 3 * 1024, "five stages of 32 KB and two Q tiles leave 3 KB");

template <int DH>
__host__ __device__ constexpr int stage_bytes() { return DH * kTile * 128; }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint64_t pack2(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t r) {
    float2 v;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(r));
    return v;
}
// a b + c.  (A packed product and a packed sum, both rounded to nearest as written,
// came out as one fused operation; a product that is to be rounded adds a zero.)
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// Per-type facts: MMA type code, the exponent bits that mark a value that is
// not finite, and a shift of the weights.
//
// Weights are rounded to the cache's type before they meet the values (their sum
// takes them unrounded): both operands of the product have one type, and 16 bits
// more of each weight would be a second product of the same size.  It costs half a
// step of a weight each, independent of one another: against 64 bits outputs of
// 64 requests are 0.0020 off in BF16 where 32-bit weights leave 0.0017 (the
// rounding of the output itself), 0.00025 and 0.00021 in FP16.  FP16 weights are
// kept 2^7 larger (at most 2^15 with the slack) so that small ones stay out of the
// subnormals.
template <typename T>
struct Facts;
template <>
struct Facts<Bf16> {
    static constexpr uint32_t mma = 1, expo = 0x7F80u;
    static constexpr float shift = 0.0f;
};
template <>
struct Facts<Fp16> {
    static constexpr uint32_t mma = 0, expo = 0x7C00u;
    static constexpr float shift = 7.0f;
};

// What is added to a row's scores (in powers of two) before they are raised.  Its
// negative is the reference of the row's weights and of their sum: past 2^17 or so
// m and the shift no longer add up in 32 bits, and only what was added counts.
// Rounded down, here and in the test, so that no weight passes 2^(slack + shift).
// A score is rounded by its scale before this is added (no fused multiply-add), as
// the maximum is: otherwise half a step of the scaled score stays in the exponent,
// a factor of two from 2^24 on, and weights overflow (FP16 there, BF16 at 2^31).
template <typename T>
__device__ __forceinline__ float base_of(float m) {
    return m == -INFINITY ? 0.0f : __fadd_rd(Facts<T>::shift, -m);
}
__device__ __forceinline__ bool passes(float mx, float m) { return mx > __fadd_rd(m, kSlack); }

template <typename T>
__device__ __forceinline__ bool half_wild(uint32_t h) {
    return (h & Facts<T>::expo) == Facts<T>::expo;
}

// A whole warp's wait; the warp's answer, so that its lanes stay together.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort, int32_t* status) {
    const bool ok = mbar_wait(bar, parity, abort, status);
    return __all_sync(0xFFFFFFFFu, ok);
}

// One lane of the warp, chosen so that the compiler knows it is one: tensor and
// copy instructions take their operands from uniform registers, and under a
// plain lane test each of them is preceded by moves that cost about 100 cycles.
__device__ __forceinline__ bool elect_one() {
    uint32_t on;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(on));
    return on != 0;
}

// Where a role stands on the axis, and the ring position it is at.
struct Ring {
    int st = 0;
    uint32_t ph = 0;
    __device__ __forceinline__ void next(int nst) {
        if (++st == nst) {
            st = 0;
            ph ^= 1;
        }
    }
};

// The columns of a row's outputs, as the calling thread has written them for a piece
// (n from x0, x0 + step, ... on; `out` 16-bit outputs, else `part`), in which a value
// that the row sees is not finite: the sum of those values takes the output's place,
// since finite terms do not change it.  The products cannot give it:
// such values were taken out where some rows must not see them, and an infinite one
// times a weight of zero (another strip's key, or one too small for 16 bits) is NaN.
template <typename T, bool kSelected>
__device__ __noinline__ void put_wild(const AttParams& p, const Piece& pc, int row, int bound, int x0, int n, int step,
                                      uint16_t* out, float* part) {
    const int from = pc.tile0 * kTile, to = min(bound, (pc.tile0 + pc.ntiles) * kTile);
    const int32_t* pages = pc.req < 0 ? p.prefix_pages : p.bt + pc.req * p.bt_stride;
    const int* list = p.list + static_cast<int64_t>(row) * p.kpad;
    for (int y = 0; x0 + y / n * step < p.dim; y += 4) {
        const int x = x0 + y / n * step + y % n;
        bool finite = true;
        for (int j = 0; j < 4; ++j) finite &= out ? !half_wild<T>(out[x + j]) : isfinite(part[x + j]);
        float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        uint32_t found = 0;
        // (where the outputs are finite only a value that was taken out can change them; nothing changes four NaNs)
        for (int k = finite ? max(from, pc.minb) : from; k < to;) {
            const int end = min(to, (k | (kPage - 1)) + 1);
            const int of_page = kSelected ? 0 : pages[k / kPage];
#pragma unroll 8
            for (; k < end; ++k) {
                const int id = kSelected ? list[k] : 0;
                const int page = !kSelected ? of_page : id < 0 ? -1 : id / kPage, token = (kSelected ? id : k) % kPage;
                uint2 v = {0, 0};
                if (page >= 0 && page < p.num_pages)
                    v = *reinterpret_cast<const uint2*>(p.vbase + page * p.vp + token * p.vt + pc.kvh * p.vh + x);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t e = (j < 2 ? v.x : v.y) >> (j & 1) * 16;
                    if (half_wild<T>(e)) sum[j] += T::unpack(e).x, found |= 1u << j;
                }
            }
            if (isnan(sum[0]) && isnan(sum[1]) && isnan(sum[2]) && isnan(sum[3])) break;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (!(found >> j & 1)) continue;
            if (out)
                out[x + j] = static_cast<uint16_t>(T::pack(sum[j], 0.0f));
            else
                part[x + j] = sum[j];
        }
    }
}

// Room for the axis of a call of few segments.
struct AxisShared {
    int64_t prefix[kPlanSegs + 1];
    int4 seg[kPlanSegs];
    int minb[kPlanSegs];
};

// Threads of a CTA: 2 producer warps and 2 MMA warps, then softmax warps: 8 a
// slot, or 4 where tiles are narrow (and 4 more a slot that copy listed keys).
template <bool kSelected, bool kNarrow>
__host__ __device__ constexpr int att_threads() { return kNarrow && !kSelected ? 384 : 640; }
// Rows up to which a tile is narrow.  (17 to 32 rows: four copies of 32 rows were
// slower than wide tiles, 488 against 471 us for 128 requests of 1 to 4 rows of
// eight heads, since the copies' join at a piece's end grows with the rows.)
constexpr int kNarrowRows = 16;
// Narrow: the part of a strip's outputs that is joined at a time, 8 rows of 64
// columns or 16 of 32, each row padded by four floats.
constexpr int kMergeFloats = 576;
constexpr int kMergeBytes = 4 * kMergeFloats * 4;    // four strips, one slot

// One CTA runs two slots, each a pipeline of its own: a producer warp (TMA), an
// MMA warp and softmax warps, a thread per tile row (the lanes of tensor memory).
//
// Wide tiles (up to 128 rows): two threads share a row, half of the tile's keys
// each, and agree on its reference.  Narrow tiles (up to 16 rows, the usual
// decode): the rows are laid four times into the 128 tile rows, one copy to each
// warp of the slot; copy j weighs only keys 32j .. 32j + 31 of a tile (its other
// weights are zero) and keeps its own reference, so the softmax of a tile, which
// every product waits for, is a quarter as long and no warp waits for another;
// the four partial outputs are added at the end of the piece.
//
// Independent slots take two shares of the axis, each with its own ring of key and value
// stages; paired slots take two row tiles of one share and read the same ring
// (the prefix of a large batch: each key tile is loaded once for 256 rows).
//
// Measured choices.  Instructions issued by an elected lane instead of lane 0: the
// paired prefix of the batch above 340 -> 280 us.  Wide tiles in half-tile steps,
// the next scores made while the softmax works on these: the whole batch 512 -> 500
// us (half tiles read Q from shared memory twice as often, but whole tiles cannot be
// made ahead, since scores and output fill tensor memory: 334 -> 362 us for 320 rows
// of 64 heads over 8 behind 32768 keys).  Narrow tiles: 64
// requests of 4096 to 8192 keys 278 -> 260 us, 64 rows of 2048 listed keys 125 ->
// 112, measured with up to 32 rows (kNarrowRows says why 16).
template <typename T, bool kPaired, bool kSelected, bool kNarrow, int DH>
__global__ void __launch_bounds__(att_threads<kSelected, kNarrow>(), 1)
    attend_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                  const __grid_constant__ CUtensorMap vmap, const AttParams p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    // (a shuffled value is uniform to the compiler, and what follows from it stays in uniform registers)
    const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int q_bytes = DH * p.q_half;                                  // one slot's Q
    uint8_t* const ring0 = smem + 2 * q_bytes;
    const int rings = kPaired ? 1 : 2;
    uint8_t* const merge_buf = ring0 + rings * p.nst * stage_bytes<DH>();
    AttShared& sh = *reinterpret_cast<AttShared*>(merge_buf + (kNarrow ? 2 * kMergeBytes : 0));
    AxisShared& axis_sh = *reinterpret_cast<AxisShared*>(reinterpret_cast<uint8_t*>(&sh) + kAttMeta);
    volatile int* const abort = &sh.abort;
    const int active = kNarrow ? 4 : (p.rows_cap + 31) / 32;            // 32-row quarters with rows
    const int softmax_warps = kNarrow ? 4 : 2 * active;                 // per slot
    // Listed keys are copied by the warps that have no rows, while the producer warp loads Q; by the
    // producer warp where every warp has rows.
    const int helpers = !kSelected ? 0 : kNarrow ? 4 : 2 * (4 - active);
    const int copiers = helpers ? helpers : 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < 2; ++s) {
            for (int i = 0; i < p.nst; ++i) {
                mbar_init(&sh.full[s][i], 1);
                mbar_init(&sh.empty[s][i], kPaired ? 2 : 1);
            }
            mbar_init(&sh.qfull[s], 1);
            mbar_init(&sh.qempty[s], 1);
            for (int i = 0; i < 2; ++i) {
                mbar_init(&sh.sfull[s][i], 2);
                mbar_init(&sh.pfull[s][i], softmax_warps);
            }
            for (int i = 0; i < 4; ++i) mbar_init(&sh.xch[s][i], 2);
            mbar_init(&sh.pvdone[s], 1);
            mbar_init(&sh.ofull[s], 2);
            mbar_init(&sh.ofree[s], softmax_warps);
            mbar_init(&sh.merge[s], softmax_warps);
            mbar_init(&sh.drain[s], 1);
        }
        sh.abort = 0;
        mbar_fence_init();
    }
    if (warp == 0) {
        if (lane == 0) {
            tma_prefetch(&qmap);
            tma_prefetch(&kmap);
            tma_prefetch(&vmap);
        }
        tc_alloc(&sh.tmem, 512);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, sh.tmem, 0);
    pdl_wait();
    pdl_launch_dependents();

    const bool copies = kSelected && (kNarrow ? warp >= 12 : warp >= 4 && (warp & 3) >= active);
    const int slot = warp < 4 ? (warp & 1) : kNarrow ? (warp >> 2) - (warp < 12 ? 1 : 3) : (warp - 4) >> 3;
    const int half = ((warp - 4) >> 2) & 1, quarter = warp & 3;         // softmax: keys of the tile (wide), tile rows
    const int rs = kPaired ? 0 : slot;                                  // whose ring
    const int x_tiles = tiles_of(p.prefix_len);
    int S = 0;
    int64_t T_all;
    Axis axis = p.axis;
    if (kPaired) {
        T_all = static_cast<int64_t>(p.x_pairs) * p.kv_heads * x_tiles;
    } else if (p.plan_in_cta) {
        // (the ring is scratch until the first copy)
        axis = Axis{axis_sh.prefix, axis_sh.seg, axis_sh.minb};
        T_all = lay_out_few<kSelected>(p, axis, reinterpret_cast<int*>(ring0 + 512), reinterpret_cast<int64_t*>(ring0),
                                       blockIdx.x == 0, &S);
        fence_proxy_async_smem();
        __syncthreads();
    } else {
        T_all = p.info[0];
        S = static_cast<int>(p.info[1]);
    }
    const int64_t W_most = kPaired ? p.x_workers : p.workers;
    const int64_t W = W_most < T_all ? W_most : T_all;
    const int worker = kPaired ? blockIdx.x : slot * gridDim.x + blockIdx.x;
    const bool works = worker < W;
    const int64_t t0 = works ? share_start(worker, T_all, W) : 0;
    const int64_t t1 = works ? share_start(worker + 1, T_all, W) : 0;
    const int rps = kPaired ? p.x_rps : p.rps;
    uint8_t* const ring = ring0 + rs * p.nst * stage_bytes<DH>();

    if (warp < 2 || copies) {
        // ------------------------------------------------- producer
        if (kPaired && slot == 1) goto done;
        const bool lead = warp < 2;                                     // loads Q and writes the pieces' records
        const int copier = lead ? 0 : kNarrow ? quarter : half * (4 - active) + quarter - active;
        Ring at;
        int64_t issued = 0;
        int npiece = 0;
        bool ok = true;
        const uint64_t once = l2_evict_first_policy();
        int s = !works || kPaired ? 0 : p.plan_in_cta ? segment_of(axis.prefix, S, t0) : p.worker[worker];
        int sb = -64;                                                   // first of 32 segments held by the lanes
        int4 rec = {0, 0, 0, 0};
        int rec_min = 0;
        int64_t rec_pre = 0, rec_next = 0;
        int64_t t = t0;
        // Q of a piece: the buffer is free once the products of the piece that had it are done.
        auto load_q = [&](const Piece& pc) {
            const uint32_t ph = npiece & 1;
            bool got = true;
#pragma unroll
            for (int x = 0; x < (kPaired ? 2 : 1); ++x) {
                const int to = kPaired ? x : slot;
                got = got && warp_wait(&sh.qempty[to], ph ^ 1, abort, p.status);
                if (got && elect_one()) {
                    // The piece's record; its readers see it through this barrier.
                    Piece w = pc;
                    if (kPaired) {
                        w.row0 = pc.row0 + x * rps;
                        w.nrows = max(0, min(rps, p.rows - w.row0));
                    }
                    sh.piece[to][npiece % kPieces] = w;
                    uint8_t* qdst = smem + to * q_bytes;
                    constexpr int kCopies = kNarrow ? 4 : 1;
                    mbar_arrive_expect_tx(&sh.qfull[to], kCopies * DH * 128 * p.group * rps);
#pragma unroll
                    for (int h = 0; h < DH * kCopies; ++h)
                        tma_load_3d(qdst + h / kCopies * p.q_half + h % kCopies * 32 * 128, &qmap, h / kCopies * 64,
                                    pc.kvh * p.group, pc.row0 + (kPaired ? x * rps : 0), &sh.qfull[to]);
                }
            }
            ++npiece;
            return got;
        };
        while (t < t1 && ok) {
            Piece pc;
            pc.poison = 0;
            if (kPaired) {
                const int64_t item = t / x_tiles;
                const int pairs = p.x_pairs;
                pc.kvh = static_cast<int>(item / pairs);
                pc.row0 = static_cast<int>(item % pairs) * 2 * rps;
                pc.req = -1;
                pc.keys = pc.minb = p.prefix_len;
                pc.tile0 = static_cast<int>(t % x_tiles);
                pc.ntiles = static_cast<int>(min(static_cast<int64_t>(x_tiles - pc.tile0), t1 - t));
                pc.slot = static_cast<int>(item + worker);
                pc.direct = 0;
            } else {
                int64_t pre, nxt;
                for (;;) {
                    if (s < sb || s >= sb + 32) {
                        sb = s;
                        const int i = s + lane;
                        if (i < S) {
                            rec = axis.seg[i];
                            rec_min = axis.minb[i];
                            rec_pre = axis.prefix[i];
                            rec_next = axis.prefix[i + 1];
                        } else {
                            rec_pre = rec_next = T_all;
                        }
                    }
                    pre = __shfl_sync(0xFFFFFFFFu, rec_pre, s - sb);
                    nxt = __shfl_sync(0xFFFFFFFFu, rec_next, s - sb);
                    if (nxt > t) break;
                    ++s;
                }
                pc.row0 = __shfl_sync(0xFFFFFFFFu, rec.x, s - sb);
                pc.nrows = __shfl_sync(0xFFFFFFFFu, rec.y, s - sb);
                pc.req = __shfl_sync(0xFFFFFFFFu, rec.z, s - sb);
                pc.keys = __shfl_sync(0xFFFFFFFFu, rec.w, s - sb);
                pc.minb = __shfl_sync(0xFFFFFFFFu, rec_min, s - sb);
                const int tph = tiles_of(pc.keys);
                const int local = static_cast<int>(t - pre);
                pc.kvh = local / tph;
                pc.tile0 = local - pc.kvh * tph;
                pc.ntiles = static_cast<int>(min(static_cast<int64_t>(tph - pc.tile0), t1 - t));
                pc.slot = (pc.req < 0 ? s : s - p.px_segs) * p.kv_heads + pc.kvh + worker;
                pc.direct = p.prefix_mode == 0 && pc.ntiles == tph;
            }
            if (kSelected && lead && helpers) {
                ok = load_q(pc);
                t += pc.ntiles;
                continue;
            }
            const int32_t* pages = pc.req < 0 ? p.prefix_pages : p.bt + pc.req * p.bt_stride;
            const int npages = (pc.keys + kPage - 1) / kPage;
            int held = 0, held_next = 0;                                // 32 page ids, one per lane
            int4 ids = {0, 0, 0, 0}, ids_next = {0, 0, 0, 0};          // listed slots 4 lane .. 4 lane + 3 of a tile
            auto listed = [&](int tile) {   // (the list's rows are whole tiles)
                const int at = tile * kTile + lane * 4;
                int4 e = *reinterpret_cast<const int4*>(p.list + static_cast<int64_t>(pc.row0) * p.kpad + at);
                if (at >= pc.keys) e.x = -1;
                if (at + 1 >= pc.keys) e.y = -1;
                if (at + 2 >= pc.keys) e.z = -1;
                if (at + 3 >= pc.keys) e.w = -1;
                return e;
            };
            auto fetch = [&](int first) {
                const int j = first + lane;
                int id = p.num_pages;                                   // outside the map: zeros
                if (j < npages) {
                    id = pages[j];
                    if (id < 0 || id >= p.num_pages) {
                        if (p.status) atomicOr(p.status, DSA_STATUS_BAD_PAGE);
                        id = p.num_pages;
                    }
                }
                return id;
            };
            if (kSelected) ids_next = listed(pc.tile0);
            for (int i = 0; i < pc.ntiles && ok; ++i) {
                const int tile = pc.tile0 + i;
                int pg0 = 0, pg1 = 0;
                if (kSelected) {
                    ids = ids_next;
                    if (i + 1 < pc.ntiles) ids_next = listed(tile + 1);
                } else {
                    if ((i & 15) == 0) {
                        held = i == 0 ? fetch(2 * tile) : held_next;
                        held_next = pc.ntiles - i > 16 ? fetch(2 * tile + 32) : 0;
                    }
                    pg0 = __shfl_sync(0xFFFFFFFFu, held, 2 * (i & 15));
                    pg1 = __shfl_sync(0xFFFFFFFFu, held, 2 * (i & 15) + 1);
                }
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    ok = warp_wait(&sh.empty[rs][at.st], at.ph ^ 1, abort, p.status);
                    if (!ok) break;
                    uint64_t* bar = &sh.full[rs][at.st];
                    uint8_t* dst = ring + at.st * stage_bytes<DH>();
                    if (kSelected) {
                        // Four listed rows a copy.  The copies' operands pass through uniform registers, which
                        // makes issuing them the cost: the slot's copiers take every copiers-th group of four.
                        const CUtensorMap* map = kv ? &vmap : &kmap;
                        const int pu = kv ? p.vpu : p.kpu, tu = kv ? p.vtu : p.ktu, none = kv ? p.v_none : p.k_none;
                        const int head = pc.kvh * (kv ? p.vhu : p.khu);
                        auto row = [&](int id) { return id < 0 ? none : (id >> 6) * pu + (id & 63) * tu + head; };
                        const int4 r = make_int4(row(ids.x), row(ids.y), row(ids.z), row(ids.w));
                        if (copier == 0 && elect_one()) mbar_arrive_expect_tx(bar, stage_bytes<DH>());
                        // (eight groups at a time, so that their operands are fetched together)
                        for (int g0 = copier; g0 < 32; g0 += 8 * copiers) {
                            int4 rg[8];
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const int g = (g0 + j * copiers) & 31;
                                rg[j] = make_int4(__shfl_sync(0xFFFFFFFFu, r.x, g), __shfl_sync(0xFFFFFFFFu, r.y, g),
                                                  __shfl_sync(0xFFFFFFFFu, r.z, g), __shfl_sync(0xFFFFFFFFu, r.w, g));
                            }
                            if (elect_one()) {
#pragma unroll
                                for (int j = 0; j < 8; ++j) {
                                    const int g = g0 + j * copiers;
                                    if (g < 32)
#pragma unroll
                                        for (int h = 0; h < DH; ++h)
                                            tma_gather4(dst + h * kTile * 128 + g * 512, map, h * 64, rg[j], bar);
                                }
                            }
                        }
                    } else if (elect_one()) {
                        const CUtensorMap* map = kv ? &vmap : &kmap;
                        mbar_arrive_expect_tx(bar, stage_bytes<DH>());
#pragma unroll
                        for (int h = 0; h < DH; ++h) {
                            // (a request's keys are read once: they leave L2 first, before the partial results;
                            // 128 requests behind a prefix 496 -> 488 us)
                            uint8_t *d0 = dst + h * kTile * 128, *d1 = d0 + kPage * 128;
                            if (!kPaired && pc.req >= 0) {
                                tma_load_4d_hint(d0, map, h * 64, 0, pc.kvh, pg0, bar, once);
                                tma_load_4d_hint(d1, map, h * 64, 0, pc.kvh, pg1, bar, once);
                            } else {
                                tma_load_4d(d0, map, h * 64, 0, pc.kvh, pg0, bar);
                                tma_load_4d(d1, map, h * 64, 0, pc.kvh, pg1, bar);
                            }
                        }
                    }
                    ++issued;
                    at.next(p.nst);
                    // Q behind its first key tile
                    if (i == 0 && kv == 0 && lead && !(ok = load_q(pc))) break;
                }
            }
            t += pc.ntiles;
        }
        // Every stage and Q buffer has been released: no arrival is still on its way when the CTA exits.
        for (int64_t i = issued > p.nst ? issued - p.nst : 0; i < issued && ok; ++i)
            ok = warp_wait(&sh.empty[rs][i % p.nst], (i / p.nst) & 1, abort, p.status);
        // (only the warp that loads Q counts pieces)
        for (int x = 0; x < (kPaired ? 2 : 1); ++x)
            if (npiece > 0 && ok)
                ok = warp_wait(&sh.qempty[kPaired ? x : slot], (npiece - 1) & 1, abort, p.status);
        if (!ok) {
            // The copies in flight land before the CTA exits.
            const unsigned long long deadline = globaltimer() + kWaitLimitNs;
            const int64_t first = issued > p.nst ? issued - p.nst : 0;
            for (int64_t i = first; i < issued; ++i)
                if (!mbar_drain(&sh.full[rs][i % p.nst], (i / p.nst) & 1, deadline, p.status)) break;
            for (int x = 0; x < (kPaired ? 2 : 1); ++x)
                // (after a failed wait Q was not copied, and its buffer's phase is one behind: already past)
                if (npiece > 0 && mbar_test_wait(&sh.qempty[kPaired ? x : slot], npiece & 1))
                    mbar_drain(&sh.qfull[kPaired ? x : slot], (npiece - 1) & 1, deadline, p.status);
        }
    } else if (warp < 4) {
        // ------------------------------------------------- MMA issuer
        const uint32_t id_s = idesc_f16(Facts<T>::mma, 128, kNarrow ? kTile : 64, 0);
        const uint32_t id_o = idesc_f16(Facts<T>::mma, 128, p.dim, 1);
        const uint32_t d_s = tmem + slot * 128, d_o = tmem + 256 + slot * 128;
        const int ksteps = p.dim / 16;
        const uint64_t q_next = (p.q_half >> 4) - 8;                    // from columns 48.. to columns 64..
        const uint64_t k_next = (kTile * 128 >> 4) - 8;
        Ring at_k, at_v;                                                // keys and values alternate in the ring
        at_v.next(p.nst);
        uint32_t ph_p = 0, ph_of = 0;                                   // (wide: one bit per half tile)
        int npiece = 0;
        bool ok = true, any = false;
        int64_t t = t0;
        while (t < t1 && ok) {
            ok = warp_wait(&sh.qfull[slot], npiece & 1, abort, p.status);
            if (!ok) break;
            any = true;
            Piece& pc = sh.piece[slot][npiece % kPieces];
            const int ntiles = pc.ntiles, tile0 = pc.tile0, keys = pc.keys, minb = pc.minb;
            const uint64_t qd = desc_sw128(smem_u32(smem + slot * q_bytes));
            // A step is a tile (narrow), or half of one (wide, the last tile's second half only where it has keys).
            constexpr int kStep = kNarrow ? 1 : 2;
            const int steps = kNarrow ? ntiles : (min(keys - tile0 * kTile, ntiles * kTile) + 63) / 64;
            // S of a step into its columns; `freed`: nothing more is read from the key stage.
            auto scores = [&](int j) {
                const int h = kNarrow ? 0 : j & 1;
                if (h == 0 && !warp_wait(&sh.full[rs][at_k.st], at_k.ph, abort, p.status)) return false;
                const bool last = j == steps - 1, freed = last || h == kStep - 1;
                if (elect_one()) {
                    tc_fence_after();
                    const uint64_t kd = desc_sw128(smem_u32(ring + at_k.st * stage_bytes<DH>())) + h * (64 * 128 >> 4);
#pragma unroll
                    for (int kk = 0; kk < DH * 4; ++kk)
                        if (kk < ksteps)
                            tc_mma_f16(d_s + h * 64, qd + 2 * kk + (kk >= 4 ? q_next : 0),
                                       kd + 2 * kk + (kk >= 4 ? k_next : 0), id_s, kk > 0);
                    tc_commit(&sh.sfull[slot][h]);
                    mbar_arrive(&sh.sfull[slot][h]);      // passes the piece's record on
                    if (freed) tc_commit(&sh.empty[rs][at_k.st]);
                    if (last) tc_commit(&sh.qempty[slot]);
                }
                if (freed) {
                    at_k.next(p.nst);
                    at_k.next(p.nst);
                }
                return true;
            };
            // Wide: the next half tile's scores are made while the softmax works on this one's.
            ok = scores(0) && (kNarrow || steps < 2 || scores(1));
            for (int j = 0; j < steps && ok; ++j) {
                const int h = kNarrow ? 0 : j & 1, i = j / kStep;
                uint8_t* va = ring + at_v.st * stage_bytes<DH>();
                if (h == 0) {
                    ok = warp_wait(&sh.full[rs][at_v.st], at_v.ph, abort, p.status);
                    if (!ok) break;
                    if (!kSelected) {
                        // Values no row may see are zeroed (0 x NaN is NaN); values only some rows may see
                        // are searched for such, which the softmax warps then look up themselves.
                        const int left = keys - (tile0 + i) * kTile;       // keys of this tile
                        const int all = minb - (tile0 + i) * kTile;        // ... that every row sees
                        if (left < kTile || all < left) {
                            const int from = min(max(all, 0), min(left, kTile));
                            for (int x = lane; x < (kTile - from) * DH * 8; x += 32) {
                                const int r = from + x / (DH * 8), c = x % (DH * 8);
                                uint8_t* at8 = va + (c >> 3) * kTile * 128 + r * 128 + (c & 7) * 16;
                                uint4* at16 = reinterpret_cast<uint4*>(at8);
                                if (r >= left) {
                                    *at16 = make_uint4(0, 0, 0, 0);
                                } else {
                                    uint4 v = *at16;
                                    uint32_t* w = &v.x;
                                    bool wild = false;
#pragma unroll
                                    for (int j = 0; j < 4; ++j) {
                                        if (half_wild<T>(w[j])) w[j] &= 0xFFFF0000u, wild = true;
                                        if (half_wild<T>(w[j] >> 16)) w[j] &= 0x0000FFFFu, wild = true;
                                    }
                                    if (wild) {
                                        *at16 = v;
                                        pc.poison = 1;
                                    }
                                }
                            }
                            fence_proxy_async_smem();
                            __syncwarp();
                        }
                    }
                }
                ok = warp_wait(&sh.pfull[slot][h], (ph_p >> h) & 1, abort, p.status);
                if (!ok) break;
                ph_p ^= 1u << h;
                if (j == 0) {   // the accumulator is free once the piece before has been read out
                    ok = warp_wait(&sh.ofree[slot], ph_of ^ 1, abort, p.status);
                    if (!ok) break;
                    ph_of ^= 1;
                }
                const bool last = j == steps - 1, freed = last || h == kStep - 1;
                if (elect_one()) {
                    tc_fence_after();
                    const uint64_t vd = desc_mn_sw128(smem_u32(va), kTile * 128);
#pragma unroll
                    for (int kk = 0; kk < kTile / 16 / kStep; ++kk)
                        tc_mma_f16_ta(d_o, d_s + h * 64 + 8 * kk, vd + 128 * (4 * h + kk), id_o, j > 0 || kk > 0);
                    if (!kNarrow) tc_commit(&sh.pvdone[slot]);
                    if (freed) tc_commit(&sh.empty[rs][at_v.st]);
                    if (last) {
                        tc_commit(&sh.ofull[slot]);
                        mbar_arrive(&sh.ofull[slot]);   // passes the record's poison mark on
                    }
                }
                if (freed) {
                    at_v.next(p.nst);
                    at_v.next(p.nst);
                }
                if (j + kStep < steps) ok = scores(j + kStep);
            }
            t += ntiles;
            ++npiece;
        }
        if (any && !ok && elect_one()) {
            // The products in flight end before the CTA exits.
            tc_commit(&sh.drain[slot]);
            mbar_drain(&sh.drain[slot], 0, globaltimer() + kWaitLimitNs, p.status);
        }
    } else if (kNarrow) {
        // ------------------------------------------------- softmax, narrow: 32 keys of a row per thread
        const int mi = lane / p.group;                                  // query row of the piece
        // the join at a piece's end: rows the buffer is laid out for, this thread's row there and its first column
        const int mrows = p.rows_cap <= 8 ? 8 : kNarrowRows;
        const int r = (quarter * 32 + lane) & (mrows - 1), col4 = (quarter * 32 + lane) / mrows * 4;
        const int ri = r / p.group, rg = r - ri * p.group, mcols = 512 / mrows;
        const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
        const uint32_t a_s = tmem + lanes + slot * 128, a_o = tmem + lanes + 256 + slot * 128;
        const float c = p.scale_log2;
        float2* const ml = reinterpret_cast<float2*>(&sh.half[0][0][0]) + slot * 128;   // [strip][row]
        float* const buf = reinterpret_cast<float*>(merge_buf + slot * kMergeBytes);    // [strip][column][row]
        uint32_t ph_s = 0, ph_o = 0, ph_m = 0;
        int npiece = 0;
        bool ok = true;
        auto meet = [&]() {                                             // the slot's four warps, bounded
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.merge[slot]);
            ok = warp_wait(&sh.merge[slot], ph_m, abort, p.status);
            ph_m ^= 1;
            return ok;
        };
        int64_t t = t0;
        while (t < t1 && ok) {
            float m_ref = -INFINITY, base = 0.0f, l = 0.0f;
            int ntiles = 1, tile0 = 0, bound = 0;
            bool on = false;
            const Piece& pc = sh.piece[slot][npiece % kPieces];
            for (int i = 0; i < ntiles; ++i) {
                ok = warp_wait(&sh.sfull[slot][0], ph_s, abort, p.status);
                if (!ok) break;
                ph_s ^= 1;
                tc_fence_after();
                if (i == 0) {
                    ntiles = pc.ntiles, tile0 = pc.tile0;
                    on = mi < pc.nrows;
                    bound = pc.keys;
                    if (on && pc.minb != pc.keys) bound = min(max(p.row_ends[pc.row0 + mi], 0), p.max_keys);
                }
                uint32_t w[32];
                tc_ld_32x32b_x32(a_s + quarter * 32, w);
                tc_wait_ld_regs<32>(w);
                const int left = bound - (tile0 + i) * kTile - quarter * 32;
                if (left < 32) {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (j >= left) w[j] = 0xFF800000u;
                }
                float m4[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) m4[j] = fmaxf(__uint_as_float(w[j]), __uint_as_float(w[j + 4]));
#pragma unroll
                for (int j = 8; j < 32; j += 8)
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        m4[x] = fmaxf(fmaxf(m4[x], __uint_as_float(w[j + x])), __uint_as_float(w[j + x + 4]));
                const float mx = __fmul_rn(fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])), c);
                const bool up = passes(mx, m_ref);
                if (__any_sync(0xFFFFFFFFu, up)) {
                    const float nb = up ? base_of<T>(mx) : base;
                    const float f = !up ? 1.0f : m_ref == -INFINITY ? 0.0f : ex2(nb - base);
                    if (up) m_ref = mx;
                    base = nb;
                    l *= f;
                    if (i > 0) {
                        // every product of this slot so far is done (they precede this tile's scores)
                        for (int x = 0; x < p.dim; x += 16) {
                            uint32_t o[16];
                            tc_ld_32x32b_x16(a_o + x, o);
                            tc_wait_ld16(o);
#pragma unroll
                            for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                            tc_st_32x32b_x16(a_o + x, o);
                        }
                    }
                }
                const uint64_t c2 = pack2(c, c), b2 = pack2(base, base);
                uint64_t s0 = 0, s1 = 0;
                uint32_t h[16];
#pragma unroll
                for (int j = 0; j < 32; j += 2) {
                    const uint64_t s2 = pack2(__uint_as_float(w[j]), __uint_as_float(w[j + 1]));
                    const float2 e = unpack2(add2(fma2(s2, c2, 0), b2));
                    const float p0 = ex2(e.x), p1 = ex2(e.y);
                    if (j & 2) s1 = add2(s1, pack2(p0, p1));
                    else s0 = add2(s0, pack2(p0, p1));
                    h[j / 2] = T::pack(p0, p1);
                }
                const float2 sum = unpack2(add2(s0, s1));
                l += sum.x + sum.y;
                // The weights take the scores' place, in this warp's own lanes: its strip, zeros elsewhere.
                uint32_t zero[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) zero[j] = 0;
#pragma unroll
                for (int x = 1; x < 4; ++x) tc_st_32x32b_x16(a_s + ((quarter + x) & 3) * 16, zero);
                tc_st_32x32b_x16(a_s + quarter * 16, h);
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.pfull[slot][0]);
            }
            if (!ok) break;
            ok = warp_wait(&sh.ofull[slot], ph_o, abort, p.status);
            if (!ok) break;
            ph_o ^= 1;
            tc_fence_after();
            // The four strips are joined, as many columns at a time as the buffer holds for this call's rows.
            // (Loops stay rolled and accesses are 16 bytes wide: this code runs once a piece, and instructions
            // that are not in the cache cost more than what they do.)  A thread writes its row's strip and adds
            // four columns of row `r`, each strip brought to the row's common reference.
            ml[quarter * 32 + lane] = make_float2(m_ref == -INFINITY ? -INFINITY : -base, l);
            if (!meet()) break;
            const bool poison = *reinterpret_cast<const volatile int*>(&pc.poison) != 0;
            const bool direct = pc.direct, own = pc.req >= 0 || kSelected;
            const bool r_on = ri < pc.nrows;
            float2 e[4];
            float top = -INFINITY, sum = 0.0f, f[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                e[x] = ml[x * 32 + r];
                top = fmaxf(top, e[x].x);
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                f[x] = e[x].x == -INFINITY ? 0.0f : ex2(e[x].x - top);
                sum += e[x].y * f[x];
            }
            const int row = pc.row0 + ri, head = pc.kvh * p.group + rg;
            uint16_t* out = p.out + row * p.orow + head * p.ohead;
            const int64_t at = static_cast<int64_t>(pc.slot) * (own ? p.own_cap : p.x_cap) + r;
            float* part = (own ? p.po : p.xo) + at * p.dim;
            if (direct) {
                const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
                for (int x = 0; x < 4; ++x) f[x] *= inv;
            }
            if (r_on && col4 == 0) {
                if (!direct)
                    (own ? p.pml : p.xml)[at] = make_float2(top, sum);
                else if (p.lse)
                    p.lse[static_cast<int64_t>(row) * p.heads + head] =
                        sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
            }
            float wild = poison ? NAN : 0.0f;
#pragma unroll 1
            for (int x = 0; x < p.dim; x += mcols) {
                if (x > 0 && !meet()) break;                            // the buffer has been read
#pragma unroll 1
                for (int y = 0; y < mcols; y += 16) {
                    if (x + y >= p.dim) break;
                    uint32_t o[16];
                    tc_ld_32x32b_x16(a_o + x + y, o);
                    tc_wait_ld16(o);
                    if (lane < mrows) {
                        uint4* to = reinterpret_cast<uint4*>(buf + quarter * kMergeFloats + lane * (mcols + 4) + y);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            to[j] = make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
                    }
                }
                if (!meet()) break;
                float4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const float4 u = *reinterpret_cast<const float4*>(buf + y * kMergeFloats + r * (mcols + 4) + col4);
                    v.x += u.x * f[y], v.y += u.y * f[y], v.z += u.z * f[y], v.w += u.w * f[y];
                }
                if (r_on && x + col4 < p.dim) {
                    // (NaN once an output is not finite)
                    wild = fmaf(v.x, 0.0f, fmaf(v.y, 0.0f, fmaf(v.z, 0.0f, fmaf(v.w, 0.0f, wild))));
                    if (direct)
                        *reinterpret_cast<uint2*>(out + x + col4) =
                            make_uint2(T::pack(v.x, v.y), T::pack(v.z, v.w));
                    else
                        *reinterpret_cast<float4*>(part + x + col4) = v;
                }
            }
            if (!ok) break;
            if (r_on && wild != 0.0f && sum > 0.0f) {
                const int sees = pc.minb == pc.keys ? pc.keys : min(max(p.row_ends[row], 0), p.max_keys);
                put_wild<T, kSelected>(p, pc, row, sees, col4, 4, mcols, direct ? out : nullptr, part);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.ofree[slot]);
            t += ntiles;
            ++npiece;
        }
    } else {
        // ------------------------------------------------- softmax, wide: half a row per thread
        if (quarter >= active) goto done;
        const int m = quarter * 32 + lane;                              // tile row
        const int mi = m / p.group, mg = m - mi * p.group;              // query row of the piece, head of the group
        const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
        const uint32_t a_s = tmem + lanes + slot * 128, a_o = tmem + lanes + 256 + slot * 128;
        const float c = p.scale_log2;
        uint32_t ph_s = 0, ph_o = 0, ph_x = 0;                          // (ph_s: one bit per half tile)
        uint32_t steps_done = 0;
        int npiece = 0;
        bool ok = true;
        // The row's two warps meet; bounded, as every wait is that another role may leave unanswered.  (At a named
        // barrier, which has no limit, 320 rows behind 32768 keys took 476 us, so 484; 17 rows behind 4001 keys 16.4
        // and 17.0.)
        auto meet = [&]() {
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.xch[slot][quarter]);
            ok = warp_wait(&sh.xch[slot][quarter], ph_x, abort, p.status);
            ph_x ^= 1;
            return ok;
        };
        // They meet, and either may say so: 0 nobody did, 1 somebody did, -1 the wait ran out.  (A place by the
        // parity of the meeting: the other warp has read it before it arrives at the next.)
        auto meet_any = [&](bool v) {
            uint8_t* const at = sh.vote[slot][quarter][ph_x];
            v = __any_sync(0xFFFFFFFFu, v);
            if (lane == 0) at[half] = v;
            if (!meet()) return -1;
            return static_cast<int>(v || *const_cast<volatile uint8_t*>(at + (half ^ 1)));
        };
        int64_t t = t0;
        while (t < t1 && ok) {
            float m_ref = -INFINITY, base = 0.0f, l = 0.0f;
            int steps = 1, ntiles = 1, tile0 = 0, bound = 0;
            bool on = false, warp_on = false;
            const Piece& pc = sh.piece[slot][npiece % kPieces];
            for (int j = 0; j < steps; ++j, ++steps_done) {
                const int h = j & 1;
                ok = warp_wait(&sh.sfull[slot][h], (ph_s >> h) & 1, abort, p.status);
                if (!ok) break;
                ph_s ^= 1u << h;
                tc_fence_after();
                if (j == 0) {
                    // the sums of the piece before, in the maxima's place, have been read
                    ok = npiece == 0 || warp_wait(&sh.ofree[slot], (npiece - 1) & 1, abort, p.status);
                    if (!ok) break;
                    ntiles = pc.ntiles, tile0 = pc.tile0;
                    steps = (min(pc.keys - tile0 * kTile, ntiles * kTile) + 63) / 64;
                    on = mi < pc.nrows;
                    warp_on = quarter * 32 < pc.nrows * p.group;
                    bound = pc.keys;
                    if (on && pc.minb != pc.keys) bound = min(max(p.row_ends[pc.row0 + mi], 0), p.max_keys);
                }
                if (warp_on) {
                    uint32_t w[32];
                    tc_ld_32x32b_x32(a_s + h * 64 + half * 32, w);
                    tc_wait_ld_regs<32>(w);
                    const int left = bound - tile0 * kTile - j * 64 - half * 32;
                    if (left < 32) {
#pragma unroll
                        for (int x = 0; x < 32; ++x)
                            if (x >= left) w[x] = 0xFF800000u;
                    }
                    float m4[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x) m4[x] = fmaxf(__uint_as_float(w[x]), __uint_as_float(w[x + 4]));
#pragma unroll
                    for (int y = 8; y < 32; y += 8)
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            m4[x] = fmaxf(fmaxf(m4[x], __uint_as_float(w[y + x])), __uint_as_float(w[y + x + 4]));
                    float mx = __fmul_rn(fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])), c);
                    // The two warps meet in any case: both have read their scores, so the weights may take the
                    // scores' columns.  Where a row's reference has to rise, they agree on it.
                    const int raise = meet_any(passes(mx, m_ref));
                    if (raise < 0) break;
                    if (raise) {
                        sh.half[slot][half][m] = mx;
                        if (!meet()) break;
                        mx = fmaxf(mx, sh.half[slot][half ^ 1][m]);
                        if (!meet()) break;
                        const bool up = passes(mx, m_ref);
                        const float nb = up ? base_of<T>(mx) : base;
                        const float f = !up ? 1.0f : m_ref == -INFINITY ? 0.0f : ex2(nb - base);
                        if (up) m_ref = mx;
                        base = nb;
                        l *= f;
                        if (j > 0) {
                            // the products of the half tile before may still be running
                            ok = warp_wait(&sh.pvdone[slot], (steps_done - 1) & 1, abort, p.status);
                            if (!ok) break;
                            tc_fence_after();
#pragma unroll 1
                            for (int x = half * 16; x < p.dim; x += 32) {
                                uint32_t o[16];
                                tc_ld_32x32b_x16(a_o + x, o);
                                tc_wait_ld16(o);
#pragma unroll
                                for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
                                tc_st_32x32b_x16(a_o + x, o);
                            }
                        }
                    }
                    const uint64_t c2 = pack2(c, c), b2 = pack2(base, base);
                    uint64_t s0 = 0, s1 = 0;
                    uint32_t e16[16];
#pragma unroll
                    for (int x = 0; x < 32; x += 2) {
                        const uint64_t s2 = pack2(__uint_as_float(w[x]), __uint_as_float(w[x + 1]));
                        const float2 e = unpack2(add2(fma2(s2, c2, 0), b2));
                        const float p0 = ex2(e.x), p1 = ex2(e.y);
                        if (x & 2) s1 = add2(s1, pack2(p0, p1));
                        else s0 = add2(s0, pack2(p0, p1));
                        e16[x / 2] = T::pack(p0, p1);
                    }
                    const float2 sum = unpack2(add2(s0, s1));
                    l += sum.x + sum.y;
                    tc_st_32x32b_x16(a_s + h * 64 + half * 16, e16);
                    tc_wait_st();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.pfull[slot][h]);
            }
            if (!ok) break;
            ok = warp_wait(&sh.ofull[slot], ph_o, abort, p.status);
            if (!ok) break;
            ph_o ^= 1;
            tc_fence_after();
            if (warp_on) {
                // (the products are done, so both warps are past the last tile's maxima)
                sh.half[slot][half][m] = l;
                if (!meet()) break;
                l = sh.half[slot][0][m] + sh.half[slot][1][m];
                const bool poison = *reinterpret_cast<const volatile int*>(&pc.poison) != 0;
                const float ref = m_ref == -INFINITY ? -INFINITY : -base;
                const int row = pc.row0 + mi, head = pc.kvh * p.group + mg;
                const bool direct = pc.direct;
                const float inv = l == 0.0f ? 0.0f : 1.0f / l;
                uint16_t* out = p.out + row * p.orow + head * p.ohead;
                float* part;
                if (kPaired) {
                    const int64_t at = (static_cast<int64_t>(pc.slot) * 2 + slot) * 128 + m;
                    part = p.xo + at * p.dim;
                    if (on && half == 0) p.xml[at] = make_float2(ref, l);
                } else {
                    const bool own = kSelected || pc.req >= 0;
                    const int64_t at = static_cast<int64_t>(pc.slot) * (own ? p.own_cap : p.x_cap) + m;
                    part = (own ? p.po : p.xo) + at * p.dim;
                    if (on && !direct && half == 0) (own ? p.pml : p.xml)[at] = make_float2(ref, l);
                }
                if (on && direct && half == 0 && p.lse)
                    p.lse[static_cast<int64_t>(row) * p.heads + head] =
                        l == 0.0f ? -INFINITY : (ref + log2f(l)) * kLn2;
                float wild = poison ? NAN : 0.0f;                       // (NaN once an output is not finite)
                for (int x = half * 16; x < p.dim; x += 32) {
                    uint32_t o[16];
                    tc_ld_32x32b_x16(a_o + x, o);
                    tc_wait_ld16(o);
#pragma unroll
                    for (int j = 0; j < 16; ++j) wild = fmaf(__uint_as_float(o[j]), 0.0f, wild);
                    if (on && direct) {
                        uint32_t h[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            h[j] = T::pack(__uint_as_float(o[2 * j]) * inv, __uint_as_float(o[2 * j + 1]) * inv);
                        *reinterpret_cast<uint4*>(out + x) = make_uint4(h[0], h[1], h[2], h[3]);
                        *reinterpret_cast<uint4*>(out + x + 8) = make_uint4(h[4], h[5], h[6], h[7]);
                    } else if (on) {
#pragma unroll
                        for (int j = 0; j < 16; j += 4)
                            *reinterpret_cast<uint4*>(part + x + j) = make_uint4(o[j], o[j + 1], o[j + 2], o[j + 3]);
                    }
                }
                if (on && wild != 0.0f && l > 0.0f)
                    put_wild<T, kSelected>(p, pc, row, bound, half * 16, 16, 32, direct ? out : nullptr, part);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.ofree[slot]);
            t += ntiles;
            ++npiece;
        }
    }
done:
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tc_dealloc(tmem, 512);
    }
}

// ----------------------------------------------------------------- join
// Joins the pieces of a (row, head): kWarps warps take every kWarps-th piece,
// four columns a lane.
template <typename T, int kWarps>
__global__ void __launch_bounds__(kWarps == 1 ? 128 : kWarps * 32) attend_join_kernel(const AttParams p) {
    constexpr int kItems = kWarps == 1 ? 4 : 1;
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // (the items fit 31 bits; 64-bit divisions here were most of the kernel's instructions)
    const uint32_t item = blockIdx.x * kItems + (kWarps == 1 ? warp : 0), heads = p.heads;
    if (item >= static_cast<uint32_t>(p.rows) * heads) return;
    const int row = item / heads, head = item - row * heads;
    const int kvh = static_cast<uint32_t>(head) / static_cast<uint32_t>(p.group), g = head - kvh * p.group;
    const RowInfo ri = p.row_info[row];
    const int64_t T_all = p.info[0];
    // two runs of pieces: the row's own keys and the prefix
    const float2 *ml0 = nullptr, *ml1 = nullptr;
    const float *po0 = nullptr, *po1 = nullptr;
    int n0 = 0, n1 = 0, step1 = p.x_cap;   // pieces; tile rows from one of the prefix's to the next
    if (ri.seg >= 0) {
        const int64_t W = p.workers < T_all ? p.workers : T_all;
        if (ri.tph > 0) {
            const int64_t first = ri.first + static_cast<int64_t>(kvh) * ri.tph;
            const int wa = worker_of(first, T_all, W), wb = worker_of(first + ri.tph - 1, T_all, W);
            const int64_t at =
                (static_cast<int64_t>(ri.seg) * p.kv_heads + kvh + wa) * p.own_cap + (row - ri.row0) * p.group + g;
            ml0 = p.pml + at;
            po0 = p.po + at * p.dim;
            n0 = wb - wa + 1;
            if (p.prefix_mode == 0 && n0 == 1) return;   // written by the attention kernel
        }
        if (p.prefix_mode != 0) {
            const int tph = tiles_of(p.prefix_len);
            const int tile = static_cast<uint32_t>(row) / static_cast<uint32_t>(p.x_rps);   // row tile
            const int in = row - tile * p.x_rps;
            int64_t at;
            if (p.prefix_mode == 1) {
                const int64_t it = static_cast<int64_t>(tile) * p.kv_heads + kvh;
                const int wa = worker_of(it * tph, T_all, W), wb = worker_of(it * tph + tph - 1, T_all, W);
                at = (it + wa) * p.x_cap + in * p.group + g;
                n1 = wb - wa + 1;
            } else {
                const int64_t T_x = static_cast<int64_t>(p.x_pairs) * p.kv_heads * tph;
                const int64_t W_x = p.x_workers < T_x ? p.x_workers : T_x;
                const int64_t it = static_cast<int64_t>(kvh) * p.x_pairs + tile / 2;
                const int wa = worker_of(it * tph, T_x, W_x), wb = worker_of(it * tph + tph - 1, T_x, W_x);
                at = ((it + wa) * 2 + tile % 2) * 128 + in * p.group + g;
                step1 = 256;
                n1 = wb - wa + 1;
            }
            ml1 = p.xml + at;
            po1 = p.xo + at * p.dim;
        }
    }
    const bool on = lane * 4 < p.dim;
    // One pass over the pieces of both runs, kAhead at a time, with a running reference.
    constexpr int kAhead = 4;
    const int all = n0 + n1;
    float top = -INFINITY, l = 0.0f;
    float4 o = {0, 0, 0, 0};
    for (int base = kWarps == 1 ? 0 : warp; base < all; base += kAhead * kWarps) {
        float2 e[kAhead];
        float4 v[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int i = base + j * kWarps;
            const bool own = i < n0;
            const int at = own ? i * p.own_cap : (i - n0) * step1;   // (at most kMaxWorkers * 256)
            e[j] = make_float2(-INFINITY, 0.0f);
            v[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (i < all) {
                e[j] = (own ? ml0 : ml1)[at];
                if (on) v[j] = *reinterpret_cast<const float4*>((own ? po0 : po1) + at * p.dim + lane * 4);
            }
        }
        float m = top;
#pragma unroll
        for (int j = 0; j < kAhead; ++j) m = fmaxf(m, e[j].x);
        const float keep = top == -INFINITY ? 0.0f : ex2(top - m);
        top = m;
        l *= keep;
        o.x *= keep, o.y *= keep, o.z *= keep, o.w *= keep;
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const float f = e[j].x == -INFINITY ? 0.0f : ex2(e[j].x - m);
            l += e[j].y * f;
            o.x += v[j].x * f, o.y += v[j].y * f, o.z += v[j].z * f, o.w += v[j].w * f;
        }
    }
    if (kWarps > 1) {
        __shared__ float2 sl[kWarps];
        __shared__ float4 so[kWarps][32];
        if (lane == 0) sl[warp] = make_float2(top, l);
        so[warp][lane] = o;
        __syncthreads();
        if (warp > 0) return;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sl[w].x);
        l = 0.0f;
        o = {0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float4 v = so[w][lane];
            const float f = sl[w].x == -INFINITY ? 0.0f : ex2(sl[w].x - top);
            l += sl[w].y * f;
            o.x += v.x * f, o.y += v.y * f, o.z += v.z * f, o.w += v.w * f;
        }
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    if (on)
        *reinterpret_cast<uint2*>(p.out + row * p.orow + head * p.ohead + lane * 4) =
            make_uint2(T::pack(o.x * inv, o.y * inv), T::pack(o.z * inv, o.w * inv));
    if (lane == 0 && p.lse)
        p.lse[item] = l == 0.0f ? -INFINITY : (top + log2f(l)) * kLn2;
}

// ----------------------------------------------------------------- host
static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

static int64_t clamp64(int64_t v, int64_t lo, int64_t hi) { return v < lo ? lo : v > hi ? hi : v; }

static AttLayout attend_layout(int64_t rows, int64_t num_requests, int64_t heads, int64_t kv_heads, int64_t dim,
                               int64_t max_query_len, int64_t k) {
    AttLayout L = {};
    const int64_t group = heads / kv_heads, most = 128 / group;
    // a request's segments: as many rows as a request is said to have, no more than fit a tile
    L.own_rps = k > 0 ? 1 : clamp64(max_query_len < rows ? max_query_len : rows, 1, most);
    const int64_t full = rows / L.own_rps + num_requests;   // every request starts a segment of its own
    const int64_t segs = k > 0 || rows < full ? rows : full;
    const int64_t px = k > 0 ? 0 : (rows + most - 1) / most;   // row tiles behind a prefix
    L.max_segs = segs + px;
    L.kpad = (k + kTile - 1) / kTile * kTile;
    size_t at = 0;
    auto take = [&](int64_t bytes) {
        const size_t here = at;
        at += (static_cast<size_t>(bytes) + 255) / 256 * 256;
        return here;
    };
    L.info = take(16);
    L.seg = take(L.max_segs * 16);
    L.minb = take(L.max_segs * 4);
    L.prefix = take((L.max_segs + 1) * 8);
    L.worker = take(kMaxWorkers * 4);
    L.row_info = take(rows * static_cast<int64_t>(sizeof(RowInfo)));
    L.count = take(k > 0 ? rows * 4 : 0);
    L.list = take(rows * L.kpad * 4);
    // a piece per item, and one more where a worker's share ends inside an item
    const int64_t slots = (segs * kv_heads + kMaxWorkers) * group * L.own_rps;
    L.po = take(slots * dim * 4);
    L.pml = take(slots * 8);
    if (k == 0) {
        // single row tiles over 2 workers a CTA, or pairs of them over one: pairs take the most room
        const int64_t xslots = px == 1 ? (kv_heads + kMaxWorkers) * group * (rows < most ? rows : most)
                                       : ((px + 1) / 2 * kv_heads + kMaxCtas) * 256;
        L.xo = take(xslots * dim * 4);
        L.xml = take(xslots * 8);
    }
    L.total = at;
    return L;
}

static bool sizes_ok(int64_t rows, int64_t num_requests, int64_t heads, int64_t kv_heads, int64_t dim) {
    return rows <= (1 << 24) && num_requests <= (1 << 24) && heads <= 65535 && dim >= 16 && dim <= 128 &&
           dim % 16 == 0 && heads / kv_heads <= 128;
}

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
    if (!sizes_ok(rows, num_requests, heads, cache->heads, cache->dim) || rows * heads > 0x7FFFFFFF)
        return DSA_ERR_UNSUPPORTED;
    if (!(scale > 0.0f) || !isfinite(scale)) return DSA_ERR_INVALID;
    if (rows == 0) return DSA_OK;
    // (a segment's tiles of all heads are counted in 31 bits)
    if (max_pages > (int64_t(1) << 24) || (max_pages / 2 + 1) * cache->heads > 0x7FFFFFFF) return DSA_ERR_UNSUPPORTED;
    if (!q || !out || !row_ends || !starts || !workspace) return DSA_ERR_INVALID;
    if (max_pages > 0 && num_requests > 0 && (!block_table || bt_stride < max_pages)) return DSA_ERR_INVALID;
    if (!aligned16(q) || !aligned16(out) || (reinterpret_cast<uintptr_t>(workspace) & 255)) return DSA_ERR_INVALID;
    if (((q_row_stride | q_head_stride | out_row_stride | out_head_stride) & 7) || q_row_stride < 0 ||
        q_head_stride < 0 || out_row_stride < 0 || out_head_stride < 0)
        return DSA_ERR_INVALID;
    if ((rows > 1 && out_row_stride == 0) || (heads > 1 && out_head_stride == 0)) return DSA_ERR_INVALID;   // one place
    return DSA_OK;
}

// TMA strides are positive; a dimension of extent 1 may come with any.
static bool fix_stride(int64_t& s, int64_t extent, int64_t instead) {
    if (s > 0) return true;
    s = instead;
    return extent <= 1;
}

struct AttCall {
    AttParams p;
    AttLayout L;
    CUtensorMap q, k, v;
    int ctas;
};

static CUtensorMapDataType map_type(int dtype) {
    return dtype == DSA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
}

static int query_map(CUtensorMap* map, const dsa_kv_cache* c, const void* q, int64_t row_stride, int64_t head_stride,
                     int64_t rows, int64_t heads, int64_t box_rows) {
    if (!fix_stride(head_stride, heads, c->dim) || !fix_stride(row_stride, rows, heads * c->dim))
        return DSA_ERR_UNSUPPORTED;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(c->dim), static_cast<cuuint64_t>(heads),
                                static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(head_stride) * 2, static_cast<cuuint64_t>(row_stride) * 2};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(heads / c->heads), static_cast<cuuint32_t>(box_rows)};
    return encode_tiled(map, map_type(c->dtype), 3, const_cast<void*>(q), dims, strides, box,
                        CU_TENSOR_MAP_SWIZZLE_128B) == CUDA_SUCCESS
               ? DSA_OK
               : DSA_ERR_CUDA;
}

// The cache the maps describe: a pool without pages (no key can be visible then)
// gets a page of the workspace that nothing loads.
static dsa_kv_cache mapped_cache(const dsa_kv_cache* cache, void* workspace) {
    dsa_kv_cache c = *cache;
    if (c.num_pages > 0) return c;
    c.k = c.v = workspace;
    c.k_head_stride = c.v_head_stride = c.dim;
    c.k_token_stride = c.v_token_stride = c.dim * c.heads;
    c.k_page_stride = c.v_page_stride = c.dim * c.heads * kPage;
    c.num_pages = 1;
    return c;
}

// How much a copy's miss in L2 brings in: at most the largest power of two that
// divides a token's columns, since what follows them may be another head's.
// (128 requests of 4096 keys, 8 heads token by token: 64 columns 258 us with 256
// bytes, 205 us with 128; 80 columns 215 us with 256, 160 us with 64.)
static CUtensorMapL2promotion promotion(const dsa_kv_cache* c) {
    return c->dim % 128 == 0  ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
           : c->dim % 64 == 0 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B
                              : CU_TENSOR_MAP_L2_PROMOTION_L2_64B;
}

// A pool as pages of 64 tokens.
static int page_map(CUtensorMap* map, const dsa_kv_cache* c, void* pool, int64_t ps, int64_t ts, int64_t hs) {
    if (!fix_stride(ps, c->num_pages, c->dim) || !fix_stride(ts, kPage, c->dim) || !fix_stride(hs, c->heads, c->dim))
        return DSA_ERR_UNSUPPORTED;
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(c->dim), kPage, static_cast<cuuint64_t>(c->heads),
                                static_cast<cuuint64_t>(c->num_pages)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(ts) * 2, static_cast<cuuint64_t>(hs) * 2,
                                   static_cast<cuuint64_t>(ps) * 2};
    const cuuint32_t box[4] = {64, kPage, 1, 1};
    return encode_tiled(map, map_type(c->dtype), 4, pool, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B,
                        promotion(c)) == CUDA_SUCCESS
               ? DSA_OK
               : DSA_ERR_CUDA;
}

static int64_t gcd64(int64_t a, int64_t b) {
    while (b) {
        const int64_t t = a % b;
        a = b;
        b = t;
    }
    return a;
}

// A pool as rows of dim columns that start every `unit` elements, the unit a
// common divisor of its strides, so that every (page, token, head) is one row.
static int row_map(CUtensorMap* map, const dsa_kv_cache* c, void* pool, int64_t ps, int64_t ts, int64_t hs, int* pu,
                   int* tu, int* hu, int* none) {
    if (!fix_stride(ps, c->num_pages, 0) || !fix_stride(ts, kPage, 0) || !fix_stride(hs, c->heads, 0))
        return DSA_ERR_UNSUPPORTED;
    int64_t unit = gcd64(gcd64(ps, ts), hs);
    if (unit == 0) unit = c->dim;
    const int64_t n = ((c->num_pages - 1) * ps + (kPage - 1) * ts + (c->heads - 1) * hs) / unit + 1;
    if (n > 0x7FFFFF00) return DSA_ERR_UNSUPPORTED;
    *pu = static_cast<int>(ps / unit), *tu = static_cast<int>(ts / unit), *hu = static_cast<int>(hs / unit);
    *none = static_cast<int>(n);
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(c->dim), static_cast<cuuint64_t>(n)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(unit) * 2};
    const cuuint32_t box[2] = {64, 1};
    return encode_tiled(map, map_type(c->dtype), 2, pool, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B,
                        promotion(c)) == CUDA_SUCCESS
               ? DSA_OK
               : DSA_ERR_CUDA;
}

constexpr int kSmemMost = 232448;   // 227 KB

// Q buffers for tiles of p.rows_cap rows, ring stages in what they leave; returns the shared memory taken.
static int fit_shared(int halves, bool paired, bool narrow, AttParams& p) {
    p.q_half = narrow ? 128 * 128 : (p.rows_cap * 128 + 1023) / 1024 * 1024;
    const int stage = halves * kTile * 128;
    const int fixed = 2 * halves * p.q_half + (narrow ? 2 * kMergeBytes : 0) + kAttMeta +
                      (p.plan_in_cta && !paired ? static_cast<int>(sizeof(AxisShared)) : 0);
    int n = (kSmemMost - fixed) / stage;
    if (!paired) n /= 2;
    p.nst = n > kMaxStages ? kMaxStages : n;
    return fixed + (paired ? 1 : 2) * p.nst * stage;
}

template <typename T, bool kPaired, bool kSelected, bool kNarrow, int DH>
static int launch_attention(const AttCall& a, int smem, cudaStream_t stream) {
    auto* kernel = attend_kernel<T, kPaired, kSelected, kNarrow, DH>;
    static bool attr_set[64] = {false};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return DSA_ERR_CUDA;
    if (!attr_set[dev]) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMost) != cudaSuccess)
            return DSA_ERR_CUDA;
        attr_set[dev] = true;
    }
    return launch_pdl(kernel, dim3(a.ctas), dim3(att_threads<kSelected, kNarrow>()), smem, stream, a.q, a.k, a.v,
                      a.p) == cudaSuccess
               ? DSA_OK
               : DSA_ERR_CUDA;
}

template <bool kPaired, bool kSelected, bool kNarrow>
static int launch_attention(AttCall& a, int dtype, cudaStream_t stream) {
    const int smem = fit_shared(a.p.dim > 64 ? 2 : 1, kPaired, kNarrow, a.p);
    if (a.p.dim > 64)
        return dtype == DSA_BF16 ? launch_attention<Bf16, kPaired, kSelected, kNarrow, 2>(a, smem, stream)
                                 : launch_attention<Fp16, kPaired, kSelected, kNarrow, 2>(a, smem, stream);
    return dtype == DSA_BF16 ? launch_attention<Bf16, kPaired, kSelected, kNarrow, 1>(a, smem, stream)
                             : launch_attention<Fp16, kPaired, kSelected, kNarrow, 1>(a, smem, stream);
}

template <typename T>
static int launch_join(const AttParams& p, cudaStream_t stream) {
    const int64_t items = static_cast<int64_t>(p.rows) * p.heads;
    // Where the workers are many to an item of the axis, its many pieces are shared by the warps of a CTA.
    // Eight warps against one: 8 items of the axis 19 and 24 us, 16: 22 and 24, 48: equal, 64: 53 and 51.  A CTA per
    // row and head costs where they are many: 24 rows of 32 heads behind 2000 keys 22 and 24 us, 32 rows of 64 heads
    // 41 and 39, 64 rows 53 and 41.
    const int64_t axis_items = static_cast<int64_t>(p.prefix_mode == 1 ? p.px_segs : p.rows) * p.kv_heads;
    const cudaError_t e = axis_items * 6 <= p.workers && items <= 4 * p.workers
                              ? launch_pdl(attend_join_kernel<T, 8>, dim3(static_cast<unsigned>(items)), dim3(256), 0,
                                           stream, p)
                              : launch_pdl(attend_join_kernel<T, 1>, dim3(static_cast<unsigned>((items + 3) / 4)),
                                           dim3(128), 0, stream, p);
    return e == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

// Plan (where the CTAs do not make it), attention over the axis, join.
template <bool kSelected>
static int launch_axis(AttCall& a, int dtype, cudaStream_t stream) {
    AttParams& p = a.p;
    if (!p.plan_in_cta && launch_pdl(attend_plan_kernel<kSelected>, dim3(1), dim3(kPlanThreads), 0, stream, p) !=
                              cudaSuccess)
        return DSA_ERR_CUDA;
    const int rc = p.rows_cap <= kNarrowRows ? launch_attention<false, kSelected, true>(a, dtype, stream)
                                    : launch_attention<false, kSelected, false>(a, dtype, stream);
    if (rc != DSA_OK) return rc;
    return dtype == DSA_BF16 ? launch_join<Bf16>(p, stream) : launch_join<Fp16>(p, stream);
}

static void fill_params(AttCall& a, const dsa_kv_cache* c, uint8_t* ws) {
    AttParams& p = a.p;
    const AttLayout& L = a.L;
    p.info = reinterpret_cast<int64_t*>(ws + L.info);
    p.axis = Axis{reinterpret_cast<int64_t*>(ws + L.prefix), reinterpret_cast<int4*>(ws + L.seg),
                  reinterpret_cast<int*>(ws + L.minb)};
    p.worker = reinterpret_cast<int*>(ws + L.worker);
    p.row_info = reinterpret_cast<RowInfo*>(ws + L.row_info);
    p.count = reinterpret_cast<int*>(ws + L.count);
    p.list = reinterpret_cast<int*>(ws + L.list);
    p.po = reinterpret_cast<float*>(ws + L.po);
    p.pml = reinterpret_cast<float2*>(ws + L.pml);
    p.xo = reinterpret_cast<float*>(ws + L.xo);
    p.xml = reinterpret_cast<float2*>(ws + L.xml);
    p.max_segs = static_cast<int>(L.max_segs);
    p.own_rps = static_cast<int>(L.own_rps);
    p.kpad = static_cast<int>(L.kpad);
    p.group = p.heads / p.kv_heads;
    p.own_cap = p.group * p.own_rps;
    p.rps = p.own_rps, p.rows_cap = p.own_cap;
    // (a plan kernel instead: 16 requests of 500 to 1000 keys 22.5 -> 24.5 us, 128 requests 78 -> 84)
    p.plan_in_cta = p.max_segs <= kPlanSegs && p.R <= kPlanSegs && p.rows <= kPlanRows;
    const int sms = device_sm_count();
    a.ctas = sms < kMaxCtas ? sms : kMaxCtas;
    p.workers = 2 * a.ctas;
    p.vbase = static_cast<const uint16_t*>(c->v);
    p.vp = c->v_page_stride, p.vt = c->v_token_stride, p.vh = c->v_head_stride;
}

}  // namespace dsa

using namespace dsa;

extern "C" size_t dsa_attend_workspace_size(int64_t rows, int64_t num_requests, int64_t heads, int64_t kv_heads,
                                            int64_t dim, int64_t max_query_len, int64_t k) {
    if (rows < 0 || num_requests < 0 || heads < 1 || kv_heads < 1 || heads % kv_heads || max_query_len < 0 || k < 0 ||
        k > (1 << 24) || !sizes_ok(rows, num_requests, heads, kv_heads, dim))
        return 0;
    return attend_layout(rows, num_requests, heads, kv_heads, dim, max_query_len, k).total;
}

extern "C" int dsa_attend_paged(const dsa_kv_cache* cache, const void* q, int64_t q_row_stride, int64_t q_head_stride,
                                int64_t heads, const int32_t* block_table, int64_t bt_stride, int64_t max_pages,
                                const int32_t* starts, const int32_t* row_ends, int64_t num_requests, int64_t rows,
                                int64_t max_query_len, const int32_t* prefix_pages, int64_t prefix_len, float scale,
                                void* out, int64_t out_row_stride, int64_t out_head_stride, float* lse,
                                void* workspace, size_t workspace_bytes, int32_t* status, void* stream_) {
    int rc = check_attend(cache, q, q_row_stride, q_head_stride, heads, block_table, bt_stride, max_pages, starts,
                          row_ends, num_requests, rows, scale, out, out_row_stride, out_head_stride, workspace);
    if (rc != DSA_OK) return rc;
    if (max_query_len < 0 || prefix_len < 0 || (prefix_len > 0 && (!prefix_pages || cache->num_pages == 0)))
        return DSA_ERR_INVALID;
    if (prefix_len > (int64_t(1) << 30) || (prefix_len / kTile + 1) * cache->heads > 0x7FFFFFFF)
        return DSA_ERR_UNSUPPORTED;
    if (rows == 0) return DSA_OK;
    AttCall a = {};
    a.L = attend_layout(rows, num_requests, heads, cache->heads, cache->dim, max_query_len, 0);
    if (workspace_bytes < a.L.total) return DSA_ERR_INVALID;
    AttParams& p = a.p;
    p.bt = block_table, p.bt_stride = bt_stride, p.starts = starts, p.row_ends = row_ends;
    p.prefix_pages = prefix_pages;
    p.out = static_cast<uint16_t*>(out), p.orow = out_row_stride, p.ohead = out_head_stride;
    p.lse = lse, p.status = status;
    p.R = static_cast<int>(num_requests), p.rows = static_cast<int>(rows), p.heads = static_cast<int>(heads);
    p.kv_heads = static_cast<int>(cache->heads), p.dim = static_cast<int>(cache->dim);
    p.max_keys = cache->num_pages > 0 ? static_cast<int>(max_pages * kPage) : 0;
    p.num_pages = static_cast<int>(cache->num_pages);
    p.prefix_len = static_cast<int>(prefix_len);
    p.scale_log2 = scale * kLog2e;
    fill_params(a, cache, static_cast<uint8_t*>(workspace));
    if (prefix_len > 0) {
        const int most = 128 / p.group;
        p.x_rps = p.rows < most ? p.rows : most;
        p.x_cap = p.group * p.x_rps;
        const int tiles = (p.rows + p.x_rps - 1) / p.x_rps;
        p.x_pairs = (tiles + 1) / 2;
        p.x_workers = a.ctas;
        // Row tiles in pairs read the prefix half as often; single ones share the axis (and the launch).
        // Pairs against the axis, 64 heads over 8, 128 rows, by the pairs' tiles a CTA: 4: 59 and 49 us, 8:
        // 67 and 61, 16: 82 and 83, 32: 116 and 129, 64: 178 and 227 (32, 64 and 256 rows, and 64
        // columns, cross between 8 and 16 too).
        p.prefix_mode = tiles > 1 && static_cast<int64_t>(p.x_pairs) * p.kv_heads * ((prefix_len + kTile - 1) / kTile) >
                                         kPairTiles * a.ctas
                            ? 2
                            : 1;
        if (p.prefix_mode == 1) {
            p.px_segs = tiles;
            p.rps = p.x_rps > p.own_rps ? p.x_rps : p.own_rps;
            p.rows_cap = p.group * p.rps;
        }
    }
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    const dsa_kv_cache c = mapped_cache(cache, workspace);
    rc = page_map(&a.k, &c, c.k, c.k_page_stride, c.k_token_stride, c.k_head_stride);
    if (rc == DSA_OK) rc = page_map(&a.v, &c, c.v, c.v_page_stride, c.v_token_stride, c.v_head_stride);
    if (rc != DSA_OK) return rc;
    if (p.prefix_mode == 2) {
        AttCall x = a;
        x.p.rows_cap = p.x_cap;
        rc = query_map(&x.q, cache, q, q_row_stride, q_head_stride, rows, heads, p.x_rps);
        if (rc == DSA_OK) rc = launch_attention<true, false, false>(x, cache->dtype, stream);
        if (rc != DSA_OK) return rc;
    }
    rc = query_map(&a.q, cache, q, q_row_stride, q_head_stride, rows, heads, p.rps);
    return rc == DSA_OK ? launch_axis<false>(a, cache->dtype, stream) : rc;
}

extern "C" int dsa_attend_selected(const dsa_kv_cache* cache, const void* q, int64_t q_row_stride,
                                   int64_t q_head_stride, int64_t heads, const int32_t* block_table, int64_t bt_stride,
                                   int64_t max_pages, const int32_t* starts, const int32_t* row_ends,
                                   int64_t num_requests, int64_t rows, const int32_t* topk, int64_t topk_stride,
                                   int64_t k, float scale, void* out, int64_t out_row_stride, int64_t out_head_stride,
                                   float* lse, void* workspace, size_t workspace_bytes, int32_t* status,
                                   void* stream_) {
    int rc = check_attend(cache, q, q_row_stride, q_head_stride, heads, block_table, bt_stride, max_pages, starts,
                          row_ends, num_requests, rows, scale, out, out_row_stride, out_head_stride, workspace);
    if (rc != DSA_OK) return rc;
    if (k < 0 || (k > 0 && rows > 0 && (!topk || topk_stride < k))) return DSA_ERR_INVALID;
    if (k > (int64_t(1) << 24) || (k / kTile + 1) * cache->heads > 0x7FFFFFFF || cache->num_pages > (1 << 25))
        return DSA_ERR_UNSUPPORTED;
    if (rows == 0) return DSA_OK;
    AttCall a = {};
    // (an empty list is one key long in the workspace: the rows still need their zeros)
    a.L = attend_layout(rows, num_requests, heads, cache->heads, cache->dim, 1, k > 0 ? k : 1);
    if (workspace_bytes < a.L.total) return DSA_ERR_INVALID;
    AttParams& p = a.p;
    p.bt = block_table, p.bt_stride = bt_stride, p.starts = starts, p.row_ends = row_ends;
    p.topk = topk, p.topk_stride = topk_stride, p.k = static_cast<int>(k);
    p.out = static_cast<uint16_t*>(out), p.orow = out_row_stride, p.ohead = out_head_stride;
    p.lse = lse, p.status = status;
    p.R = static_cast<int>(num_requests), p.rows = static_cast<int>(rows), p.heads = static_cast<int>(heads);
    p.kv_heads = static_cast<int>(cache->heads), p.dim = static_cast<int>(cache->dim);
    p.max_keys = cache->num_pages > 0 ? static_cast<int>(max_pages * kPage) : 0;
    p.num_pages = static_cast<int>(cache->num_pages);
    p.scale_log2 = scale * kLog2e;
    fill_params(a, cache, static_cast<uint8_t*>(workspace));
    rc = query_map(&a.q, cache, q, q_row_stride, q_head_stride, rows, heads, 1);
    const dsa_kv_cache c = mapped_cache(cache, workspace);
    if (rc == DSA_OK)
        rc = row_map(&a.k, &c, c.k, c.k_page_stride, c.k_token_stride, c.k_head_stride, &p.kpu, &p.ktu, &p.khu,
                     &p.k_none);
    if (rc == DSA_OK)
        rc = row_map(&a.v, &c, c.v, c.v_page_stride, c.v_token_stride, c.v_head_stride, &p.vpu, &p.vtu, &p.vhu,
                     &p.v_none);
    if (rc != DSA_OK) return rc;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    if (launch_pdl(attend_list_kernel, dim3(static_cast<unsigned>(rows)), dim3(kListThreads), 0, stream, p) !=
        cudaSuccess)
        return DSA_ERR_CUDA;
    return launch_axis<true>(a, cache->dtype, stream);
}
