// dsa_attend_paged_fp4 and dsa_attend_selected_fp4: decode attention over the
// 4-bit key/value cache.
//
//   o = sum_t softmax_t(c q . k_t) v_t, one pass: p = 2^(c (s - m)), l += sum p,
//   O += p v with the running maximum m; pieces of a row's keys taken by different
//   warps are joined by their (m, l, O).
//
// Every warp streams its own sections (64 keys and values of one head) through its
// own ring in shared memory and multiplies what it streams: no warp waits for
// another.  A page's section is one bulk copy; listed keys are gathered row by row.
// The units (64 keys of one item: a key head of a request under 8, 16 or 32 query
// rows) lie on one axis, of which every warp takes an equal share; an item that several
// warps share is joined by a last, small kernel.
//
// The products are mma.sync m16n8k16 on FP16, so that codes become operands in
// registers, without a way through memory.  Neither product cares in what order the
// summed index is taken, which leaves the layouts free: a thread's bytes of a key are
// those of its own operand rows.  Codes times scales are exact in FP16 (6 bits).
//
// What bounds it: a unit of 128 columns is 9216 bytes, 392 cycles of an SM's share of
// the memory.  Converting its codes and multiplying them by their scales takes 252
// cycles whatever the rows (256 conversions and 256 products a warp wide, two of either
// a cycle on one SM); the matrix products of 8 rows hide behind that, 16 rows bring a
// unit to 435 cycles, 32 to 670.  Measured: 413, 653 and 712 cycles.  So up to 8 rows
// the memory bounds (64 requests of 4096 to 8192 keys, 32 heads over 8: 82 us, 82 % of
// the copy rate with 5 us until the first unit), under 32 the pipes, the matrix products
// alone with 512 cycles (128 requests of 1 to 4 rows, 64 heads over 8, 64 to 8192 keys: 243
// us, 11 of them the join).  Under 16 rows no pipe that was counted is active more than 31 % of
// the time, and what the 218 cycles past the count go into is not known (8 x 131071 keys,
// 16 heads over 1: 50 us).
//
// tcgen05 was tried for 9 to 32 rows and not kept: operands made by some warps and put
// into tensor memory, products issued by another, the softmax in four more.  It was right
// and slower as far as it got (8 x 131071 keys under 16 rows 95 us against 52, the 128
// requests 555 against 257): 1190 instructions an SMSP for 128 keys at 37 % issue, most
// stalls for instructions to be fetched.  That is no bound of the form; the codes'
// conversions are the same in both.
#pragma once

#include <cooperative_groups.h>
#include <math.h>

#include <atomic>

#include "elem16.cuh"
#include "fp4_cache.cuh"
#include "host.h"

namespace dsa {

constexpr int kUnit = kPage;            // keys of a unit
constexpr int kMaxCtas4 = 160;          // workspaces are sized for at most this many CTAs
constexpr int kMaxWarps4 = 12;          // ... of this many warps
// Up to this many requests (and 4096 rows) every CTA lays out the axis itself; past
// them a launch of its own does, and what the CTAs would read grows with the batch.
constexpr int kCtaRequests = 256;
constexpr int kPlan4Threads = 512;
constexpr int kOwnRows = 32;            // a request's rows are read by one thread up to here, by its warp past it
// Units a warp under which the axis counts units alone: a share is then a unit or a few,
// and a share without a unit wastes a warp, which costs more than an uneven start does.
constexpr int kFewUnits = 8;
constexpr int kList4Threads = 256;
constexpr int kBitmapKeys = 1 << 20;    // positions that a list is put in order by
// Listed sections' bytes from which lists are put in order first (a launch, 6 to 7 us).
// Lists of 2048 of 4096 to 8192 positions, 8 heads, in order and not: 18 MB 28.3 and
// 25.2 us, 36 MB 36.5 and 37.5, 72 MB 48.8 and 57, 144 MB 66 and 91, 576 MB 163 and 303.
// The rule does not know how dense a list is, and sparse ones gain less: 151 MB of lists of
// 2048 of 8192 positions 52 and 76, of 32768 69 and 84, of 131072 88 and 88; 75 MB of 8192
// 37 and 42, of 65536 50 and 49, of 131072 56 and 50.  Nor do lists of four rows a request
// that share its keys, 59 MB of 2000 of 8192 positions and 4 heads of 64: 38 and 31.
constexpr int64_t kPackBytes = 32 << 20;
constexpr float kLog2e4 = 1.4426950408889634f;
constexpr float kLn2_4 = 0.6931471805599453f;
// Weights are kept times 2^6: FP16 then holds them from 2^-30 of the largest on.
constexpr float kLift = 6.0f;
// ... and a row's reference is raised when a score passes it by 2^8, which leaves
// them below 2^14 (the score's limit is rounded down: where a step of FP32 is several
// powers of two, up would let a weight pass FP16); until then what there is needs no
// rescaling.
constexpr float kSlack4 = 8.0f;

// Where the join finds a row's pieces.
struct Row4 {
    int64_t first;          // where the row's request starts on the axis
    int pages, tiles;       // units an item, row tiles a head
    int place;              // the row's place in its request
    int weight, start;      // what a unit, and an item's start, take of the axis
    int pad;
};

struct Att4Layout {
    size_t info;            // int64[2]: the axis' length, whether it counts units alone
    size_t prefix, units, pages;   // the axis in global memory: int64[R + 1] twice, int[R]
    size_t list;            // int[rows][kpad]: slots of the listed keys
    size_t rows;            // Row4[rows]
    size_t po, pml;         // float[slots][cap][dim], float2[slots][cap]: partial results
    size_t total;
    int cap;                // query rows of a tile, and of a slot
    int tiles;              // row tiles of the longest request, as far as max_query_len tells
};

// The requests on the axis: where each starts, units before it, and pages an item of it has.
struct Axis4 {
    int64_t* prefix;
    int64_t* units;
    int* pages;
    int light, heavy, start;   // what units of up to 16 query rows, and of more, and an item's start take of the axis
};

struct Att4Params {
    const uint8_t* cache;
    int64_t page_stride, head_stride;
    const uint16_t* q;
    int64_t qrow, qhead;
    uint16_t* out;
    int64_t orow, ohead;
    float* lse;
    const int32_t* bt;
    int64_t bt_stride;
    const int32_t* starts;
    const int32_t* row_ends;
    const int32_t* topk;
    int64_t topk_stride;
    int64_t* info;
    Axis4 axis;
    int* list;
    Row4* row_info;
    float* po;
    float2* pml;
    int32_t* status;
    int R, rows, heads, group, kv_heads, dim, max_keys, num_pages;
    int k, list_units, list_tiles;   // listed keys: units an item, row tiles a head
    int packed;                      // ... and slots in `list`, in order, instead of positions in `topk`
    int cap, warps;                  // query rows of a tile; warps of the whole grid
    int bf16;                        // type of q and out (else FP16)
    int section, stage;              // bytes of a section, and of a ring stage
    int plan_in_cta;
    float c, v_scale;                // scale * k_scale * log2(e)
};

// q and out: the type is looked up, since it matters once an item only.
__device__ __forceinline__ float2 unpack2(const Att4Params& p, uint32_t w) {
    return p.bf16 ? Bf16::unpack(w) : Fp16::unpack(w);
}
__device__ __forceinline__ uint32_t pack2(const Att4Params& p, float lo, float hi) {
    return p.bf16 ? Bf16::pack(lo, hi) : Fp16::pack(lo, hi);
}

// ----------------------------------------------------------------- the axis
// Worker w of W has the units that start in [w T / W, (w + 1) T / W).
__device__ __forceinline__ int64_t share4(int64_t w, int64_t T, int64_t W) {
    if ((w + 1) * T < (int64_t(1) << 32)) return static_cast<uint32_t>(w * T) / static_cast<uint32_t>(W);
    return w * T / W;
}
__device__ __forceinline__ int worker_at(int64_t u, int64_t T, int64_t W) {
    if ((u + 1) * W < (int64_t(1) << 32) && T < (int64_t(1) << 32))
        return static_cast<int>((static_cast<uint32_t>(u + 1) * static_cast<uint32_t>(W) - 1) /
                                static_cast<uint32_t>(T));
    return static_cast<int>(((u + 1) * W - 1) / T);
}

__device__ __forceinline__ int64_t div64(int64_t a, int64_t b) {   // (a 64-bit division takes five times as long)
    return (a | b) < (int64_t(1) << 32) ? static_cast<uint32_t>(a) / static_cast<uint32_t>(b) : a / b;
}

// How many warps share an axis of length T on which units are at most `most` apart: every share has one.
__device__ __forceinline__ int64_t sharers(const Att4Params& p, int64_t T, int most) {
    return max(min(static_cast<int64_t>(p.warps), div64(T, most)), static_cast<int64_t>(T > 0));
}

// The last request that starts at or before v.
template <typename I>
__device__ __forceinline__ int last_at_most(const I* starts, int n, I v) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (starts[mid] <= v) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// (Row, head) pairs of a key head in request j, from row *row0 on.
__device__ __forceinline__ int pairs_of(const Att4Params& p, int j, int* row0) {
    *row0 = min(max(p.starts[j], 0), p.rows);
    return (min(max(p.starts[j + 1], *row0), p.rows) - *row0) * p.group;
}

// An item of n units takes start + n weight of the axis: its first unit is at its
// beginning, unit k behind that at start + k weight.
__device__ __forceinline__ int64_t item_length(int n, int weight, int start) {
    return n > 0 ? start + static_cast<int64_t>(n) * weight : 0;
}

// Units before the first that is at or behind place c of the axis.
__device__ __forceinline__ int64_t unit_at(const Att4Params& p, const Axis4& x, int64_t c) {
    if (c >= x.prefix[p.R]) return x.units[p.R];
    const int j = last_at_most(x.prefix, p.R, c);
    int row0;
    const int weight = pairs_of(p, j, &row0) <= 16 ? x.light : x.heavy, n = x.pages[j];
    const int64_t length = item_length(n, weight, x.start), in = c - x.prefix[j];
    const int64_t item = div64(in, length), rest = in - item * length;
    const int64_t k = rest == 0 ? 0 : rest <= x.start ? 1 : max(div64(rest - x.start + weight - 1, weight), int64_t(1));
    return x.units[j] + item * n + k;
}

// The axis of few units counts them alone: a share is a unit or a few then.
__device__ __forceinline__ void count_units(Axis4& x) {
    x.prefix = x.units;
    x.light = x.heavy = 1, x.start = 0;
}

// Lays out the requests (whole block).  `tmp`: 66 int64 of shared scratch.
// `write`: also what the join reads.
static __device__ void lay_out4(const Att4Params& p, Axis4& x, int64_t* tmp, bool write) {
    const int nt = blockDim.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    bool bad = false;
    // (on their way while the starts are read)
    for (int r = threadIdx.x * 32; r < p.rows; r += nt * 32)
        asm volatile("prefetch.global.L1 [%0];" ::"l"(p.row_ends + r));
    if (write)
        for (int r = threadIdx.x; r < p.rows; r += nt) p.row_info[r] = Row4{0, 0, 1, 0, 1, 0, 0};
    int64_t carry = 0, carry_units = 0;
    for (int base = 0; base < p.R; base += nt) {
        const int j = base + threadIdx.x;
        int s0 = 0, s1 = 0, most = 0;
        if (j < p.R) {
            const int a = p.starts[j], b = p.starts[j + 1];
            if (a < 0 || b < a || b > p.rows) bad = true;
            s0 = min(max(a, 0), p.rows);
            s1 = min(max(b, s0), p.rows);
        }
        auto bound = [&](int r) {
            const int given = p.row_ends[r], e = min(max(given, 0), p.max_keys);
            if (e != given) bad = true;
            return e;
        };
        if (s1 - s0 <= kOwnRows)
            for (int r = s0; r < s1; ++r) most = max(most, bound(r));
        for (uint32_t many = __ballot_sync(0xFFFFFFFFu, s1 - s0 > kOwnRows); many; many &= many - 1) {
            const int whose = __ffs(many) - 1, to = __shfl_sync(0xFFFFFFFFu, s1, whose);
            int all = 0;
#pragma unroll 4
            for (int r = __shfl_sync(0xFFFFFFFFu, s0, whose) + lane; r < to; r += 32) all = max(all, bound(r));
            all = __reduce_max_sync(0xFFFFFFFFu, all);
            if (lane == whose) most = all;
        }
        const int n = (most + kUnit - 1) / kUnit;
        const int64_t all = static_cast<int64_t>(s1 - s0) * p.group;
        const int tiles = static_cast<int>((all + p.cap - 1) / p.cap), weight = all <= 16 ? x.light : x.heavy;
        const int64_t items = static_cast<int64_t>(tiles) * p.kv_heads;
        const int64_t units = n * items, cost = item_length(n, weight, x.start) * items;
        int64_t v = cost, y = units;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t o = __shfl_up_sync(0xFFFFFFFFu, v, d), q = __shfl_up_sync(0xFFFFFFFFu, y, d);
            if (lane >= d) v += o, y += q;
        }
        if (lane == 31) tmp[warp] = v, tmp[33 + warp] = y;
        __syncthreads();
        if (warp < 2) {
            int64_t* const t = tmp + 33 * warp;
            int64_t z = lane < nt / 32 ? t[lane] : 0;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int64_t o = __shfl_up_sync(0xFFFFFFFFu, z, d);
                if (lane >= d) z += o;
            }
            t[lane] = z;
            if (lane == 31) t[32] = z;
        }
        __syncthreads();
        const int64_t before = carry + v - cost + (warp > 0 ? tmp[warp - 1] : 0);
        if (j < p.R) {
            x.prefix[j] = before;
            x.units[j] = carry_units + y - units + (warp > 0 ? tmp[33 + warp - 1] : 0);
            x.pages[j] = n;
        }
        carry += tmp[32];
        carry_units += tmp[65];
        __syncthreads();
    }
    if (threadIdx.x == 0) x.prefix[p.R] = carry, x.units[p.R] = carry_units;
    const bool few = carry_units < kFewUnits * static_cast<int64_t>(p.warps);
    __syncthreads();
    if (few) count_units(x);
    if (write) {
        if (threadIdx.x == 0) p.info[0] = x.prefix[p.R], p.info[1] = few;
        for (int base = 0; base < p.R; base += nt) {
            const int j = base + threadIdx.x;
            int row0 = 0, n = 0;
            Row4 info = {};
            if (j < p.R) {
                const int all = pairs_of(p, j, &row0);
                n = all / p.group;
                info = Row4{x.prefix[j], x.pages[j], max((all + p.cap - 1) / p.cap, 1), 0,
                            all <= 16 ? x.light : x.heavy, x.start, 0};
            }
            if (n <= kOwnRows)
                for (; info.place < n; ++info.place) p.row_info[row0 + info.place] = info;
            for (uint32_t many = __ballot_sync(0xFFFFFFFFu, n > kOwnRows); many; many &= many - 1) {
                const int whose = __ffs(many) - 1;
                Row4 its;
                its.first = __shfl_sync(0xFFFFFFFFu, info.first, whose);
                its.pages = __shfl_sync(0xFFFFFFFFu, info.pages, whose);
                its.tiles = __shfl_sync(0xFFFFFFFFu, info.tiles, whose);
                its.weight = __shfl_sync(0xFFFFFFFFu, info.weight, whose);
                its.start = __shfl_sync(0xFFFFFFFFu, info.start, whose);
                its.pad = 0;
                const int first = __shfl_sync(0xFFFFFFFFu, row0, whose), count = __shfl_sync(0xFFFFFFFFu, n, whose);
                for (its.place = lane; its.place < count; its.place += 32) p.row_info[first + its.place] = its;
            }
        }
    }
    if (write && bad && p.status) atomicOr(p.status, DSA_STATUS_BAD_GEOMETRY);
    __syncthreads();
}

template <bool kSelected>
__global__ void __launch_bounds__(kPlan4Threads) attend_fp4_plan_kernel(const Att4Params p) {
    pdl_wait();
    pdl_launch_dependents();
    __shared__ int64_t tmp[66];
    Axis4 axis = p.axis;
    lay_out4(p, axis, tmp, true);
}

// Listed keys as slots (page * 64 + token), in the order of their positions, so that
// neighbours in a page are read one behind the other: the memory opens a row for every
// key that stands alone, and 64-byte pieces in a random order get a third of its rate.
// One CTA a row, latency (6 to 7 us).  The order comes from a bitmap of the row's
// positions; where a position is listed twice (it counts twice), or where there are
// more positions than the bitmap holds, the slots stay in the list's order.
template <bool kSelected>
__global__ void __launch_bounds__(kList4Threads) attend_fp4_list_kernel(const Att4Params p) {
    pdl_wait();
    pdl_launch_dependents();
    extern __shared__ uint32_t bitmap[];
    __shared__ int sums[kList4Threads / 32 + 1];
    __shared__ int s_req, s_twice;
    const int row = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int32_t* src = p.topk + row * p.topk_stride;
    int* const dst = p.list + static_cast<int64_t>(row) * p.list_units * kUnit;
    // (the first entries are on their way while the row's request is looked up)
    constexpr int kFirst = 8;
    int first[kFirst];
#pragma unroll
    for (int i = 0; i < kFirst; ++i) {
        const int at = threadIdx.x + i * kList4Threads;
        first[i] = at < p.k ? src[at] : -1;
    }
    const int e = p.row_ends[row], bound = min(max(e, 0), p.max_keys);
    const bool ordered = p.max_keys <= kBitmapKeys;
    const int words = ordered ? (bound + 31) / 32 : 0;
    if (threadIdx.x == 0) s_req = -1, s_twice = 0;
    for (int i = threadIdx.x; i < words; i += kList4Threads) bitmap[i] = 0;
    __syncthreads();
    bool bad = false, bad_page = false;
    for (int j = threadIdx.x; j < p.R; j += kList4Threads) {
        const int a = p.starts[j], b = p.starts[j + 1];
        if (a < 0 || b < a || b > p.rows) bad = true;
        if (a <= row && row < b) atomicMax(&s_req, j);
    }
    bool past = false;
    auto mark = [&](int t) {
        past |= t >= bound;
        if (ordered && t >= 0 && t < bound && (atomicOr(&bitmap[t >> 5], 1u << (t & 31)) >> (t & 31) & 1)) s_twice = 1;
    };
#pragma unroll
    for (int i = 0; i < kFirst; ++i)
        if (first[i] >= 0) mark(first[i]);
    for (int i = threadIdx.x + kFirst * kList4Threads; i < p.k; i += kList4Threads) mark(src[i]);
    __syncthreads();
    const int req = s_req;
    const int32_t* const table = p.bt + (req >= 0 ? req : 0) * p.bt_stride;
    auto slot_of = [&](int t) {
        const int page = table[t / kPage];
        const bool ok = page >= 0 && page < p.num_pages;
        bad_page |= !ok;
        return ok ? page * kPage + t % kPage : -1;
    };
    int count = 0;
    if (req >= 0) {
        if (e != bound || past) bad = true;
        const bool by_map = ordered && !s_twice;
        // positions: a run of the bitmap's words a thread; entries: one a thread and round
        const int each = (words + kList4Threads - 1) / kList4Threads;
        const int from = min(threadIdx.x * each, words), to = min(from + each, words);
        const int rounds = by_map ? 1 : (p.k + kList4Threads - 1) / kList4Threads;
        for (int round = 0; round < rounds; ++round) {
            int n = 0, t = -1;
            if (by_map) {
                for (int i = from; i < to; ++i) n += __popc(bitmap[i]);
            } else if (round * kList4Threads + threadIdx.x < p.k) {
                t = src[round * kList4Threads + threadIdx.x];
                n = t >= 0 && t < bound;
            }
            int inc = n;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(0xFFFFFFFFu, inc, d);
                if (lane >= d) inc += o;
            }
            if (lane == 31) sums[warp] = inc;
            __syncthreads();
            int before = count + inc - n, all = count;
            for (int i = 0; i < kList4Threads / 32; ++i) {
                if (i < warp) before += sums[i];
                all += sums[i];
            }
            if (by_map) {
                for (int i = from; i < to; ++i)
                    for (uint32_t bits = bitmap[i]; bits; bits &= bits - 1)
                        dst[before++] = slot_of(i * 32 + __ffs(bits) - 1);
            } else if (n) {
                dst[before] = slot_of(t);
            }
            count = all;
            __syncthreads();
        }
    }
    for (int i = count + threadIdx.x; i < p.list_units * kUnit; i += kList4Threads) dst[i] = -1;
    if (bad && p.status) atomicOr(p.status, DSA_STATUS_BAD_GEOMETRY);
    if (bad_page && p.status) atomicOr(p.status, DSA_STATUS_BAD_PAGE);
}

// ----------------------------------------------------------------- attention
constexpr int kSmemMost4 = 227 * 1024;

// The forms of a head: 128 columns, 64 columns, others up to 128, others up to 64.
enum Form { kForm128 = 0, kForm64 = 1, kFormAny128 = 2, kFormAny64 = 3 };
constexpr bool wide(Form f) { return f == kForm128 || f == kFormAny128; }

// Tiles of 8, 16 or 32 query rows; warps of a CTA and stages of a warp's ring.  Warps
// are limited by registers (a row's sums of 128 columns), stages by shared memory: 12
// rings of 2 sections.  16 rows with 12 warps, for which the rings had to be cut in
// halves, took 61 us where 8 warps take 52; 3 stages for 64 columns 34 us for 31.
template <Form kForm, int kRows>
struct Shape4 {
    static constexpr int kWarps = kRows == 8 ? 12 : kRows == 16 ? (wide(kForm) ? 8 : 12) : 8;
    static constexpr int kStages = 2;
};

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ float ex2_4(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
template <typename V>
__device__ __forceinline__ V lds(const uint8_t* a) {
    return *reinterpret_cast<const V*>(a);
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src, uint32_t src_bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
__device__ __forceinline__ void cp_async16s(uint32_t dst, const void* src, uint32_t src_bytes) {
    asm volatile("cp.async.cg.shared.global.L2::64B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
// NaN among four E4M3 bytes (not zero if so).
__device__ __forceinline__ uint32_t nan4(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

// A unit of a worker's share, as a lane works it out.
struct Unit4 {
    int page;           // its page, -1: none in the pool (listed keys: the row's request, -1: none)
    int kvh;            // key head
    int at, row;        // listed keys: its place in its item, the row (pages: row tiles that read it),
    int bound;          // ... and the positions from which on keys are not the row's
};

// An item: query rows (row0 + (first + n) / group, head kvh * group + (first + n) % group), n < nq.
struct Item4 {
    int row0, first, nq, kvh;
    int at, n;          // the unit asked for, and the item's units
};

// What a warp keeps in shared memory besides its ring.
template <int kSteps, int kRows>
struct QueryDesk {
    uint4 q[kSteps][kRows / 16][32];      // query operands: step, tile of 16 rows, lane
};
template <int kSteps>
struct QueryDesk<kSteps, 8> {};           // (those of 8 rows are in registers)

template <Form kForm, int kRows, bool kSelected>
struct Desk4 : QueryDesk<wide(kForm) ? 8 : 4, kRows> {
    uint64_t full[Shape4<kForm, kRows>::kStages];        // pages: copies that landed
    uint64_t listed[Shape4<kForm, kRows>::kStages];      // which of a unit's keys there are
    int64_t rows[kSelected ? kUnit : 1];                 // where listed tokens' codes are
    int ends[8];                                         // tiles of 8 rows: their bounds
    int abort;
};

// What the tiles of 8 rows and those of more share: the layout of a section, and
// codes as operands.
template <Form kForm, int kRows, bool kSelected>
struct Base4 {
    using Desk = Desk4<kForm, kRows, kSelected>;
    static constexpr int kBlocks = wide(kForm) ? 8 : 4;        // blocks of 16 columns in registers
    static constexpr int kSteps = kBlocks;                     // steps of the scores' product, a block's worth each

    const Att4Params& p;
    Desk& desk;
    int lane, g, t;
    Item4 item;
    int least, most;                  // the smallest and the largest bound of the item's rows

    __device__ __forceinline__ Base4(const Att4Params& params, Desk& d) : p(params), desk(d) {
        lane = threadIdx.x & 31;
        g = lane >> 2, t = lane & 3;
    }

    __device__ __forceinline__ int nblk() const { return kForm == kForm128 ? 8 : kForm == kForm64 ? 4 : p.dim / 16; }
    __device__ __forceinline__ int row_bytes() const { return 8 * nblk(); }
    __device__ __forceinline__ int scale_row() const { return wide(kForm) ? 8 : 4; }
    __device__ __forceinline__ int v_off() const { return kPage * row_bytes(); }
    __device__ __forceinline__ int s_off() const { return 2 * kPage * row_bytes(); }
    static constexpr bool kFull = kForm == kForm128 || kForm == kForm64;   // no block is missing

    // Which key of eight is operand row (or column) i: neighbours differ in parity, and so do those two apart
    // (rows of keys and of values then meet in fewer banks).
    static __device__ __forceinline__ int key_of(int i) { return i ^ ((i >> 1) & 1); }

    // The block of 16 columns that a thread has in step s of the scores' product (four columns of it).
    __device__ __forceinline__ int step_block(int s) const {
        return kForm == kForm128 ? 2 * t + (s >> 2) : t + (s & 4);
    }

    // A query row's columns for the thread's steps, times the power of two that puts the largest of the row next to
    // 2^14; *c: what the row's scores are multiplied by then (log2(e) scale, the power taken back).
    __device__ __forceinline__ void load_query(const uint16_t* src, bool on, float (&f)[kSteps][4], float* c) {
        uint32_t top = 0;
#pragma unroll
        for (int b = 0; b < kBlocks / 4; ++b) {   // the thread's blocks: steps 4b .. 4b + 3
            const int blk = step_block(4 * b);
            uint4 w[2] = {};
            if (on && blk < nblk()) {
                w[0] = __ldg(reinterpret_cast<const uint4*>(src + 16 * blk));
                w[1] = __ldg(reinterpret_cast<const uint4*>(src + 16 * blk + 8));
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 y = unpack2(p, (&w[i >> 2].x)[i & 3]);
                f[4 * b + i / 2][2 * (i & 1)] = y.x;
                f[4 * b + i / 2][2 * (i & 1) + 1] = y.y;
                top = max(top, max(__float_as_uint(y.x) & 0x7FFFFFFFu, __float_as_uint(y.y) & 0x7FFFFFFFu));
            }
        }
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
        // 2^(14 - power) for the exponent of the row's largest |q|
        const int power = max(static_cast<int>(top >> 23) - 127, -112);
        const float up = __int_as_float((127 + 14 - power) << 23);
        const float down = power >= 14 ? __int_as_float((127 + power - 14) << 23) : 1.0f / up;
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i) f[s][i] *= up;
        *c = fminf(fmaxf(p.c * down, 1e-37f), 3e38f);
    }

    // The rows of 64 listed tokens (two a lane: their place in page[h], that a position chose, -1 for none) into a
    // stage, asynchronously.
    __device__ __forceinline__ void gather(uint8_t* stage, int index, const int (&pos)[2], const int (&page)[2],
                                           int kvh) const {
        // rows of codes are cut into pieces of 16 bytes (8 where rows are not multiples of 16)
        constexpr int kPiece = kFull ? 16 : 8;
        constexpr int kLanes = kForm == kForm128 ? 4 : kForm == kForm64 ? 2 : wide(kForm) ? 8 : 4;   // of a row
        uint32_t there[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const bool on = page[h] >= 0 && page[h] < p.num_pages;
            if (pos[h] >= 0 && !on && p.status) atomicOr(p.status, DSA_STATUS_BAD_PAGE);
            // (tokens that are not there: any codes, and scales of zero)
            const int token = pos[h] % kPage, sr = 2 * scale_row();
            const int64_t section = on ? page[h] * p.page_stride + kvh * p.head_stride : 0;
            desk.rows[lane + 32 * h] = section + (on ? token * row_bytes() : 0);
            const uint8_t* src = p.cache + section + s_off() + (on ? token * sr : 0);
            const uint32_t to = smem_u32(stage + s_off() + (lane + 32 * h) * sr);
            if (p.num_pages > 0) {
                if (sr == 16) cp_async16s(to, src, on ? 16 : 0);
                else cp_async8(to, src, on ? 8 : 0);
            }
            there[h] = __ballot_sync(0xFFFFFFFFu, on);
        }
        if (lane == 0) desk.listed[index] = static_cast<uint64_t>(there[1]) << 32 | there[0];
        __syncwarp();
        const int part = lane % kLanes;
        if ((there[0] | there[1]) && part * kPiece < row_bytes()) {
#pragma unroll
            for (int c = 0; c < 2 * kLanes; ++c) {
                const int token = c * (32 / kLanes) + lane / kLanes;
                const uint8_t* src = p.cache + desk.rows[token] + part * kPiece;
                const uint32_t to = smem_u32(stage + token * row_bytes() + part * kPiece);
                if (kPiece == 16) {
                    cp_async16s(to, src, 16);
                    cp_async16s(to + v_off(), src + v_off(), 16);
                } else {
                    cp_async8(to, src, 8);
                    cp_async8(to + v_off(), src + v_off(), 8);
                }
            }
        }
        __syncwarp();   // (all have read the places before the next unit's are written over them)
    }

    // The (row, head) pair n of the item's tile.
    __device__ __forceinline__ void pair(int n, int* row, int* head) const {
        const int at = item.first + n;
        *row = item.row0 + at / p.group;
        *head = item.kvh * p.group + at % p.group;
    }

    // Code words (8 columns each) of a key for the thread's steps, and its scales, each twice.
    __device__ __forceinline__ void key_words(const uint8_t* stage, int key, uint32_t (&w)[kBlocks / 2],
                                              uint32_t (&sc)[kBlocks / 4]) const {
        const uint8_t* row = stage + key * row_bytes();
        const uint8_t* scales = stage + s_off() + key * 2 * scale_row();
        if constexpr (kForm == kForm128) {
            const uint4 x = lds<uint4>(row + 16 * t);
            w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
            const uint32_t two = e4m3x2_f16(lds<uint16_t>(scales + 2 * t));
            sc[0] = __byte_perm(two, 0, 0x1010);
            sc[1] = __byte_perm(two, 0, 0x3232);
        } else {
#pragma unroll
            for (int b = 0; b < kBlocks / 4; ++b) {
                const int blk = t + 4 * b;
                uint2 x = {0, 0};
                uint32_t one = 0;
                if (kFull || blk < nblk()) {
                    x = lds<uint2>(row + 8 * blk);
                    one = lds<uint8_t>(scales + blk);
                }
                w[2 * b] = x.x, w[2 * b + 1] = x.y;
                sc[b] = __byte_perm(e4m3x2_f16(one), 0, 0x1010);
            }
        }
    }

    // Values of keys 2t, 2t + 1, 2t + 8, 2t + 9 (as operands count them) of key tile i, in the thread's columns (2
    // kBlocks one behind the other from 2 kBlocks g): pairs of the first two keys and of the others, even columns and
    // odd ones.  `use(x, z, ...)` gets columns 8x + 2z and 8x + 2z + 1.
    template <typename Use>
    __device__ __forceinline__ void value_words(const uint8_t* stage, int i, Use use) const {
        const int blk = kBlocks == 8 ? g : g >> 1;
        uint2 v[4];
        uint32_t one[4];
#pragma unroll
        for (int z = 0; z < 4; ++z) {
            const int key = 16 * i + 8 * (z >> 1) + key_of(2 * t + (z & 1));
            const uint8_t* row = stage + v_off() + key * row_bytes() + g * kBlocks;
            const uint8_t* scales = stage + s_off() + (key * 2 + 1) * scale_row();
            v[z] = make_uint2(0, 0);
            one[z] = 0;
            if (kFull || blk < nblk()) {
                if constexpr (kBlocks == 8) v[z] = lds<uint2>(row);
                else v[z].x = lds<uint32_t>(row);
                one[z] = lds<uint8_t>(scales + blk);
            }
        }
        const uint32_t sa = e4m3x2_f16(one[0] | one[1] << 8), sb = e4m3x2_f16(one[2] | one[3] << 8);
#pragma unroll
        for (int x = 0; x < kBlocks / 4; ++x) {
            const uint32_t k0 = x ? v[0].y : v[0].x, k1 = x ? v[1].y : v[1].x;
            const uint32_t k2 = x ? v[2].y : v[2].x, k3 = x ? v[3].y : v[3].x;
            uint32_t a0[4], a1[4], a2[4], a3[4];
            e2m1x8((k0 & 0x0F0F0F0Fu) | (k1 << 4 & 0xF0F0F0F0u), a0);
            e2m1x8((k0 >> 4 & 0x0F0F0F0Fu) | (k1 & 0xF0F0F0F0u), a1);
            e2m1x8((k2 & 0x0F0F0F0Fu) | (k3 << 4 & 0xF0F0F0F0u), a2);
            e2m1x8((k2 >> 4 & 0x0F0F0F0Fu) | (k3 & 0xF0F0F0F0u), a3);
#pragma unroll
            for (int z = 0; z < 4; ++z)
                use(x, z, hmul2(a0[z], sa), hmul2(a1[z], sa), hmul2(a2[z], sb), hmul2(a3[z], sb));
        }
    }

    // Whether a value scale is NaN (two keys a lane); the padding of a scale row holds anything.
    __device__ __forceinline__ bool any_nan(const uint8_t* stage) const {
        uint32_t bad = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint8_t* at = stage + s_off() + ((lane + 32 * h) * 2 + 1) * scale_row();
            bad |= nan4(lds<uint32_t>(at) & scale_bytes(0));
            if (wide(kForm)) bad |= nan4(lds<uint32_t>(at + 4) & scale_bytes(4));
        }
        return __any_sync(0xFFFFFFFFu, bad != 0);
    }
    __device__ __forceinline__ uint32_t scale_bytes(int first) const {
        return kFull || nblk() >= first + 4 ? ~0u : nblk() <= first ? 0u : (1u << 8 * (nblk() - first)) - 1;
    }
    __device__ __forceinline__ bool nan_at(const uint8_t* stage, int key, int blk) const {
        return blk < nblk() && (lds<uint8_t>(stage + s_off() + (key * 2 + 1) * scale_row() + blk) & 0x7F) == 0x7F;
    }
    // Their bytes become zero (the columns they enter have become NaN for the rows that see the key, and for nobody
    // else).
    __device__ __forceinline__ void clear_nan(uint8_t* stage) const {
        __syncwarp();
#pragma unroll 1
        for (int i = lane; i < kUnit * nblk(); i += 32) {
            const int key = i / nblk(), blk = i - key * nblk();
            if (nan_at(stage, key, blk)) stage[s_off() + (key * 2 + 1) * scale_row() + blk] = 0;
        }
        __syncwarp();
        fence_proxy_async_smem();   // (the next copy into the stage is the asynchronous proxy's)
    }

    // kCols columns from col on of pair n's output, or of a piece's (po).
    template <int kCols>
    __device__ __forceinline__ void write(float* po, int n, int col, const float (&o)[kCols], float inv) const {
        if (po) {
            float* dst = po + n * p.dim + col;
#pragma unroll
            for (int i = 0; i < kCols; i += 4)
                *reinterpret_cast<float4*>(dst + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
        } else {
            int row, head;
            pair(n, &row, &head);
            uint16_t* dst = p.out + row * p.orow + head * p.ohead + col;
#pragma unroll
            for (int i = 0; i < kCols; i += 8)
                *reinterpret_cast<uint4*>(dst + i) =
                    make_uint4(pack2(p, o[i] * inv, o[i + 1] * inv), pack2(p, o[i + 2] * inv, o[i + 3] * inv),
                               pack2(p, o[i + 4] * inv, o[i + 5] * inv), pack2(p, o[i + 6] * inv, o[i + 7] * inv));
        }
    }
    // Pair n's reference (times c) and sum of weights.
    __device__ __forceinline__ void write_sum(float2* pml, int n, float top, float sum) const {
        if (pml) {
            pml[n] = make_float2(sum == 0.0f ? -INFINITY : top, sum);
        } else if (p.lse) {
            int row, head;
            pair(n, &row, &head);
            p.lse[static_cast<int64_t>(row) * p.heads + head] =
                sum == 0.0f ? -INFINITY : (top + log2f(sum) - kLift) * kLn2_4;
        }
    }
};

// Up to 8 query rows: keys (then value columns) are the 16 operand rows and query
// rows the 8 columns, so that few rows waste nothing.  The scores' accumulators
// become the values' second operand by a transposition in registers.  64 keys' scores
// are in registers at once: the loads and conversions of one tile hide the products of
// another.
template <Form kForm, bool kSelected>
struct Few4 : Base4<kForm, 8, kSelected> {
    using B = Base4<kForm, 8, kSelected>;
    using B::p, B::desk, B::lane, B::g, B::t, B::item, B::least, B::most, B::nblk, B::key_of;
    static constexpr int kBlocks = B::kBlocks, kSteps = B::kSteps;
    static constexpr int kMT = kUnit / 16;

    uint2 q[kSteps];                       // query operands
    float o[kBlocks][4];                   // columns' tiles: rows g and g + 8 are columns 2i and 2i + 1
    float ref[2], l[2], c[2], limit[2];    // query rows 2t, 2t + 1: reference, sum, factor, where the reference is raised

    __device__ __forceinline__ Few4(const Att4Params& params, typename B::Desk& d) : B(params, d) {}

    __device__ __forceinline__ void begin(const Item4& x) {
        item = x;
        const bool on = g < x.nq;
        int row, head;
        B::pair(on ? g : 0, &row, &head);
        float f[kSteps][4], cj;
        B::load_query(p.q + row * p.qrow + head * p.qhead, on, f, &cj);
#pragma unroll
        for (int s = 0; s < kSteps; ++s) q[s] = make_uint2(Fp16::pack(f[s][0], f[s][1]), Fp16::pack(f[s][2], f[s][3]));
        const int e = on ? min(max(p.row_ends[row], 0), p.max_keys) : 0x7FFFFFFF;
        if (t == 0) desk.ends[g] = e;
        least = __reduce_min_sync(0xFFFFFFFFu, e);
        most = __reduce_max_sync(0xFFFFFFFFu, on ? e : 0);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            c[i] = __shfl_sync(0xFFFFFFFFu, cj, (2 * t + i) * 4);
            ref[i] = l[i] = 0.0f;
            limit[i] = -INFINITY;
        }
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
        __syncwarp();
    }

    __device__ __forceinline__ bool sees(int e, int key, int key_base, uint64_t listed) const {
        return kSelected ? (listed >> key & 1) : key_base + key < desk.ends[2 * t + e];
    }

    __device__ __forceinline__ void unit(uint8_t* stage, int key_base, uint64_t listed) {
        if (B::any_nan(stage)) {
#pragma unroll 1
            for (int key = 0; key < kUnit; ++key)
                if (B::nan_at(stage, key, kBlocks == 8 ? g : g >> 1))
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        if (sees(e, key, key_base, listed))
#pragma unroll
                            for (int i = 0; i < kBlocks; ++i) o[i][e] = o[i][e + 2] = __int_as_float(0x7FC00000);
            B::clear_nan(stage);
        }
        float s[kMT][4];
#pragma unroll
        for (int i = 0; i < kMT; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.0f;
        uint32_t w[kMT][2][kBlocks / 2], sc[kMT][2][kBlocks / 4];   // keys g and g + 8 of a tile
#pragma unroll
        for (int i = 0; i < kMT; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) B::key_words(stage, 16 * i + 8 * h + key_of(g), w[i][h], sc[i][h]);
#pragma unroll
        for (int x = 0; x < kSteps / 2; ++x)   // a word: two steps
#pragma unroll
            for (int i = 0; i < kMT; ++i) {
                uint32_t a[4], b[4];
                e2m1x8(w[i][0][x], a);
                e2m1x8(w[i][1][x], b);
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    a[z] = hmul2(a[z], sc[i][0][x / 2]);
                    b[z] = hmul2(b[z], sc[i][1][x / 2]);
                }
#pragma unroll
                for (int z = 0; z < 2; ++z)
                    mma16816(s[i], a[2 * z], b[2 * z], a[2 * z + 1], b[2 * z + 1], q[2 * x + z].x, q[2 * x + z].y);
            }
        if (kSelected ? listed != ~0ull : key_base + kUnit > least) {
#pragma unroll
            for (int i = 0; i < kMT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (!sees(e & 1, 16 * i + 8 * (e >> 1) + key_of(g), key_base, listed)) s[i][e] = -INFINITY;
        }
        // The reference is raised when a score passes it by kSlack powers of two; until then O and l stay.
        float top[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            top[e] = fmaxf(s[0][e], s[0][e + 2]);
#pragma unroll
            for (int i = 1; i < kMT; ++i) top[e] = fmaxf(top[e], fmaxf(s[i][e], s[i][e + 2]));
        }
        if (__any_sync(0xFFFFFFFFu, top[0] > limit[0] || top[1] > limit[1])) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) top[e] = fmaxf(top[e], __shfl_xor_sync(0xFFFFFFFFu, top[e], d));
                if (top[e] > limit[e]) {
                    const float keep = limit[e] == -INFINITY ? 0.0f : ex2_4((ref[e] - top[e]) * c[e]);
                    ref[e] = top[e];
                    limit[e] = __fadd_rd(top[e], kSlack4 / c[e]);
                    l[e] *= keep;
#pragma unroll
                    for (int i = 0; i < kBlocks; ++i) o[i][e] *= keep, o[i][e + 2] *= keep;
                }
            }
        }
        uint32_t pb[kMT][2];
#pragma unroll
        for (int i = 0; i < kMT; ++i) {
            float y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                // (the difference first: a large score times c would leave its rounding in the exponent)
                y[e] = ex2_4(__fmaf_rn(s[i][e] - ref[e & 1], c[e & 1], kLift));
                l[e & 1] += y[e];
            }
            pb[i][0] = transpose8x8(Fp16::pack(y[0], y[1]));
            pb[i][1] = transpose8x8(Fp16::pack(y[2], y[3]));
        }
#pragma unroll
        for (int i = 0; i < kMT; ++i)
            B::value_words(stage, i, [&](int x, int z, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
                mma16816(o[4 * x + z], a0, a1, a2, a3, pb[i][0], pb[i][1]);
            });
    }

    // The item's result, or a piece's: sums [row][column] to po, references and sums of weights to pml.
    __device__ __forceinline__ void finish(float* po, float2* pml) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float sum = l[e];
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
            const int n = 2 * t + e;
            if (n >= item.nq) continue;
            float y[2 * kBlocks];
#pragma unroll
            for (int i = 0; i < kBlocks; ++i) y[2 * i] = o[i][e], y[2 * i + 1] = o[i][e + 2];
            if (B::kFull || (kBlocks == 8 ? g : g >> 1) < nblk())
                B::write(po, n, g * 2 * kBlocks, y, sum == 0.0f ? 0.0f : p.v_scale / sum);
            if (g == 0) B::write_sum(pml, n, ref[e] * c[e], sum);
        }
    }
};

// 16 or 32 query rows: they are the operand rows, keys (then value columns) the
// columns, and the scores' accumulators are the values' first operand as they are (with
// keys as the operand rows, as for 8 query rows, the 128 requests took 322 us instead of
// 283).  32 rows take 16 keys at a time, since their sums alone are 128 registers: with 64
// keys the same took 314.
template <Form kForm, int kRows, bool kSelected>
struct Many4 : Base4<kForm, kRows, kSelected> {
    using B = Base4<kForm, kRows, kSelected>;
    using B::p, B::desk, B::lane, B::g, B::t, B::item, B::least, B::most, B::nblk, B::key_of;
    static constexpr int kBlocks = B::kBlocks, kSteps = B::kSteps;
    static constexpr int kTiles = kRows / 16;
    static constexpr int kOT = 2 * kBlocks;                  // tiles of 8 value columns: column n * kOT + i is n of tile i
    static constexpr int kMT = kRows == 16 ? 4 : 1;          // tiles of 16 keys whose scores are in registers at once

    float o[kOT][kTiles][4];
    // query rows 16r + g and 16r + g + 8: reference, sum, factor, where the reference is raised, bound
    float ref[kTiles][2], l[kTiles][2], c[kTiles][2], limit[kTiles][2];
    int end[kTiles][2];

    __device__ __forceinline__ Many4(const Att4Params& params, typename B::Desk& d) : B(params, d) {}

    __device__ __forceinline__ void begin(const Item4& x) {
        item = x;
        least = 0x7FFFFFFF, most = 0;
#pragma unroll
        for (int r = 0; r < kTiles; ++r) {
            uint2 a[2][kSteps];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int n = 16 * r + 8 * h + g;
                const bool on = n < x.nq;
                int row, head;
                B::pair(on ? n : 0, &row, &head);
                float f[kSteps][4];
                B::load_query(p.q + row * p.qrow + head * p.qhead, on, f, &c[r][h]);
#pragma unroll
                for (int s = 0; s < kSteps; ++s)
                    a[h][s] = make_uint2(Fp16::pack(f[s][0], f[s][1]), Fp16::pack(f[s][2], f[s][3]));
                end[r][h] = on ? min(max(p.row_ends[row], 0), p.max_keys) : 0x7FFFFFFF;
                least = min(least, end[r][h]), most = max(most, on ? end[r][h] : 0);
                ref[r][h] = l[r][h] = 0.0f;
                limit[r][h] = -INFINITY;
            }
#pragma unroll
            for (int s = 0; s < kSteps; ++s) desk.q[s][r][lane] = make_uint4(a[0][s].x, a[1][s].x, a[0][s].y, a[1][s].y);
#pragma unroll
            for (int i = 0; i < kOT; ++i) o[i][r][0] = o[i][r][1] = o[i][r][2] = o[i][r][3] = 0.0f;
        }
        least = __reduce_min_sync(0xFFFFFFFFu, least), most = __reduce_max_sync(0xFFFFFFFFu, most);
        __syncwarp();
    }

    __device__ __forceinline__ bool sees(int r, int h, int key, int key_base, uint64_t listed) const {
        return kSelected ? (listed >> key & 1) : key_base + key < end[r][h];
    }

    // The unit's keys under the first R tiles of 16 rows.
    template <int R>
    __device__ __forceinline__ void unit(uint8_t* stage, int key_base, uint64_t listed) {
        if (B::any_nan(stage)) {
#pragma unroll 1
            for (int key = 0; key < kUnit; ++key)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    if (B::nan_at(stage, key, kBlocks == 8 ? 2 * t + e : t))
#pragma unroll
                        for (int r = 0; r < R; ++r)
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                if (sees(r, h, key, key_base, listed))
#pragma unroll
                                    for (int i = 0; i < kOT; ++i) o[i][r][2 * h + e] = __int_as_float(0x7FC00000);
            B::clear_nan(stage);
        }
        const bool all_see = kSelected ? listed == ~0ull : key_base + kUnit <= least;
#pragma unroll 1
        for (int first = 0; first < kUnit / 16; first += kMT) {   // tiles of 16 keys, two of 8 each
            float s[2 * kMT][R][4];
#pragma unroll
            for (int i = 0; i < 2 * kMT; ++i)
#pragma unroll
                for (int r = 0; r < R; ++r) s[i][r][0] = s[i][r][1] = s[i][r][2] = s[i][r][3] = 0.0f;
            uint32_t w[2 * kMT][kBlocks / 2], sc[2 * kMT][kBlocks / 4];
#pragma unroll
            for (int i = 0; i < 2 * kMT; ++i) B::key_words(stage, 16 * first + 8 * i + key_of(g), w[i], sc[i]);
#pragma unroll
            for (int x = 0; x < kSteps / 2; ++x) {   // a word: two steps
                uint4 q[2][R];
#pragma unroll
                for (int z = 0; z < 2; ++z)
#pragma unroll
                    for (int r = 0; r < R; ++r) q[z][r] = desk.q[2 * x + z][r][lane];
#pragma unroll
                for (int i = 0; i < 2 * kMT; ++i) {
                    uint32_t b[4];
                    e2m1x8(w[i][x], b);
#pragma unroll
                    for (int z = 0; z < 4; ++z) b[z] = hmul2(b[z], sc[i][x / 2]);
#pragma unroll
                    for (int z = 0; z < 2; ++z)
#pragma unroll
                        for (int r = 0; r < R; ++r)
                            mma16816(s[i][r], q[z][r].x, q[z][r].y, q[z][r].z, q[z][r].w, b[2 * z], b[2 * z + 1]);
                }
            }
            if (!all_see) {
#pragma unroll
                for (int i = 0; i < 2 * kMT; ++i)
#pragma unroll
                    for (int r = 0; r < R; ++r)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (!sees(r, e >> 1, 16 * first + 8 * i + key_of(2 * t + (e & 1)), key_base, listed))
                                s[i][r][e] = -INFINITY;
            }
            // The reference is raised when a score passes it by kSlack powers of two; until then O and l stay.
            float top[R][2];
            bool raised = false;
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    top[r][h] = fmaxf(s[0][r][2 * h], s[0][r][2 * h + 1]);
#pragma unroll
                    for (int i = 1; i < 2 * kMT; ++i)
                        top[r][h] = fmaxf(top[r][h], fmaxf(s[i][r][2 * h], s[i][r][2 * h + 1]));
                    raised |= top[r][h] > limit[r][h];
                }
            if (__any_sync(0xFFFFFFFFu, raised)) {
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        top[r][h] = fmaxf(top[r][h], __shfl_xor_sync(0xFFFFFFFFu, top[r][h], 1));
                        top[r][h] = fmaxf(top[r][h], __shfl_xor_sync(0xFFFFFFFFu, top[r][h], 2));
                        if (top[r][h] > limit[r][h]) {
                            const float keep =
                                limit[r][h] == -INFINITY ? 0.0f : ex2_4((ref[r][h] - top[r][h]) * c[r][h]);
                            ref[r][h] = top[r][h];
                            limit[r][h] = __fadd_rd(top[r][h], kSlack4 / c[r][h]);
                            l[r][h] *= keep;
#pragma unroll
                            for (int i = 0; i < kOT; ++i) o[i][r][2 * h] *= keep, o[i][r][2 * h + 1] *= keep;
                        }
                    }
            }
            uint32_t a[2 * kMT][R][2];
#pragma unroll
            for (int i = 0; i < 2 * kMT; ++i)
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float y[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            // (the difference first: a large score times c would leave its rounding in the exponent)
                            y[e] = ex2_4(__fmaf_rn(s[i][r][2 * h + e] - ref[r][h], c[r][h], kLift));
                            l[r][h] += y[e];
                        }
                        a[i][r][h] = Fp16::pack(y[0], y[1]);
                    }
#pragma unroll
            for (int i = 0; i < kMT; ++i)
                B::value_words(stage, first + i, [&](int x, int z, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        mma16816(o[8 * x + 2 * z][r], a[2 * i][r][0], a[2 * i][r][1], a[2 * i + 1][r][0],
                                 a[2 * i + 1][r][1], a0, a2);
                        mma16816(o[8 * x + 2 * z + 1][r], a[2 * i][r][0], a[2 * i][r][1], a[2 * i + 1][r][0],
                                 a[2 * i + 1][r][1], a1, a3);
                    }
                });
        }
    }
    __device__ __forceinline__ void unit(uint8_t* stage, int key_base, uint64_t listed) {
        if (kTiles == 2 && item.nq > 16) unit<kTiles>(stage, key_base, listed);
        else unit<1>(stage, key_base, listed);
    }

    __device__ __forceinline__ void finish(float* po, float2* pml) {
#pragma unroll
        for (int r = 0; r < kTiles; ++r)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float sum = l[r][h];
                sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
                sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
                const int n = 16 * r + 8 * h + g;
                if (n >= item.nq) continue;
                const float inv = sum == 0.0f ? 0.0f : p.v_scale / sum;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float y[kOT];
#pragma unroll
                    for (int i = 0; i < kOT; ++i) y[i] = o[i][r][2 * h + e];
                    if (B::kFull || (kBlocks == 8 ? 2 * t + e : t) < nblk()) B::write(po, n, (2 * t + e) * kOT, y, inv);
                }
                if (t == 0) B::write_sum(pml, n, ref[r][h] * c[r][h], sum);
            }
    }
};

template <Form kForm, int kRows, bool kSelected>
struct Worker4 : Many4<kForm, kRows, kSelected> {
    using Many4<kForm, kRows, kSelected>::Many4;
};
template <Form kForm, bool kSelected>
struct Worker4<kForm, 8, kSelected> : Few4<kForm, kSelected> {
    using Few4<kForm, kSelected>::Few4;
};

constexpr int kAxisBytes4 = (2 * (kCtaRequests + 1) + 66) * 8 + kCtaRequests * 4;

// A head's row tiles lie on the axis from both ends of the request in turn: where rows
// see ever more keys (a prompt's), units past the bounds of a tile's rows are not
// multiplied, and two neighbours together have as many as any others (4096 rows of 4096
// keys, 32 heads over 8: 732 us, 1051 with the tiles in order).
__device__ __forceinline__ int tile_at(int i, int tiles) { return i & 1 ? tiles - 1 - i / 2 : i / 2; }
__device__ __forceinline__ int place_of(int tile, int tiles) {
    return 2 * tile < tiles ? 2 * tile : 2 * (tiles - 1 - tile) + 1;
}

// Unit u: what a lane has to know of it, and its item.
__device__ __forceinline__ Unit4 paged_unit(const Att4Params& p, const Axis4& axis, int64_t u, Item4* y = nullptr) {
    Unit4 x;
    const int j = last_at_most(axis.units, p.R, u);
    const int64_t in = u - axis.units[j];
    const int n = axis.pages[j];
    const int item = in < (int64_t(1) << 32) ? static_cast<int>(static_cast<uint32_t>(in) / static_cast<uint32_t>(n))
                                             : static_cast<int>(in / n);
    x.at = static_cast<int>(in - static_cast<int64_t>(item) * n);
    int page = 0;
    if (!y) page = p.bt[j * p.bt_stride + x.at];
    int row0;
    const int all = pairs_of(p, j, &row0), tiles = (all + p.cap - 1) / p.cap;
    x.kvh = item / tiles;
    if (y) {
        const int first = tile_at(item - x.kvh * tiles, tiles) * p.cap;
        *y = Item4{row0, first, min(p.cap, all - first), x.kvh, x.at, n};
        return x;
    }
    x.page = page >= 0 && page < p.num_pages ? page : -1;
    if (x.page < 0 && p.status) atomicOr(p.status, DSA_STATUS_BAD_PAGE);
    x.row = tiles;
    x.bound = 0;
    return x;
}

__device__ __forceinline__ Unit4 listed_unit(const Att4Params& p, const int* starts, int64_t u, Item4* y = nullptr) {
    Unit4 x;
    const int per_row = p.kv_heads * p.list_tiles * p.list_units;
    x.row = static_cast<int>(u / per_row);
    const int in = static_cast<int>(u - static_cast<int64_t>(x.row) * per_row);
    const int item = in / p.list_units;
    x.at = in - item * p.list_units;
    x.kvh = item / p.list_tiles;
    if (y) {
        const int first = (item - x.kvh * p.list_tiles) * p.cap;
        *y = Item4{x.row, first, min(p.cap, p.group - first), x.kvh, x.at, p.list_units};
        return x;
    }
    x.page = x.bound = 0;
    if (p.packed) return x;
    const int e = p.row_ends[x.row];
    const int j = p.R > 0 ? last_at_most(starts, p.R, x.row) : -1;
    x.page = j >= 0 && starts[j] <= x.row && x.row < starts[j + 1] ? j : -1;
    x.bound = min(max(e, 0), p.max_keys);
    if (x.page >= 0 && e != x.bound && p.status) atomicOr(p.status, DSA_STATUS_BAD_GEOMETRY);
    return x;
}

// Shared memory: the warps' rings, their desks, then the axis.
template <Form kForm, int kRows, bool kSelected>
__global__ void __launch_bounds__((Shape4<kForm, kRows>::kWarps * 32), 1) attend_fp4_kernel(const Att4Params p) {
    using S4 = Shape4<kForm, kRows>;
    using W4 = Worker4<kForm, kRows, kSelected>;
    using Desk = Desk4<kForm, kRows, kSelected>;
    constexpr int kStages = S4::kStages;
    extern __shared__ __align__(128) uint8_t smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    pdl_launch_dependents();
    uint8_t* const ring = smem + warp * kStages * p.stage;
    Desk& desk = reinterpret_cast<Desk*>(smem + S4::kWarps * kStages * p.stage)[warp];
    W4 k(p, desk);
    if (lane == 0) {
        if (!kSelected) {
            for (int i = 0; i < kStages; ++i) mbar_init(&desk.full[i], 1);
            mbar_fence_init();
        }
        desk.abort = 0;
    }
    Axis4 axis = p.axis;
    const int* starts = p.starts;
    uint8_t* const table = smem + S4::kWarps * (kStages * p.stage + sizeof(Desk));
    if (!kSelected && p.plan_in_cta) {
        axis.prefix = reinterpret_cast<int64_t*>(table);
        axis.units = axis.prefix + kCtaRequests + 1;
        axis.pages = reinterpret_cast<int*>(axis.units + kCtaRequests + 1 + 66);
        lay_out4(p, axis, axis.units + kCtaRequests + 1, blockIdx.x == 0);
    } else if (!kSelected && p.info[1]) {
        count_units(axis);
    }
    if (kSelected && !p.packed) {
        bool bad = false;
        if (p.R <= kCtaRequests) starts = reinterpret_cast<int*>(table);
        if (p.R <= kCtaRequests || blockIdx.x == 0)
            for (int j = threadIdx.x; j <= p.R; j += blockDim.x) {
                const int a = p.starts[j];
                if (p.R <= kCtaRequests) reinterpret_cast<int*>(table)[j] = a;
                if (blockIdx.x == 0) bad |= a < 0 || (j > 0 && a < p.starts[j - 1]) || a > p.rows;
            }
        if (bad && p.status) atomicOr(p.status, DSA_STATUS_BAD_GEOMETRY);
        __syncthreads();
    }
    __syncwarp();
    const int64_t total = kSelected ? static_cast<int64_t>(p.rows) * p.kv_heads * p.list_tiles * p.list_units
                                    : axis.prefix[p.R];
    const int64_t W = sharers(p, total, kSelected ? 1 : axis.heavy + axis.start);
    const int w = warp * gridDim.x + blockIdx.x;   // (neighbouring shares on different SMs)
    if (w >= W) return;
    int64_t u0 = share4(w, total, W), u1 = share4(w + 1, total, W);
    if (!kSelected) u0 = unit_at(p, axis, u0), u1 = unit_at(p, axis, u1);
    const int count = static_cast<int>(u1 - u0);

    // The share's units are looked up 32 at a time, one a lane.
    Unit4 mine;
    auto look_up = [&](int base) {
        if (base + lane < count)
            mine = kSelected ? listed_unit(p, starts, u0 + base + lane) : paged_unit(p, axis, u0 + base + lane);
    };
    const uint64_t once = l2_evict_first_policy();
    // A page's copy, by the unit's lane.
    auto copy_page = [&](int i) {
        if (i >= count) return;
        if (i % 32 == 0) look_up(i);
        if (lane == i % 32) {
            uint64_t* const bar = &desk.full[i % kStages];
            desk.listed[i % kStages] = mine.page >= 0;
            if (mine.page >= 0) {
                mbar_arrive_expect_tx(bar, p.section);
                const uint8_t* src = p.cache + mine.page * p.page_stride + mine.kvh * p.head_stride;
                // (a page that one row tile reads is not needed again in this call)
                if (mine.row == 1) bulk_load_hint(ring + (i % kStages) * p.stage, src, p.section, bar, once);
                else bulk_load(ring + (i % kStages) * p.stage, src, p.section, bar);
            } else {
                mbar_arrive(bar);
            }
        }
    };

    // Listed keys, two tokens a lane: while a unit is in work, the pages of the unit kStages on are looked up and the
    // positions of the one behind it loaded.
    int pos[2], page[2], ahead[2];
    struct List {
        int req, kvh, bound;
    } next, later;                       // the units of pos / page, and of ahead
    auto load_positions = [&](int i) {   // into ahead / later
#pragma unroll
        for (int h = 0; h < 2; ++h) ahead[h] = -1;
        if (i >= count) return;
        if (i % 32 == 0) look_up(i);
        const int at = __shfl_sync(0xFFFFFFFFu, mine.at, i % 32), row = __shfl_sync(0xFFFFFFFFu, mine.row, i % 32);
        later.req = __shfl_sync(0xFFFFFFFFu, mine.page, i % 32);
        later.kvh = __shfl_sync(0xFFFFFFFFu, mine.kvh, i % 32);
        later.bound = __shfl_sync(0xFFFFFFFFu, mine.bound, i % 32);
        if (later.req < 0) return;
        const int32_t* list =
            p.packed ? p.list + static_cast<int64_t>(row) * p.list_units * kUnit : p.topk + row * p.topk_stride;
        const int most = p.packed ? p.list_units * kUnit : p.k;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int e = at * kUnit + lane + 32 * h;
            if (e < most) ahead[h] = list[e];
        }
    };
    auto load_pages = [&]() {            // ahead / later become pos, page / next
        next = later;
        bool bad = false;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            pos[h] = ahead[h];
            page[h] = -1;
            if (p.packed) {   // a slot
                if (pos[h] >= 0) page[h] = pos[h] / kPage;
                continue;
            }
            if (pos[h] >= next.bound) {
                bad |= pos[h] >= 0;
                pos[h] = -1;
            }
            if (pos[h] >= 0) page[h] = p.bt[next.req * p.bt_stride + pos[h] / kPage];
        }
        if (bad && p.status) atomicOr(p.status, DSA_STATUS_BAD_GEOMETRY);
    };
    auto gather = [&](int i) {           // the unit of pos / page into its stage
        if (i < count) k.gather(ring + (i % kStages) * p.stage, i % kStages, pos, page, next.kvh);
        cp_async_commit();
    };

    if constexpr (kSelected) {
        for (int i = 0; i < kStages; ++i) {
            load_positions(i);
            load_pages();
            gather(i);
        }
        load_positions(kStages);
    } else {
        for (int i = 0; i < kStages; ++i) copy_page(i);
    }
    int i = 0;
    bool gave_up = false;
    Item4 x, behind;
    auto item_of = [&](int at, Item4* y) {
        if (kSelected) listed_unit(p, starts, u0 + at, y);
        else paged_unit(p, axis, u0 + at, y);
    };
    if (count > 0) item_of(0, &behind);
    while (i < count && !gave_up) {
        // The part of an item that is in the share: units at .. until - 1 of its n.
        x = behind;
        k.begin(x);
        const int until = min(x.n, x.at + count - i);
        // The next item's queries are on their way to L2 meanwhile.
        if (i + until - x.at < count) {
            item_of(i + until - x.at, &behind);
            if (lane < behind.nq) {
                const int n = behind.first + lane;
                const uint16_t* src =
                    p.q + (behind.row0 + n / p.group) * p.qrow + (behind.kvh * p.group + n % p.group) * p.qhead;
                for (int c = 0; c < p.dim; c += 64) asm volatile("prefetch.global.L2 [%0];" ::"l"(src + c));
            }
        }
        for (int at = x.at; at < until; ++at, ++i) {
            uint8_t* const stage = ring + (i % kStages) * p.stage;
            if constexpr (kSelected) {
                load_pages();                     // of unit i + kStages
                load_positions(i + kStages + 1);
                cp_async_wait<kStages - 1>();
                __syncwarp();
            } else {
                const bool landed = mbar_wait(&desk.full[i % kStages], (i / kStages) & 1, &desk.abort, p.status);
                if (!__all_sync(0xFFFFFFFFu, landed)) {
                    gave_up = true;
                    break;
                }
            }
            const uint64_t listed = desk.listed[i % kStages];
            if (listed != 0 && (kSelected || at * kUnit < k.most)) k.unit(stage, at * kUnit, listed);
            __syncwarp();
            if constexpr (kSelected) gather(i + kStages);
            else copy_page(i + kStages);
            __syncwarp();
        }
        // slot 2w + 1: the item's first piece; 2w: a later one (a share has at most one of each)
        const int64_t slot = 2 * static_cast<int64_t>(w) + (x.at == 0 ? 1 : 0);
        const bool whole = x.at == 0 && until == x.n;
        if (!gave_up) k.finish(whole ? nullptr : p.po + slot * p.cap * p.dim, whole ? nullptr : p.pml + slot * p.cap);
    }
    if constexpr (kSelected) {
        cp_async_wait<0>();
    } else if (gave_up) {   // the copies in flight land before the CTA ends
        const unsigned long long deadline = globaltimer() + kWaitLimitNs;
        for (int j = i; j < min(i + kStages, count); ++j)
            mbar_drain(&desk.full[j % kStages], (j / kStages) & 1, deadline, p.status);
    }
}

// Few items with few units: eight CTAs, a cluster, have an item (four, two or one where
// the items are too many for more), and its units go round their warps.  What the warps
// have is joined through the cluster's shared memory, so one launch does it all, and the
// first page is on its way before the item's length is known.  Bound by latency (as
// graphs, and by the axis and a join; 32 heads over 8): one request of 1000 keys 7.0 and
// 10.9 us, of 6000 8.7 and 12.6, 9 of 1000 7.8 and 12.5, 19 of 3000 16.8 and 23.5, lists of
// 2048 for one row 7.5 and 10.5, for 19 rows 16.8 and 24.4.  Taken where all clusters run
// at once, as far as the GPU has room for them (15 of eight CTAs; a second turn took 14.4
// us for 8.5 with four), and a warp has at most kClusterUnits units: there the two meet (10
// requests of 6000 keys 24.8 and 24.6, 4 of 12000 16.9 and 20.1), past it the axis shares them better.
// Lengths are on the device, so the units are those of the block table's width (or of the
// list): under a table of 2048 pages one request of 1000 keys takes the axis, 10.9 us for 6.9.
constexpr int kCluster = 8;        // CTAs of a cluster at most
constexpr int kClusterUnits = 4;   // units of a warp at most
// A request's row tiles take turns in its cluster, 11 to 25 us each, while the axis spreads
// them: the longest request that max_query_len allows has this many at most (30 requests of
// 1000 keys, 16 heads over 1, a row each 11.2 us and by the axis 17.5, one of them with two
// tiles 26.2 and 19.0, with three 38.6 and 19.0; 63 of 4096 keys with a row each beside one of
// 67 rows 990 and 50).
constexpr int kClusterTiles = 2;

template <Form kForm, int kRows, bool kSelected>
__global__ void __launch_bounds__((Shape4<kForm, kRows>::kWarps * 32), 1)
attend_fp4_cluster_kernel(const Att4Params p) {
    using S4 = Shape4<kForm, kRows>;
    using W4 = Worker4<kForm, kRows, kSelected>;
    using Desk = Desk4<kForm, kRows, kSelected>;
    constexpr int kStages = S4::kStages, kWarps = S4::kWarps;
    namespace cg = cooperative_groups;
    const cg::cluster_group cluster = cg::this_cluster();
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float2 ml[kWarps][kRows], joined[kRows];   // references and sums of the warps, of the CTA
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rank = cluster.block_rank(), ctas = cluster.num_blocks(), item = blockIdx.x / ctas;
    const int sharers = kWarps * ctas;
    pdl_wait();
    pdl_launch_dependents();
    uint8_t* const ring = smem + warp * kStages * p.stage;
    Desk& desk = reinterpret_cast<Desk*>(smem + kWarps * kStages * p.stage)[warp];
    W4 k(p, desk);
    if (lane == 0) {
        for (int i = 0; i < kStages; ++i) mbar_init(&desk.full[i], 1);
        mbar_fence_init();
        desk.abort = 0;
    }
    __syncwarp();
    const int sharer = warp * ctas + rank;   // (an item's first units are on different SMs)

    // The item, and its units: those of this warp are sharer, sharer + sharers, ...
    int row0 = 0, all = 0, kvh, units = 0, req = -1, bound = 0;
    bool bad = false;
    int first_page = -1, first_pos[2] = {-1, -1};   // the first unit's page, its positions
    if (kSelected) {
        const int per_row = p.kv_heads * p.list_tiles;
        row0 = item / per_row;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int e = sharer * kUnit + lane + 32 * h;
            if (e < p.k) first_pos[h] = p.topk[row0 * p.topk_stride + e];
        }
        kvh = (item - row0 * per_row) / p.list_tiles;
        units = p.list_units;
        const int j = p.R > 0 ? last_at_most(p.starts, p.R, row0) : -1;
        if (j >= 0 && p.starts[j] <= row0 && row0 < p.starts[j + 1]) req = j;
        const int e = p.row_ends[row0];
        bound = min(max(e, 0), p.max_keys);
        bad = req >= 0 && e != bound;
        if (req < 0) units = 0;
    } else {
        req = item / p.kv_heads;
        kvh = item - req * p.kv_heads;
        if (lane == 0 && sharer * kPage < p.max_keys) {
            // (a copy that the item turns out not to need is waited for like any other)
            const int page = p.bt[req * p.bt_stride + sharer];
            first_page = page >= 0 && page < p.num_pages ? page : -1;
            if (first_page >= 0) {
                mbar_arrive_expect_tx(&desk.full[0], p.section);
                bulk_load(ring, p.cache + first_page * p.page_stride + kvh * p.head_stride, p.section, &desk.full[0]);
            }
        }
        all = pairs_of(p, req, &row0);
        int most = 0;
        for (int r = row0 + lane; r < row0 + all / p.group; r += 32) {
            const int given = p.row_ends[r], e = min(max(given, 0), p.max_keys);
            bad |= e != given;
            most = max(most, e);
        }
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, d));
        units = (most + kUnit - 1) / kUnit;
    }
    // what the geometry says wrong, and rows outside every request (a warp that has units last, or none)
    if (warp == kWarps - 1) {
        if (blockIdx.x == 0)
            for (int j = lane; j <= p.R; j += 32) {
                const int a = p.starts[j];
                bad |= a < 0 || (j > 0 && a < p.starts[j - 1]) || a > p.rows;
            }
        if (!kSelected)
            for (int base = blockIdx.x * 32; base < p.rows; base += gridDim.x * 32) {
                const int j = last_at_most(p.starts, p.R, base + lane);
                const bool mine = p.starts[j] <= base + lane && base + lane < p.starts[j + 1];
                for (uint32_t others = __ballot_sync(0xFFFFFFFFu, !mine && base + lane < p.rows); others;
                     others &= others - 1) {
                    const int r = base + __ffs(others) - 1;
                    for (int i = lane; i < p.heads * (p.dim / 8); i += 32) {
                        const int head = i / (p.dim / 8), col = i - head * (p.dim / 8);
                        *reinterpret_cast<uint4*>(p.out + r * p.orow + head * p.ohead + col * 8) =
                            make_uint4(0, 0, 0, 0);
                        if (col == 0 && p.lse) p.lse[static_cast<int64_t>(r) * p.heads + head] = -INFINITY;
                    }
                }
            }
    }
    if (bad && p.status) atomicOr(p.status, DSA_STATUS_BAD_GEOMETRY);

    int count = sharer < units ? (units - sharer + sharers - 1) / sharers : 0;
    const int tiles = kSelected ? 1 : (all + p.cap - 1) / p.cap;
    int pos[2], page[2];
    auto copy = [&](int tile, int i) {   // unit i of the warp into its stage
        uint8_t* const stage = ring + (i % kStages) * p.stage;
        if constexpr (kSelected) {
            if (i < count) {
                const int32_t* list = p.topk + row0 * p.topk_stride;
                const int from = (sharer + i * sharers) * kUnit + lane;
                bool past = false;
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    pos[h] = i == 0 ? first_pos[h] : from + 32 * h < p.k ? list[from + 32 * h] : -1;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (pos[h] >= bound) past |= pos[h] >= 0, pos[h] = -1;
                    page[h] = pos[h] >= 0 ? p.bt[req * p.bt_stride + pos[h] / kPage] : -1;
                }
                if (past && p.status) atomicOr(p.status, DSA_STATUS_BAD_GEOMETRY);
                k.gather(stage, i % kStages, pos, page, kvh);
            }
            cp_async_commit();
        } else if (lane == 0 && i < count && !(tile == 0 && i == 0 && first_page >= 0)) {
            const int at = p.bt[req * p.bt_stride + sharer + i * sharers];
            const bool ok = at >= 0 && at < p.num_pages;
            desk.listed[i % kStages] = ok;
            if (ok) {
                mbar_arrive_expect_tx(&desk.full[i % kStages], p.section);
                bulk_load(stage, p.cache + at * p.page_stride + kvh * p.head_stride, p.section,
                          &desk.full[i % kStages]);
            } else {
                mbar_arrive(&desk.full[i % kStages]);
                if (p.status) atomicOr(p.status, DSA_STATUS_BAD_PAGE);
            }
        } else if (lane == 0 && tile == 0 && i == 0 && first_page >= 0) {
            desk.listed[0] = 1;
        }
    };
    // Parities of the stages' barriers: a copy that was not needed took one of stage 0 too.
    int turns[kStages] = {};
    for (int tile = 0; tile < max(tiles, 1); ++tile) {
        Item4 x;
        if (kSelected) {
            const int first = (item % p.list_tiles) * p.cap;
            x = Item4{row0, first, min(p.cap, p.group - first), kvh, 0, 0};
        } else {
            x = Item4{row0, tile * p.cap, min(p.cap, all - tile * p.cap), kvh, 0, 0};
        }
        for (int i = 0; i < kStages; ++i) copy(tile, i);
        __syncwarp();
        if (x.nq > 0 && count > 0) k.begin(x);
        for (int i = 0; i < count && x.nq > 0; ++i) {
            uint8_t* const stage = ring + (i % kStages) * p.stage;
            if constexpr (kSelected) {
                cp_async_wait<kStages - 1>();
                __syncwarp();
            } else {
                int parity = 0;
#pragma unroll
                for (int s = 0; s < kStages; ++s)
                    if (i % kStages == s) parity = turns[s]++ & 1;
                const bool ok = mbar_wait(&desk.full[i % kStages], parity, &desk.abort, p.status);
                if (!__all_sync(0xFFFFFFFFu, ok)) {   // the copies in flight land before their place is used again
                    const unsigned long long deadline = globaltimer() + kWaitLimitNs;
                    for (int j = i; j < min(i + kStages, count); ++j) {
#pragma unroll
                        for (int s = 0; s < kStages; ++s)
                            if (j % kStages == s) parity = (turns[s] - (j == i)) & 1;
                        mbar_drain(&desk.full[j % kStages], parity, deadline, p.status);
                    }
                    count = 0;   // (no more copies: those of a later tile would have other parities than `turns`)
                    break;
                }
            }
            const uint64_t listed = desk.listed[i % kStages];
            const int first = (sharer + i * sharers) * kUnit;
            if (listed != 0 && (kSelected || first < k.most)) k.unit(stage, first, listed);
            __syncwarp();
            copy(tile, i + kStages);
            __syncwarp();
        }
        if (kSelected) cp_async_wait<0>();
        // (the copy that was not needed)
        if (!kSelected && tile == 0 && sharer >= units && lane == 0 && first_page >= 0)
            mbar_drain(&desk.full[0], 0, globaltimer() + kWaitLimitNs, p.status);
        __syncwarp();
        // The warp's results take the place of its ring; the CTA's are joined in its first warp's, the cluster's from
        // there.
        if (x.nq > 0 && count > 0) k.finish(reinterpret_cast<float*>(ring), ml[warp]);
        fence_proxy_async_smem();   // (the next tile's copies take the results' place)
        __syncthreads();
        const int pieces = min(units, sharers), vectors = x.nq * (p.dim / 4);
        const int held = pieces > rank ? (pieces - rank + ctas - 1) / ctas : 0;   // warps with results
        for (int i = threadIdx.x; i < vectors; i += blockDim.x) {
            const int n = i / (p.dim / 4);
            float top = -INFINITY, l = 0.0f;
            float4 o = {0, 0, 0, 0};
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                if (w < held) top = fmaxf(top, ml[w][n].x);
#pragma unroll 4
            for (int w = 0; w < held; ++w) {
                const float2 e = ml[w][n];
                const float4 v = reinterpret_cast<const float4*>(smem + w * kStages * p.stage)[i];
                const float f = e.x == -INFINITY ? 0.0f : ex2_4(e.x - top);
                l += e.y * f;
                o.x += v.x * f, o.y += v.y * f, o.z += v.z * f, o.w += v.w * f;
            }
            reinterpret_cast<float4*>(smem)[i] = o;
            if (i == n * (p.dim / 4)) joined[n] = make_float2(top, l);
        }
        fence_proxy_async_smem();
        cluster.sync();
        for (int i = (warp * ctas + rank) * 32 + lane; i < vectors; i += ctas * blockDim.x) {
            const int n = i / (p.dim / 4), col = (i - n * (p.dim / 4)) * 4;
            float2 e[kCluster];
            float4 v[kCluster];
#pragma unroll
            for (int c = 0; c < kCluster; ++c) {
                e[c] = make_float2(-INFINITY, 0.0f);
                v[c] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (c < min(pieces, ctas)) {
                    e[c] = *cluster.map_shared_rank(&joined[n], c);
                    v[c] = *cluster.map_shared_rank(reinterpret_cast<const float4*>(smem) + i, c);
                }
            }
            float top = e[0].x, l = 0.0f;
            float4 o = {0, 0, 0, 0};
#pragma unroll
            for (int c = 1; c < kCluster; ++c) top = fmaxf(top, e[c].x);
#pragma unroll
            for (int c = 0; c < kCluster; ++c) {
                const float f = e[c].x == -INFINITY ? 0.0f : ex2_4(e[c].x - top);
                l += e[c].y * f;
                o.x += v[c].x * f, o.y += v[c].y * f, o.z += v[c].z * f, o.w += v[c].w * f;
            }
            const float inv = l == 0.0f ? 0.0f : p.v_scale / l;
            const int row = x.row0 + (x.first + n) / p.group, head = kvh * p.group + (x.first + n) % p.group;
            *reinterpret_cast<uint2*>(p.out + row * p.orow + head * p.ohead + col) =
                make_uint2(pack2(p, o.x * inv, o.y * inv), pack2(p, o.z * inv, o.w * inv));
            if (col == 0 && p.lse)
                p.lse[static_cast<int64_t>(row) * p.heads + head] =
                    l == 0.0f ? -INFINITY : (top + log2f(l) - kLift) * kLn2_4;
        }
        cluster.sync();   // (what the others read of this CTA stays until they are done)
    }
}

// ----------------------------------------------------------------- join
// Joins the pieces of a (row, head), and writes the rows that no unit reached:
// kWarps warps take every kWarps-th piece, four columns a lane.  Bound by the pieces'
// way through L2 and by its launch: 5 us behind 64 rows of 32 heads, 11 behind 320 of 64.
// A warp by itself takes kHeads neighbouring heads of a row, which lie in one tile.
template <int kWarps, int kHeads, bool kSelected>
__global__ void __launch_bounds__(kWarps == 1 ? 128 : kWarps * 32) attend_fp4_join_kernel(const Att4Params p) {
    constexpr int kItems = kWarps == 1 ? 4 : 1;
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t item = (blockIdx.x * kItems + (kWarps == 1 ? warp : 0)) * kHeads, heads = p.heads;
    if (item >= static_cast<uint32_t>(p.rows) * heads) return;
    const int row = item / heads, head = item - row * heads;
    const int kvh = static_cast<uint32_t>(head) / static_cast<uint32_t>(p.group), in_group = head - kvh * p.group;
    Row4 ri;
    int64_t total;
    if (kSelected) {
        const int64_t per_row = static_cast<int64_t>(p.kv_heads) * p.list_tiles * p.list_units;
        total = p.rows * per_row;
        ri = Row4{row * per_row, p.list_units, p.list_tiles, 0, 1, 0, 0};
    } else {
        ri = p.row_info[row];
        total = p.info[0];
    }
    int pieces = 0, cap_row = 0;
    int64_t slot = 0;   // of the second piece; the first's is the one before
    if (ri.pages > 0 && total > 0) {
        const int n = ri.place * p.group + in_group;
        const int tile = n / p.cap;
        cap_row = n - tile * p.cap;
        const int64_t W = sharers(p, total, kSelected || p.info[1] ? 1 : p.axis.heavy + p.axis.start);
        const int64_t length = item_length(ri.pages, ri.weight, ri.start);
        const int64_t a = min(
            ri.first + (static_cast<int64_t>(kvh) * ri.tiles + (kSelected ? tile : place_of(tile, ri.tiles))) * length,
            total - 1);
        const int64_t last = min(ri.pages > 1 ? a + length - ri.weight : a, total - 1);
        const int wa = worker_at(a, total, W), wb = worker_at(last, total, W);
        pieces = wb - wa + 1;
        if (pieces == 1) return;   // written by the attention kernel
        slot = 2 * static_cast<int64_t>(wa + 1);
    }
    const bool on = lane * 4 < p.dim;
    constexpr int kAhead = kWarps > 1 ? 8 : kHeads > 1 ? 2 : 4;   // pieces a warp has in flight
    float top[kHeads], l[kHeads];
    float4 o[kHeads];
#pragma unroll
    for (int h = 0; h < kHeads; ++h) top[h] = -INFINITY, l[h] = 0.0f, o[h] = {0, 0, 0, 0};
    for (int base = kWarps == 1 ? 0 : warp; base < pieces; base += kAhead * kWarps) {
        float2 e[kHeads][kAhead];
        float4 v[kHeads][kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int i = base + j * kWarps;
            const int64_t at = (i == 0 ? slot - 1 : slot + 2 * (i - 1)) * p.cap + cap_row;
#pragma unroll
            for (int h = 0; h < kHeads; ++h) {
                e[h][j] = make_float2(-INFINITY, 0.0f);
                v[h][j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (i < pieces) {
                    e[h][j] = p.pml[at + h];
                    if (on) v[h][j] = *reinterpret_cast<const float4*>(p.po + (at + h) * p.dim + lane * 4);
                }
            }
        }
#pragma unroll
        for (int h = 0; h < kHeads; ++h) {
            float m = top[h];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) m = fmaxf(m, e[h][j].x);
            const float keep = top[h] == -INFINITY ? 0.0f : ex2_4(top[h] - m);
            top[h] = m;
            l[h] *= keep;
            o[h].x *= keep, o[h].y *= keep, o[h].z *= keep, o[h].w *= keep;
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const float f = e[h][j].x == -INFINITY ? 0.0f : ex2_4(e[h][j].x - m);
                l[h] += e[h][j].y * f;
                o[h].x += v[h][j].x * f, o[h].y += v[h][j].y * f, o[h].z += v[h][j].z * f, o[h].w += v[h][j].w * f;
            }
        }
    }
    if (kWarps > 1) {
        static_assert(kWarps == 1 || kHeads == 1, "several warps join one head");
        __shared__ float2 sl[kWarps];
        __shared__ float4 so[kWarps][32];
        if (lane == 0) sl[warp] = make_float2(top[0], l[0]);
        so[warp][lane] = o[0];
        __syncthreads();
        if (warp > 0) return;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) top[0] = fmaxf(top[0], sl[i].x);
        l[0] = 0.0f;
        o[0] = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
            const float4 v = so[i][lane];
            const float f = sl[i].x == -INFINITY ? 0.0f : ex2_4(sl[i].x - top[0]);
            l[0] += sl[i].y * f;
            o[0].x += v.x * f, o[0].y += v.y * f, o[0].z += v.z * f, o[0].w += v.w * f;
        }
    }
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
        const float inv = l[h] == 0.0f ? 0.0f : p.v_scale / l[h];
        if (on)
            *reinterpret_cast<uint2*>(p.out + row * p.orow + (head + h) * p.ohead + lane * 4) =
                make_uint2(pack2(p, o[h].x * inv, o[h].y * inv), pack2(p, o[h].z * inv, o[h].w * inv));
        if (lane == 0 && p.lse)
            p.lse[item + h] = l[h] == 0.0f ? -INFINITY : (top[h] + log2f(l[h]) - kLift) * kLn2_4;
    }
}

// ----------------------------------------------------------------- host
static bool aligned16_4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

static Att4Layout attend4_layout(int64_t rows, int64_t num_requests, int64_t heads, int64_t kv_heads, int64_t dim,
                                 int64_t max_query_len, int64_t k) {
    Att4Layout L = {};
    const int64_t group = heads / kv_heads;
    int64_t each = k > 0 ? 1 : max_query_len < rows ? max_query_len : rows;   // rows that share keys
    if (each < 1) each = 1;
    L.cap = static_cast<int>(group * each < 32 ? group * each : 32);
    L.tiles = k > 0 ? 1 : static_cast<int>((group * each + L.cap - 1) / L.cap);
    size_t at = 0;
    auto take = [&](int64_t bytes) {
        const size_t here = at;
        at += (static_cast<size_t>(bytes) + 255) / 256 * 256;
        return here;
    };
    L.info = take(16);
    L.prefix = take(k > 0 ? 0 : (num_requests + 1) * 8);
    L.units = take(k > 0 ? 0 : (num_requests + 1) * 8);
    L.list = take(k > 0 ? rows * ((k + kUnit - 1) / kUnit * kUnit) * 4 : 0);
    L.pages = take(k > 0 ? 0 : num_requests * 4);
    L.rows = take(k > 0 ? 0 : rows * static_cast<int64_t>(sizeof(Row4)));
    const int64_t slots = 2 * kMaxCtas4 * kMaxWarps4;
    L.po = take(slots * L.cap * dim * 4);
    L.pml = take(slots * L.cap * 8);
    L.total = at;
    return L;
}

static bool sizes4_ok(int64_t rows, int64_t num_requests, int64_t heads, int64_t kv_heads, int64_t dim) {
    return rows <= (1 << 24) && num_requests <= (1 << 24) && heads <= 65535 && dim >= 16 && dim <= kFp4MaxDim &&
           dim % 16 == 0 && heads / kv_heads <= 128;
}

static int check_attend4(const dsa_kv_cache_fp4* cache, int32_t dtype, const void* q, int64_t q_row_stride,
                         int64_t q_head_stride, int64_t heads, const int32_t* block_table, int64_t bt_stride,
                         int64_t max_pages, const int32_t* starts, const int32_t* row_ends, int64_t num_requests,
                         int64_t rows, float scale, const void* out, int64_t out_row_stride, int64_t out_head_stride,
                         const void* workspace) {
    const int rc = check_kv_cache_fp4(cache);
    if (rc != DSA_OK) return rc;
    if (dtype != DSA_BF16 && dtype != DSA_FP16) return DSA_ERR_UNSUPPORTED;
    if (heads < 1 || rows < 0 || num_requests < 0 || max_pages < 0) return DSA_ERR_INVALID;
    if (heads % cache->heads) return DSA_ERR_INVALID;
    // (rows by heads, and so a request's items, key heads by row tiles, are counted in 31 bits)
    if (!sizes4_ok(rows, num_requests, heads, cache->heads, cache->dim) || rows * heads > 0x7FFFFFFF)
        return DSA_ERR_UNSUPPORTED;
    if (!(scale > 0.0f) || !isfinite(scale)) return DSA_ERR_INVALID;
    if (rows == 0) return DSA_OK;
    if (max_pages > (int64_t(1) << 24)) return DSA_ERR_UNSUPPORTED;
    if (!q || !out || !row_ends || !starts || !workspace) return DSA_ERR_INVALID;
    if (max_pages > 0 && num_requests > 0 && (!block_table || bt_stride < max_pages)) return DSA_ERR_INVALID;
    if (!aligned16_4(q) || !aligned16_4(out) || (reinterpret_cast<uintptr_t>(workspace) & 255)) return DSA_ERR_INVALID;
    if (((q_row_stride | q_head_stride | out_row_stride | out_head_stride) & 7) || q_row_stride < 0 ||
        q_head_stride < 0 || out_row_stride < 0 || out_head_stride < 0)
        return DSA_ERR_INVALID;
    if ((rows > 1 && out_row_stride == 0) || (heads > 1 && out_head_stride == 0)) return DSA_ERR_INVALID;   // one place
    return DSA_OK;
}

template <Form kForm, int kRows, bool kSelected>
static int launch_attend4(Att4Params& p, int ctas, cudaStream_t stream) {
    static_assert(Shape4<kForm, kRows>::kWarps <= kMaxWarps4, "workspaces are sized for it");
    using S4 = Shape4<kForm, kRows>;
    auto* kernel = attend_fp4_kernel<kForm, kRows, kSelected>;
    const int smem = S4::kWarps * (S4::kStages * p.stage + static_cast<int>(sizeof(Desk4<kForm, kRows, kSelected>))) +
                     (kSelected ? (kCtaRequests + 1) * 4 : p.plan_in_cta ? kAxisBytes4 : 0);
    static bool attr_set[64] = {false};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return DSA_ERR_CUDA;
    if (!attr_set[dev]) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMost4) != cudaSuccess)
            return DSA_ERR_CUDA;
        attr_set[dev] = true;
    }
    return launch_pdl(kernel, dim3(ctas), dim3(S4::kWarps * 32), smem, stream, p) == cudaSuccess ? DSA_OK
                                                                                               : DSA_ERR_CUDA;
}

// Returns DSA_ERR_UNSUPPORTED, with nothing launched, where the GPU has no room for `items` clusters at once.
template <Form kForm, int kRows, bool kSelected>
static int launch_cluster4(Att4Params& p, int items, int sms, int most_units, cudaStream_t stream) {
    using S4 = Shape4<kForm, kRows>;
    auto* kernel = attend_fp4_cluster_kernel<kForm, kRows, kSelected>;
    static bool attr_set[64] = {false};
    // Clusters of 8, 4, 2 CTAs and CTAs that run at once, and one, for heads of 16, 32, ... columns (what they keep in
    // shared memory differs); host threads may come at the same time and find the same.
    static std::atomic<int> room[64][kFp4MaxDim / 16][4];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return DSA_ERR_CUDA;
    if (!attr_set[dev]) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMost4 - 4096) != cudaSuccess)
            return DSA_ERR_CUDA;
        attr_set[dev] = true;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(S4::kWarps * 32);
    cfg.dynamicSmemBytes =
        S4::kWarps * (S4::kStages * p.stage + static_cast<int>(sizeof(Desk4<kForm, kRows, kSelected>)));
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    for (int i = 0; i < 4; ++i) {
        const int ctas = kCluster >> i;
        if (items * ctas > sms || most_units > S4::kWarps * ctas * kClusterUnits) continue;
        cfg.gridDim = dim3(items * ctas);
        attr[0].val.clusterDim.x = ctas;
        std::atomic<int>& known = room[dev][p.dim / 16 - 1][i];
        int n = known.load(std::memory_order_relaxed) - 1;
        if (n < 0) {
            cfg.numAttrs = 1;
            if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) return DSA_ERR_CUDA;
            known.store(n + 1, std::memory_order_relaxed);
        }
        if (items > n) continue;
        cfg.numAttrs = 2;
        return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
    }
    return DSA_ERR_UNSUPPORTED;
}

template <bool kSelected, int kRows>
static int launch_cluster_form4(Att4Params& p, int items, int sms, int most_units, cudaStream_t stream) {
    return p.dim == 128  ? launch_cluster4<kForm128, kRows, kSelected>(p, items, sms, most_units, stream)
           : p.dim == 64 ? launch_cluster4<kForm64, kRows, kSelected>(p, items, sms, most_units, stream)
           : p.dim > 64  ? launch_cluster4<kFormAny128, kRows, kSelected>(p, items, sms, most_units, stream)
                         : launch_cluster4<kFormAny64, kRows, kSelected>(p, items, sms, most_units, stream);
}

template <bool kSelected, int kRows>
static int launch_form4(Att4Params& p, int ctas, cudaStream_t stream) {
    return p.dim == 128  ? launch_attend4<kForm128, kRows, kSelected>(p, ctas, stream)
           : p.dim == 64 ? launch_attend4<kForm64, kRows, kSelected>(p, ctas, stream)
           : p.dim > 64  ? launch_attend4<kFormAny128, kRows, kSelected>(p, ctas, stream)
                         : launch_attend4<kFormAny64, kRows, kSelected>(p, ctas, stream);
}

template <bool kSelected>
static int launch_all4(Att4Params& p, int most_tiles, cudaStream_t stream) {
    int ctas = device_sm_count();
    if (ctas > kMaxCtas4) ctas = kMaxCtas4;
    // A cluster an item, where there are few and their units few, and a request has a row tile or hardly more, on
    // average and at most.
    const int64_t items_all = kSelected ? static_cast<int64_t>(p.rows) * p.kv_heads * p.list_tiles
                                        : static_cast<int64_t>(p.R) * p.kv_heads;
    const int most_units = kSelected ? p.list_units : p.max_keys / kUnit;
    if (items_all > 0 && items_all <= ctas && most_tiles <= kClusterTiles &&
        (kSelected || static_cast<int64_t>(p.rows) * p.group <= static_cast<int64_t>(p.R + 1) * p.cap)) {
        const int n = static_cast<int>(items_all);
        const int rc = p.cap <= 8    ? launch_cluster_form4<kSelected, 8>(p, n, ctas, most_units, stream)
                       : p.cap <= 16 ? launch_cluster_form4<kSelected, 16>(p, n, ctas, most_units, stream)
                                     : launch_cluster_form4<kSelected, 32>(p, n, ctas, most_units, stream);
        if (rc != DSA_ERR_UNSUPPORTED) return rc;
    }
    const bool wide_head = p.dim > 64;
    p.warps = ctas * (p.cap <= 8    ? Shape4<kForm128, 8>::kWarps
                      : p.cap <= 16 ? (wide_head ? Shape4<kForm128, 16>::kWarps : Shape4<kForm64, 16>::kWarps)
                                    : Shape4<kForm128, 32>::kWarps);
    if constexpr (kSelected) {
        if (p.packed) {
            const int bitmap = p.max_keys <= kBitmapKeys ? (p.max_keys + 31) / 32 * 4 : 0;
            auto* kernel = attend_fp4_list_kernel<kSelected>;
            static bool attr_set[64] = {false};
            int dev = 0;
            if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return DSA_ERR_CUDA;
            if (!attr_set[dev]) {
                if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBitmapKeys / 8) !=
                    cudaSuccess)
                    return DSA_ERR_CUDA;
                attr_set[dev] = true;
            }
            if (launch_pdl(kernel, dim3(p.rows), dim3(kList4Threads), bitmap, stream, p) != cudaSuccess)
                return DSA_ERR_CUDA;
        }
    } else if (!p.plan_in_cta && launch_pdl(attend_fp4_plan_kernel<kSelected>, dim3(1), dim3(kPlan4Threads), 0, stream,
                                            p) != cudaSuccess) {
        return DSA_ERR_CUDA;
    }
    const int rc = p.cap <= 8    ? launch_form4<kSelected, 8>(p, ctas, stream)
                   : p.cap <= 16 ? launch_form4<kSelected, 16>(p, ctas, stream)
                                 : launch_form4<kSelected, 32>(p, ctas, stream);
    if (rc != DSA_OK) return rc;
    const int64_t items = static_cast<int64_t>(p.rows) * p.heads;
    // Few rows and heads have many pieces each, which the warps of a CTA share; many leave a warp several heads, for
    // which it looks up the pieces once (the whole call, 4 heads a warp and one: 400 rows of 64 heads 81 and 85 us, 64
    // rows of 32 heads 88.0 and 87.3).
    const cudaError_t e =
        items <= 4 * ctas
            ? launch_pdl(attend_fp4_join_kernel<8, 1, kSelected>, dim3(static_cast<unsigned>(items)), dim3(256), 0,
                         stream, p)
        : items >= 32 * ctas && p.group % 4 == 0
            ? launch_pdl(attend_fp4_join_kernel<1, 4, kSelected>, dim3(static_cast<unsigned>((items + 15) / 16)),
                         dim3(128), 0, stream, p)
            : launch_pdl(attend_fp4_join_kernel<1, 1, kSelected>, dim3(static_cast<unsigned>((items + 3) / 4)),
                         dim3(128), 0, stream, p);
    return e == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

static Att4Params params4(const dsa_kv_cache_fp4* c, const Att4Layout& L, uint8_t* ws, float scale) {
    Att4Params p = {};
    p.cache = static_cast<const uint8_t*>(c->data);
    p.page_stride = c->page_stride, p.head_stride = c->head_stride;
    p.kv_heads = static_cast<int>(c->heads), p.dim = static_cast<int>(c->dim);
    p.num_pages = static_cast<int>(c->num_pages);
    p.section = fp4_section_bytes(p.dim);
    p.stage = (p.section + 127) / 128 * 128;
    p.info = reinterpret_cast<int64_t*>(ws + L.info);
    p.axis = Axis4{reinterpret_cast<int64_t*>(ws + L.prefix), reinterpret_cast<int64_t*>(ws + L.units),
                   reinterpret_cast<int*>(ws + L.pages), 1, 1, 0};
    p.list = reinterpret_cast<int*>(ws + L.list);
    p.row_info = reinterpret_cast<Row4*>(ws + L.rows);
    p.po = reinterpret_cast<float*>(ws + L.po);
    p.pml = reinterpret_cast<float2*>(ws + L.pml);
    p.cap = L.cap;
    p.c = scale * c->k_scale * kLog2e4, p.v_scale = c->v_scale;
    return p;
}

}  // namespace dsa
