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
// The units (64 keys of one item: a key head of a request, up to 8 NT query rows)
// lie on one axis, of which every warp takes an equal share; an item that several
// warps share is joined by a last, small kernel.
//
// The products are mma.sync m16n8k16 on FP16: keys (then value columns) are the 16
// rows, query rows the 8 columns, so that the few rows of a decode step fill the
// tile, and codes become operands in registers, without a way through memory.
// Neither product cares in what order the summed index is taken, which leaves the
// layouts free: a thread's bytes of a key are those of its own operand rows.
// Codes times scales are exact in FP16 (6 bits).
#include <math.h>

#include "elem16.cuh"
#include "fp4_cache.cuh"
#include "host.h"

namespace dsa {

constexpr int kUnit = kPage;            // keys of a unit
constexpr int kMaxCtas4 = 160;          // workspaces are sized for at most this many CTAs
constexpr int kMaxWorkers4 = 12;        // ... of this many workers
constexpr int kCtaRequests = 256;       // up to this many requests every CTA lays out the axis itself
constexpr int kPlan4Threads = 512;
constexpr int kList4Threads = 256;
constexpr int kBitmapKeys = 1 << 20;    // positions that a list is put in order by
constexpr int64_t kPackBytes = 64 << 20;   // listed sections' bytes from which lists are put in order first
constexpr float kLog2e4 = 1.4426950408889634f;
constexpr float kLn2_4 = 0.6931471805599453f;
// Weights are kept times 2^6: FP16 then holds them from 2^-30 of the largest on.
constexpr float kLift = 6.0f;

// Where the join finds a row's pieces.
struct Row4 {
    int64_t first;          // where the row's request starts on the axis
    int pages, tiles;       // units an item, row tiles a head
    int place, weight;      // the row's place in its request, what a unit of it takes of the axis
};

struct Att4Layout {
    size_t info;            // int64: the axis' length
    size_t prefix, units, pages;   // the axis in global memory: int64[R + 1] twice, int[R]
    size_t list;            // int[rows][kpad]: slots of the listed keys
    size_t rows;            // Row4[rows]
    size_t po, pml;         // float[slots][cap][dim], float2[slots][cap]: partial results
    size_t total;
    int nt, cap;            // column tiles of 8 query rows; rows of a slot
};

// The requests on the axis: where each starts, units before it, and pages an item of it has.
struct Axis4 {
    int64_t* prefix;
    int64_t* units;
    int* pages;
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
    int light, heavy;                // what units of up to 16 query rows, and of more, take of the axis
    int nt, cap, workers;            // workers: of the whole grid
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

// How many workers share an axis of length T: no more than leave a unit's start to every share.
__device__ __forceinline__ int64_t sharers(const Att4Params& p, int64_t T) {
    return max(min(static_cast<int64_t>(p.workers), T / p.heavy), static_cast<int64_t>(T > 0));
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

// Units before the first that starts at or behind place c of the axis.
__device__ __forceinline__ int64_t unit_at(const Att4Params& p, const Axis4& x, int64_t c) {
    if (c >= x.prefix[p.R]) return x.units[p.R];
    const int j = last_at_most(x.prefix, p.R, c);
    int row0;
    const int weight = pairs_of(p, j, &row0) <= 16 ? p.light : p.heavy;
    const int64_t in = c - x.prefix[j] + weight - 1;
    return x.units[j] + (weight == 1                 ? in
                         : in < (int64_t(1) << 32) ? static_cast<uint32_t>(in) / static_cast<uint32_t>(weight)
                                                   : in / weight);
}

// Lays out the requests (whole block).  `tmp`: 66 int64 of shared scratch.
// `write`: also what the join reads.
__device__ void lay_out4(const Att4Params& p, const Axis4& x, int64_t* tmp, bool write) {
    const int nt = blockDim.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    bool bad = false;
    // (on their way while the starts are read)
    for (int r = threadIdx.x * 32; r < p.rows; r += nt * 32)
        asm volatile("prefetch.global.L1 [%0];" ::"l"(p.row_ends + r));
    if (write)
        for (int r = threadIdx.x; r < p.rows; r += nt) p.row_info[r] = Row4{0, 0, 1, 0, 1};
    int64_t carry = 0, carry_units = 0;
    if (write) __syncthreads();
    for (int base = 0; base < p.R; base += nt) {
        const int j = base + threadIdx.x;
        int s0 = 0, s1 = 0, most = 0;
        if (j < p.R) {
            const int a = p.starts[j], b = p.starts[j + 1];
            if (a < 0 || b < a || b > p.rows) bad = true;
            s0 = min(max(a, 0), p.rows);
            s1 = min(max(b, s0), p.rows);
            for (int r = s0; r < s1; ++r) {
                const int given = p.row_ends[r], e = min(max(given, 0), p.max_keys);
                if (e != given) bad = true;
                most = max(most, e);
            }
        }
        const int n = (most + kUnit - 1) / kUnit;
        const int64_t all = static_cast<int64_t>(s1 - s0) * p.group;
        const int tiles = static_cast<int>((all + p.cap - 1) / p.cap), weight = all <= 16 ? p.light : p.heavy;
        const int64_t units = static_cast<int64_t>(n) * tiles * p.kv_heads, cost = units * weight;
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
            if (write)
                for (int r = s0; r < s1; ++r) p.row_info[r] = Row4{before, n, max(tiles, 1), r - s0, weight};
        }
        carry += tmp[32];
        carry_units += tmp[65];
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        x.prefix[p.R] = carry;
        x.units[p.R] = carry_units;
        if (write) p.info[0] = carry;
    }
    if (write && bad && p.status) atomicOr(p.status, DSA_STATUS_BAD_GEOMETRY);
    __syncthreads();
}

__global__ void __launch_bounds__(kPlan4Threads) attend_fp4_plan_kernel(const Att4Params p) {
    pdl_wait();
    pdl_launch_dependents();
    __shared__ int64_t tmp[66];
    lay_out4(p, p.axis, tmp, true);
}

// Listed keys as slots (page * 64 + token), in the order of their positions, so that
// neighbours in a page are read one behind the other: 64 rows of 2048 out of 4096 to
// 8192 keys take DRAM 15 us less than in a random order.  One CTA a row.  The order
// comes from a bitmap of the row's positions; where a position is listed twice (it
// counts twice), or where there are more positions than the bitmap holds, the slots
// stay in the list's order.
__global__ void __launch_bounds__(kList4Threads) attend_fp4_list_kernel(const Att4Params p) {
    pdl_wait();
    pdl_launch_dependents();
    extern __shared__ uint32_t bitmap[];
    __shared__ int sums[kList4Threads / 32 + 1];
    __shared__ int s_req, s_twice;
    const int row = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int32_t* src = p.topk + row * p.topk_stride;
    int* const dst = p.list + static_cast<int64_t>(row) * p.list_units * kUnit;
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
    if (ordered)
        for (int i = threadIdx.x; i < p.k; i += kList4Threads) {
            const int t = src[i];
            if (t >= 0 && t < bound && (atomicOr(&bitmap[t >> 5], 1u << (t & 31)) >> (t & 31) & 1)) s_twice = 1;
        }
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
        if (e != bound) bad = true;
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
        for (int i = threadIdx.x; i < p.k; i += kList4Threads) bad |= src[i] >= bound;
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

// NT column tiles of 8 query rows.  A worker is a warp, or for wide heads under
// more than 8 query rows a team of two: each scores half of a unit's keys and has
// the values of half of the columns, so that neither the codes are converted twice
// nor the accumulators (8 NT registers for 16 columns) leave the registers.
template <Form kForm, int NT, bool kSelected>
struct Shape4 {
    static constexpr int kTeam = NT > 1 && wide(kForm) ? 2 : 1;
    static constexpr int kWarps = kTeam == 2 ? (NT == 2 ? 16 : 12) : NT == 4 ? 8 : 12;
    static constexpr int kStages = 2;
    static constexpr int kWorkers = kWarps / kTeam;
    static constexpr int kLead = kTeam == 2 ? kStages - 1 : kStages;   // units whose copies are ahead of the one begun
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

// What a worker keeps in shared memory besides its ring.
template <int kSteps, int NT>
struct QueryDesk {
    uint2 q[kSteps][NT][32];              // query operands: step, column tile, lane
};
template <int kSteps>
struct QueryDesk<kSteps, 1> {};           // (one column tile's are in registers)
template <int NT, bool kTeamed>
struct TeamDesk {
    uint2 p[4][NT][32];                   // weights as operands: key tile, column tile, lane
    float top[2][8 * NT], sum[2][8 * NT]; // maxima and sums of the two warps' keys
};
template <int NT>
struct TeamDesk<NT, false> {};
template <bool kSelected>
struct ListDesk {
    int64_t rows[kSelected ? kUnit : 1];  // where listed tokens' codes are
};

template <Form kForm, int NT, bool kSelected>
struct Desk4 : QueryDesk<wide(kForm) ? 8 : 4, NT>,
               TeamDesk<NT, Shape4<kForm, NT, kSelected>::kTeam == 2>,
               ListDesk<kSelected> {
    float c[8 * NT];                      // log2(e) scale of the query rows' scores
    int ends[8 * NT];                     // their bounds
    uint64_t full[Shape4<kForm, NT, kSelected>::kStages];       // pages: copies that landed
    uint32_t listed[Shape4<kForm, NT, kSelected>::kStages][2];  // which of a unit's keys are listed
    int abort;
};

template <Form kForm, int NT, bool kSelected>
struct Worker4 {
    using S4 = Shape4<kForm, NT, kSelected>;
    using Desk = Desk4<kForm, NT, kSelected>;
    static constexpr int kTeam = S4::kTeam;
    static constexpr int kBlocks = wide(kForm) ? 8 : 4;        // blocks of 16 columns in the scores' product
    static constexpr int kSteps = kBlocks;                     // ... a step each
    static constexpr int kMT = kUnit / 16 / kTeam;             // key tiles of 16 that the warp scores
    static constexpr int kOT = kBlocks / kTeam;                // tiles of 16 value columns that it has

    const Att4Params& p;
    Desk& desk;
    int lane, g, t, half;
    uint2 q1[NT == 1 ? kSteps : 1];   // query operands of one column tile
    float o[kOT][NT][4];
    float m[NT][2], l[NT][2], c[NT][2];
    Item4 item;
    int least;                        // the smallest bound of the item's rows

    __device__ __forceinline__ Worker4(const Att4Params& params, Desk& d) : p(params), desk(d) {
        lane = threadIdx.x & 31;
        g = lane >> 2, t = lane & 3;
        half = kTeam == 2 ? (threadIdx.x >> 5) & 1 : 0;
    }

    __device__ __forceinline__ int nblk() const { return kForm == kForm128 ? 8 : kForm == kForm64 ? 4 : p.dim / 16; }
    __device__ __forceinline__ int row_bytes() const { return 8 * nblk(); }
    __device__ __forceinline__ int scale_row() const { return wide(kForm) ? 8 : 4; }
    __device__ __forceinline__ int codes_bytes() const { return kPage * row_bytes(); }
    __device__ __forceinline__ int v_off() const { return codes_bytes(); }
    __device__ __forceinline__ int s_off() const { return 2 * codes_bytes(); }

    // The warps of the worker have all come here.
    __device__ __forceinline__ void meet() const {
        if constexpr (kTeam == 2)
            asm volatile("bar.sync %0, 64;" ::"r"(static_cast<int>(threadIdx.x >> 6) + 1) : "memory");
        else
            __syncwarp();
    }

    // Which key of eight is operand row i: neighbours differ in parity, and so do those two apart
    // (rows of keys and of values then meet in fewer banks).
    static __device__ __forceinline__ int key_of(int i) { return i ^ ((i >> 1) & 1); }

    // The block of 16 columns that a thread has in step s of the scores' product (four columns of it).
    __device__ __forceinline__ int step_block(int s) const {
        return kForm == kForm128 ? 2 * t + (s >> 2) : t + (s & 4);
    }
    // The thread's value columns, 2 kOT one behind the other, and their block.
    __device__ __forceinline__ int columns() const { return half * 64 + g * 2 * kOT; }
    __device__ __forceinline__ int block() const { return kOT == 8 ? g : half * 4 + (g >> 1); }

    // Query operands, bounds and factors of an item.
    __device__ __forceinline__ void begin(const Item4& x) {
        item = x;
#pragma unroll
        for (int j0 = 0; j0 < NT; j0 += kTeam) {
            const int j = j0 + half;
            const int n = 8 * j + g;
            const bool on = n < x.nq;
            const int at = x.first + (on ? n : 0);
            const int row = x.row0 + at / p.group, head = x.kvh * p.group + at % p.group;
            const uint16_t* src = p.q + row * p.qrow + head * p.qhead;
            float f[kSteps][4];
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
            // 2^(14 - power) for the exponent of the head's largest |q|
            const int power = max(static_cast<int>(top >> 23) - 127, -112);
            const float up = __int_as_float((127 + 14 - power) << 23);
            const float down = power >= 14 ? __int_as_float((127 + power - 14) << 23) : 1.0f / up;
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
            {
                const uint2 b =
                    make_uint2(Fp16::pack(f[s][0] * up, f[s][1] * up), Fp16::pack(f[s][2] * up, f[s][3] * up));
                if constexpr (NT == 1) q1[s] = b;
                else desk.q[s][j][lane] = b;
            }
            if (t == 0) {
                desk.c[n] = fminf(fmaxf(p.c * down, 1e-37f), 3e38f);
                desk.ends[n] = on ? min(max(p.row_ends[row], 0), p.max_keys) : 0x7FFFFFFF;
            }
        }
        meet();
        least = 0x7FFFFFFF;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int n = 8 * j + 2 * t + e;
                c[j][e] = desk.c[n];
                least = min(least, desk.ends[n]);
                m[j][e] = -INFINITY;
                l[j][e] = 0.0f;
            }
        least = min(least, __shfl_xor_sync(0xFFFFFFFFu, least, 1));
        least = min(least, __shfl_xor_sync(0xFFFFFFFFu, least, 2));
#pragma unroll
        for (int i = 0; i < kOT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j) o[i][j][0] = o[i][j][1] = o[i][j][2] = o[i][j][3] = 0.0f;
    }

    // The scores of the warp's keys under the first N column tiles.
    template <int N>
    __device__ __forceinline__ void scores(const uint8_t* stage, float (&s)[kMT][N][4]) {
#pragma unroll
        for (int i = 0; i < kMT; ++i)
#pragma unroll
            for (int j = 0; j < N; ++j) s[i][j][0] = s[i][j][1] = s[i][j][2] = s[i][j][3] = 0.0f;
        uint32_t w[kMT][2][kBlocks / 2];   // words of 8 codes: rows g and g + 8
        uint32_t sc[kMT][2][kBlocks / 4];  // a scale twice
#pragma unroll
        for (int i = 0; i < kMT; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int key = 16 * (half * kMT + i) + 8 * h + key_of(g);
                const uint8_t* row = stage + key * row_bytes();
                const uint8_t* scales = stage + s_off() + key * 2 * scale_row();
                if constexpr (kForm == kForm128) {
                    const uint4 x = lds<uint4>(row + 16 * t);
                    w[i][h][0] = x.x, w[i][h][1] = x.y, w[i][h][2] = x.z, w[i][h][3] = x.w;
                    const uint32_t two = e4m3x2_f16(lds<uint16_t>(scales + 2 * t));
                    sc[i][h][0] = __byte_perm(two, 0, 0x1010);
                    sc[i][h][1] = __byte_perm(two, 0, 0x3232);
                } else {
#pragma unroll
                    for (int b = 0; b < kBlocks / 4; ++b) {
                        const int blk = t + 4 * b;
                        uint2 x = {0, 0};
                        uint32_t one = 0;
                        if (kForm == kForm64 || blk < nblk()) {
                            x = lds<uint2>(row + 8 * blk);
                            one = lds<uint8_t>(scales + blk);
                        }
                        w[i][h][2 * b] = x.x, w[i][h][2 * b + 1] = x.y;
                        sc[i][h][b] = __byte_perm(e4m3x2_f16(one), 0, 0x1010);
                    }
                }
            }
#pragma unroll
        for (int x = 0; x < kSteps / 2; ++x) {   // a word: two steps
            uint2 qs[2][N];
#pragma unroll
            for (int z = 0; z < 2; ++z)
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    if constexpr (NT == 1) qs[z][j] = q1[2 * x + z];
                    else qs[z][j] = desk.q[2 * x + z][j][lane];
                }
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
#pragma unroll
                    for (int j = 0; j < N; ++j)
                        mma16816(s[i][j], a[2 * z], b[2 * z], a[2 * z + 1], b[2 * z + 1], qs[z][j].x, qs[z][j].y);
            }
        }
    }

    __device__ __forceinline__ bool sees(int j, int e, int key, int key_base, uint64_t listed) const {
        return kSelected ? (listed >> key & 1) : key_base + key < desk.ends[8 * j + 2 * t + e];
    }

    // Scores of keys that a row does not see.
    template <int N>
    __device__ __forceinline__ void mask(int key_base, uint64_t listed, float (&s)[kMT][N][4]) {
        if (kSelected ? listed == ~0ull : key_base + kUnit <= least) return;
#pragma unroll
        for (int i = 0; i < kMT; ++i)
#pragma unroll
            for (int j = 0; j < N; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int key = 16 * (half * kMT + i) + 8 * (e >> 1) + key_of(g);
                    if (!sees(j, e & 1, key, key_base, listed)) s[i][j][e] = -INFINITY;
                }
    }

    // The largest score of each column among the warp's keys.
    template <int N>
    __device__ __forceinline__ void maxima(const float (&s)[kMT][N][4], float (&x)[N][2]) {
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                x[j][e] = fmaxf(s[0][j][e], s[0][j][e + 2]);
#pragma unroll
                for (int i = 1; i < kMT; ++i) x[j][e] = fmaxf(x[j][e], fmaxf(s[i][j][e], s[i][j][e + 2]));
                x[j][e] = fmaxf(x[j][e], __shfl_xor_sync(0xFFFFFFFFu, x[j][e], 4));
                x[j][e] = fmaxf(x[j][e], __shfl_xor_sync(0xFFFFFFFFu, x[j][e], 8));
                x[j][e] = fmaxf(x[j][e], __shfl_xor_sync(0xFFFFFFFFu, x[j][e], 16));
            }
    }

    // The weights of the warp's keys as operands, under the columns' maxima x of the unit; what there is so far is
    // brought to the new maxima.
    template <int N>
    __device__ __forceinline__ void weights(const float (&s)[kMT][N][4], const float (&x)[N][2],
                                            uint2 (&pb)[kMT][N]) {
        bool raised = false;
        float ref[N][2], keep[N][2];
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float top = fmaxf(x[j][e], m[j][e]);
                raised |= top > m[j][e];
                ref[j][e] = top == -INFINITY ? 0.0f : top;
                keep[j][e] = ex2_4((m[j][e] - ref[j][e]) * c[j][e]);
                m[j][e] = top;
            }
        if (__any_sync(0xFFFFFFFFu, raised)) {
#pragma unroll
            for (int j = 0; j < N; ++j) {
                l[j][0] *= keep[j][0], l[j][1] *= keep[j][1];
#pragma unroll
                for (int i = 0; i < kOT; ++i) {
                    o[i][j][0] *= keep[j][0], o[i][j][2] *= keep[j][0];
                    o[i][j][1] *= keep[j][1], o[i][j][3] *= keep[j][1];
                }
            }
        }
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
            for (int i = 0; i < kMT; ++i) {
                float w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    // (the difference first: a large score times c would leave its rounding in the exponent)
                    w[e] = ex2_4(__fmaf_rn(s[i][j][e] - ref[j][e & 1], c[j][e & 1], kLift));
                    l[j][e & 1] += w[e];
                }
                pb[i][j] = make_uint2(transpose8x8(Fp16::pack(w[0], w[1])), transpose8x8(Fp16::pack(w[2], w[3])));
            }
    }

    // The values of key tile i under its weights.
    template <int N>
    __device__ __forceinline__ void values(const uint8_t* stage, int i, const uint2 (&pb)[N]) {
        uint2 v[4];          // codes of keys 2t, 2t + 1, 2t + 8, 2t + 9 (operand rows), the thread's columns
        uint32_t one[4];
#pragma unroll
        for (int z = 0; z < 4; ++z) {
            const int key = 16 * i + 8 * (z >> 1) + key_of(2 * t + (z & 1));
            const uint8_t* row = stage + v_off() + key * row_bytes() + columns() / 2;
            const uint8_t* scales = stage + s_off() + (key * 2 + 1) * scale_row();
            v[z] = make_uint2(0, 0);
            one[z] = 0;
            if (kForm == kForm128 || kForm == kForm64 || block() < nblk()) {
                if constexpr (kOT == 8) v[z] = lds<uint2>(row);
                else v[z].x = lds<uint32_t>(row);
                one[z] = lds<uint8_t>(scales + block());
            }
        }
        const uint32_t sa = e4m3x2_f16(one[0] | one[1] << 8), sb = e4m3x2_f16(one[2] | one[3] << 8);
#pragma unroll
        for (int x = 0; x < kOT / 4; ++x) {   // a word: four column tiles
            const uint32_t k0 = x ? v[0].y : v[0].x, k1 = x ? v[1].y : v[1].x;
            const uint32_t k2 = x ? v[2].y : v[2].x, k3 = x ? v[3].y : v[3].x;
            uint32_t a0[4], a1[4], a2[4], a3[4];   // even columns (operand rows 0-7), odd columns (8-15)
            e2m1x8((k0 & 0x0F0F0F0Fu) | (k1 << 4 & 0xF0F0F0F0u), a0);
            e2m1x8((k0 >> 4 & 0x0F0F0F0Fu) | (k1 & 0xF0F0F0F0u), a1);
            e2m1x8((k2 & 0x0F0F0F0Fu) | (k3 << 4 & 0xF0F0F0F0u), a2);
            e2m1x8((k2 >> 4 & 0x0F0F0F0Fu) | (k3 & 0xF0F0F0F0u), a3);
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                a0[z] = hmul2(a0[z], sa), a1[z] = hmul2(a1[z], sa);
                a2[z] = hmul2(a2[z], sb), a3[z] = hmul2(a3[z], sb);
#pragma unroll
                for (int j = 0; j < N; ++j)
                    mma16816(o[4 * x + z][j], a0[z], a1[z], a2[z], a3[z], pb[j].x, pb[j].y);
            }
        }
    }

    // Value scales that are NaN: the columns they enter become NaN for the rows that see the key, and the bytes zero,
    // so that nobody else's do.
    template <int N>
    __device__ __forceinline__ void poison(uint8_t* stage, int key_base, uint64_t listed) {
        const int blk = block();
#pragma unroll 1
        for (int key = 0; key < kUnit; ++key) {
            uint8_t* const at = stage + s_off() + (key * 2 + 1) * scale_row() + blk;
            const bool bad = blk < nblk() && (lds<uint8_t>(at) & 0x7F) == 0x7F;
#pragma unroll
            for (int j = 0; j < N; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    if (bad && sees(j, e, key, key_base, listed))
#pragma unroll
                        for (int i = 0; i < kOT; ++i) o[i][j][e] = o[i][j][e + 2] = __int_as_float(0x7FC00000);
            __syncwarp();
            if (bad) *at = 0;
        }
        __syncwarp();
        fence_proxy_async_smem();   // (the next copy into the stage is the asynchronous proxy's)
    }

    // Looks for value scales that are NaN among the warp's blocks, two keys a lane.
    template <int N>
    __device__ __forceinline__ void check(uint8_t* stage, int key_base, uint64_t listed) {
        constexpr bool kBoth = wide(kForm) && kTeam == 1;   // two words of four blocks, or the warp's one
        const int from = kTeam == 2 ? half * 4 : 0;
        uint32_t bad = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint8_t* at = stage + s_off() + ((lane + 32 * h) * 2 + 1) * scale_row();
            bad |= nan4(lds<uint32_t>(at + from) & scale_bytes(from));
            if (kBoth) bad |= nan4(lds<uint32_t>(at + 4) & scale_bytes(4));
        }
        if (__any_sync(0xFFFFFFFFu, bad != 0)) poison<N>(stage, key_base, listed);
    }
    // The bytes of a scale row's word from `first` on that are scales (the row's padding holds anything).
    __device__ __forceinline__ uint32_t scale_bytes(int first) const {
        return kForm == kForm128 || kForm == kForm64 || nblk() >= first + 4 ? ~0u
               : nblk() <= first                                             ? 0u
                                                                             : (1u << 8 * (nblk() - first)) - 1;
    }

    // A unit that has landed in its stage (or not in time: true is returned).  `issue` orders the copies that the
    // unit's progress makes room for.
    template <int N, typename Issue>
    __device__ __forceinline__ bool unit(uint8_t* stage, int key_base, uint64_t listed, bool any, Issue issue) {
        float s[kMT][N][4], x[N][2];
        uint2 pb[kMT][N];
        if constexpr (kTeam == 1) {
            __syncwarp();
            if (!kSelected && *static_cast<volatile int*>(&desk.abort)) return true;
            if (any) {
                check<N>(stage, key_base, listed);
                scores<N>(stage, s);
                mask<N>(key_base, listed, s);
                maxima<N>(s, x);
                weights<N>(s, x, pb);
#pragma unroll
                for (int i = 0; i < kMT; ++i) values<N>(stage, i, pb[i]);
            }
            __syncwarp();
            issue();
            __syncwarp();
        } else {
            if (any) {
                scores<N>(stage, s);
                mask<N>(key_base, listed, s);
                maxima<N>(s, x);
                if (g == 0)
#pragma unroll
                    for (int j = 0; j < N; ++j)
                        *reinterpret_cast<float2*>(&desk.top[half][8 * j + 2 * t]) = make_float2(x[j][0], x[j][1]);
            }
            meet();
            // (seen alike by both warps: neither waits for the next unit before they have met again)
            const bool gave_up = !kSelected && *static_cast<volatile int*>(&desk.abort) != 0;
            if (!gave_up) issue();
            if (gave_up || !any) {
                meet();
                return gave_up;
            }
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const float2 y = *reinterpret_cast<const float2*>(&desk.top[half ^ 1][8 * j + 2 * t]);
                x[j][0] = fmaxf(x[j][0], y.x), x[j][1] = fmaxf(x[j][1], y.y);
            }
            check<N>(stage, key_base, listed);
            weights<N>(s, x, pb);
#pragma unroll
            for (int i = 0; i < kMT; ++i)
#pragma unroll
                for (int j = 0; j < N; ++j) desk.p[half * kMT + i][j][lane] = pb[i][j];
            meet();
#pragma unroll
            for (int i = 0; i < 2 * kMT; ++i) {
                uint2 w[N];
#pragma unroll
                for (int j = 0; j < N; ++j) w[j] = desk.p[i][j][lane];
                values<N>(stage, i, w);
            }
        }
        return false;
    }

    // The item's result, or the partial one of a piece (slot >= 0).
    __device__ __forceinline__ void finish(int64_t slot) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                l[j][e] += __shfl_xor_sync(0xFFFFFFFFu, l[j][e], 4);
                l[j][e] += __shfl_xor_sync(0xFFFFFFFFu, l[j][e], 8);
                l[j][e] += __shfl_xor_sync(0xFFFFFFFFu, l[j][e], 16);
                if constexpr (kTeam == 2)
                    if (g == 0) desk.sum[half][8 * j + 2 * t + e] = l[j][e];
            }
        if constexpr (kTeam == 2) meet();
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int n = 8 * j + 2 * t + e;
                if (n >= item.nq) continue;
                float sum = l[j][e];
                if constexpr (kTeam == 2) sum = desk.sum[0][n] + desk.sum[1][n];
                const bool cols = kForm == kForm128 || kForm == kForm64 || block() < nblk();
                const bool first = g == 0 && half == 0;
                const float top = m[j][e] * c[j][e];
                if (slot >= 0) {
                    float* dst = p.po + (slot * p.cap + n) * p.dim + columns();
                    if (cols)
#pragma unroll
                        for (int i = 0; i < kOT; i += 2)
                            *reinterpret_cast<float4*>(dst + 2 * i) =
                                make_float4(o[i][j][e], o[i][j][e + 2], o[i + 1][j][e], o[i + 1][j][e + 2]);
                    if (first) p.pml[slot * p.cap + n] = make_float2(m[j][e] == -INFINITY ? -INFINITY : top, sum);
                } else {
                    const int row = item.row0 + (item.first + n) / p.group;
                    const int head = item.kvh * p.group + (item.first + n) % p.group;
                    const float inv = sum == 0.0f ? 0.0f : p.v_scale / sum;
                    uint16_t* dst = p.out + row * p.orow + head * p.ohead + columns();
                    if (cols)
#pragma unroll
                        for (int i = 0; i < kOT; i += 4)
                            *reinterpret_cast<uint4*>(dst + 2 * i) =
                                make_uint4(pack2(p, o[i][j][e] * inv, o[i][j][e + 2] * inv),
                                           pack2(p, o[i + 1][j][e] * inv, o[i + 1][j][e + 2] * inv),
                                           pack2(p, o[i + 2][j][e] * inv, o[i + 2][j][e + 2] * inv),
                                           pack2(p, o[i + 3][j][e] * inv, o[i + 3][j][e + 2] * inv));
                    if (first && p.lse)
                        p.lse[static_cast<int64_t>(row) * p.heads + head] =
                            sum == 0.0f ? -INFINITY : (top + log2f(sum) - kLift) * kLn2_4;
                }
            }
    }
};

constexpr int kAxisBytes4 = (2 * (kCtaRequests + 1) + 66) * 8 + kCtaRequests * 4;

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
        const int first = (item - x.kvh * tiles) * p.cap;
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

// Shared memory: the workers' rings, their desks, then the axis.
template <Form kForm, int NT, bool kSelected>
__global__ void __launch_bounds__((Shape4<kForm, NT, kSelected>::kWarps * 32), 1)
attend_fp4_kernel(const Att4Params p) {
    using S4 = Shape4<kForm, NT, kSelected>;
    using W4 = Worker4<kForm, NT, kSelected>;
    using Desk = Desk4<kForm, NT, kSelected>;
    constexpr int kTeam = S4::kTeam, kStages = S4::kStages, kLead = S4::kLead;
    extern __shared__ __align__(128) uint8_t smem[];
    const int lane = threadIdx.x & 31, worker = threadIdx.x / (32 * kTeam);
    pdl_wait();
    pdl_launch_dependents();
    uint8_t* const ring = smem + worker * kStages * p.stage;
    Desk& desk = reinterpret_cast<Desk*>(smem + S4::kWorkers * kStages * p.stage)[worker];
    W4 k(p, desk);
    const bool leads = k.half == 0;      // the warp that looks units up and orders pages
    if (leads && lane == 0) {
        if (!kSelected) {
            for (int i = 0; i < kStages; ++i) mbar_init(&desk.full[i], 1);
            mbar_fence_init();
        }
        desk.abort = 0;
    }
    Axis4 axis = p.axis;
    const int* starts = p.starts;
    uint8_t* const table = smem + S4::kWorkers * (kStages * p.stage + sizeof(Desk));
    if (!kSelected && p.plan_in_cta) {
        axis.prefix = reinterpret_cast<int64_t*>(table);
        axis.units = axis.prefix + kCtaRequests + 1;
        axis.pages = reinterpret_cast<int*>(axis.units + kCtaRequests + 1 + 66);
        lay_out4(p, axis, axis.units + kCtaRequests + 1, blockIdx.x == 0);
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
    k.meet();
    const int64_t total = kSelected ? static_cast<int64_t>(p.rows) * p.kv_heads * p.list_tiles * p.list_units
                                    : axis.prefix[p.R];
    const int64_t W = sharers(p, total);
    const int w = worker * gridDim.x + blockIdx.x;   // (neighbouring shares on different SMs)
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
            desk.listed[i % kStages][0] = mine.page >= 0;
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

    // Listed keys: two tokens a lane, or one where two warps share them.  While a unit is in work, the pages of the
    // unit kLead on are looked up and the positions of the one behind it loaded.
    constexpr int kTokens = 2 / kTeam;
    int pos[kTokens], page[kTokens], ahead[kTokens];
    struct List {
        int req, kvh, bound;
    } next, later;                       // the units of pos / page, and of ahead
    const int token0 = k.half * 32 + lane;
    auto load_positions = [&](int i) {   // into ahead / later
#pragma unroll
        for (int h = 0; h < kTokens; ++h) ahead[h] = -1;
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
        for (int h = 0; h < kTokens; ++h) {
            const int e = at * kUnit + token0 + 32 * h;
            if (e < most) ahead[h] = list[e];
        }
    };
    auto load_pages = [&]() {            // ahead / later become pos, page / next
        next = later;
        bool bad = false;
#pragma unroll
        for (int h = 0; h < kTokens; ++h) {
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
    // Rows of codes are cut into pieces of 16 bytes (8 where rows are not multiples of 16).
    constexpr int kPiece = kForm == kForm128 || kForm == kForm64 ? 16 : 8;
    constexpr int kLanes = kForm == kForm128 ? 4 : kForm == kForm64 ? 2 : wide(kForm) ? 8 : 4;   // of a row
    auto gather = [&](int i) {           // the unit of pos / page into its stage
        if (i < count) {
            uint8_t* const stage = ring + (i % kStages) * p.stage;
            uint32_t any = 0;
#pragma unroll
            for (int h = 0; h < kTokens; ++h) {
                const bool on = page[h] >= 0 && page[h] < p.num_pages;
                if (pos[h] >= 0 && !on && p.status) atomicOr(p.status, DSA_STATUS_BAD_PAGE);
                // (tokens that are not there: any codes, and scales of zero)
                const int token = pos[h] % kPage, sr = 2 * k.scale_row();
                const int64_t section = on ? page[h] * p.page_stride + next.kvh * p.head_stride : 0;
                desk.rows[token0 + 32 * h] = section + (on ? token * k.row_bytes() : 0);
                const uint8_t* src = p.cache + section + k.s_off() + (on ? token * sr : 0);
                const uint32_t to = smem_u32(stage + k.s_off() + (token0 + 32 * h) * sr);
                if (p.num_pages > 0) {
                    if (sr == 16) cp_async16s(to, src, on ? 16 : 0);
                    else cp_async8(to, src, on ? 8 : 0);
                }
                const uint32_t mask = __ballot_sync(0xFFFFFFFFu, on);
                any |= mask;
                if (lane == 0) desk.listed[i % kStages][k.half + h] = mask;
            }
            __syncwarp();
            const int part = lane % kLanes;
            if (any && part * kPiece < k.row_bytes()) {
#pragma unroll
                for (int c = 0; c < kTokens * kLanes; ++c) {
                    const int token = k.half * 32 + c * (32 / kLanes) + lane / kLanes;
                    const uint8_t* src = p.cache + desk.rows[token] + part * kPiece;
                    const uint32_t to = smem_u32(stage + token * k.row_bytes() + part * kPiece);
                    if (kPiece == 16) {
                        cp_async16s(to, src, 16);
                        cp_async16s(to + k.v_off(), src + k.v_off(), 16);
                    } else {
                        cp_async8(to, src, 8);
                        cp_async8(to + k.v_off(), src + k.v_off(), 8);
                    }
                }
            }
        }
        cp_async_commit();
    };

    if constexpr (kSelected) {
        for (int i = 0; i < kLead; ++i) {
            load_positions(i);
            load_pages();
            gather(i);
        }
        load_positions(kLead);
    } else if (leads) {
        for (int i = 0; i < kLead; ++i) copy_page(i);
    }
    int i = 0;
    bool gave_up = false;
    while (i < count && !gave_up) {
        // The part of an item that is in the share: units at .. until - 1 of its n.
        Item4 x;
        if (kSelected) listed_unit(p, starts, u0 + i, &x);
        else paged_unit(p, axis, u0 + i, &x);
        k.begin(x);
        const int until = min(x.n, x.at + count - i);
        for (int at = x.at; at < until; ++at, ++i) {
            uint8_t* const stage = ring + (i % kStages) * p.stage;
            if constexpr (kSelected) {
                load_pages();                     // of unit i + kLead
                load_positions(i + kLead + 1);
                cp_async_wait<kLead - 1>();
                __syncwarp();
            } else {
                mbar_wait(&desk.full[i % kStages], (i / kStages) & 1, &desk.abort, p.status);
            }
            // (written where the unit's copies were ordered, and the worker has met since)
            uint64_t listed = 0;
            bool any;
            if constexpr (kSelected) {
                listed = static_cast<uint64_t>(desk.listed[i % kStages][1]) << 32 | desk.listed[i % kStages][0];
                any = kTeam == 2 || listed != 0;
            } else {
                any = desk.listed[i % kStages][0] != 0;
            }
            auto issue = [&]() {
                if constexpr (kSelected) gather(i + kLead);
                else if (leads) copy_page(i + kLead);
            };
            if constexpr (NT == 4) {
                gave_up = x.nq <= 16 ? k.template unit<2>(stage, at * kUnit, listed, any, issue)
                                     : k.template unit<4>(stage, at * kUnit, listed, any, issue);
            } else {
                gave_up = k.template unit<NT>(stage, at * kUnit, listed, any, issue);
            }
            if (gave_up) break;
        }
        // slot 2w + 1: the item's first piece; 2w: a later one (a share has at most one of each)
        if (!gave_up) k.finish(x.at == 0 && until == x.n ? -1 : 2 * static_cast<int64_t>(w) + (x.at == 0 ? 1 : 0));
        k.meet();
    }
    if constexpr (kSelected) {
        cp_async_wait<0>();
    } else if (gave_up && leads) {   // the copies in flight land before the CTA ends
        const unsigned long long deadline = globaltimer() + kWaitLimitNs;
        for (int j = i; j < min(i + kLead + 1, count); ++j)
            mbar_drain(&desk.full[j % kStages], (j / kStages) & 1, deadline, p.status);
    }
}

// ----------------------------------------------------------------- join
// Joins the pieces of a (row, head), and writes the rows that no unit reached:
// kWarps warps take every kWarps-th piece, four columns a lane.
template <int kWarps, bool kSelected>
__global__ void __launch_bounds__(kWarps == 1 ? 128 : kWarps * 32) attend_fp4_join_kernel(const Att4Params p) {
    constexpr int kItems = kWarps == 1 ? 4 : 1;
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t item = blockIdx.x * kItems + (kWarps == 1 ? warp : 0), heads = p.heads;
    if (item >= static_cast<uint32_t>(p.rows) * heads) return;
    const int row = item / heads, head = item - row * heads;
    const int kvh = static_cast<uint32_t>(head) / static_cast<uint32_t>(p.group), in_group = head - kvh * p.group;
    Row4 ri;
    int64_t total;
    if (kSelected) {
        const int64_t per_row = static_cast<int64_t>(p.kv_heads) * p.list_tiles * p.list_units;
        total = p.rows * per_row;
        ri = Row4{row * per_row, p.list_units, p.list_tiles, 0, 1};
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
        const int64_t W = sharers(p, total);
        const int64_t a =
            min(ri.first + (static_cast<int64_t>(kvh) * ri.tiles + tile) * ri.pages * ri.weight, total - 1);
        const int64_t last = min(a + static_cast<int64_t>(ri.pages - 1) * ri.weight, total - 1);
        const int wa = worker_at(a, total, W), wb = worker_at(last, total, W);
        pieces = wb - wa + 1;
        if (pieces == 1) return;   // written by the attention kernel
        slot = 2 * static_cast<int64_t>(wa + 1);
    }
    const bool on = lane * 4 < p.dim;
    constexpr int kAhead = 4;
    float top = -INFINITY, l = 0.0f;
    float4 o = {0, 0, 0, 0};
    for (int base = kWarps == 1 ? 0 : warp; base < pieces; base += kAhead * kWarps) {
        float2 e[kAhead];
        float4 v[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int i = base + j * kWarps;
            e[j] = make_float2(-INFINITY, 0.0f);
            v[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (i < pieces) {
                const int64_t at = (i == 0 ? slot - 1 : slot + 2 * (i - 1)) * p.cap + cap_row;
                e[j] = p.pml[at];
                if (on) v[j] = *reinterpret_cast<const float4*>(p.po + at * p.dim + lane * 4);
            }
        }
        float m = top;
#pragma unroll
        for (int j = 0; j < kAhead; ++j) m = fmaxf(m, e[j].x);
        const float keep = top == -INFINITY ? 0.0f : ex2_4(top - m);
        top = m;
        l *= keep;
        o.x *= keep, o.y *= keep, o.z *= keep, o.w *= keep;
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const float f = e[j].x == -INFINITY ? 0.0f : ex2_4(e[j].x - m);
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
        for (int i = 0; i < kWarps; ++i) top = fmaxf(top, sl[i].x);
        l = 0.0f;
        o = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
            const float4 v = so[i][lane];
            const float f = sl[i].x == -INFINITY ? 0.0f : ex2_4(sl[i].x - top);
            l += sl[i].y * f;
            o.x += v.x * f, o.y += v.y * f, o.z += v.z * f, o.w += v.w * f;
        }
    }
    const float inv = l == 0.0f ? 0.0f : p.v_scale / l;
    if (on)
        *reinterpret_cast<uint2*>(p.out + row * p.orow + head * p.ohead + lane * 4) =
            make_uint2(pack2(p, o.x * inv, o.y * inv), pack2(p, o.z * inv, o.w * inv));
    if (lane == 0 && p.lse) p.lse[item] = l == 0.0f ? -INFINITY : (top + log2f(l) - kLift) * kLn2_4;
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
    L.nt = L.cap <= 8 ? 1 : L.cap <= 16 ? 2 : 4;
    size_t at = 0;
    auto take = [&](int64_t bytes) {
        const size_t here = at;
        at += (static_cast<size_t>(bytes) + 255) / 256 * 256;
        return here;
    };
    L.info = take(8);
    L.prefix = take(k > 0 ? 0 : (num_requests + 1) * 8);
    L.units = take(k > 0 ? 0 : (num_requests + 1) * 8);
    L.list = take(k > 0 ? rows * ((k + kUnit - 1) / kUnit * kUnit) * 4 : 0);
    L.pages = take(k > 0 ? 0 : num_requests * 4);
    L.rows = take(k > 0 ? 0 : rows * static_cast<int64_t>(sizeof(Row4)));
    const int64_t slots = 2 * kMaxCtas4 * kMaxWorkers4;
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
    if (!sizes4_ok(rows, num_requests, heads, cache->heads, cache->dim) || rows * heads > 0x7FFFFFFF)
        return DSA_ERR_UNSUPPORTED;
    if (!(scale > 0.0f) || !isfinite(scale)) return DSA_ERR_INVALID;
    if (rows == 0) return DSA_OK;
    // (an item's number in its request is counted in 31 bits: key heads by row tiles of 32, at least 4 rows of heads)
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

template <Form kForm, int NT, bool kSelected>
static int launch_attend4(Att4Params& p, int ctas, cudaStream_t stream) {
    static_assert(Shape4<kForm, NT, kSelected>::kWorkers <= kMaxWorkers4, "workspaces are sized for it");
    using S4 = Shape4<kForm, NT, kSelected>;
    auto* kernel = attend_fp4_kernel<kForm, NT, kSelected>;
    const int smem = S4::kWorkers * (S4::kStages * p.stage + static_cast<int>(sizeof(Desk4<kForm, NT, kSelected>))) +
                     (kSelected ? (kCtaRequests + 1) * 4 : p.plan_in_cta ? kAxisBytes4 : 0);
    static bool attr_set[64] = {false};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return DSA_ERR_CUDA;
    if (!attr_set[dev]) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMost4) != cudaSuccess)
            return DSA_ERR_CUDA;
        attr_set[dev] = true;
    }
    p.workers = ctas * S4::kWorkers;
    return launch_pdl(kernel, dim3(ctas), dim3(S4::kWarps * 32), smem, stream, p) == cudaSuccess ? DSA_OK
                                                                                               : DSA_ERR_CUDA;
}

template <bool kSelected, int NT>
static int launch_form4(Att4Params& p, int ctas, cudaStream_t stream) {
    return p.dim == 128  ? launch_attend4<kForm128, NT, kSelected>(p, ctas, stream)
           : p.dim == 64 ? launch_attend4<kForm64, NT, kSelected>(p, ctas, stream)
           : p.dim > 64  ? launch_attend4<kFormAny128, NT, kSelected>(p, ctas, stream)
                         : launch_attend4<kFormAny64, NT, kSelected>(p, ctas, stream);
}

template <bool kSelected>
static int launch_all4(Att4Params& p, cudaStream_t stream) {
    int ctas = device_sm_count();
    if (ctas > kMaxCtas4) ctas = kMaxCtas4;
    if (kSelected && p.packed) {
        const int bitmap = p.max_keys <= kBitmapKeys ? (p.max_keys + 31) / 32 * 4 : 0;
        static bool attr_set[64] = {false};
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return DSA_ERR_CUDA;
        if (!attr_set[dev]) {
            if (cudaFuncSetAttribute(attend_fp4_list_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     kBitmapKeys / 8) != cudaSuccess)
                return DSA_ERR_CUDA;
            attr_set[dev] = true;
        }
        if (launch_pdl(attend_fp4_list_kernel, dim3(p.rows), dim3(kList4Threads), bitmap, stream, p) != cudaSuccess)
            return DSA_ERR_CUDA;
    }
    if (!kSelected && !p.plan_in_cta &&
        launch_pdl(attend_fp4_plan_kernel, dim3(1), dim3(kPlan4Threads), 0, stream, p) != cudaSuccess)
        return DSA_ERR_CUDA;
    const int rc = p.nt == 1   ? launch_form4<kSelected, 1>(p, ctas, stream)
                   : p.nt == 2 ? launch_form4<kSelected, 2>(p, ctas, stream)
                               : launch_form4<kSelected, 4>(p, ctas, stream);
    if (rc != DSA_OK) return rc;
    const int64_t items = static_cast<int64_t>(p.rows) * p.heads;
    // Few rows and heads have many pieces each, which the warps of a CTA share.
    const cudaError_t e =
        items <= 4 * ctas
            ? launch_pdl(attend_fp4_join_kernel<8, kSelected>, dim3(static_cast<unsigned>(items)), dim3(256), 0,
                         stream, p)
            : launch_pdl(attend_fp4_join_kernel<1, kSelected>, dim3(static_cast<unsigned>((items + 3) / 4)),
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
                   reinterpret_cast<int*>(ws + L.pages)};
    p.list = reinterpret_cast<int*>(ws + L.list);
    p.light = p.heavy = 1;
    p.row_info = reinterpret_cast<Row4*>(ws + L.rows);
    p.po = reinterpret_cast<float*>(ws + L.po);
    p.pml = reinterpret_cast<float2*>(ws + L.pml);
    p.nt = L.nt, p.cap = L.cap;
    p.c = scale * c->k_scale * kLog2e4, p.v_scale = c->v_scale;
    return p;
}

}  // namespace dsa

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
    if (p.nt == 4) p.light = 2, p.heavy = 3;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    return launch_all4<false>(p, stream);
}

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
    return launch_all4<true>(p, stream);
}
