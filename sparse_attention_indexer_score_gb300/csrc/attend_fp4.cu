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
constexpr int kCtaRequests = 512;       // up to this many requests every CTA lays out the axis itself
constexpr int kPlan4Threads = 512;
constexpr float kLog2e4 = 1.4426950408889634f;
constexpr float kLn2_4 = 0.6931471805599453f;
// Weights are kept times 2^6: FP16 then holds them from 2^-30 of the largest on.
constexpr float kLift = 6.0f;

// Where the join finds a row's pieces.
struct Row4 {
    int64_t first;          // first unit of the row's request
    int pages, tiles;       // units an item, row tiles a head
    int place, pad;         // the row's place in its request
};

struct Att4Layout {
    size_t info;            // int64: units on the axis
    size_t prefix, pages;   // the axis in global memory: int64[R + 1], int[R]
    size_t rows;            // Row4[rows]
    size_t po, pml;         // float[slots][cap][dim], float2[slots][cap]: partial results
    size_t total;
    int nt, cap;            // column tiles of 8 query rows; rows of a slot
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
    int64_t* prefix;
    int* pages;
    Row4* row_info;
    float* po;
    float2* pml;
    int32_t* status;
    int R, rows, heads, group, kv_heads, dim, max_keys, num_pages;
    int k, list_units, list_tiles;   // listed keys: units an item, row tiles a head
    int nt, cap, warps;              // warps: of the whole grid
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
// Warp w of W takes units [w T / W, (w + 1) T / W).
__device__ __forceinline__ int64_t share4(int64_t w, int64_t T, int64_t W) {
    if ((w + 1) * T < (int64_t(1) << 32)) return static_cast<uint32_t>(w * T) / static_cast<uint32_t>(W);
    return w * T / W;
}
__device__ __forceinline__ int warp_of(int64_t u, int64_t T, int64_t W) {
    if ((u + 1) * W < (int64_t(1) << 32) && T < (int64_t(1) << 32))
        return static_cast<int>((static_cast<uint32_t>(u + 1) * static_cast<uint32_t>(W) - 1) /
                                static_cast<uint32_t>(T));
    return static_cast<int>(((u + 1) * W - 1) / T);
}

// Lays out the requests (whole block): prefix[j] units before request j, pages[j].
// `tmp`: 33 int64 of shared scratch.  `write`: also what the join reads.
__device__ void lay_out4(const Att4Params& p, int64_t* prefix, int* pages, int64_t* tmp, bool write) {
    const int nt = blockDim.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    bool bad = false;
    if (write)
        for (int r = threadIdx.x; r < p.rows; r += nt) p.row_info[r] = Row4{0, 0, 1, 0, 0};
    int64_t carry = 0;
    __syncthreads();
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
        const int tiles = static_cast<int>((static_cast<int64_t>(s1 - s0) * p.group + p.cap - 1) / p.cap);
        const int64_t units = static_cast<int64_t>(n) * tiles * p.kv_heads;
        int64_t v = units;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t o = __shfl_up_sync(0xFFFFFFFFu, v, d);
            if (lane >= d) v += o;
        }
        if (lane == 31) tmp[warp] = v;
        __syncthreads();
        if (warp == 0) {
            int64_t s = lane < nt / 32 ? tmp[lane] : 0;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int64_t o = __shfl_up_sync(0xFFFFFFFFu, s, d);
                if (lane >= d) s += o;
            }
            tmp[lane] = s;
            if (lane == 31) tmp[32] = s;
        }
        __syncthreads();
        const int64_t before = carry + v - units + (warp > 0 ? tmp[warp - 1] : 0);
        if (j < p.R) {
            prefix[j] = before;
            pages[j] = n;
            if (write)
                for (int r = s0; r < s1; ++r) p.row_info[r] = Row4{before, n, max(tiles, 1), r - s0, 0};
        }
        carry += tmp[32];
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        prefix[p.R] = carry;
        if (write) p.info[0] = carry;
    }
    if (write && bad && p.status) atomicOr(p.status, DSA_STATUS_BAD_GEOMETRY);
    __syncthreads();
}

__global__ void __launch_bounds__(kPlan4Threads) attend_fp4_plan_kernel(const Att4Params p) {
    pdl_wait();
    pdl_launch_dependents();
    __shared__ int64_t tmp[33];
    lay_out4(p, p.prefix, p.pages, tmp, true);
}

// ----------------------------------------------------------------- attention
// The forms of a head: 128 columns, 64 columns, any other (in the place of 128).
enum Form { kForm128 = 0, kForm64 = 1, kFormAny = 2 };

template <int NT, bool kSelected>
struct Shape4 {
    static constexpr bool kQShared = NT > 2;               // query operands in shared memory, not in registers
    static constexpr int kWarps = NT == 1 ? 12 : 8;
    static constexpr int kStages = NT == 2 ? 3 : 2;
    static constexpr int kMT = NT > 2 ? 2 : 4;             // key tiles of 16 whose scores are in registers at once
};

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ float ex2_4(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
    uint32_t v;
    asm volatile("{\n\t.reg .u16 t;\n\tld.shared.u16 t, [%1];\n\tcvt.u32.u16 %0, t;\n\t}" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ void sts64(uint32_t a, uint32_t x, uint32_t y) {
    asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(a), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void sts8(uint32_t a, uint32_t x) {
    asm volatile("st.shared.u8 [%0], %1;" ::"r"(a), "r"(x) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src, uint32_t src_bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
__device__ __forceinline__ void cp_async16s(uint32_t dst, const void* src, uint32_t src_bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
// NaN among four E4M3 bytes (not zero if so).
__device__ __forceinline__ uint32_t nan4(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

// A unit of a warp's share: worked out by a lane, read by the warp.
struct __align__(16) Unit4 {
    int page;               // its page, -1: none in the pool (listed keys: the row's request, -1: none)
    int at, n;              // unit of its item, units of the item
    int kvh;                // key head
    int row0, first, nq;    // first query row of the request; first (row, head) of the tile, how many
    int bound;              // listed keys: positions from here on are not the row's
    uint64_t listed;        // which of the unit's keys are listed
    uint64_t pad;
};

template <Form kForm, int NT, bool kSelected>
struct Worker4 {
    using S4 = Shape4<NT, kSelected>;
    static constexpr int kBlocks = kForm == kForm64 ? 4 : 8;   // blocks of 16 columns in registers
    static constexpr int kSteps = kBlocks;                     // steps of 16 columns of the scores' product
    static constexpr int kOT = kBlocks;                        // tiles of 16 value columns
    static constexpr int kQ = S4::kQShared ? 1 : kSteps;

    const Att4Params& p;
    int lane, g, t;
    // the item
    uint32_t qf[kQ][S4::kQShared ? 1 : NT][2];
    uint32_t q_smem;                  // query operands in shared memory
    float o[kOT][NT][4];
    float m[NT][2], l[NT][2], c[NT][2];
    int end[NT][2];
    int row0, first, nq, kvh;         // first query row of the request, first (row, head) of the tile, how many, key head
    int least, most;                  // bounds of the tile's rows

    __device__ __forceinline__ explicit Worker4(const Att4Params& params) : p(params) {
        lane = threadIdx.x & 31;
        g = lane >> 2, t = lane & 3;
    }

    __device__ __forceinline__ int nblk() const { return kForm == kForm128 ? 8 : kForm == kForm64 ? 4 : p.dim / 16; }
    __device__ __forceinline__ int row_bytes() const { return kForm == kForm128 ? 64 : kForm == kForm64 ? 32 : p.dim / 2; }
    __device__ __forceinline__ int scale_row() const { return kForm == kForm128 ? 8 : kForm == kForm64 ? 4 : fp4_scale_row(p.dim); }
    // The bytes of a scale row's word from `first` on that are scales (the row's padding holds anything).
    __device__ __forceinline__ uint32_t scale_bytes(int first) const {
        return kForm != kFormAny || nblk() >= first + 4 ? ~0u : (1u << 8 * (nblk() - first)) - 1;
    }
    __device__ __forceinline__ int k_off() const { return 0; }
    __device__ __forceinline__ int v_off() const { return kPage * row_bytes(); }
    __device__ __forceinline__ int s_off() const { return 2 * kPage * row_bytes(); }

    // Which key of eight is operand row i: neighbours differ in parity, and so do those two apart
    // (rows of keys and of values then meet in fewer banks).
    static __device__ __forceinline__ int key_of(int i) { return i ^ ((i >> 1) & 1); }

    // The block of 16 columns that a thread has in step s of the scores' product (four columns of it).
    __device__ __forceinline__ int step_block(int s) const {
        return kForm == kForm128 ? 2 * t + (s >> 2) : kForm == kForm64 ? t : t + (s & 4);
    }

    // Query operands, bounds and factors of the item: rows first .. first + nq - 1 of (row, head) pairs of the
    // request whose rows start at row0.
    __device__ __forceinline__ void begin(int row0_, int first_, int nq_, int kvh_) {
        row0 = row0_, first = first_, nq = nq_, kvh = kvh_;
        least = 0x7FFFFFFF, most = 0;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const int n = 8 * j + g;
            const bool on = n < nq;
            const int at = first + (on ? n : 0);
            const int row = row0 + at / p.group, head = kvh * p.group + at % p.group;
            const uint16_t* src = p.q + row * p.qrow + head * p.qhead;
            float f[kSteps][4];
            uint32_t top = 0;
#pragma unroll
            for (int b = 0; b < kBlocks / 4; ++b) {   // the thread's blocks: steps 4b .. 4b + 3
                const int block = step_block(4 * b);
                uint4 w[2] = {};
                if (on && block < nblk()) {
                    w[0] = __ldg(reinterpret_cast<const uint4*>(src + 16 * block));
                    w[1] = __ldg(reinterpret_cast<const uint4*>(src + 16 * block + 8));
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float2 x = unpack2(p, (&w[i >> 2].x)[i & 3]);
                    f[4 * b + i / 2][2 * (i & 1)] = x.x;
                    f[4 * b + i / 2][2 * (i & 1) + 1] = x.y;
                    top = max(top, max(__float_as_uint(x.x) & 0x7FFFFFFFu, __float_as_uint(x.y) & 0x7FFFFFFFu));
                }
            }
            top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
            top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
            // 2^(14 - x) for the exponent x of the head's largest |q|
            const int x = max(static_cast<int>(top >> 23) - 127, -112);
            const float up = __int_as_float((127 + 14 - x) << 23);
            const float down = x >= 14 ? __int_as_float((127 + x - 14) << 23) : 1.0f / up;
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                const uint32_t b0 = Fp16::pack(f[s][0] * up, f[s][1] * up), b1 = Fp16::pack(f[s][2] * up, f[s][3] * up);
                if constexpr (S4::kQShared) {
                    sts64(q_smem + ((s * NT + j) * 32 + lane) * 8, b0, b1);
                } else {
                    qf[s][j][0] = b0, qf[s][j][1] = b1;
                }
            }
            const float cj = fminf(fmaxf(p.c * down, 1e-37f), 3e38f);
            int e = 0;
            if (on) {
                e = min(max(p.row_ends[row], 0), p.max_keys);
                least = min(least, e);
                most = max(most, e);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                c[j][i] = __shfl_sync(0xFFFFFFFFu, cj, (2 * t + i) * 4);
                end[j][i] = __shfl_sync(0xFFFFFFFFu, e, (2 * t + i) * 4);
                m[j][i] = -INFINITY;
                l[j][i] = 0.0f;
            }
#pragma unroll
            for (int i = 0; i < kOT; ++i) o[i][j][0] = o[i][j][1] = o[i][j][2] = o[i][j][3] = 0.0f;
        }
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) {
            least = min(least, __shfl_xor_sync(0xFFFFFFFFu, least, d));
            most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, d));
        }
        __syncwarp();
    }

    // A key's codes as operands of a step: two FP16 pairs of the thread's columns.
    // Keys key0 .. of the stage, MT tiles of 16; scores in s.
    __device__ __forceinline__ void scores(uint32_t stage, int key0, int nt, float (&s)[S4::kMT][NT][4]) {
#pragma unroll
        for (int i = 0; i < S4::kMT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j) s[i][j][0] = s[i][j][1] = s[i][j][2] = s[i][j][3] = 0.0f;
        uint32_t w[S4::kMT][2][kBlocks / 2];   // words of 8 codes: rows g and g + 8
        uint32_t sc[S4::kMT][2][kBlocks / 4];  // a scale twice
#pragma unroll
        for (int i = 0; i < S4::kMT; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int key = key0 + 16 * i + 8 * h + key_of(g);
                const uint32_t row = stage + k_off() + key * row_bytes();
                const uint32_t scales = stage + s_off() + key * 2 * scale_row();
                if constexpr (kForm == kForm128) {
                    const uint4 x = lds128(row + 16 * t);
                    w[i][h][0] = x.x, w[i][h][1] = x.y, w[i][h][2] = x.z, w[i][h][3] = x.w;
                    const uint32_t two = e4m3x2_f16(lds16(scales + 2 * t));
                    sc[i][h][0] = __byte_perm(two, 0, 0x1010);
                    sc[i][h][1] = __byte_perm(two, 0, 0x3232);
                } else {
#pragma unroll
                    for (int b = 0; b < kBlocks / 4; ++b) {
                        const int block = t + 4 * b;
                        uint2 x = {0, 0};
                        uint32_t one = 0;
                        if (kForm == kForm64 || block < nblk()) {
                            x = lds64(row + 8 * block);
                            one = lds8(scales + block);
                        }
                        w[i][h][2 * b] = x.x, w[i][h][2 * b + 1] = x.y;
                        sc[i][h][b] = __byte_perm(e4m3x2_f16(one), 0, 0x1010);
                    }
                }
            }
#pragma unroll
        for (int x = 0; x < kSteps / 2; ++x) {   // a word: two steps
            if (kForm == kFormAny && x >= 2 && nblk() <= 4) break;
#pragma unroll
            for (int i = 0; i < S4::kMT; ++i) {
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
                    for (int j = 0; j < NT; ++j) {
                        if (j > 0 && j >= nt) break;
                        uint2 qb;
                        if constexpr (S4::kQShared) {
                            qb = lds64(q_smem + (((2 * x + z) * NT + j) * 32 + lane) * 8);
                        } else {
                            qb = make_uint2(qf[2 * x + z][j][0], qf[2 * x + z][j][1]);
                        }
                        mma16816(s[i][j], a[2 * z], b[2 * z], a[2 * z + 1], b[2 * z + 1], qb.x, qb.y);
                    }
            }
        }
    }

    // Weights of the scores, and the values under them.
    __device__ __forceinline__ void values(uint32_t stage, int key0, int nt, float (&s)[S4::kMT][NT][4]) {
        bool raised = false;
        float ref[NT][2], keep[NT][2];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            if (j > 0 && j >= nt) break;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x = fmaxf(s[0][j][e], s[0][j][e + 2]);
#pragma unroll
                for (int i = 1; i < S4::kMT; ++i) x = fmaxf(x, fmaxf(s[i][j][e], s[i][j][e + 2]));
                x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 4));
                x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 8));
                x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 16));
                x = fmaxf(x, m[j][e]);
                raised |= x > m[j][e];
                ref[j][e] = x == -INFINITY ? 0.0f : x;
                keep[j][e] = ex2_4((m[j][e] - ref[j][e]) * c[j][e]);
                m[j][e] = x;
            }
        }
        if (__any_sync(0xFFFFFFFFu, raised)) {
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                if (j > 0 && j >= nt) break;
                l[j][0] *= keep[j][0], l[j][1] *= keep[j][1];
#pragma unroll
                for (int i = 0; i < kOT; ++i) {
                    o[i][j][0] *= keep[j][0], o[i][j][2] *= keep[j][0];
                    o[i][j][1] *= keep[j][1], o[i][j][3] *= keep[j][1];
                }
            }
        }
        uint32_t pb[S4::kMT][NT][2];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            if (j > 0 && j >= nt) break;
#pragma unroll
            for (int i = 0; i < S4::kMT; ++i) {
                float w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    // (the difference first: a large score times c would leave its rounding in the exponent)
                    w[e] = ex2_4(__fmaf_rn(s[i][j][e] - ref[j][e & 1], c[j][e & 1], kLift));
                    l[j][e & 1] += w[e];
                }
                pb[i][j][0] = transpose8x8(Fp16::pack(w[0], w[1]));
                pb[i][j][1] = transpose8x8(Fp16::pack(w[2], w[3]));
            }
        }
#pragma unroll
        for (int i = 0; i < S4::kMT; ++i) {
            uint2 v[4];          // codes of keys 2t, 2t + 1, 2t + 8, 2t + 9 (operand rows), the thread's columns
            uint32_t one[4];
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                const int key = key0 + 16 * i + 8 * (z >> 1) + key_of(2 * t + (z & 1));
                const uint32_t row = stage + v_off() + key * row_bytes();
                const uint32_t scales = stage + s_off() + key * 2 * scale_row() + scale_row();
                if constexpr (kForm == kForm64) {
                    v[z] = make_uint2(lds32(row + 4 * g), 0);
                    one[z] = lds8(scales + (g >> 1));
                } else if (kForm == kForm128 || g < nblk()) {
                    v[z] = lds64(row + 8 * g);
                    one[z] = lds8(scales + g);
                } else {
                    v[z] = make_uint2(0, 0);
                    one[z] = 0;
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
                    for (int j = 0; j < NT; ++j) {
                        if (j > 0 && j >= nt) break;
                        mma16816(o[4 * x + z][j], a0[z], a1[z], a2[z], a3[z], pb[i][j][0], pb[i][j][1]);
                    }
                }
            }
        }
    }

    __device__ __forceinline__ bool sees(int j, int e, int key, int key_base, uint64_t listed) const {
        return kSelected ? (listed >> key & 1) : key_base + key < end[j][e];
    }

    // Value scales that are NaN: the columns they enter become NaN for the rows that see the key, and the bytes zero,
    // so that nobody else's do.
    __device__ __forceinline__ void poison(uint32_t stage, int nt, int key_base, uint64_t listed) {
        const int block = kForm == kForm64 ? g >> 1 : g;
#pragma unroll 1
        for (int key = 0; key < kUnit; ++key) {
            const uint32_t at = stage + s_off() + (key * 2 + 1) * scale_row() + block;
            const bool bad = block < nblk() && (lds8(at) & 0x7F) == 0x7F;
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    if (bad && j < nt && sees(j, e, key, key_base, listed))
#pragma unroll
                        for (int i = 0; i < kOT; ++i) o[i][j][e] = o[i][j][e + 2] = __int_as_float(0x7FC00000);
            __syncwarp();
            if (bad) sts8(at, 0);
        }
        __syncwarp();
        fence_proxy_async_smem();   // (the next copy into the stage is the asynchronous proxy's)
    }

    // 64 keys of the stage; `listed`: which of them are listed.
    __device__ __forceinline__ void unit(uint32_t stage, int key_base, uint64_t listed) {
        const int nt = NT == 1 ? 1 : (nq + 7) / 8;
        {   // two keys' value scales a lane
            uint32_t bad = 0;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t at = stage + s_off() + ((lane + 32 * h) * 2 + 1) * scale_row();
                bad |= nan4(lds32(at) & scale_bytes(0));
                if (kForm == kForm128 || (kForm == kFormAny && nblk() > 4)) bad |= nan4(lds32(at + 4) & scale_bytes(4));
            }
            if (__any_sync(0xFFFFFFFFu, bad != 0)) poison(stage, nt, key_base, listed);
        }
#pragma unroll
        for (int key0 = 0; key0 < kUnit; key0 += 16 * S4::kMT) {
            float s[S4::kMT][NT][4];
            scores(stage, key0, nt, s);
            if (kSelected ? listed != ~0ull : key_base + kUnit > least) {
#pragma unroll
                for (int i = 0; i < S4::kMT; ++i)
#pragma unroll
                    for (int j = 0; j < NT; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int key = key0 + 16 * i + 8 * (e >> 1) + key_of(g);
                            if (!sees(j, e & 1, key, key_base, listed)) s[i][j][e] = -INFINITY;
                        }
            }
            values(stage, key0, nt, s);
        }
    }

    // The item's result, or the partial one of a piece (slot >= 0).
    __device__ __forceinline__ void finish(int64_t slot) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float sum = l[j][e];
                sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 4);
                sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 8);
                sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 16);
                const int n = 8 * j + 2 * t + e;
                if (n >= nq) continue;
                constexpr int kCols = 2 * kOT;   // the thread's columns, one behind the other
                const bool cols = kForm != kFormAny || g < nblk();
                const float top = m[j][e] * c[j][e];
                if (slot >= 0) {
                    float* dst = p.po + (slot * p.cap + n) * p.dim + g * kCols;
                    if (cols)
#pragma unroll
                        for (int i = 0; i < kOT; i += 2)
                            *reinterpret_cast<float4*>(dst + 2 * i) =
                                make_float4(o[i][j][e], o[i][j][e + 2], o[i + 1][j][e], o[i + 1][j][e + 2]);
                    if (g == 0) p.pml[slot * p.cap + n] = make_float2(m[j][e] == -INFINITY ? -INFINITY : top, sum);
                } else {
                    const int row = row0 + (first + n) / p.group, head = kvh * p.group + (first + n) % p.group;
                    const float inv = sum == 0.0f ? 0.0f : p.v_scale / sum;
                    uint16_t* dst = p.out + row * p.orow + head * p.ohead + g * kCols;
                    if (cols)
#pragma unroll
                        for (int i = 0; i < kOT; i += 4)
                            *reinterpret_cast<uint4*>(dst + 2 * i) =
                                make_uint4(pack2(p, o[i][j][e] * inv, o[i][j][e + 2] * inv),
                                           pack2(p, o[i + 1][j][e] * inv, o[i + 1][j][e + 2] * inv),
                                           pack2(p, o[i + 2][j][e] * inv, o[i + 2][j][e + 2] * inv),
                                           pack2(p, o[i + 3][j][e] * inv, o[i + 3][j][e + 2] * inv));
                    if (g == 0 && p.lse)
                        p.lse[static_cast<int64_t>(row) * p.heads + head] =
                            sum == 0.0f ? -INFINITY : (top + log2f(sum) - kLift) * kLn2_4;
                }
            }
    }
};

constexpr int kAxisBytes4 = (kCtaRequests + 1 + 33) * 8 + kCtaRequests * 4;

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

// Unit u of the axis.
__device__ __forceinline__ Unit4 paged_unit(const Att4Params& p, const int64_t* prefix, const int* pages, int64_t u) {
    Unit4 x;
    const int j = last_at_most(prefix, p.R, u);
    const int64_t in = u - prefix[j];
    x.n = pages[j];
    const int item = in < (int64_t(1) << 32) ? static_cast<int>(static_cast<uint32_t>(in) / static_cast<uint32_t>(x.n))
                                             : static_cast<int>(in / x.n);
    x.at = static_cast<int>(in - static_cast<int64_t>(item) * x.n);
    const int page = p.bt[j * p.bt_stride + x.at];
    x.page = page >= 0 && page < p.num_pages ? page : -1;
    if (x.page < 0 && p.status) atomicOr(p.status, DSA_STATUS_BAD_PAGE);
    x.row0 = min(max(p.starts[j], 0), p.rows);
    const int all = (min(max(p.starts[j + 1], x.row0), p.rows) - x.row0) * p.group;
    const int tiles = (all + p.cap - 1) / p.cap;
    x.kvh = item / tiles;
    x.first = (item - x.kvh * tiles) * p.cap;
    x.nq = min(p.cap, all - x.first);
    x.bound = 0;
    x.listed = 0;
    return x;
}

__device__ __forceinline__ Unit4 listed_unit(const Att4Params& p, int64_t u) {
    Unit4 x;
    const int per_row = p.kv_heads * p.list_tiles * p.list_units;
    const int row = static_cast<int>(u / per_row);
    const int in = static_cast<int>(u - static_cast<int64_t>(row) * per_row);
    const int item = in / p.list_units;
    x.n = p.list_units;
    x.at = in - item * p.list_units;
    x.kvh = item / p.list_tiles;
    x.first = (item - x.kvh * p.list_tiles) * p.cap;
    x.nq = min(p.cap, p.group - x.first);
    x.row0 = row;
    const int j = p.R > 0 ? last_at_most(p.starts, p.R, row) : -1;
    x.page = j >= 0 && p.starts[j] <= row && row < p.starts[j + 1] ? j : -1;
    const int e = p.row_ends[row];
    x.bound = min(max(e, 0), p.max_keys);
    if (x.page >= 0 && e != x.bound && p.status) atomicOr(p.status, DSA_STATUS_BAD_GEOMETRY);
    x.listed = 0;
    return x;
}

template <Form kForm, int NT, bool kSelected>
__global__ void __launch_bounds__((Shape4<NT, kSelected>::kWarps * 32), 1) attend_fp4_kernel(const Att4Params p) {
    using S4 = Shape4<NT, kSelected>;
    using W4 = Worker4<kForm, NT, kSelected>;
    constexpr int kStages = S4::kStages, kWarps = S4::kWarps;
    constexpr int kQBytes = S4::kQShared ? W4::kSteps * NT * 32 * 8 : 0;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t full[kWarps][kStages];
    __shared__ Unit4 units[kWarps][kStages];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    pdl_launch_dependents();
    // ring stages, query operands, then the axis
    uint8_t* const ring = smem + warp * kStages * p.stage;
    uint8_t* const queries = smem + kWarps * kStages * p.stage;
    if (!kSelected && lane == 0) {
        for (int i = 0; i < kStages; ++i) mbar_init(&full[warp][i], 1);
        mbar_fence_init();
    }
    __syncwarp();
    const int64_t* prefix = p.prefix;
    const int* pages = p.pages;
    if (!kSelected && p.plan_in_cta) {
        int64_t* const px = reinterpret_cast<int64_t*>(queries + kWarps * kQBytes);
        int* const pg = reinterpret_cast<int*>(px + kCtaRequests + 1 + 33);
        lay_out4(p, px, pg, px + kCtaRequests + 1, blockIdx.x == 0);
        prefix = px, pages = pg;
    }
    if (kSelected && blockIdx.x == 0 && p.status) {
        bool bad = false;
        for (int j = threadIdx.x; j < p.R; j += blockDim.x) {
            const int a = p.starts[j], b = p.starts[j + 1];
            bad |= a < 0 || b < a || b > p.rows;
        }
        if (bad) atomicOr(p.status, DSA_STATUS_BAD_GEOMETRY);
    }
    const int64_t total = kSelected ? static_cast<int64_t>(p.rows) * p.kv_heads * p.list_tiles * p.list_units
                                    : prefix[p.R];
    const int64_t W = p.warps < total ? p.warps : total;
    const int w = warp * gridDim.x + blockIdx.x;   // (neighbouring shares on different SMs)
    if (w >= W) return;
    const int64_t u0 = share4(w, total, W);
    const int count = static_cast<int>(share4(w + 1, total, W) - u0);

    W4 k(p);
    k.q_smem = smem_u32(queries) + warp * kQBytes;
    // The share's units are looked up 32 at a time, one a lane; a unit's lane writes its record to its stage.
    Unit4 mine;
    auto look_up = [&](int base) {
        if (base + lane < count)
            mine = kSelected ? listed_unit(p, u0 + base + lane) : paged_unit(p, prefix, pages, u0 + base + lane);
    };
    // Unit i of the share: its item's results so far, then its keys.
    bool whole = true;   // the piece of the item begins with it
    int begun = 0;       // ... and with this unit of the share
    auto work = [&](int i, const Unit4& x, uint32_t stage, bool any) {
        if (i == 0 || x.at == 0) {
            whole = x.at == 0;
            begun = i;
            k.begin(x.row0, x.first, x.nq, x.kvh);
        }
        if (any) k.unit(stage, x.at * kUnit, x.listed);
        // slot 2w: the piece that the share starts with; 2w + 1: one that starts inside it and does not end there
        if (x.at == x.n - 1)
            k.finish(whole ? -1 : 2 * static_cast<int64_t>(w));
        else if (i == count - 1)
            k.finish(2 * static_cast<int64_t>(w) + (begun > 0 ? 1 : 0));
    };

    if constexpr (!kSelected) {
        int abort = 0;
        auto issue = [&](int i) {
            if (i >= count) return;
            if (i % 32 == 0) look_up(i);
            if (lane == i % 32) {
                const int s = i % kStages;
                units[warp][s] = mine;
                if (mine.page >= 0) {
                    mbar_arrive_expect_tx(&full[warp][s], p.section);
                    bulk_load(ring + s * p.stage, p.cache + mine.page * p.page_stride + mine.kvh * p.head_stride,
                              p.section, &full[warp][s]);
                } else {
                    mbar_arrive(&full[warp][s]);
                }
            }
        };
        for (int i = 0; i < kStages; ++i) issue(i);
        __syncwarp();
        int i = 0;
        for (; i < count; ++i) {
            const int s = i % kStages;
            const Unit4 x = units[warp][s];
            const bool landed = mbar_wait(&full[warp][s], (i / kStages) & 1, &abort, p.status);
            if (!__all_sync(0xFFFFFFFFu, landed)) break;
            work(i, x, smem_u32(ring + s * p.stage), x.page >= 0);
            __syncwarp();
            issue(i + kStages);
            __syncwarp();
        }
        if (i < count) {   // gave up: the copies in flight land before the CTA ends
            const unsigned long long deadline = globaltimer() + kWaitLimitNs;
            const int issued = min(i + kStages, count);
            for (; i < issued; ++i) mbar_drain(&full[warp][i % kStages], (i / kStages) & 1, deadline, p.status);
        }
    } else {
        // Unit i + 2's rows of the pool are looked up and unit i + 3's positions loaded while unit i is in work.
        int pos[2], page[2], ahead[2];
        Unit4 next, later;   // the units of pos/page, and of ahead
        auto shuffled = [&](int i) {
            if (i % 32 == 0) look_up(i);
            Unit4 x;
            x.page = __shfl_sync(0xFFFFFFFFu, mine.page, i % 32);
            x.at = __shfl_sync(0xFFFFFFFFu, mine.at, i % 32);
            x.n = mine.n;
            x.kvh = __shfl_sync(0xFFFFFFFFu, mine.kvh, i % 32);
            x.row0 = __shfl_sync(0xFFFFFFFFu, mine.row0, i % 32);
            x.first = __shfl_sync(0xFFFFFFFFu, mine.first, i % 32);
            x.nq = __shfl_sync(0xFFFFFFFFu, mine.nq, i % 32);
            x.bound = __shfl_sync(0xFFFFFFFFu, mine.bound, i % 32);
            x.listed = 0;
            return x;
        };
        auto load_positions = [&](int i) {   // into ahead / later
            ahead[0] = ahead[1] = -1;
            if (i >= count) return;
            later = shuffled(i);
            if (later.page < 0) return;
            const int32_t* list = p.topk + later.row0 * p.topk_stride;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int e = later.at * kUnit + lane + 32 * h;
                if (e < p.k) ahead[h] = list[e];
            }
        };
        auto load_pages = [&]() {            // ahead / later become pos, page / next
            next = later;
            bool bad = false;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                pos[h] = ahead[h];
                page[h] = -1;
                if (pos[h] >= next.bound) {
                    bad |= pos[h] >= 0;
                    pos[h] = -1;
                }
                if (pos[h] >= 0) page[h] = p.bt[next.page * p.bt_stride + pos[h] / kPage];
            }
            if (bad && p.status) atomicOr(p.status, DSA_STATUS_BAD_GEOMETRY);
        };
        auto copy = [&](int i) {             // the rows of pos, page into the stage
            if (i < count) {
                const int s = i % kStages;
                const uint32_t stage = smem_u32(ring + s * p.stage);
                int64_t at[2];
                bool on[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    on[h] = page[h] >= 0 && page[h] < p.num_pages;
                    if (pos[h] >= 0 && !on[h] && p.status) atomicOr(p.status, DSA_STATUS_BAD_PAGE);
                    at[h] = on[h] ? page[h] * p.page_stride + next.kvh * p.head_stride : 0;
                }
                const uint32_t lo = __ballot_sync(0xFFFFFFFFu, on[0]), hi = __ballot_sync(0xFFFFFFFFu, on[1]);
                next.listed = static_cast<uint64_t>(hi) << 32 | lo;
                if (lane == 0) {
                    next.n = p.list_units;
                    units[warp][s] = next;
                }
                if (next.listed) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int sr = 2 * k.scale_row();
                        const uint8_t* src = p.cache + at[h] + (on[h] ? k.s_off() + (pos[h] % kPage) * sr : 0);
                        const uint32_t dst = stage + k.s_off() + (lane + 32 * h) * sr;
                        if (sr == 16) cp_async16s(dst, src, on[h] ? 16 : 0);
                        else cp_async8(dst, src, on[h] ? 8 : 0);
                        at[h] += on[h] ? (pos[h] % kPage) * k.row_bytes() : 0;
                    }
                    // rows of codes, cut into pieces of 16 bytes (8 where rows are not multiples of 16)
                    constexpr int kPiece = kForm == kFormAny ? 8 : 16;
                    constexpr int kLanes = kForm == kForm128 ? 4 : kForm == kForm64 ? 2 : 8;   // of a row
                    const int part = lane & (kLanes - 1), row = lane / kLanes;
                    const bool mine_too = part * kPiece < k.row_bytes();
#pragma unroll 4
                    for (int c = 0; c < kUnit / (32 / kLanes); ++c) {
                        const int token = c * (32 / kLanes) + row;
                        const int64_t a = __shfl_sync(0xFFFFFFFFu, c < kLanes ? at[0] : at[1], token & 31);
                        const bool real = next.listed >> token & 1;
                        const uint32_t dst = stage + token * k.row_bytes() + part * kPiece;
                        const uint8_t* src = p.cache + a + (real ? part * kPiece : 0);
                        if (mine_too) {
                            if (kPiece == 16) {
                                cp_async16s(dst, src, real ? 16 : 0);
                                cp_async16s(dst + k.v_off(), src + (real ? k.v_off() : 0), real ? 16 : 0);
                            } else {
                                cp_async8(dst, src, real ? 8 : 0);
                                cp_async8(dst + k.v_off(), src + (real ? k.v_off() : 0), real ? 8 : 0);
                            }
                        }
                    }
                }
            }
            cp_async_commit();
        };
        for (int i = 0; i < kStages; ++i) {
            load_positions(i);
            load_pages();
            copy(i);
        }
        load_positions(kStages);
        for (int i = 0; i < count; ++i) {
            load_pages();                         // unit i + kStages
            load_positions(i + kStages + 1);
            cp_async_wait<kStages - 1>();
            __syncwarp();
            const Unit4 x = units[warp][i % kStages];
            work(i, x, smem_u32(ring + (i % kStages) * p.stage), x.listed != 0);
            __syncwarp();
            copy(i + kStages);
        }
        cp_async_wait<0>();
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
        ri = Row4{row * per_row, p.list_units, p.list_tiles, 0, 0};
    } else {
        ri = p.row_info[row];
        total = p.info[0];
    }
    int pieces = 0, cap_row = 0;
    int64_t slot = 0, second = 0;   // slots of the first piece and of the second
    if (ri.pages > 0 && total > 0) {
        const int n = ri.place * p.group + in_group;
        const int tile = n / p.cap;
        cap_row = n - tile * p.cap;
        const int64_t W = p.warps < total ? p.warps : total;
        const int64_t a = min(ri.first + (static_cast<int64_t>(kvh) * ri.tiles + tile) * ri.pages, total - 1);
        const int wa = warp_of(a, total, W), wb = warp_of(min(a + ri.pages, total) - 1, total, W);
        pieces = wb - wa + 1;
        if (pieces == 1) return;   // written by the attention kernel
        slot = 2 * static_cast<int64_t>(wa) + (share4(wa, total, W) < a ? 1 : 0);
        second = 2 * static_cast<int64_t>(wa + 1);
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
                const int64_t at = (i == 0 ? slot : second + 2 * (i - 1)) * p.cap + cap_row;
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
    L.pages = take(k > 0 ? 0 : num_requests * 4);
    L.rows = take(k > 0 ? 0 : rows * static_cast<int64_t>(sizeof(Row4)));
    const int64_t slots = 2 * kMaxCtas4 * (L.nt == 1 ? Shape4<1, false>::kWarps : Shape4<2, false>::kWarps);
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
    using S4 = Shape4<NT, kSelected>;
    using W4 = Worker4<kForm, NT, kSelected>;
    auto* kernel = attend_fp4_kernel<kForm, NT, kSelected>;
    const int smem = S4::kWarps * (S4::kStages * p.stage + (S4::kQShared ? W4::kSteps * NT * 32 * 8 : 0)) +
                     (!kSelected && p.plan_in_cta ? kAxisBytes4 : 0);
    static bool attr_set[64] = {false};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return DSA_ERR_CUDA;
    if (!attr_set[dev]) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 230400) != cudaSuccess)
            return DSA_ERR_CUDA;
        attr_set[dev] = true;
    }
    p.warps = ctas * S4::kWarps;
    return launch_pdl(kernel, dim3(ctas), dim3(S4::kWarps * 32), smem, stream, p) == cudaSuccess ? DSA_OK
                                                                                               : DSA_ERR_CUDA;
}

template <bool kSelected, int NT>
static int launch_form4(Att4Params& p, int ctas, cudaStream_t stream) {
    return p.dim == 128  ? launch_attend4<kForm128, NT, kSelected>(p, ctas, stream)
           : p.dim == 64 ? launch_attend4<kForm64, NT, kSelected>(p, ctas, stream)
                         : launch_attend4<kFormAny, NT, kSelected>(p, ctas, stream);
}

template <bool kSelected>
static int launch_all4(Att4Params& p, cudaStream_t stream) {
    int ctas = device_sm_count();
    if (ctas > kMaxCtas4) ctas = kMaxCtas4;
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
    p.prefix = reinterpret_cast<int64_t*>(ws + L.prefix);
    p.pages = reinterpret_cast<int*>(ws + L.pages);
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
    if (static_cast<int64_t>(p.kv_heads) * p.list_tiles * p.list_units > 0x7FFFFFFF) return DSA_ERR_UNSUPPORTED;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    return launch_all4<true>(p, stream);
}
