// dsa_kv_append_fp4 and dsa_kv_read_fp4: new keys and values into the 4-bit cache
// (rotated and quantised on the way), and back out of it.
//
// A block of 16 columns x becomes s = E4M3(max |x| / (6 g)) and the codes
// E2M1(x / (s g)); a code c reads as (c s) g.  Both kernels move 16-bit elements
// once on one side and 9/16 of a byte an element on the other and are bound by
// memory: 16384 tokens of 32 query and 2 x 8 cache heads of 128 columns, appended and
// read back, take 79 us (84 % of the copy rate), 65536 tokens of 2 x 8 heads read back 61
// (83 %).  Few tokens are bound by the launch and two loads that depend on each other.
#include <math.h>

#include "elem16.cuh"
#include "fp4_cache.cuh"
#include "host.h"

namespace dsa {

constexpr int kAppend4Threads = 128;
constexpr int kAppend4Batch = 6;   // most head rows a thread has in flight
constexpr int kRead4Threads = 256;

struct Append4Args {
    const uint16_t* k;
    const uint16_t* v;
    const uint16_t* q;
    uint16_t* q_out;
    uint8_t* cache;
    int64_t kt, kh, vt, vh, qt, qh, ot, oh;   // element strides: token, head
    int64_t page_stride, head_stride;         // bytes
    const int64_t* slots;
    const int64_t* positions;
    const float* cos_sin;
    int64_t cs_stride, max_pos, num_slots, n;
    int q_heads, kv_heads, dim, units, rot_units, half, row_lanes, head_lanes, tokens_per_cta, batch;
    float k_scale, v_scale, k_six, v_six;     // g and 6 g
    int32_t* status;
};

// Streaming: read or written once, first to leave L2.
template <bool kStreams>
__device__ __forceinline__ uint4 ld_row(const uint16_t* p) {
    const uint4* v = reinterpret_cast<const uint4*>(p);
    return kStreams ? __ldcs(v) : *v;
}
template <bool kStreams>
__device__ __forceinline__ void st_row(uint16_t* p, uint4 v) {
    if (kStreams)
        __stcs(reinterpret_cast<uint4*>(p), v);
    else
        *reinterpret_cast<uint4*>(p) = v;
}

template <typename T>
__device__ __forceinline__ void unpack8(const uint4& w, float (&f)[8]) {
    const uint32_t* p = &w.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 x = T::unpack(p[i]);
        f[2 * i] = x.x, f[2 * i + 1] = x.y;
    }
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(T::pack(f[0], f[1]), T::pack(f[2], f[3]), T::pack(f[4], f[5]), T::pack(f[6], f[7]));
}

// The pair (a, b) turned: two rounded products, one rounded sum, as dsa_kv_append.
__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
    const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
    b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
    a = x;
}

// The larger of two magnitudes, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}
__device__ __forceinline__ float amax8(const float (&x)[8]) {
    float m = fabsf(x[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) m = max_nan(m, fabsf(x[i]));
    return m;
}

// A block's scale byte from its largest magnitude, 6 g given.
__device__ __forceinline__ uint32_t block_scale(float amax, float six) {
    const float s = __fdiv_rn(amax, six);
    uint16_t two;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two) : "f"(0.0f), "f"(s));
    return two & 0xFFu;
}

// Eight codes of x / (s g).  The quotient is correctly rounded without a division
// an element: q0 = x inv(d) with the correctly rounded reciprocal, its remainder
// (negated, so that the quotient of -0 stays -0) exactly by a fused multiply-add, one
// correction (Markstein).  Under the largest scale |x| is first cut to 8 d, past the
// largest code, so that nothing overflows; under the others |x| is not above 9 d (the
// smallest scale stands for up to one and a half of itself), and what is past the
// largest code becomes it.
__device__ __forceinline__ uint32_t codes8(const float (&x)[8], uint32_t scale_byte, float g) {
    const float d = __fmul_rn(half2_float2(e4m3x2_f16(scale_byte)).x, g);
    uint32_t w = 0;
    if (scale_byte == 0) {   // nothing but zeros; their signs stay
#pragma unroll
        for (int i = 0; i < 8; ++i) w |= (__float_as_uint(x[i]) >> 31) << (4 * i + 3);
        return w;
    }
    const float inv = __frcp_rn(d);
    float a[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = x[i];
    if (scale_byte >= 0x7E) {
        const float most = 8.0f * d;
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] = fminf(fmaxf(a[i], -most), most);
    }
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        float y[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float q0 = __fmul_rn(a[i + j], inv);
            y[j] = __fmaf_rn(-__fmaf_rn(q0, d, -a[i + j]), inv, q0);
        }
        uint32_t two;
        asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %2, %1;\n\tcvt.u32.u8 %0, t;\n\t}"
            : "=r"(two)
            : "f"(y[0]), "f"(y[1]));
        w |= two << (4 * i);
    }
    return w;
}

// A head row is cut into vectors of 8 columns; vectors 2b and 2b + 1 are block b.
// A row has `units` threads of two vectors each (row_lanes of them, the next power
// of two, so that a row stays within a warp): unit u < rot_units of a rotated row of
// halves has vectors u and u + rot_units, which turn together, any other row or unit
// 2u and 2u + 1.  In the first form a block's two vectors may be in two threads,
// which tell each other their largest magnitudes.  A token has row_lanes x head_lanes
// threads; a thread keeps its unit's eight angles and walks the token's heads in steps
// of head_lanes.  Queries and keys with values have CTAs of their own: the two take
// different registers, and short code.
struct Place4 {
    int64_t tok, slot;
    int unit, lane;            // of the row; row of the step
    bool on, cached, turns;
    int v0, v1;                // vectors of a rotated row
};

template <bool kInterleaved>
__device__ __forceinline__ Place4 place(const Append4Args& a, int64_t block, bool flags, float (&c)[8], float (&s)[8]) {
    Place4 x;
    const int per_token = a.row_lanes * a.head_lanes;
    const int sub = threadIdx.x / per_token;
    x.tok = block * a.tokens_per_cta + sub;
    const int in = threadIdx.x - sub * per_token;
    x.unit = in & (a.row_lanes - 1), x.lane = in / a.row_lanes;
    // (threads without work stay: rows' threads shuffle as whole warps)
    x.on = sub < a.tokens_per_cta && x.tok < a.n && x.unit < a.units;
    x.slot = x.on ? a.slots[x.tok] : -1;
    x.cached = x.slot >= 0 && x.slot < a.num_slots;
    if (flags && x.slot >= a.num_slots && in == 0 && a.status) atomicOr(a.status, DSA_STATUS_BAD_SLOT);
    x.turns = x.on && x.unit < a.rot_units;
    const bool halves = x.turns && !kInterleaved;
    x.v0 = halves ? x.unit : 2 * x.unit, x.v1 = halves ? x.unit + a.rot_units : 2 * x.unit + 1;
    if (x.turns) {
        int64_t p = a.positions[x.tok];
        if (p < 0 || p >= a.max_pos) {
            if (flags && x.slot >= 0 && in == 0 && a.status) atomicOr(a.status, DSA_STATUS_BAD_GEOMETRY);
            p = p < 0 ? 0 : a.max_pos - 1;
        }
        const float* row = a.cos_sin + p * a.cs_stride + x.unit * 8;
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
            *reinterpret_cast<float4*>(c + i) = __ldg(reinterpret_cast<const float4*>(row + i));
            *reinterpret_cast<float4*>(s + i) = __ldg(reinterpret_cast<const float4*>(row + a.half + i));
        }
    }
    return x;
}

template <bool kInterleaved>
__device__ __forceinline__ void turn_row(float (&f)[8], float (&g)[8], const float (&c)[8], const float (&s)[8]) {
    if (kInterleaved) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            turn(f[2 * j], f[2 * j + 1], c[j], s[j]);
            turn(g[2 * j], g[2 * j + 1], c[4 + j], s[4 + j]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) turn(f[j], g[j], c[j], s[j]);
    }
}

template <typename T, bool kInterleaved, bool kStreams>
__device__ __forceinline__ void append_queries(const Append4Args& a, int64_t block) {
    float c[8], s[8];
    const Place4 x = place<kInterleaved>(a, block, false, c, s);
    if (!x.on) return;
    for (int base = x.lane; base < a.q_heads; base += a.batch * a.head_lanes) {
        uint4 w[kAppend4Batch], y[kAppend4Batch];
#pragma unroll
        for (int i = 0; i < kAppend4Batch; ++i) {
            const int h = base + i * a.head_lanes;
            if (i >= a.batch || h >= a.q_heads) continue;
            const uint16_t* src = a.q + x.tok * a.qt + h * a.qh;
            w[i] = ld_row<kStreams>(src + x.v0 * 8);
            y[i] = ld_row<kStreams>(src + x.v1 * 8);
        }
#pragma unroll
        for (int i = 0; i < kAppend4Batch; ++i) {
            const int h = base + i * a.head_lanes;
            if (i >= a.batch || h >= a.q_heads) continue;
            if (x.turns) {
                float f[8], g[8];
                unpack8<T>(w[i], f);
                unpack8<T>(y[i], g);
                turn_row<kInterleaved>(f, g, c, s);
                w[i] = pack8<T>(f);
                y[i] = pack8<T>(g);
            }
            uint16_t* dst = a.q_out + x.tok * a.ot + h * a.oh;
            st_row<kStreams>(dst + x.v0 * 8, w[i]);
            st_row<kStreams>(dst + x.v1 * 8, y[i]);
        }
    }
}

template <typename T, bool kInterleaved, bool kStreams>
__device__ __forceinline__ void append_keys_values(const Append4Args& a, int64_t block) {
    float c[8], s[8];
    const Place4 x = place<kInterleaved>(a, block, true, c, s);
    const bool halves = x.turns && !kInterleaved;
    // where the other vectors of the thread's blocks are: lane and vector of the pair there
    const int row_base = (threadIdx.x & 31) - x.unit;
    auto owner = [&](int v, bool* second) {
        const bool h = !kInterleaved && v < 2 * a.rot_units;
        *second = h ? v >= a.rot_units : v & 1;
        return row_base + (h ? (v >= a.rot_units ? v - a.rot_units : v) : v >> 1);
    };
    bool second0, second1;
    const int mate0 = owner(x.v0 ^ 1, &second0), mate1 = owner(x.v1 ^ 1, &second1);
    const int off = static_cast<int>(x.slot & 63), sr = fp4_scale_row(a.dim);
    uint8_t* const section = a.cache + (x.cached ? (x.slot >> 6) * a.page_stride : 0);
#pragma unroll 1
    for (int base = 0; base < a.kv_heads; base += a.head_lanes) {
        const int h = base + x.lane;
        const bool on = x.cached && h < a.kv_heads;
        uint4 kw = {}, ky = {}, vw = {}, vy = {};
        if (on) {
            const uint16_t* k = a.k + x.tok * a.kt + h * a.kh;
            const uint16_t* v = a.v + x.tok * a.vt + h * a.vh + x.unit * 16;
            kw = ld_row<kStreams>(k + x.v0 * 8);
            ky = ld_row<kStreams>(k + x.v1 * 8);
            vw = ld_row<kStreams>(v);
            vy = ld_row<kStreams>(v + 8);
        }
        uint8_t* const at = section + h * a.head_stride;
        uint8_t* const scales = at + fp4_scales(a.dim, off);
        float f[8], g[8];
        unpack8<T>(kw, f);
        unpack8<T>(ky, g);
        if (x.turns) turn_row<kInterleaved>(f, g, c, s);
        float m0 = amax8(f), m1 = amax8(g);
        if (!kInterleaved && a.rot_units > 0) {
            const float a0 = __shfl_sync(0xFFFFFFFFu, m0, mate0), a1 = __shfl_sync(0xFFFFFFFFu, m1, mate0);
            const float b0 = __shfl_sync(0xFFFFFFFFu, m0, mate1), b1 = __shfl_sync(0xFFFFFFFFu, m1, mate1);
            m0 = max_nan(m0, second0 ? a1 : a0);
            m1 = max_nan(m1, second1 ? b1 : b0);
        } else {
            m0 = m1 = max_nan(m0, m1);
        }
        if (!on) continue;
        {
            const uint32_t s0 = block_scale(m0, a.k_six), s1 = halves ? block_scale(m1, a.k_six) : s0;
            const uint32_t w0 = codes8(f, s0, a.k_scale), w1 = codes8(g, s1, a.k_scale);
            uint8_t* const codes = at + fp4_k_row(a.dim, off);
            if (halves) {
                *reinterpret_cast<uint32_t*>(codes + x.v0 * 4) = w0;
                *reinterpret_cast<uint32_t*>(codes + x.v1 * 4) = w1;
                if (!(x.v0 & 1)) scales[x.v0 >> 1] = static_cast<uint8_t>(s0);
                if (!(x.v1 & 1)) scales[x.v1 >> 1] = static_cast<uint8_t>(s1);
            } else {
                *reinterpret_cast<uint2*>(codes + x.unit * 8) = make_uint2(w0, w1);
                scales[x.unit] = static_cast<uint8_t>(s0);
            }
        }
        unpack8<T>(vw, f);
        unpack8<T>(vy, g);
        const uint32_t s0 = block_scale(max_nan(amax8(f), amax8(g)), a.v_six);
        const uint32_t w0 = codes8(f, s0, a.v_scale), w1 = codes8(g, s0, a.v_scale);
        *reinterpret_cast<uint2*>(at + fp4_v_row(a.dim, off) + x.unit * 8) = make_uint2(w0, w1);
        scales[sr + x.unit] = static_cast<uint8_t>(s0);
    }
}

template <typename T, bool kInterleaved, bool kStreams>
__global__ void __launch_bounds__(kAppend4Threads) kv_append_fp4_kernel(const Append4Args a) {
    pdl_wait();
    pdl_launch_dependents();
    // every other CTA, so that both kinds are on the GPU together
    const int64_t block = a.q ? blockIdx.x >> 1 : blockIdx.x;
    if (a.q && blockIdx.x & 1)
        append_queries<T, kInterleaved, kStreams>(a, block);
    else
        append_keys_values<T, kInterleaved, kStreams>(a, block);
}

struct Read4Args {
    const uint8_t* cache;
    int64_t page_stride, head_stride;
    const int64_t* slots;
    int64_t n, num_slots;
    uint16_t* k;
    uint16_t* v;
    int64_t kt, kh, vt, vh;
    int heads, dim, units;
    float k_scale, v_scale;
    int32_t* status;
};

// 16 columns, first to leave L2: in one store where they are a sector (32-byte
// alignment).  A sector that is written in two halves may leave L2 between them, and
// what is missing is then read.
template <bool kSectors>
__device__ __forceinline__ void st_block(uint16_t* dst, const uint32_t (&w)[8]) {
    if constexpr (kSectors) {
        asm volatile("st.global.cs.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]),
                     "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        __stcs(reinterpret_cast<uint4*>(dst), make_uint4(w[0], w[1], w[2], w[3]));
        __stcs(reinterpret_cast<uint4*>(dst + 8), make_uint4(w[4], w[5], w[6], w[7]));
    }
}

template <typename T, bool kSectors>
__device__ __forceinline__ void write_block(uint16_t* dst, uint2 codes, uint32_t scale, float g) {
    const float s = half2_float2(e4m3x2_f16(scale)).x;
    uint32_t out[8];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t h[4];
        e2m1x8(i ? codes.y : codes.x, h);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = half2_float2(h[j]);
            out[4 * i + j] = T::pack(__fmul_rn(__fmul_rn(f.x, s), g), __fmul_rn(__fmul_rn(f.y, s), g));
        }
    }
    st_block<kSectors>(dst, out);
}

// A thread reads the block of 16 columns of a token's head out of keys and values.
template <typename T, bool kSectors>
__global__ void __launch_bounds__(kRead4Threads) kv_read_fp4_kernel(const Read4Args a) {
    pdl_wait();
    pdl_launch_dependents();
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kRead4Threads + threadIdx.x;
    const int per_token = a.heads * a.units;
    const int64_t tok = i < (int64_t(1) << 32) ? static_cast<uint32_t>(i) / static_cast<uint32_t>(per_token)
                                               : i / per_token;
    if (tok >= a.n) return;
    const int in = static_cast<int>(i - tok * per_token);
    const int head = in / a.units, unit = in - head * a.units;
    const int64_t slot = a.slots[tok];
    const bool real = slot >= 0 && slot < a.num_slots;
    if (slot >= a.num_slots && in == 0 && a.status) atomicOr(a.status, DSA_STATUS_BAD_SLOT);
    uint2 kc = {0, 0}, vc = {0, 0};
    uint32_t ks = 0, vs = 0;
    if (real) {
        const uint8_t* section = a.cache + (slot >> 6) * a.page_stride + head * a.head_stride;
        const int off = static_cast<int>(slot & 63);
        const uint8_t* scales = section + fp4_scales(a.dim, off) + unit;
        kc = *reinterpret_cast<const uint2*>(section + fp4_k_row(a.dim, off) + unit * 8);
        vc = *reinterpret_cast<const uint2*>(section + fp4_v_row(a.dim, off) + unit * 8);
        ks = scales[0];
        vs = scales[fp4_scale_row(a.dim)];
    }
    write_block<T, kSectors>(a.k + tok * a.kt + head * a.kh + unit * 16, kc, ks, a.k_scale);
    write_block<T, kSectors>(a.v + tok * a.vt + head * a.vh + unit * 16, vc, vs, a.v_scale);
}

template <typename T>
static cudaError_t launch_append4(const Append4Args& a, dim3 grid, bool interleaved, bool streams,
                                  cudaStream_t stream) {
    auto* kernel = interleaved ? (streams ? kv_append_fp4_kernel<T, true, true> : kv_append_fp4_kernel<T, true, false>)
                               : (streams ? kv_append_fp4_kernel<T, false, true>
                                          : kv_append_fp4_kernel<T, false, false>);
    return launch_pdl(kernel, grid, dim3(kAppend4Threads), 0, stream, a);
}

int check_kv_cache_fp4(const dsa_kv_cache_fp4* c) {
    if (!c) return DSA_ERR_INVALID;
    if (c->num_pages < 0 || c->heads < 1 || c->dim < 16) return DSA_ERR_INVALID;
    if (c->dim % 16 || c->dim > kFp4MaxDim || c->heads > 65535 || c->num_pages > 0x7FFFFFFF)
        return DSA_ERR_UNSUPPORTED;
    if (c->num_pages > 0 && !c->data) return DSA_ERR_INVALID;
    if ((reinterpret_cast<uintptr_t>(c->data) & 15) || c->page_stride < 0 || c->head_stride < 0 ||
        c->page_stride % 16 || c->head_stride % 16)
        return DSA_ERR_INVALID;
    const int64_t section = fp4_section_bytes(static_cast<int>(c->dim));
    if ((c->num_pages > 1 && c->page_stride < section) || (c->heads > 1 && c->head_stride < section))
        return DSA_ERR_INVALID;
    const float least = ldexpf(1.0f, -64), most = ldexpf(1.0f, 64);
    for (float g : {c->k_scale, c->v_scale})
        if (!(g >= least && g <= most)) return DSA_ERR_INVALID;
    return DSA_OK;
}

// A dimension of several elements written to one place.
static bool one_place(int64_t extent, int64_t stride) { return extent > 1 && stride == 0; }

}  // namespace dsa

using namespace dsa;

extern "C" size_t dsa_kv_section_bytes_fp4(int64_t dim) {
    return dim < 16 || dim > kFp4MaxDim || dim % 16 ? 0 : fp4_section_bytes(static_cast<int>(dim));
}

extern "C" int dsa_kv_append_fp4(const dsa_kv_cache_fp4* cache, int32_t dtype, const void* k, int64_t k_token_stride,
                                 int64_t k_head_stride, const void* v, int64_t v_token_stride, int64_t v_head_stride,
                                 const void* q, int64_t q_token_stride, int64_t q_head_stride, int64_t q_heads,
                                 void* q_out, int64_t qo_token_stride, int64_t qo_head_stride, int64_t n,
                                 const int64_t* slots, const int64_t* positions, const float* cos_sin,
                                 int64_t cs_stride, int64_t max_pos, int64_t rot_dim, int interleaved, int32_t* status,
                                 void* stream_) {
    const int rc = check_kv_cache_fp4(cache);
    if (rc != DSA_OK) return rc;
    if (dtype != DSA_BF16 && dtype != DSA_FP16) return DSA_ERR_UNSUPPORTED;
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
    if (q && (one_place(n, qo_token_stride) || one_place(q_heads, qo_head_stride))) return DSA_ERR_INVALID;

    Append4Args a;
    a.k = static_cast<const uint16_t*>(k);
    a.v = static_cast<const uint16_t*>(v);
    a.q = static_cast<const uint16_t*>(q);
    a.q_out = static_cast<uint16_t*>(q_out);
    a.cache = static_cast<uint8_t*>(cache->data);
    a.kt = k_token_stride, a.kh = k_head_stride, a.vt = v_token_stride, a.vh = v_head_stride;
    a.qt = q_token_stride, a.qh = q_head_stride, a.ot = qo_token_stride, a.oh = qo_head_stride;
    a.page_stride = cache->page_stride, a.head_stride = cache->head_stride;
    a.slots = slots;
    a.positions = positions;
    a.cos_sin = cos_sin;
    a.cs_stride = cs_stride, a.max_pos = max_pos, a.num_slots = cache->num_pages * kPage, a.n = n;
    a.q_heads = q ? static_cast<int>(q_heads) : 0;
    a.kv_heads = static_cast<int>(cache->heads);
    a.dim = static_cast<int>(cache->dim);
    a.units = a.dim / 16;
    a.rot_units = static_cast<int>(rot_dim / 16);
    a.half = static_cast<int>(rot_dim / 2);
    a.k_scale = cache->k_scale, a.v_scale = cache->v_scale;
    a.k_six = 6.0f * a.k_scale, a.v_six = 6.0f * a.v_scale;
    a.status = status;
    // The longer the append, the fewer threads a token, so that a thread turns more
    // heads with the angles it holds: short ones a CTA a token of each kind (latency),
    // 16384 tokens of 32 + 2 x 8 heads 131, 91, 84 to 87 and 84 us with 128, 64, 32 and
    // 16 threads (the call and the reading back of what it wrote).
    const int64_t sms = device_sm_count();
    const bool streams = n >= 4 * sms;
    const int want = n >= 32 * sms ? 16 : streams ? 64 : kAppend4Threads;
    a.row_lanes = 1;
    while (a.row_lanes < a.units) a.row_lanes *= 2;
    a.head_lanes = want / a.row_lanes;
    // the query heads of a thread in equal rounds
    const int each = a.q ? (a.q_heads + a.head_lanes - 1) / a.head_lanes : 1;
    const int rounds = (each + kAppend4Batch - 1) / kAppend4Batch;
    a.batch = (each + rounds - 1) / rounds;
    a.tokens_per_cta = kAppend4Threads / want;
    const int64_t blocks = (n + a.tokens_per_cta - 1) / a.tokens_per_cta * (a.q ? 2 : 1);
    if (blocks > 0x7FFFFFFF) return DSA_ERR_UNSUPPORTED;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    const dim3 grid(static_cast<unsigned>(blocks));
    const cudaError_t err = dtype == DSA_BF16 ? launch_append4<Bf16>(a, grid, interleaved, streams, stream)
                                              : launch_append4<Fp16>(a, grid, interleaved, streams, stream);
    return err == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

extern "C" int dsa_kv_read_fp4(const dsa_kv_cache_fp4* cache, int32_t dtype, const int64_t* slots, int64_t n,
                               void* k_out, int64_t k_token_stride, int64_t k_head_stride, void* v_out,
                               int64_t v_token_stride, int64_t v_head_stride, int32_t* status, void* stream_) {
    const int rc = check_kv_cache_fp4(cache);
    if (rc != DSA_OK) return rc;
    if (dtype != DSA_BF16 && dtype != DSA_FP16) return DSA_ERR_UNSUPPORTED;
    if (n < 0) return DSA_ERR_INVALID;
    if (n == 0) return DSA_OK;
    if (!slots || !k_out || !v_out) return DSA_ERR_INVALID;
    if ((reinterpret_cast<uintptr_t>(k_out) | reinterpret_cast<uintptr_t>(v_out)) & 15) return DSA_ERR_INVALID;
    const int64_t strides[2][2] = {{k_token_stride, k_head_stride}, {v_token_stride, v_head_stride}};
    for (int i = 0; i < 2; ++i)
        if (((strides[i][0] | strides[i][1]) & 7) || one_place(n, strides[i][0]) ||
            one_place(cache->heads, strides[i][1]))
            return DSA_ERR_INVALID;
    Read4Args a;
    a.cache = static_cast<const uint8_t*>(cache->data);
    a.page_stride = cache->page_stride, a.head_stride = cache->head_stride;
    a.slots = slots, a.n = n, a.num_slots = cache->num_pages * kPage;
    a.k = static_cast<uint16_t*>(k_out), a.v = static_cast<uint16_t*>(v_out);
    a.kt = k_token_stride, a.kh = k_head_stride, a.vt = v_token_stride, a.vh = v_head_stride;
    a.heads = static_cast<int>(cache->heads), a.dim = static_cast<int>(cache->dim), a.units = a.dim / 16;
    a.k_scale = cache->k_scale, a.v_scale = cache->v_scale;
    a.status = status;
    if (n > (int64_t(1) << 40)) return DSA_ERR_UNSUPPORTED;
    const int64_t blocks = (n * a.heads * a.units + kRead4Threads - 1) / kRead4Threads;
    if (blocks > 0x7FFFFFFF) return DSA_ERR_UNSUPPORTED;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    const dim3 grid(static_cast<unsigned>(blocks));
    const bool sectors = ((reinterpret_cast<uintptr_t>(k_out) | reinterpret_cast<uintptr_t>(v_out)) & 31) == 0 &&
                         ((k_token_stride | k_head_stride | v_token_stride | v_head_stride) & 15) == 0;
    auto* kernel = dtype == DSA_BF16 ? (sectors ? kv_read_fp4_kernel<Bf16, true> : kv_read_fp4_kernel<Bf16, false>)
                                     : (sectors ? kv_read_fp4_kernel<Fp16, true> : kv_read_fp4_kernel<Fp16, false>);
    const cudaError_t err = launch_pdl(kernel, grid, dim3(kRead4Threads), 0, stream, a);
    return err == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}
